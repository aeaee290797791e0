// Sampling a token from each row of logits: temperature, top-k, top-p, min-p
// and a draw from a given uniform number.
//
// w_i = exp((l_i - max l) / T), tokens ordered by (l descending, i ascending).
// top-k keeps the first k; top-p the shortest prefix whose sum reaches p times
// the top-k sum; min-p the tokens with w >= min_p (the largest w is 1). The
// token is the first i, in vocabulary order, whose running sum of kept weights
// passes u times their total. Both cuts are prefixes of one order, so the set
// that they leave is (key of the last kept logit, how many of its equals), and
// no row is ever sorted.
//
// One thread-block cluster takes a row: its CTAs hold a slice each in shared
// memory, so the logits are read from memory once, and histograms and totals
// meet through distributed shared memory.
//
// Mostly a short list settles a row, which the first CTA ranks and finishes by
// itself. For a small top-k a histogram of the threads' largest logits (one
// addition to a thread) gives a bound that the k-th largest token cannot lie
// below. Else a cut is found by a histogram of all tokens over equal steps of
// (max l - l) / T (1024 of them, down to weights of 2^-46), whose bins a
// vocabulary's logits fill evenly, so that few of a warp's additions meet in one
// word; if what top-p keeps fits the list, it is listed, else the cut's bin alone
// is ranked, or cut further by histograms over its keys until it holds at most
// kList tokens or equal logits only. What bounds it: the passes over the slices in
// shared memory (some 35 instructions a token where weights are summed) and, for one
// row, the barriers between them. Measured (a graph's launch included): one row of
// 151936 with temperature, top-k 20, top-p 0.95 and min-p 14.4 us; 64 such rows 37 us,
// without a cut 37 us (39 MB, 1.1 TB/s), with top-p alone 55 us where that keeps few
// tokens, 92 us at 0.92 of a spread-out row and 111 us at 0.92 of a flat one.
//
// Sums are taken in 64-bit fixed point (2^46 for the largest weight): they are
// the same whatever the order of the additions, so one input gives one token.
#include <algorithm>
#include <type_traits>

#include "qw3_internal.cuh"

namespace qw3 {

namespace {

using u64 = unsigned long long;

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 2 * kThreads;   // two to a thread
constexpr int kList = 256;      // tokens that the first CTA ranks
constexpr int kMaxCluster = 16;

// The largest weight in fixed point: 2^46 while 64 bits hold the sum of a vocabulary of
// them (and 32 bits the digit sums of a slice), else 2^40. Weights are odd: cut to a
// multiple of 2, and half of that added, so that the sums lean to neither side (what
// cutting alone takes from 150,000 small weights moves the draw of one row in 40,000
// at 2^46, and of one in 500 at 2^40).
constexpr int kFineVocab = 1 << 18, kFineBits = 46, kCoarseBits = 40;

// Order of logits as unsigned keys; the two zeros are one value.
__device__ __forceinline__ uint32_t logit_key(float v) { return float_order_key(v + 0.0f); }

// e in [0, 1] times 2^bits, cut to an integer, or (up) the next one where that cuts
// something off: from its bits (a conversion of f32 to 64 bits runs on the f64 units,
// which are few).
__device__ __forceinline__ u64 fixed_point(float e, int bits, bool up = false) {
    const uint32_t x = __float_as_uint(e);
    if (!(e > 0.0f)) return 0ull;
    const int shift = static_cast<int>(x >> 23) - 150 + bits;   // e = mantissa * 2^(shift - bits)
    const u64 m = (x & 0x7fffffu) | (x >> 23 ? 0x800000u : 0u);
    const u64 v = shift >= 0 ? m << shift : (shift > -24 ? m >> -shift : 0ull);
    return v + (up && shift < 0 && (shift <= -24 || (m & ((1ull << -shift) - 1ull)) != 0ull));
}

// f x for f in [0, 1], to the integer below or (up) above, exactly: equal weights are
// parted where f says, which a product in f64 would miss by what it rounds off.
__device__ __forceinline__ u64 share_of(float f, u64 x, bool up) {
    if (!(f > 0.0f)) return 0ull;
    if (f >= 1.0f) return x;
    const uint32_t b = __float_as_uint(f);
    const u64 m = (b & 0x7fffffu) | (b >> 23 ? 0x800000u : 0u);
    const int e = 150 - max(static_cast<int>(b >> 23), 1);   // f = m 2^-e, e >= 24
    const u64 hi = __umul64hi(m, x), lo = m * x;
    if (e >= 64) return (e < 128 ? hi >> (e - 64) : 0ull) + (up && x > 0 && (e >= 128 || lo || (hi & ((1ull << (e - 64)) - 1ull))));
    return (lo >> e | hi << (64 - e)) + (up && (lo & ((1ull << e) - 1ull)));
}

// 2^30 * 2^(j / 256), rounded: made when this file is compiled, by the series of exp.
struct Powers {
    uint32_t v[256];
    constexpr Powers() : v() {
        for (int j = 0; j < 256; ++j) {
            const double x = j * (0.69314718055994530942 / 256);
            double term = 1.0, sum = 1.0;
            for (int i = 1; i < 24; ++i) {
                term *= x / i;
                sum += term;
            }
            v[j] = static_cast<uint32_t>(sum * 1073741824.0 + 0.5);
        }
    }
};
__device__ const Powers kPowers{};

__device__ __forceinline__ void remote_st(uint32_t addr, u64 v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ uint32_t remote_ld32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t remote_add(uint32_t addr, uint32_t v) {
    uint32_t o;
    asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(o) : "r"(addr), "r"(v) : "memory");
    return o;
}

// The cluster barrier wants each warp in one piece.
__device__ __forceinline__ void sync_cluster() {
    __syncwarp();
    hw_cluster_sync();
}

struct Shared {
    // this CTA's histogram: counts, and weights as sums of their digits (16 bits at
    // 2^46 with up to 45056 tokens to a slice, 14 at 2^40 with up to 2^18: no sum
    // passes 32 bits)
    uint32_t cnt[kBins], digit[3][kBins];
    // the row's
    uint32_t tcnt[kBins];
    u64 tw[kBins];
    // tokens of a small bin, in the first CTA: key and ~index, weight
    u64 list[kList], list_w[kList];
    u64 peer[kMaxCluster];    // a word from each CTA
    u64 peer2[kMaxCluster];
    u64 red[2 * kWarps + 2];
    uint32_t n_list;
    int row;           // which row this cluster takes
    uint64_t bar;      // the slice has arrived
    uint32_t lost;     // it did not in time
    // what a search found
    uint32_t bin, found, last_rank, sent;
    u64 above_cnt, above_w;
    u64 res[4];   // cut, ties, weight of the prefix, ties left out
    uint32_t pow2[256];   // kPowers
};

// Sums over the threads below this one, of a and b at once, and in ta and tb
// over the block.
__device__ __forceinline__ void scan2(u64 &a, u64 &b, u64 &ta, u64 &tb, Shared &s) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    u64 x = a, y = b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 p = __shfl_up_sync(0xffffffffu, x, o), q = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) {
            x += p;
            y += q;
        }
    }
    __syncthreads();
    if (lane == 31) {
        s.red[warp] = x;
        s.red[kWarps + warp] = y;
    }
    __syncthreads();
    u64 bx = 0, by = 0;
    ta = tb = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const u64 p = s.red[w], q = s.red[kWarps + w];
        if (w < warp) {
            bx += p;
            by += q;
        }
        ta += p;
        tb += q;
    }
    a = bx + x - a;
    b = by + y - b;
}

constexpr float kNats = 32.0f, kCoarseNats = 28.0f;   // exp(-32) < 2^-46, exp(-28) < 2^-40: beyond, no weight

// Largest word of the block.
__device__ __forceinline__ uint32_t block_max(uint32_t v, Shared &s) {
    v = __reduce_max_sync(0xffffffffu, v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s.red[threadIdx.x >> 5] = v;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v = max(v, static_cast<uint32_t>(s.red[w]));
    return v;
}

// Weights: 2^(x / 256) with x = (l - max l) 256 log2(e) / T, the 256 powers of a table
// and a polynomial between them (a published way to exp: P. Tang, "Table-driven
// implementation of the exponential function in IEEE floating-point arithmetic",
// 1989). l c - max c, c = 256 log2(e) / T, is had with c in two floats, its whole part
// taken off within the fma, so that what is left, at most 1, keeps an error of some
// 2^-24; the weight is then within 2^-29 of exact, besides its rounding to an odd
// integer. It takes some 25 instructions. A single f32 weight (ex2.approx of an argument
// rounded twice: 10 instructions, 4e-6 off at most) gave another token than 64 bits in
// one row of 600 over a whole vocabulary; its times: 64 rows of 151936 with mixed
// settings 45 us against 47.5, without a cut 32 against 37.
struct Row {
    const float *l;   // this CTA's slice, in shared or global memory
    int n, base;      // its length, and its first token
    float top, step;  // the largest logit; bins per unit of logit
    uint32_t rank, size;      // in the cluster
    float c, c_lo;            // c in two floats
    float x;                  // less the fraction of max c; its whole part
    int whole;
    float least;              // logits below have no weight
    bool wide;                // max c is too large for that: the difference first
    int bits;                 // the largest weight is 2^bits
    const uint32_t *pow2;

    // the temperature's part, while the slice is on its way, and the largest logit's
    __device__ __forceinline__ void set_temperature(float T) {
        constexpr float kL = 369.32993f;   // 256 log2(e) in two floats
        constexpr float kLlo = static_cast<float>(256.0 * 1.4426950408889634074 - static_cast<double>(kL));
        c = __fdiv_rn(kL, T);
        c_lo = __fdiv_rn(__fadd_rn(__fmaf_rn(-c, T, kL), kLlo), T);
        step = kBins / kNats / T;
    }
    __device__ __forceinline__ void set_top(float highest, float T) {
        top = highest;
        wide = !(fabsf(__fmul_rn(top, c)) < 2097152.0f);
        const float m = __fmaf_rn(top, c, kMagic);
        whole = __float_as_int(m);
        x = -__fmaf_rn(top, c_lo, __fmaf_rn(top, c, -__fsub_rn(m, kMagic)));
        least = fmaxf(top - (bits == kFineBits ? kNats : kCoarseNats) * T, -3.4028235e38f);
    }
    static constexpr float kMagic = 12582912.0f;   // 1.5 * 2^23: a number added to it is rounded to an integer
    // The weight of a logit (of the row's: at most top, or -inf) in fixed point.
    __device__ __forceinline__ u64 weight(float v) const { return wide ? weight<true>(v) : weight<false>(v); }
    template <bool WIDE>
    __device__ __forceinline__ u64 weight(float v) const {
        float f;
        int k;
        if constexpr (!WIDE) {
            const float m = __fmaf_rn(v, c, kMagic);
            f = __fadd_rn(__fmaf_rn(v, c_lo, __fmaf_rn(v, c, -__fsub_rn(m, kMagic))), x);
            k = __float_as_int(m) - whole;
        } else {
            // v - top as two floats (Knuth's two-sum), then its product with c
            const float s = __fsub_rn(v, top), b = __fsub_rn(s, v);
            const float e = __fsub_rn(__fsub_rn(v, __fsub_rn(s, b)), __fadd_rn(top, b));
            const float m = __fmaf_rn(s, c, kMagic);
            f = __fmaf_rn(e, c, __fmaf_rn(s, c_lo, __fmaf_rn(s, c, -__fsub_rn(m, kMagic))));
            k = __float_as_int(m) - __float_as_int(kMagic);
        }
        // 2^(f / 256) - 1, |f| <= 1, as a multiple of 2^-30: what the sum with a number of 2^-7 keeps
        constexpr double kG = 0.69314718055994530942 / 256;
        constexpr float kA1 = static_cast<float>(kG), kA2 = static_cast<float>(kG * kG / 2);
        constexpr float kA3 = static_cast<float>(kG * kG * kG / 6), kSplit = 1.5f / 128.0f;
        constexpr uint32_t kSplitBits = 0x3c400000u;   // kSplit's
        const float y = __fmul_rn(f, __fmaf_rn(f, __fmaf_rn(f, kA3, kA2), kA1));
        const uint32_t one_y = __float_as_uint(__fadd_rn(y, kSplit)) + ((1u << 30) - kSplitBits);
        // 2^60 times the weight less its power of two (where `least` was rounded down, k
        // may be past the last bit)
        const u64 m = static_cast<u64>(pow2[k & 255]) * one_y;
        return v >= least ? m >> min(60 - bits - (k >> 8), 63) | 1ull : 0ull;
    }
    // Bin of a logit, kBins or more for one that has no weight: the float
    // operations are monotone, so the bins follow the order of the logits.
    __device__ __forceinline__ int bin(float v) const {
        return static_cast<int>(fminf((top - v) * step, static_cast<float>(kBins)));
    }
    // bin(v) <= b, for b < kBins
    __device__ __forceinline__ bool within(float v, int b) const { return (top - v) * step < static_cast<float>(b + 1); }
};

// Shares a word of this CTA with its cluster: afterwards slot[r] holds CTA r's.
__device__ __forceinline__ void share(const Row &row, u64 *slot, u64 v) {
    if (threadIdx.x < row.size) remote_st(dsmem_map(&slot[row.rank], threadIdx.x), v);
    sync_cluster();
}

__device__ __forceinline__ int digit_bits(const Row &row) { return row.bits == kFineBits ? 16 : 14; }

__device__ __forceinline__ void clear_histogram(bool weigh, Shared &s) {
    for (int i = threadIdx.x; i < kBins; i += kThreads) {
        if (weigh) s.digit[0][i] = s.digit[1][i] = s.digit[2][i] = 0u;
        else s.cnt[i] = 0u;
    }
    __syncthreads();
}

// As many tokens at most as bin b of the first histogram holds, if they weigh w
// together: its weights lie within 3.2 percent of each other, and 0.1 percent
// covers the roundings of bins and weights. (2^20 where weights are so small that
// being rounded to integers counts.)
__device__ __forceinline__ uint32_t most_in_bin(u64 w, int b, int bits) {
    const float least = exp2f(static_cast<float>(bits) - kNats / kBins * 1.4426950408889634f * (b + 1.0f)) * 0.999f;
    return w == 0 ? 0u : least < 4096.0f ? 1u << 20 : static_cast<uint32_t>(fminf(static_cast<float>(w) / least, 1048576.0f));
}

// The cluster's histograms added up, in every CTA's tcnt and tw; with weights
// tcnt is what most_in_bin says.
__device__ __forceinline__ void add_histograms(const Row &row, bool weigh, Shared &s) {
    const int d = digit_bits(row);
    if (row.size == 1) {
        __syncthreads();
        for (int i = threadIdx.x; i < kBins; i += kThreads) {
            const u64 w = weigh ? (static_cast<u64>(s.digit[2][i]) << (2 * d)) + (static_cast<u64>(s.digit[1][i]) << d) + s.digit[0][i] : 0;
            s.tcnt[i] = weigh ? most_in_bin(w, i, row.bits) : s.cnt[i];
            s.tw[i] = w;
        }
        __syncthreads();
        return;
    }
    sync_cluster();
    // each CTA adds its share of the bins over the cluster and hands it to all:
    // size / 2 neighbouring threads to a bin, two CTAs to each
    const int parts = static_cast<int>(row.size) / 2, part = static_cast<int>(threadIdx.x) % parts;
    const int bin = static_cast<int>(row.rank) * (kBins / static_cast<int>(row.size)) + static_cast<int>(threadIdx.x) / parts;
    uint32_t c = 0;
    u64 w = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t p = 2 * part + h;
        if (!weigh) {
            c += remote_ld32(dsmem_map(&s.cnt[bin], p));
        } else {
            w += static_cast<u64>(remote_ld32(dsmem_map(&s.digit[2][bin], p))) << (2 * d);
            w += static_cast<u64>(remote_ld32(dsmem_map(&s.digit[1][bin], p))) << d;
            w += remote_ld32(dsmem_map(&s.digit[0][bin], p));
        }
    }
    for (int o = 1; o < parts; o <<= 1) {
        if (!weigh) c += __shfl_xor_sync(0xffffffffu, c, o);
        else w += __shfl_xor_sync(0xffffffffu, w, o);
    }
    if (weigh) c = most_in_bin(w, bin, row.bits);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t p = 2 * part + h;
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(dsmem_map(&s.tcnt[bin], p)), "r"(c) : "memory");
        remote_st(dsmem_map(&s.tw[bin], p), w);
    }
    sync_cluster();
}

// Histogram of the row, of counts or (weigh) of weights: bin_of(logit) gives a
// bin or a negative number for a token left out.
template <bool WIDE, typename F>
__device__ __forceinline__ void weigh_slice(const Row &row, Shared &s, F bin_of) {
    const int d = digit_bits(row);
    const uint32_t mask = (1u << d) - 1u;
#pragma unroll 4
    for (int i = threadIdx.x; i < row.n; i += kThreads) {
        const float v = row.l[i];
        const int bin = bin_of(v);
        if (bin < 0) continue;
        const u64 w = row.weight<WIDE>(v);
        const uint32_t d0 = static_cast<uint32_t>(w) & mask, d1 = static_cast<uint32_t>(w >> d) & mask;
        const uint32_t d2 = static_cast<uint32_t>(w >> (2 * d));
        if (d0) atomicAdd(&s.digit[0][bin], d0);
        if (d1) atomicAdd(&s.digit[1][bin], d1);
        if (d2) atomicAdd(&s.digit[2][bin], d2);
    }
}
template <typename F>
__device__ __forceinline__ void histogram(const Row &row, bool weigh, Shared &s, F bin_of) {
    clear_histogram(weigh, s);
    if (weigh) {
        if (row.wide) weigh_slice<true>(row, s, bin_of);
        else weigh_slice<false>(row, s, bin_of);
    } else {
#pragma unroll 4
        for (int i = threadIdx.x; i < row.n; i += kThreads) {
            const int bin = bin_of(row.l[i]);
            if (bin >= 0) atomicAdd(&s.cnt[bin], 1u);
        }
    }
    add_histograms(row, weigh, s);
}

// The bin in which the running sum (of counts, or of weights) of the row's
// histogram, over above_c and above_w, reaches target.
struct Found {
    bool some;
    int bin;
    u64 n;                         // tokens in the bin (of weights: as many at most)
    u64 w, above_c, above_w;       // its weight; counts and weight before it
    u64 total_c, total_w;          // of all bins
};

__device__ __forceinline__ Found find(bool by_weight, u64 target, u64 above_c, u64 above_w, Shared &s) {
    // thread t looks at bins 2 t and 2 t + 1
    const int b0 = 2 * threadIdx.x;
    u64 c = static_cast<u64>(s.tcnt[b0]) + s.tcnt[b0 + 1], w = s.tw[b0] + s.tw[b0 + 1];
    Found f;
    scan2(c, w, f.total_c, f.total_w, s);
    if (threadIdx.x == 0) s.found = 0u;
    __syncthreads();
    c += above_c;
    w += above_w;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const u64 nc = c + s.tcnt[b0 + h], nw = w + s.tw[b0 + h];
        if (by_weight ? (w < target && nw >= target) : (c < target && nc >= target)) {
            s.found = 1u;
            s.bin = b0 + h;
            s.above_cnt = c;
            s.above_w = w;
        }
        c = nc;
        w = nw;
    }
    __syncthreads();
    f.some = s.found != 0u;
    f.bin = f.some ? static_cast<int>(s.bin) : 0;
    f.n = s.tcnt[f.bin];
    f.w = s.tw[f.bin];
    f.above_c = s.above_cnt;
    f.above_w = s.above_w;
    return f;
}

// The tokens that `in` picks, at most kList in the row, into the first CTA's
// list; the list's length there is s.n_list. All CTAs leave together.
template <typename F>
__device__ __forceinline__ void gather(const Row &row, Shared &s, F in) {
    const uint32_t n_at = dsmem_map(&s.n_list, 0u), list_at = dsmem_map(s.list, 0u);
    for (int i = threadIdx.x; i < row.n; i += kThreads) {
        const float v = row.l[i];
        if (in(v)) {
            const uint32_t at = remote_add(n_at, 1u);
            if (at < kList)
                remote_st(list_at + 8u * at,
                          static_cast<u64>(logit_key(v)) << 32 | (0xffffffffu - static_cast<uint32_t>(row.base + i)));
        }
    }
    if (row.size > 1) sync_cluster();
    else __syncthreads();
}

struct Cut {
    uint32_t key;      // kept: keys above, and the first `ties` equal to it
    u64 ties;
    u64 w;             // weight of what is kept (by_weight cuts only)
    bool some;         // equals of the key are left out
};

// The tokens of a bin of weight w in which no token's exact weight lies below that
// of `one`: as many at most (with room for that weight's roundings).
__device__ __forceinline__ u64 most_tokens(u64 w, u64 one) {
    const u64 low = one - (one >> 14) - 1;
    return one > 1 ? w / low + 1 : ~0ull;
}

// The shortest prefix of the row's order that holds `target` tokens or
// (by_weight) reaches `target` weight, its end known to lie in the bin f of the
// first histogram; keys below floor_key are out.
__device__ Cut cut_in_bin(const Row &row, Found f, bool by_weight, u64 target, uint32_t floor_key, Shared &s) {
    const int bin0 = f.bin;
    // keys that the bin can hold, with room for the rounding of its float operations
    const float slack = 4.0f * 1.2e-7f * (fabsf(row.top) + (bin0 + 2.0f) / row.step);
    uint32_t hi = logit_key(row.top - static_cast<float>(bin0) / row.step + slack);
    uint32_t lo = logit_key(row.top - (static_cast<float>(bin0) + 1.0f) / row.step - slack);
    hi = min(hi, logit_key(row.top));
    lo = min(max(lo, floor_key), hi);
    if (by_weight) f.n = most_tokens(f.w, fixed_point(exp2f(-kNats / kBins * 1.4426950408889634f * (bin0 + 1.0f)), row.bits));
    while (f.n > kList) {
        if (lo == hi) {
            // equal logits, each of weight `one`
            const u64 one = row.weight(float_from_order_key(lo));
            const u64 m = by_weight ? (target - f.above_w - 1) / one + 1 : target - f.above_c;
            return Cut{lo, m, f.above_w + m * one, by_weight ? m * one < f.w : m < f.n};
        }
        const int bits = 32 - __clz(hi - lo), shift = bits > 10 ? bits - 10 : 0;
        histogram(row, by_weight, s, [&](float v) {
            const uint32_t k = logit_key(v);
            return row.bin(v) == bin0 && k >= lo && k <= hi ? static_cast<int>((hi - k) >> shift) : -1;
        });
        f = find(by_weight, target, f.above_c, f.above_w, s);
        hi -= static_cast<uint32_t>(f.bin) << shift;
        const uint32_t width = (1u << shift) - 1u;
        lo = hi - lo >= width ? hi - width : lo;
        if (by_weight) f.n = most_tokens(f.w, row.weight(float_from_order_key(lo)));
    }
    gather(row, s, [&](float v) {
        const uint32_t k = logit_key(v);
        return row.bin(v) == bin0 && k >= lo && k <= hi;
    });
    if (row.rank == 0) {
        const int n = static_cast<int>(min(s.n_list, static_cast<uint32_t>(kList)));
        // two threads to a token, each looking at every other one
        const int i = static_cast<int>(threadIdx.x) >> 1, half = static_cast<int>(threadIdx.x) & 1;
        if (threadIdx.x == 0) s.last_rank = 0u;
        u64 before_w = 0, mine = 0, w = 0;
        if (i < n) {
            mine = s.list[i];
            w = row.weight(float_from_order_key(static_cast<uint32_t>(mine >> 32)));
            s.list_w[i] = w;
        }
        __syncthreads();
        uint32_t rank = 0, same = 0, equal = 0;
        if (i < n) {
            const uint32_t key = static_cast<uint32_t>(mine >> 32);
#pragma unroll 4
            for (int j = half; j < n; j += 2) {
                const u64 x = s.list[j], xw = s.list_w[j];
                const bool above = x > mine, eq = static_cast<uint32_t>(x >> 32) == key;
                rank += above;
                before_w += above ? xw : 0;
                same += above && eq;
                equal += eq;
            }
        }
        rank += __shfl_xor_sync(0xffffffffu, rank, 1);
        same += __shfl_xor_sync(0xffffffffu, same, 1);
        equal += __shfl_xor_sync(0xffffffffu, equal, 1);
        before_w += __shfl_xor_sync(0xffffffffu, before_w, 1) + f.above_w;
        const bool kept = i < n && (by_weight ? before_w < target : f.above_c + rank < target);
        if (kept) atomicMax(&s.last_rank, rank);
        __syncthreads();
        if (kept && !half && rank == s.last_rank) {
            s.res[0] = mine >> 32;
            s.res[1] = same + 1;
            s.res[2] = before_w + w;
            s.res[3] = equal - same - 1;
        }
        if (threadIdx.x == 0) s.n_list = 0u;
        __syncthreads();
        if (threadIdx.x < row.size * 4u && threadIdx.x >= 4u)
            remote_st(dsmem_map(&s.res[threadIdx.x & 3], threadIdx.x >> 2), s.res[threadIdx.x & 3]);
    }
    if (row.size > 1) sync_cluster();
    else __syncthreads();
    const Cut cut{static_cast<uint32_t>(s.res[0]), s.res[1], s.res[2], s.res[3] != 0};
    __syncthreads();
    return cut;
}

// The answer: token, and its weight's share of the total. (v - top) / T in two
// parts, so that the probability is good to a few f32 roundings.
__device__ __forceinline__ void answer(const SampleArgs &a, int b, int token, float v, const Row &row, u64 total) {
    a.token[b] = token;
    if (a.next) a.next[b] = token;
    if (a.prob) {
        const float T = a.temperature ? fmaxf(a.temperature[b], 1e-30f) : 1.0f;
        // v - top as two floats (Knuth's two-sum): rounded, 20 below the largest costs 6e-7
        const float d = __fsub_rn(v, row.top), z = __fsub_rn(d, v);
        const float lo = __fsub_rn(__fsub_rn(v, __fsub_rn(d, z)), __fadd_rn(row.top, z));
        const float q = __fdiv_rn(d, T), r = __fdiv_rn(__fadd_rn(__fmaf_rn(-q, T, d), lo), T);
        const float e = expf(q);
        a.prob[b] = fmaf(e, r, e) * (exp2f(static_cast<float>(row.bits)) / static_cast<float>(total));
    }
}

// The row from its list alone (the first CTA): the top-k tokens are all in it,
// or (k = 0) the tokens of weight p of the row's total `all`. Two threads to a
// token, each looking at every other one.
__device__ void finish_list(const SampleArgs &a, int b, const Row &row, u64 k, float p, u64 mp, u64 all, Shared &s) {
    const int n = static_cast<int>(min(s.n_list, static_cast<uint32_t>(kList))), i = threadIdx.x >> 1, half = threadIdx.x & 1;
    u64 mine = 0, w = 0;
    float v = 0.0f;
    if (i < n) {
        mine = s.list[i];
        v = float_from_order_key(static_cast<uint32_t>(mine >> 32));
        w = row.weight(v);
        s.list_w[i] = w;
    }
    __syncthreads();
    u64 before = 0;
    uint32_t rank = 0;
    if (i < n)
        for (int j = half; j < n; j += 2)
            if (s.list[j] > mine) {
                ++rank;
                before += s.list_w[j];
            }
    rank += __shfl_xor_sync(0xffffffffu, rank, 1);
    before += __shfl_xor_sync(0xffffffffu, before, 1);
    bool kept = i < n && (k == 0 || rank < k);
    if (p < 1.0f) {
        if (k > 0) {
            u64 x = kept && !half ? w : 0, y = 0, none;
            scan2(x, y, all, none, s);
        }
        const u64 target = share_of(p, all, true);
        kept = kept && (rank == 0 || before < target);
    }
    kept = kept && w >= mp;
    __syncthreads();
    if (i < n) s.list_w[i] = kept ? w : 0;
    u64 x = kept && !half ? w : 0, y = 0, total, none;
    scan2(x, y, total, none, s);   // its barriers also show everyone the kept weights
    const uint32_t idx = static_cast<uint32_t>(mine);   // ~index: the larger, the earlier
    u64 first = 0;
    if (kept)
        for (int j = half; j < n; j += 2)
            if (static_cast<uint32_t>(s.list[j]) > idx) first += s.list_w[j];
    first += __shfl_xor_sync(0xffffffffu, first, 1);
    const float u = a.u[b];
    u64 at = share_of(u, total, false);
    if (at >= total) at = total - 1;
    if (kept && !half && first <= at && at < first + w) answer(a, b, static_cast<int>(0xffffffffu - idx), v, row, total);
}

// Lists the row's largest tokens in the first CTA, the `want` largest among
// them, where that takes at most kList: a bin that `want` of the threads' largest
// logits (thread_top) reach holds, with those above it, at least so many tokens.
// Every CTA returns the same.
__device__ __forceinline__ bool try_list(const Row &row, float thread_top, u64 want, Shared &s) {
    if (threadIdx.x == 0) s.sent = 0u;
    clear_histogram(false, s);
    const int mine = row.bin(thread_top);
    if (mine < kBins) atomicAdd(&s.cnt[mine], 1u);
    add_histograms(row, false, s);
    const Found f = find(false, want, 0, 0, s);
    if (!f.some) return false;
    const uint32_t n_at = dsmem_map(&s.n_list, 0u), list_at = dsmem_map(s.list, 0u);
    u64 count = 0;
#pragma unroll 4
    for (int i = threadIdx.x; i < row.n; i += kThreads) {
        const float v = row.l[i];
        if (row.within(v, f.bin)) {
            ++count;
            // a CTA with more than the list holds (equal logits, say) need not send them
            if (atomicAdd(&s.sent, 1u) < kList) {
                const uint32_t at = remote_add(n_at, 1u);
                if (at < kList)
                    remote_st(list_at + 8u * at,
                              static_cast<u64>(logit_key(v)) << 32 | (0xffffffffu - static_cast<uint32_t>(row.base + i)));
            }
        }
    }
    u64 none = 0, total, zero;
    scan2(count, none, total, zero, s);
    if (row.size > 1) {
        share(row, s.peer, total);   // the list has arrived too
        total = 0;
        for (uint32_t p = 0; p < row.size; ++p) total += s.peer[p];
    }
    const bool fits = total <= kList;
    __syncthreads();
    if (!fits && threadIdx.x == 0) s.n_list = 0u;   // a later gather starts over
    return fits;
}

// The row of the cluster that starts as the c-th of n <= kThreads: rows that take
// longest first, so that no such row is begun last (cuts over the whole
// vocabulary, then long lists, then the rest).
__device__ int row_of(const SampleArgs &a, int n, int c, Shared &s) {
    const int i = static_cast<int>(threadIdx.x);
    int kind = -1;
    if (i < n) {
        const int k = a.top_k ? a.top_k[i] : 0;
        const bool has_k = k > 0 && k < a.V, greedy = a.temperature && a.temperature[i] <= 0.0f;
        const bool whole = has_k ? k > kList : a.top_p && a.top_p[i] < 1.0f;
        kind = greedy ? 0 : whole ? 2 : has_k && k > 64 ? 1 : 0;
    }
    u64 x2 = kind == 2, x1 = kind == 1, n2, n1;
    scan2(x2, x1, n2, n1, s);
    const u64 at = kind == 2 ? x2 : kind == 1 ? n2 + x1 : n2 + n1 + static_cast<u64>(i) - x2 - x1;
    if (kind >= 0 && at == static_cast<u64>(c)) s.row = i;
    __syncthreads();
    return s.row;
}

template <bool kHeld>
__global__ void __launch_bounds__(kThreads) k_sample(SampleArgs a, int slice, bool reorder) {
    extern __shared__ __align__(16) float held[];
    __shared__ Shared s;
    const int tid = threadIdx.x;
    const uint32_t power = kPowers.v[tid & 255];
    pdl_wait();
    const int size = static_cast<int>(gridDim.x);   // one cluster along x
    Row row;
    row.rank = size > 1 ? cluster_rank() : 0u;
    // a CTA's shared memory may be written by its peers once it has started: waited
    // for at the first share below, behind the slice's load
    if (size > 1) cluster_arrive_release();
    row.size = static_cast<uint32_t>(size);
    const int b = reorder ? row_of(a, static_cast<int>(gridDim.y), static_cast<int>(blockIdx.y), s) : static_cast<int>(blockIdx.y);
    row.base = static_cast<int>(row.rank) * slice;
    row.n = max(0, min(slice, a.V - row.base));
    const float *src = a.logits + b * a.stride + row.base;
    row.l = src;
    row.bits = a.V < kFineVocab ? kFineBits : kCoarseBits;
    row.pow2 = s.pow2;
    const float T = a.temperature ? a.temperature[b] : 1.0f;

    // ---- the slice into shared memory: the 16-byte aligned middle as one bulk
    // copy, the ends by themselves, each value as far from a 16-byte boundary as in memory
    if constexpr (kHeld) {
        const int shift = static_cast<int>((reinterpret_cast<uintptr_t>(src) / 4) & 3);
        float *to = held + shift;
        row.l = to;
        const int head = min(row.n, (4 - shift) & 3), mid = (row.n - head) / 4 * 4;
        if (tid == 0) {
            mbar_init(&s.bar, 1);
            fence_mbar_init();
            if (mid > 0) {
                mbar_arrive_expect_tx(&s.bar, static_cast<uint32_t>(mid) * 4u);
                bulk_g2s(to + head, src + head, static_cast<uint32_t>(mid) * 4u, &s.bar, policy_evict_first());
            }
        }
        for (int i = tid; i < head; i += kThreads) to[i] = src[i];
        for (int i = head + mid + tid; i < row.n; i += kThreads) to[i] = src[i];
        if (tid == 0) s.lost = 0u;
        row.set_temperature(fmaxf(T, 1e-30f));
        __syncthreads();
        if (mid > 0 && !mbar_wait_bounded(&s.bar, 0u)) {
            // the copy did not arrive in a second: what there is of it is taken
            // (every thread saw the wait run out, or sees the data now)
            s.lost = 1u;
        }
        __syncthreads();
        if (s.lost && tid == 0) {
            record_status(a.status, QW3_ERR_TIMEOUT);
            (void)mbar_wait_bounded(&s.bar, 0u);
        }
    }

    if constexpr (!kHeld) row.set_temperature(fmaxf(T, 1e-30f));
    if (tid < 256) s.pow2[tid] = power;   // (barriers follow before its first use)
    // ---- the largest logit; a NaN counts above all
    float top = -INFINITY;
    bool nan = false;
    if (tid == 0) s.n_list = 0u;
#pragma unroll 4
    for (int i = tid; i < row.n; i += kThreads) {
        const float v = row.l[i];
        nan |= v != v;
        top = fmaxf(top, v);
    }
    u64 best = block_max(nan ? ~0u : logit_key(top), s);
    if (size > 1) {
        __syncwarp();
        cluster_wait_acquire();   // every CTA of the cluster runs
        share(row, s.peer, best);
        for (int p = 0; p < size; ++p) best = s.peer[p] > best ? s.peer[p] : best;
    }
    row.top = float_from_order_key(static_cast<uint32_t>(best));
    const float p = a.top_p ? a.top_p[b] : 1.0f, min_p = a.min_p ? a.min_p[b] : 0.0f;
    const bool greedy = T <= 0.0f;
    // a setting that is not a number has no answer
    const bool bad = best == ~0u || row.top == -INFINITY || !(fabsf(T) < INFINITY) ||
                     (!greedy && (row.top == INFINITY || p != p || min_p != min_p));
    if (bad || greedy) {
        u64 first = ~0ull;   // the lowest index of the largest logit
        if (!bad) {
            uint32_t at = ~0u;
            for (int i = tid; i < row.n; i += kThreads)
                if (row.l[i] == row.top) at = min(at, static_cast<uint32_t>(row.base + i));
            first = ~0u - block_max(~0u - at, s);
            if (size > 1) {
                share(row, s.peer2, first);
                for (int p = 0; p < size; ++p) first = s.peer2[p] < first ? s.peer2[p] : first;
            }
        }
        if (row.rank == 0 && tid == 0) {
            if (bad) record_status(a.status, QW3_ERR_NONFINITE);
            a.token[b] = bad ? -1 : static_cast<int>(first);
            if (a.next) a.next[b] = bad ? 0 : static_cast<int>(first);
            if (a.prob) a.prob[b] = bad ? 0.0f : 1.0f;
        }
        return;
    }
    row.set_top(row.top, fmaxf(T, 1e-30f));
    const int k = a.top_k ? a.top_k[b] : 0;
    const u64 mp = fixed_point(fminf(min_p, 1.0f), row.bits, true);
    // kept: every token with a weight, until a cut says otherwise
    Cut cut{0u, ~0ull, 0, false};
    const bool has_k = k > 0 && k < a.V;
    if (has_k && k <= kList && try_list(row, top, static_cast<u64>(k), s)) {
        if (row.rank == 0) finish_list(a, b, row, static_cast<u64>(k), p, mp, 0, s);
        return;
    }
    if (has_k) {
        histogram(row, false, s, [&](float v) {
            const int i = row.bin(v);
            return i < kBins ? i : -1;
        });
        const Found f = find(false, static_cast<u64>(k), 0, 0, s);
        if (f.some) cut = cut_in_bin(row, f, false, static_cast<u64>(k), 0u, s);
    }
    if (p < 1.0f) {
        // weights of what top-k left; of the equals of its last logit all are
        // counted, which matters only where the cut falls among them
        histogram(row, true, s, [&](float v) {
            const int i = row.bin(v);
            return i < kBins && logit_key(v) >= cut.key ? i : -1;
        });
        u64 x = s.tw[2 * tid] + s.tw[2 * tid + 1], y = 0, total, none;
        scan2(x, y, total, none, s);
        if (cut.some) {
            const u64 one = row.weight(float_from_order_key(cut.key));
            u64 equals = 0;
            for (int i = tid; i < row.n; i += kThreads) equals += logit_key(row.l[i]) == cut.key;
            u64 z = 0, all;
            scan2(equals, z, all, none, s);
            if (size > 1) {
                share(row, s.peer2, all);
                all = 0;
                for (int q = 0; q < size; ++q) all += s.peer2[q];
            }
            total -= (all - cut.ties) * one;
        }
        u64 target = share_of(p, total, true);
        target = target < 1 ? 1 : (target < total ? target : total);
        __syncthreads();
        const Found f = find(true, target, 0, 0, s);
        if (f.above_c + f.n <= kList) {
            gather(row, s, [&](float v) { return row.within(v, f.bin) && logit_key(v) >= cut.key; });
            if (row.rank == 0) finish_list(a, b, row, 0, p, mp, total, s);
            return;
        }
        const Cut c = cut_in_bin(row, f, true, target, cut.key, s);
        if (c.key > cut.key) cut = c;
        else if (c.ties < cut.ties) cut = Cut{c.key, c.ties, 0, true};
    }
    // ---- the draw: tokens in vocabulary order, a run of them to each thread;
    // an odd length keeps the threads' runs in different banks
    const int run = ((row.n + kThreads - 1) / kThreads) | 1, i0 = min(row.n, tid * run), i1 = min(row.n, i0 + run);
    u64 n0 = 0;
    if (cut.some) {
        // only the first equals of the cut key are kept: number them
        u64 none = 0, t0, t1;
        for (int i = i0; i < i1; ++i) n0 += logit_key(row.l[i]) == cut.key;
        scan2(n0, none, t0, t1, s);
        if (size > 1) {
            share(row, s.peer, t0);
            for (uint32_t q = 0; q < row.rank; ++q) n0 += s.peer[q];
        }
    }
    // kept weight of a token; nth: its number among the equals of the cut's logit
    const float edge = cut.key ? float_from_order_key(cut.key) : -INFINITY;
    row.least = fmaxf(row.least, edge);
    const auto weight = [&](float v, u64 nth) -> u64 {
        const u64 e = row.weight(v);
        return (v > edge || (v == edge && nth < cut.ties)) && e >= mp ? e : 0ull;
    };
    u64 w = 0, none = 0, t0, t1;
    if (cut.some) {
        u64 seen = n0;
        for (int i = i0; i < i1; ++i) {
            const float v = row.l[i];
            w += weight(v, seen);
            seen += logit_key(v) == cut.key;
        }
    } else {
        const auto sum = [&](auto wide) {
#pragma unroll 4
            for (int i = i0; i < i1; ++i) {
                const float v = row.l[i];
                const u64 e = row.weight<decltype(wide)::value>(v);
                w += e >= mp ? e : 0ull;
            }
        };
        if (row.wide) sum(std::true_type{});
        else sum(std::false_type{});
    }
    const u64 mine = w;
    scan2(w, none, t0, t1, s);
    u64 total = t0, before = 0;
    if (size > 1) {
        __syncthreads();
        share(row, s.peer2, t0);
        total = 0;
        for (int q = 0; q < size; ++q) {
            if (q < static_cast<int>(row.rank)) before += s.peer2[q];
            total += s.peer2[q];
        }
    }
    const float u = a.u[b];
    u64 at = share_of(u, total, false);
    if (at >= total) at = total - 1;
    w += before;
    // the warp whose lane holds the place looks through that lane's run, 32 tokens at a time
    const unsigned holder = __ballot_sync(0xffffffffu, w <= at && at < w + mine);
    if (!holder) return;
    const int from = __ffs(static_cast<int>(holder)) - 1, lane = tid & 31;
    const int first = __shfl_sync(0xffffffffu, i0, from), last = __shfl_sync(0xffffffffu, i1, from);
    u64 sum = __shfl_sync(0xffffffffu, w, from), nth = __shfl_sync(0xffffffffu, n0, from);
    for (int i = first; i < last; i += 32) {
        const bool in = i + lane < last;
        const float v = in ? row.l[i + lane] : -INFINITY;
        const unsigned equals = __ballot_sync(0xffffffffu, in && logit_key(v) == cut.key);
        const u64 x = in ? weight(v, cut.some ? nth + __popc(equals & ((1u << lane) - 1u)) : 0) : 0;
        u64 run = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const u64 y = __shfl_up_sync(0xffffffffu, run, o);
            if (lane >= o) run += y;
        }
        const unsigned past = __ballot_sync(0xffffffffu, sum + run > at);
        if (past) {
            if (lane == __ffs(static_cast<int>(past)) - 1) answer(a, b, row.base + i + lane, v, row, total);
            return;
        }
        sum += __shfl_sync(0xffffffffu, run, 31);
        nth += __popc(equals);
    }
}

// CTAs per row and the tokens of one: a small vocabulary stays in one CTA (64
// rows of 8192 with top-k and top-p 10.3 us, 12.3 in two CTAs), a large one is
// cut into slices of which two fit an SM (up to 20224 tokens, 79 KB: 64 rows of
// 151936 with settings of their own 47 us, 71 in 4 CTAs each that take an SM
// each), or finer, to 16 CTAs, while the rows together leave SMs free (one row
// without a cut 12.3 us in 16 CTAs, 13.9 in 8; 64 rows 52 and 37); beyond 16 slices
// of what one SM holds the row is read again from memory (L2) at every pass.
constexpr int kOneCta = 8192, kSlice = 20224, kMaxHeld = 45056;

}  // namespace

cudaError_t configure_sample() {
    cudaError_t e = cudaFuncSetAttribute(k_sample<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxHeld * 4 + 16);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(k_sample<true>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(k_sample<false>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    return e;
}

cudaError_t launch_sample(const SampleArgs &a, int B, bool pdl, cudaStream_t s) {
    if (B <= 0) return cudaSuccess;
    int size = 1;
    if (a.V > kOneCta)
        while (size < kMaxCluster && ((a.V + size - 1) / size > (size < 8 ? kSlice : kMaxHeld) ||
                                      (static_cast<int64_t>(B) * size * 2 <= 152 && a.V / size > kOneCta)))
            size *= 2;
    const int slice = (a.V + size - 1) / size;
    const bool is_held = slice <= kMaxHeld;
    // Settings that differ from row to row, in more than one wave (two CTAs to an
    // SM): 64 rows of 151936 47 us against 62, 400 of 32000 58 against 61, 512 of
    // 8192 29 against 32. Finding its row costs a CTA two microseconds, which rows
    // of the same settings pay for nothing: 37 us against 34, 51 against 46, 27
    // against 24.
    const bool reorder = static_cast<int64_t>(B) * size > 2 * 152 && B <= kThreads && (a.top_p || a.top_k);
    for (int b0 = 0; b0 < B; b0 += 65535) {
        SampleArgs x = a;
        x.logits += b0 * a.stride;
        if (x.temperature) x.temperature += b0;
        if (x.top_k) x.top_k += b0;
        if (x.top_p) x.top_p += b0;
        if (x.min_p) x.min_p += b0;
        x.u += b0;
        x.token += b0;
        if (x.next) x.next += b0;
        if (x.prob) x.prob += b0;
        const cudaError_t e = launch_pdl(pdl, is_held ? k_sample<true> : k_sample<false>, dim3(size, std::min(65535, B - b0)),
                                         kThreads, is_held ? static_cast<size_t>(slice) * 4 + 16 : 0, size, s, x, slice, reorder);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace qw3
