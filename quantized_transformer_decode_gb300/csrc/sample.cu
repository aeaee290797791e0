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
// meet through distributed shared memory. A cut is found by histograms over
// ranges of keys (1024 bins, counts and weights), each level inside the bin of
// the one before, until the bin holds at most kList tokens; these are ranked
// directly. A row with few distinct logits ends at a bin of one key instead.
//
// Sums are taken in 64-bit fixed point (2^40 for the largest weight): they are
// the same whatever the order of the additions, so one input gives one token.
#include <algorithm>

#include "qw3_internal.cuh"

namespace qw3 {

namespace {

using u64 = unsigned long long;

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 1024;
constexpr int kList = 256;
constexpr int kMaxCluster = 8;
constexpr float kOne = 1099511627776.0f;   // 2^40

// Order of logits as unsigned keys; the two zeros are one value.
__device__ __forceinline__ uint32_t logit_key(float v) { return float_order_key(v + 0.0f); }

// e in [0, 1] times 2^40, cut to an integer, from its bits (a conversion of
// f32 to 64 bits runs on the f64 units, which are few).
__device__ __forceinline__ u64 fixed_weight(float e) {
    const uint32_t x = __float_as_uint(e);
    const int shift = static_cast<int>(x >> 23) - 110;   // 2^40 e = mantissa * 2^shift
    const u64 m = (x & 0x7fffffu) | 0x800000u;
    return shift >= 0 ? m << shift : (shift > -24 ? m >> -shift : 0ull);
}

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
    // this CTA's histogram: counts, and weights as 32-bit halves with carries
    uint32_t cnt[kBins], wlo[kBins], whi[kBins];
    // the row's
    uint32_t tcnt[kBins];
    u64 tw[kBins];
    // tokens of a small bin, in the first CTA: key and ~index, weight
    u64 list[kList], list_w[kList];
    u64 peer[kMaxCluster];    // a word from each CTA
    u64 peer2[kMaxCluster];
    u64 red[2 * kWarps + 2];
    uint32_t n_list;
    // what a search found
    uint32_t bin, found, last_rank;
    u64 above_cnt, above_w;
    u64 res[4];   // cut, ties, weight of the prefix, ties left out
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

struct Row {
    const float *l;   // this CTA's slice, in shared or global memory
    int n, base;      // its length, and its first token
    float top, inv_t;
    uint32_t rank, size;   // in the cluster
    __device__ __forceinline__ float weight(float v) const { return expf((v - top) * inv_t); }
};

// Shares a word of this CTA with its cluster: afterwards slot[r] holds CTA r's.
__device__ __forceinline__ void share(const Row &row, u64 *slot, u64 v) {
    if (threadIdx.x < row.size) remote_st(dsmem_map(&slot[row.rank], threadIdx.x), v);
    sync_cluster();
}

// Histogram of the row's keys in [lo, hi], the highest keys in bin 0.
__device__ void histogram(const Row &row, uint32_t lo, uint32_t hi, int shift, Shared &s) {
    for (int i = threadIdx.x; i < kBins; i += kThreads) s.cnt[i] = s.wlo[i] = s.whi[i] = 0u;
    __syncthreads();
    for (int i = threadIdx.x; i < row.n; i += kThreads) {
        const float v = row.l[i];
        const uint32_t k = logit_key(v);
        if (k < lo || k > hi) continue;
        const uint32_t bin = (hi - k) >> shift;
        const u64 w = fixed_weight(row.weight(v));
        atomicAdd(&s.cnt[bin], 1u);
        const uint32_t wl = static_cast<uint32_t>(w), old = atomicAdd(&s.wlo[bin], wl);
        const uint32_t wh = static_cast<uint32_t>(w >> 32) + (old + wl < old ? 1u : 0u);
        if (wh) atomicAdd(&s.whi[bin], wh);
    }
    if (row.size == 1) {
        __syncthreads();
        for (int i = threadIdx.x; i < kBins; i += kThreads) {
            s.tcnt[i] = s.cnt[i];
            s.tw[i] = static_cast<u64>(s.whi[i]) << 32 | s.wlo[i];
        }
        __syncthreads();
        return;
    }
    sync_cluster();
    // each CTA adds its share of the bins over the cluster and hands it to all
    const int share_n = kBins / static_cast<int>(row.size);
    for (int i = threadIdx.x; i < share_n; i += kThreads) {
        const int bin = static_cast<int>(row.rank) * share_n + i;
        uint32_t c = 0;
        u64 w = 0;
        for (uint32_t p = 0; p < row.size; ++p) {
            c += remote_ld32(dsmem_map(&s.cnt[bin], p));
            w += static_cast<u64>(remote_ld32(dsmem_map(&s.whi[bin], p))) << 32;
            w += remote_ld32(dsmem_map(&s.wlo[bin], p));
        }
        for (uint32_t p = 0; p < row.size; ++p) {
            asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(dsmem_map(&s.tcnt[bin], p)), "r"(c) : "memory");
            remote_st(dsmem_map(&s.tw[bin], p), w);
        }
    }
    sync_cluster();
}

struct Cut {
    uint32_t key;      // kept: keys above, and the first `ties` equal to it
    u64 ties;
    u64 w;             // weight of what is kept
    bool some;         // equals of the key are left out
};

// The shortest prefix of the row's order, among keys in [lo, hi], that holds
// `target` tokens or (by_weight) reaches `target` weight. Where the whole range
// does not, all of it. target >= 1.
__device__ Cut prefix(const Row &row, uint32_t lo, uint32_t hi, bool by_weight, u64 target, Shared &s) {
    u64 above_c = 0, above_w = 0;
    const uint32_t floor_key = lo;
    while (true) {
        const uint32_t range = hi - lo;
        const int bits = 32 - __clz(range), shift = bits > 10 ? bits - 10 : 0;
        histogram(row, lo, hi, shift, s);
        // thread t looks at bins 2 t and 2 t + 1
        const int b0 = 2 * threadIdx.x;
        u64 c = static_cast<u64>(s.tcnt[b0]) + s.tcnt[b0 + 1], w = s.tw[b0] + s.tw[b0 + 1], tc, tw;
        scan2(c, w, tc, tw, s);
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
        if (!s.found) return Cut{floor_key, ~0ull, above_w + tw, false};
        const uint32_t bin = s.bin, n = s.tcnt[bin];
        above_c = s.above_cnt;
        above_w = s.above_w;
        const u64 bw = s.tw[bin];
        hi = hi - (bin << shift);
        lo = (shift == 0) ? hi : (hi - lo >= (1u << shift) - 1u ? hi - ((1u << shift) - 1u) : lo);
        if (n <= kList) break;
        if (lo == hi) {
            // n equal logits
            const u64 one = bw / n;
            const u64 m = by_weight ? (target - above_w + one - 1) / one : target - above_c;
            __syncthreads();
            return Cut{lo, m, above_w + m * one, m < n};
        }
        __syncthreads();
    }
    // ---- rank the bin's tokens in the first CTA
    if (threadIdx.x == 0) {
        s.n_list = 0u;
        s.last_rank = 0u;
    }
    if (row.size > 1) sync_cluster();
    else __syncthreads();
    const uint32_t n_at = dsmem_map(&s.n_list, 0u), list_at = dsmem_map(s.list, 0u);
    for (int i = threadIdx.x; i < row.n; i += kThreads) {
        const uint32_t k = logit_key(row.l[i]);
        if (k >= lo && k <= hi) {
            const uint32_t at = remote_add(n_at, 1u);
            if (at < kList)
                remote_st(list_at + 8u * at, static_cast<u64>(k) << 32 | (0xffffffffu - static_cast<uint32_t>(row.base + i)));
        }
    }
    if (row.size > 1) sync_cluster();
    else __syncthreads();
    if (row.rank == 0) {
        const int n = static_cast<int>(min(s.n_list, static_cast<uint32_t>(kList)));
        bool kept = false;
        u64 before_w = above_w, same = 0, left = 0, mine = 0;
        uint32_t rank = 0;
        if (static_cast<int>(threadIdx.x) < n) {
            mine = s.list[threadIdx.x];
            s.list_w[threadIdx.x] = fixed_weight(row.weight(float_from_order_key(static_cast<uint32_t>(mine >> 32))));
        }
        __syncthreads();
        if (static_cast<int>(threadIdx.x) < n) {
            for (int j = 0; j < n; ++j) {
                const u64 x = s.list[j];
                if (x > mine) {
                    ++rank;
                    before_w += s.list_w[j];
                    same += (x >> 32) == (mine >> 32);
                } else if (x < mine) {
                    left += (x >> 32) == (mine >> 32);
                }
            }
            kept = by_weight ? before_w < target : above_c + rank < target;
            if (kept) atomicMax(&s.last_rank, rank);
        }
        __syncthreads();
        if (kept && rank == s.last_rank) {
            const uint32_t k = static_cast<uint32_t>(mine >> 32);
            s.res[0] = k;
            s.res[1] = same + 1;
            s.res[2] = before_w + s.list_w[threadIdx.x];
            s.res[3] = left;
        }
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

template <bool kHeld>
__global__ void __launch_bounds__(kThreads) k_sample(SampleArgs a, int slice) {
    extern __shared__ float held[];
    __shared__ Shared s;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int size = static_cast<int>(gridDim.x);   // one cluster along x
    Row row;
    row.rank = size > 1 ? cluster_rank() : 0u;
    row.size = static_cast<uint32_t>(size);
    const int b = blockIdx.y;
    row.base = static_cast<int>(row.rank) * slice;
    row.n = max(0, min(slice, a.V - row.base));
    const float *src = a.logits + b * a.stride + row.base;
    row.l = kHeld ? held : src;

    // ---- the largest logit, the lowest index among equals; a NaN above all
    u64 best = 0;
#pragma unroll 8
    for (int i = tid; i < row.n; i += kThreads) {
        const float v = src[i];
        if (kHeld) held[i] = v;
        const u64 k = v != v ? ~0ull : argmax_pack(v + 0.0f, row.base + i);
        best = k > best ? k : best;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const u64 k = __shfl_xor_sync(0xffffffffu, best, o);
        best = k > best ? k : best;
    }
    if (lane == 0) s.red[warp] = best;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) best = s.red[w] > best ? s.red[w] : best;
    if (size > 1) {
        share(row, s.peer, best);
        for (int p = 0; p < size; ++p) best = s.peer[p] > best ? s.peer[p] : best;
    }
    row.top = float_from_order_key(static_cast<uint32_t>(best >> 32));
    const float T = a.temperature ? a.temperature[b] : 1.0f;
    const bool greedy = T <= 0.0f;
    const bool bad = best == ~0ull || row.top == -INFINITY || !(T < INFINITY) || (!greedy && row.top == INFINITY);
    if (bad || greedy) {
        if (row.rank == 0 && tid == 0) {
            if (bad) record_status(a.status, QW3_ERR_NONFINITE);
            const int arg = bad ? -1 : static_cast<int>(0xffffffffu - static_cast<uint32_t>(best));
            a.token[b] = arg;
            if (a.next) a.next[b] = max(arg, 0);
            if (a.prob) a.prob[b] = bad ? 0.0f : 1.0f;
        }
        return;
    }
    row.inv_t = 1.0f / fmaxf(T, 1e-30f);
    const int k = a.top_k ? a.top_k[b] : 0;
    const float p = a.top_p ? a.top_p[b] : 1.0f, mp = a.min_p ? fminf(a.min_p[b], 1.0f) : 0.0f;
    // below: weights that round to zero (exp(-29) < 2^-41)
    const uint32_t hi = logit_key(row.top), lo = logit_key(row.top - 29.0f * fmaxf(T, 1e-30f));
    Cut cut{lo, ~0ull, 0, false};
    if (k > 0 && k < a.V) cut = prefix(row, lo, hi, false, static_cast<u64>(k), s);
    if (p < 1.0f) {
        u64 total = cut.w;
        if (total == 0) {
            // no top-k: the whole row's weight
            u64 w = 0, none = 0, t0, t1;
            for (int i = tid; i < row.n; i += kThreads) w += fixed_weight(row.weight(row.l[i]));
            scan2(w, none, t0, t1, s);
            total = t0;
            if (size > 1) {
                share(row, s.peer2, t0);
                total = 0;
                for (int q = 0; q < size; ++q) total += s.peer2[q];
            }
        }
        const u64 target = static_cast<u64>(ceil(static_cast<double>(fmaxf(p, 0.0f)) * static_cast<double>(total)));
        const Cut c = prefix(row, cut.key, hi, true, target > 0 ? (target < total ? target : total) : 1ull, s);
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
    auto weight = [&](int i, u64 &seen) -> u64 {
        const float v = row.l[i];
        const uint32_t key = logit_key(v);
        if (key < cut.key || (key == cut.key && cut.some && seen++ >= cut.ties)) return 0ull;
        const float e = row.weight(v);
        return e >= mp ? fixed_weight(e) : 0ull;
    };
    u64 w = 0, seen = n0, none = 0, t0, t1;
    for (int i = i0; i < i1; ++i) w += weight(i, seen);
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
    u64 at = static_cast<u64>(static_cast<double>(u > 0.0f ? u : 0.0f) * static_cast<double>(total));
    if (at >= total) at = total - 1;
    w += before;
    if (w <= at && at < w + mine) {
        seen = n0;
        for (int i = i0; i < i1; ++i) {
            w += weight(i, seen);
            if (w > at) {
                a.token[b] = row.base + i;
                if (a.next) a.next[b] = row.base + i;
                if (a.prob)
                    a.prob[b] = static_cast<float>(exp((static_cast<double>(row.l[i]) - row.top) / fmaxf(T, 1e-30f)) *
                                                   static_cast<double>(kOne) / static_cast<double>(total));
                break;
            }
        }
    }
}

// CTAs per row and the tokens of one: a small vocabulary stays in one CTA, a
// large one is cut into slices of which two fit an SM (up to 20480 tokens, 80
// KB); beyond 8 slices of what one SM holds the row is read again from memory
// (L2) at every pass.
constexpr int kOneCta = 8192, kSlice = 20480, kMaxHeld = 45056;

}  // namespace

cudaError_t configure_sample() {
    return cudaFuncSetAttribute(k_sample<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxHeld * 4);
}

cudaError_t launch_sample(const SampleArgs &a, int B, cudaStream_t s) {
    if (B <= 0) return cudaSuccess;
    int size = 1;
    if (a.V > kOneCta)
        while (size < kMaxCluster && (a.V + size - 1) / size > kSlice) size *= 2;
    const int slice = (a.V + size - 1) / size;
    const bool is_held = slice <= kMaxHeld;
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
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(size, std::min(65535, B - b0));
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = is_held ? static_cast<size_t>(slice) * 4 : 0;
        cfg.stream = s;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = static_cast<unsigned>(size);
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        const cudaError_t e = is_held ? cudaLaunchKernelEx(&cfg, k_sample<true>, x, slice)
                                      : cudaLaunchKernelEx(&cfg, k_sample<false>, x, slice);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace qw3
