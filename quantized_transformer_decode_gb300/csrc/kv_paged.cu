// The paged KV cache: rows of a ragged batch appended (with the per-head Q/K
// RMSNorm and the rotation in the same pass) and attended over.
//
// Layout: f16 [page][K|V][kv head][page_size][hd], page_size a power of two
// from 16 to 256: what one head reads of a page is one contiguous run of whole
// 128-byte lines, and 16 positions never straddle two pages.
#include <algorithm>
#include <cstdint>

#include "qw3_internal.cuh"

namespace qw3 {

namespace {

// ---------------------------------------------------------------- append

// A lane holds V values (16 bytes) of a head's first half and the V of its second
// half that the rotation pairs them with: L = HD / 2 / V lanes to a head, 32 / L
// heads to a warp at once, and no value has to change lanes.
template <typename T>
struct PgVec {
    static constexpr int V = 16 / sizeof(T);
};

// 16 bytes as f32 values, and back.
template <typename T>
__device__ __forceinline__ void pg_cvt(float *v, uint4 t) {
    const uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) {
            v[i] = __uint_as_float(w[i]);
        } else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
}
template <int N>
__device__ __forceinline__ void pg_st_half(__half *p, const float *v) {
    uint32_t w[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    if constexpr (N == 8) *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void pg_st(float *p, const float *v) { *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]); }
__device__ __forceinline__ void pg_st(__half *p, const float *v) { pg_st_half<8>(p, v); }

template <int L>
__device__ __forceinline__ float pg_sum(float v) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// x / sqrt(mean x^2 + eps) of the lane's head in f64.
template <int L, int N>
__device__ __noinline__ void pg_norm_f64(const float (&x)[N], float eps, float (&y)[N]) {
    double ss = 0.0;
#pragma unroll
    for (int e = 0; e < N; ++e) ss += static_cast<double>(x[e]) * x[e];
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const double r = 1.0 / sqrt(ss / (L * N) + static_cast<double>(eps));
#pragma unroll
    for (int e = 0; e < N; ++e) y[e] = static_cast<float>(x[e] * r);
}

// Bound by reads that wait for the ones before them: 4096 rows of 32/8 heads (186
// MB) take 41 us, 0.68 of the copy rate; one row of 16/8 heads 2.5 us.
//
// Warp w of a row's per_row takes passes w, w + per_row, .. (of 32 / L heads), NP at
// most, whose loads are all issued before the row's place is looked up.
template <typename T, int HD, int NP>
__global__ void __launch_bounds__(128) k_paged_append(const KvPagedAppendArgs a, int per_row, long long units) {
    constexpr int V = PgVec<T>::V, L = HD / 2 / V, H = 32 / L;
    const int lane = threadIdx.x & 31;
    const long long unit = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    __shared__ __align__(16) float s_w[2][HD];   // the norms' weights (4-byte loads for every head were what bounded this)
    pdl_trigger();
    pdl_wait();
    for (int e = threadIdx.x; e < HD; e += 128) {
        s_w[0][e] = a.q_norm ? a.q_norm[e] : 1.0f;
        s_w[1][e] = a.k_norm ? a.k_norm[e] : 1.0f;
    }
    __syncthreads();
    if (unit >= units) return;
    const int row = static_cast<int>(unit / per_row), pass0 = static_cast<int>(unit % per_row);
    const int nkv = a.c.nkv, heads = a.nh + 2 * nkv, at = lane % L * V;
    const T *src = static_cast<const T *>(a.qkv) + row * a.qkv_stride + at;
    uint4 raw[NP][2];
#pragma unroll
    for (int k = 0; k < NP; ++k) {
        const int h = (pass0 + k * per_row) * H + lane / L;
        raw[k][0] = raw[k][1] = make_uint4(0, 0, 0, 0);
        if (h < heads) {
            raw[k][0] = __ldcs(reinterpret_cast<const uint4 *>(src + static_cast<size_t>(h) * HD));
            raw[k][1] = __ldcs(reinterpret_cast<const uint4 *>(src + static_cast<size_t>(h) * HD + HD / 2));
        }
    }
    const int i = kv_seq_of(a.b, row, lane);
    if (i < 0) return;
    // its position: row t of n rows (kv_seq's n may be cut, this one is not)
    const int s0 = min(max(a.b.starts[i], 0), a.b.M), s1 = min(max(a.b.starts[i + 1], 0), a.b.M);
    if (row < s0 || row >= s1) return;
    const int p = a.b.lens[i] - (s1 - row);
    const int page = p >= 0 && p < a.rope_len ? kv_page(a.b, a.c, i, p) : -1;
    float2 cs[V];
#pragma unroll
    for (int e = 0; e < V; ++e) cs[e] = make_float2(0.0f, 0.0f);
    if (page >= 0) {
        const float4 *r = reinterpret_cast<const float4 *>(a.rope + static_cast<size_t>(p) * (HD / 2) + at);
#pragma unroll
        for (int e = 0; e < V / 2; ++e) {
            const float4 t = r[e];
            cs[2 * e] = make_float2(t.x, t.y);
            cs[2 * e + 1] = make_float2(t.z, t.w);
        }
    }
    bool bad = false;
#pragma unroll
    for (int k = 0; k < NP; ++k) {
        const int h = (pass0 + k * per_row) * H + lane / L;
        if ((pass0 + k * per_row) * H >= heads) break;
        float y[2 * V];   // the first half's values, then the second's
        pg_cvt<T>(y, raw[k][0]);
        pg_cvt<T>(y + V, raw[k][1]);
        const bool turned = h < a.nh + nkv;
        const bool w = h < a.nh ? a.q_norm != nullptr : turned && a.k_norm;
        if (__any_sync(0xffffffffu, w)) {
            float ss = 0.0f;
#pragma unroll
            for (int e = 0; e < 2 * V; ++e) ss = fmaf(y[e], y[e], ss);
            const float mean = pg_sum<L>(ss) * (1.0f / HD) + a.eps;
            float wv[2 * V];
            const float *sw = s_w[h < a.nh ? 0 : 1] + at;
#pragma unroll
            for (int e = 0; e < 2 * V; e += 4) {
                const float4 t = *reinterpret_cast<const float4 *>(sw + (e < V ? e : HD / 2 - V + e));
                wv[e] = t.x; wv[e + 1] = t.y; wv[e + 2] = t.z; wv[e + 3] = t.w;
            }
            // where the squares, or their sum, leave f32 the head is normalised in f64
            if (__any_sync(0xffffffffu, w && !(mean > 0x1p-100f && mean < 0x1p120f))) {
                float z[2 * V];
                pg_norm_f64<L, 2 * V>(y, a.eps, z);
                if (w) {
#pragma unroll
                    for (int e = 0; e < 2 * V; ++e) y[e] = z[e] * wv[e];
                }
            } else if (w) {
                const float r = rsqrtf(mean), r1 = r * fmaf(-0.5f * mean * r, r, 1.5f);   // one Newton step: within a rounding
#pragma unroll
                for (int e = 0; e < 2 * V; ++e) y[e] = y[e] * r1 * wv[e];
            }
        }
        if (turned) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float u = y[e], v = y[V + e];
                y[e] = u * cs[e].x - v * cs[e].y;
                y[V + e] = v * cs[e].x + u * cs[e].y;
            }
        }
        // a head of K or V that f16 does not hold
        bool over = false;
#pragma unroll
        for (int e = 0; e < 2 * V; ++e) over |= !(fabsf(y[e]) < 65520.0f);
        const unsigned head = (1u << (L & 31)) - 1;
        over = (__ballot_sync(0xffffffffu, over) & head << (lane / L * L)) != 0;
        if (h < a.nh) {
            if (page < 0) {
#pragma unroll
                for (int e = 0; e < 2 * V; ++e) y[e] = 0.0f;
            }
            T *to = static_cast<T *>(a.q_out) + row * a.q_stride + static_cast<size_t>(h) * HD + at;
            pg_st(to, y);
            pg_st(to + HD / 2, y + V);
        } else if (h < heads && page >= 0) {
            if (over) {
                bad = true;
#pragma unroll
                for (int e = 0; e < 2 * V; ++e) y[e] = 0.0f;
            }
            const int g = h - a.nh;
            __half *to = kv_paged_row<HD>(a.c, page, g >= nkv, g >= nkv ? g - nkv : g, p) + at;
            pg_st_half<V>(to, y);
            pg_st_half<V>(to + HD / 2, y + V);
        }
        __syncwarp();
    }
    if (bad) record_status(a.status, QW3_ERR_NONFINITE);
}

template <typename T, int HD>
cudaError_t append_t(const KvPagedAppendArgs &a, bool pdl, cudaStream_t s) {
    constexpr int V = PgVec<T>::V, H = 32 / (HD / 2 / V);
    constexpr int NP = 2;   // 4096 rows of 32/8 heads, f32: 46 us with 1, 42 with 2, 47 with 4 (floor 28)
    const int passes = (a.nh + 2 * a.c.nkv + H - 1) / H;
    // few rows: a warp to a pass
    const bool few = static_cast<long long>(a.b.M) * passes <= 152 * 32;
    const int per_row = few ? passes : (passes + NP - 1) / NP;
    const long long units = static_cast<long long>(a.b.M) * per_row;
    const dim3 grid(static_cast<unsigned>((units + 3) / 4));
    return few ? launch_pdl(pdl, k_paged_append<T, HD, 1>, grid, 128, 0, 1, s, a, per_row, units)
               : launch_pdl(pdl, k_paged_append<T, HD, NP>, grid, 128, 0, 1, s, a, per_row, units);
}

// ---------------------------------------------------------------- attention of few rows
//
// Decoding, and verify blocks of a few rows: bound by the K and V that have to
// be read. The rows of a sequence that share a kv head are columns j = t * G + h
// (G query heads to a kv head); a unit is up to W columns of one kv head of one
// sequence, a step 16 positions of it (they lie in one page). The steps of all
// units are dealt to the CTAs in equal shares, so ragged lengths fill the GPU
// evenly; a unit cut between CTAs leaves parts (maximum, sum, output) in the
// workspace that a second kernel joins.
//
// A warp takes every eighth step of its CTA's share, through a ring of its own
// in shared memory that cp.async fills three steps ahead, over the units' ends
// too. Scores S = Q K^T and outputs O = P V are mma.sync.m16n8k16: 16 rows of A
// are 8 columns in two f16 parts (f32 activations; hi + lo, 22 bits) or 16
// columns (f16), K is B as it lies (8 positions x 16 dimensions, the dimensions
// in an order that gives a thread 16 contiguous bytes), and so is V after
// setting pairs of positions side by side (one byte permutation to a register).
// f16 activations: a weight is rounded to f16, once, as the product with V asks
// (2^-11 of it at most beside the output's own rounding; sums are of the weights
// before it).
// tcgen05.mma has no part here: a tile of 128 rows would be filled by 2 to 16,
// and reading K and V is what takes the time, not the products.
//
// Bound by HBM: 64 sequences of 1 to 4101, 16/8 heads of 128, f32 (537 MB) take 98
// us, 0.81 of the copy rate; one of 32768, 32/8 heads, f16 (134 MB) 34 us with its
// join, 0.58. Short ones by the latency of a warp's steps: 517 positions 9.9 us.

constexpr int kTokWarps = 8, kTokStages = 3, kTokKeys = 16;
// What a unit's ends cost, in steps (loading its queries, joining the warps),
// where there are more units than CTAs: 64 sequences of 1 to 4101 take 135 us
// with 0, 112 with 10, 98 with 24, 99 with 40. Fewer units: a CTA has two at
// most, and shares may be short.
constexpr int kTokUnit = 24;
// Few short units: a CTA to each, and nothing to join. (One token of one sequence,
// 16/8 heads: 517 positions 9.9 us instead of 12.2, 1000 positions 13.3 instead of 12.5.)
constexpr int kTokWhole = 48;
constexpr int kTokCols = 32;      // columns of a sequence's kv head that these kernels take

template <typename T, int HD>
struct TokSizes {
    static constexpr bool split = sizeof(T) == 4;
    static constexpr int W = split ? 8 : 16;                    // columns of a unit
    static constexpr int part = HD + 4;                         // floats of a column's part: output, maximum, sum
    static constexpr uint32_t half = kTokKeys * HD * 2;         // bytes of a step's K, or V
    static constexpr uint32_t ring = kTokStages * 2 * half;     // of a warp
    static constexpr uint32_t smem = kTokWarps * (ring + 8 * part * 4);
};

// The steps of a sequence's units: its first `sinks` positions, then the
// window's (or all). Rows 0 .. n - 1 are at p0 ..; where no row sees anything
// there is one step, for the zeros.
struct TokSeq {
    int start, n, p0, cols, sink_steps, first, steps;
    __device__ __forceinline__ int key_step(int k) const { return k < sink_steps ? k : k - sink_steps + first; }
};
__device__ __forceinline__ TokSeq tok_seq(const KvPagedAttnArgs &a, int i, int G) {
    const KvSeq q = kv_seq(a.b, i);
    TokSeq s;
    s.start = q.start;
    s.n = q.n;
    s.p0 = q.p0;
    s.cols = q.n * G;
    if (s.cols > kTokCols) s.n = s.cols = 0;   // another kernel's
    const int last = s.p0 + s.n - 1;
    const int lo = a.window > 0 ? max(0, s.p0 - a.window + 1) : 0;
    s.first = lo / kTokKeys;
    s.sink_steps = a.window > 0 ? min((min(a.sinks, lo) + kTokKeys - 1) / kTokKeys, s.first) : 0;
    s.steps = last < 0 ? 1 : s.sink_steps + last / kTokKeys - s.first + 1;
    return s;
}

__device__ __forceinline__ void cp_async16(uint32_t to, const void *from, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float2 unpack_half2(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2 *>(&v)); }
__device__ __forceinline__ bool half2_nonfinite(uint32_t v) {
    return (v & 0x7c00u) == 0x7c00u || (v & 0x7c000000u) == 0x7c000000u;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The shares are of work: a unit's is `ends` (kTokUnit or 0) and then its steps; or
// (ends < 0) one, and a CTA has one unit.
// Where a CTA (or a warp's loads, ahead of it) is: unit `u` of sequence i, its
// steps k .. end - 1 among them, and `left` of the share behind those.
struct TokAt {
    TokSeq s;
    int i, u, units, k, end;
    long long left;
};
// The units of sequence i, for all kv heads.
template <int W>
__device__ __forceinline__ int tok_units(const TokSeq &s, int nkv) { return (s.cols + W - 1) / W * nkv; }

// The next unit of which the share has a step; i = -1 behind the last one.
template <int W>
__device__ __forceinline__ void tok_next(TokAt &t, const KvPagedAttnArgs &a, int G, int ends) {
    while (t.left > 0) {
        if (++t.u >= t.units) {
            t.u = -1;
            if (++t.i >= a.b.B) break;
            t.s = tok_seq(a, t.i, G);
            t.units = tok_units<W>(t.s, a.c.nkv);
            continue;
        }
        t.left -= ends;
        if (t.left <= 0) break;   // (its steps begin in the next share)
        t.k = 0;
        t.end = static_cast<int>(min(static_cast<long long>(t.s.steps), t.left));
        t.left -= t.end;
        return;
    }
    t.left = 0;
    t.i = -1;
}

// The CTAs that a unit is cut between: the first and the last, with bit 31 of
// `last` where it begins in the first one's own first piece; first = -1 for a
// unit that one CTA has whole.
struct TokCut {
    int first;
    uint32_t last;
};

template <typename T, int HD>
__global__ void __launch_bounds__(kTokWarps * 32, 1) k_paged_tokens(const KvPagedAttnArgs a, int G, int max_cb, int ends, int min_share, int beside) {
    using Z = TokSizes<T, HD>;
    constexpr int W = Z::W, KS = HD / 16, NT = HD / 8, CH = HD / 8;
    constexpr float kOff = 12.0f, kLazy = 3.0f;   // a weight is 2^(s - ref + 12), at most 2^15
    extern __shared__ __align__(128) uint8_t tok_smem[];
    __shared__ long long s_sum[kTokWarps];
    __shared__ int s_i, s_off_u, s_off_k;
    __shared__ float s_m[kTokWarps][8], s_l[kTokWarps][8];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, gid = lane >> 2, tig = lane & 3;
    const int nkv = a.c.nkv;
    // beside: the kernel before this one works on other sequences and has waited for what came before itself; this one
    // runs beside it, and ends after it
    pdl_trigger();
    if (!beside) pdl_wait();

    // ---- the share of this CTA: x0 .. x1 - 1 of all the work
    const int per = (a.b.B + kTokWarps * 32 - 1) / (kTokWarps * 32);
    const int i0 = min(a.b.B, tid * per), i1 = min(a.b.B, i0 + per);
    long long mine = 0;
    for (int i = i0; i < i1; ++i) {
        const TokSeq s = tok_seq(a, i, G);
        mine += static_cast<long long>(tok_units<W>(s, nkv)) * (ends < 0 ? 1 : ends + s.steps);
    }
    long long upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
    }
    if (lane == 31) s_sum[warp] = upto;
    __syncthreads();
    long long total = 0, before = upto - mine;
    for (int w = 0; w < kTokWarps; ++w) {
        if (w < warp) before += s_sum[w];
        total += s_sum[w];
    }
    const long long share = max((total + gridDim.x - 1) / gridDim.x, static_cast<long long>(min_share));
    const long long x0 = share * blockIdx.x, x1 = min(total, x0 + share);
    if (x0 >= before && x0 < before + mine) {
        long long at = before;
        for (int i = i0; i < i1; ++i) {
            const TokSeq s = tok_seq(a, i, G);
            const int unit = ends < 0 ? 1 : ends + s.steps;
            const long long n = static_cast<long long>(tok_units<W>(s, nkv)) * unit;
            if (x0 < at + n) {
                s_i = i;
                s_off_u = static_cast<int>((x0 - at) / unit);
                s_off_k = ends < 0 ? 0 : static_cast<int>((x0 - at) % unit) - ends;
                break;
            }
            at += n;
        }
    }
    __syncthreads();
    if (x0 >= total) {
        if (beside) pdl_wait();
        return;
    }

    TokAt t;   // what the CTA computes
    t.i = s_i;
    t.s = tok_seq(a, t.i, G);
    t.units = tok_units<W>(t.s, nkv);
    t.u = s_off_u;
    t.k = max(0, s_off_k);
    long long x = x0 + max(0, -s_off_k);   // where this piece's steps begin
    if (x >= x1) {                         // (only at the end of all the work: min_share > ends)
        if (beside) pdl_wait();
        return;
    }
    t.end = ends < 0 ? t.s.steps : static_cast<int>(min(static_cast<long long>(t.s.steps), t.k + (x1 - x)));
    t.left = ends < 0 ? 0 : x1 - x - (t.end - t.k);

    // ---- this warp's loads: the next step to fetch, its page known one step ahead
    const uint32_t ring = smem_u32(tok_smem) + warp * Z::ring;
    TokAt f = t;
    int fk = f.k + warp, fpage = -1;
    uint32_t paged = 0;   // bit per stage: its step has a page
    auto settle = [&]() {   // fk to a step of the share, if there is one
        while (f.i >= 0 && fk >= f.end) {
            tok_next<W>(f, a, G, ends);
            fk = f.k + warp;
        }
        fpage = f.i >= 0 ? kv_page(a.b, a.c, f.i, f.s.key_step(fk) * kTokKeys) : -1;
    };
    auto fetch = [&](int stage) {
        if (f.i >= 0) {
            const int j0 = f.s.key_step(fk) * kTokKeys, g = f.u / ((f.s.cols + W - 1) / W);
            const bool there = fpage >= 0;
            paged = (paged & ~(1u << stage)) | static_cast<uint32_t>(there) << stage;
            const uint8_t *k = reinterpret_cast<const uint8_t *>(kv_paged_row<HD>(a.c, there ? fpage : 0, 0, g, j0));
            const uint8_t *v = reinterpret_cast<const uint8_t *>(kv_paged_row<HD>(a.c, there ? fpage : 0, 1, g, j0));
            const uint32_t to = ring + stage * 2 * Z::half;
#pragma unroll
            for (int n = 0; n < kTokKeys * CH / 32; ++n) {
                const int c = n * 32 + lane, r = c / CH, ch = c % CH;
                cp_async16(to + (r * CH + (ch ^ ((r & 1) << 2))) * 16, k + c * 16, there);
                cp_async16(to + Z::half + (r * CH + (ch ^ ((r >> 1 & 3) << 1))) * 16, v + c * 16, there);
            }
            fk += kTokWarps;
            settle();
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    settle();
#pragma unroll
    for (int n = 0; n < kTokStages; ++n) fetch(n);
    int stage = 0;

    const float scale2 = a.scale * 1.4426950408889634f;   // softmax in base 2
    float *slots = static_cast<float *>(a.ws);
    TokCut *cuts = reinterpret_cast<TokCut *>(slots + static_cast<size_t>(gridDim.x) * 2 * W * Z::part);
    for (int piece = 0; t.i >= 0; ++piece) {
        const int blocks = (t.s.cols + W - 1) / W, g = t.u / blocks, cb = t.u % blocks, col0 = cb * W;
        const int pmin = t.s.p0 + col0 / G, pmax = t.s.p0 + (min(t.s.cols, col0 + W) - 1) / G;
        // ---- the queries as A, and this thread's columns: gid (and gid + 8)
        uint32_t qf[KS][4];
        float cscale[2];
        int p[2];
#pragma unroll
        for (int e = 0; e < (Z::split ? 1 : 2); ++e) {
            const int col = col0 + gid + 8 * e;
            const bool real = col < t.s.cols;
            p[e] = real ? t.s.p0 + col / G : pmax;   // (a column that is none sees what the last one sees)
            const T *src = static_cast<const T *>(a.q) + (t.s.start + (real ? col / G : 0)) * a.q_stride +
                           static_cast<size_t>(g * G + (real ? col % G : 0)) * HD + 8 * tig;
            if constexpr (Z::split) {
                float v[HD / 32][8], amax = 0.0f;
#pragma unroll
                for (int c = 0; c < HD / 32; ++c) {
                    const float4 u0 = *reinterpret_cast<const float4 *>(src + 32 * c), u1 = *reinterpret_cast<const float4 *>(src + 32 * c + 4);
                    v[c][0] = u0.x; v[c][1] = u0.y; v[c][2] = u0.z; v[c][3] = u0.w;
                    v[c][4] = u1.x; v[c][5] = u1.y; v[c][6] = u1.z; v[c][7] = u1.w;
#pragma unroll
                    for (int d = 0; d < 8; ++d) amax = fmaxf(amax, fabsf(v[c][d]));
                }
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                // the power of two that takes the largest into [2^14, 2^15)
                const int ex = min(126, 14 + 127 - static_cast<int>(__float_as_uint(amax) >> 23 & 0xffu));
                const float up = pow2_f32(ex);
                cscale[0] = pow2_f32(-ex) * scale2;
#pragma unroll
                for (int c = 0; c < HD / 32; ++c) {
                    float w[8];
#pragma unroll
                    for (int d = 0; d < 8; ++d) w[d] = real ? v[c][d] * up : 0.0f;
                    uint4 hi, lo;
                    split8_f16(w, hi, lo);
                    qf[2 * c][0] = hi.x; qf[2 * c][1] = lo.x; qf[2 * c][2] = hi.y; qf[2 * c][3] = lo.y;
                    qf[2 * c + 1][0] = hi.z; qf[2 * c + 1][1] = lo.z; qf[2 * c + 1][2] = hi.w; qf[2 * c + 1][3] = lo.w;
                }
            } else {
                cscale[e] = scale2;
#pragma unroll
                for (int c = 0; c < HD / 32; ++c) {
                    const uint4 u = real ? *reinterpret_cast<const uint4 *>(src + 32 * c) : make_uint4(0, 0, 0, 0);
                    qf[2 * c][e] = u.x; qf[2 * c][2 + e] = u.y;
                    qf[2 * c + 1][e] = u.z; qf[2 * c + 1][2 + e] = u.w;
                }
            }
        }

        float acc[NT][4], ref[2] = {-INFINITY, -INFINITY}, sum[2] = {0.0f, 0.0f};
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[n][e] = 0.0f;

        for (int k = t.k + warp; k < t.end; k += kTokWarps) {
            const int j0 = t.s.key_step(k) * kTokKeys;
            const bool held = paged >> stage & 1;
            asm volatile("cp.async.wait_group %0;" ::"n"(kTokStages - 1) : "memory");
            __syncwarp();
            const uint32_t at = ring + stage * 2 * Z::half;
            // ---- scores of 2 x 8 positions
            float s[2][4];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                s[b][0] = s[b][1] = s[b][2] = s[b][3] = 0.0f;
#pragma unroll
                for (int c = 0; c < HD / 32; ++c) {
                    const int r = 8 * b + gid, ch = 4 * c + tig;
                    const uint4 u = lds128(at + (r * CH + (ch ^ ((r & 1) << 2))) * 16);
                    mma16816(s[b], qf[2 * c], u.x, u.y);
                    mma16816(s[b], qf[2 * c + 1], u.z, u.w);
                }
            }
            // every column sees all 16 positions?
            const bool open = held && j0 + kTokKeys - 1 <= pmin && (a.window == 0 || pmax - j0 < a.window || j0 + kTokKeys <= a.sinks);
            // s[b][2 h + e]: column gid + 8 h, position j0 + 8 b + 2 tig + e
            constexpr int NC = Z::split ? 1 : 2;
            float z[NC][4];
#pragma unroll
            for (int h = 0; h < NC; ++h)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float raw = Z::split ? s[e >> 1][e & 1] + s[e >> 1][2 + (e & 1)] : s[e >> 1][2 * h + (e & 1)];
                    z[h][e] = raw * cscale[h];
                    const int j = j0 + 8 * (e >> 1) + 2 * tig + (e & 1);
                    if (!open && !(held && kv_sees(p[h], j, a.window, a.sinks))) z[h][e] = -INFINITY;
                }
            // ---- the reference follows the maximum when it is passed by more than 2^kLazy
            bool far = false;
            float mx[NC];
#pragma unroll
            for (int h = 0; h < NC; ++h) {
                mx[h] = fmaxf(fmaxf(z[h][0], z[h][1]), fmaxf(z[h][2], z[h][3]));
                far |= mx[h] > ref[h] + kLazy;
            }
            if (__any_sync(0xffffffffu, far)) {
#pragma unroll
                for (int h = 0; h < NC; ++h) {
                    float m = mx[h];
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
                    if (m > ref[h] + kLazy) {
                        const float c = ref[h] == -INFINITY ? 0.0f : ex2(ref[h] - m);
                        ref[h] = m;
                        sum[h] *= c;
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            acc[n][2 * h] *= c;
                            acc[n][2 * h + 1] *= c;
                            if constexpr (Z::split) {
                                acc[n][2] *= c;
                                acc[n][3] *= c;
                            }
                        }
                    }
                }
            }
            uint32_t pf[4];
#pragma unroll
            for (int h = 0; h < NC; ++h) {
                const float base = (ref[h] == -INFINITY ? 0.0f : ref[h]) - kOff;
                float w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    w[e] = ex2(z[h][e] - base);
                    sum[h] += w[e];
                }
                if constexpr (Z::split) {
                    pf[0] = pack_half2(w[0], w[1]);
                    pf[2] = pack_half2(w[2], w[3]);
                    const float2 h0 = unpack_half2(pf[0]), h1 = unpack_half2(pf[2]);
                    pf[1] = pack_half2(w[0] - h0.x, w[1] - h0.y);
                    pf[3] = pack_half2(w[2] - h1.x, w[3] - h1.y);
                } else {
                    pf[h] = pack_half2(w[0], w[1]);
                    pf[2 + h] = pack_half2(w[2], w[3]);
                }
            }
            // ---- O += P V
#pragma unroll
            for (int hh = 0; hh < HD / 64; ++hh) {
                uint32_t v[4][4];   // positions 2 tig, + 1, + 8, + 9; dimensions 64 hh + 8 gid ..
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int r = 2 * tig + (e & 1) + 8 * (e >> 1), ch = 8 * hh + gid;
                    const uint4 u = lds128(at + Z::half + (r * CH + (ch ^ ((r >> 1 & 3) << 1))) * 16);
                    v[e][0] = u.x; v[e][1] = u.y; v[e][2] = u.z; v[e][3] = u.w;
                }
                bool slow = false;
                if (!open) {
                    // what no column sees is zeros (its weights are 0, but 0 * NaN is not); what some do not
                    // see has to be finite, or the columns are taken one by one
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int j = j0 + 2 * tig + (e & 1) + 8 * (e >> 1);
                        const bool any = held && j <= pmax && kv_sees(max(j, pmin), j, a.window, a.sinks);
#pragma unroll
                        for (int d = 0; d < 4; ++d) {
                            v[e][d] = any ? v[e][d] : 0u;
                            slow |= half2_nonfinite(v[e][d]);
                        }
                    }
                    slow = __any_sync(0xffffffffu, slow);
                }
                if (!slow) {
#pragma unroll
                    for (int d = 0; d < 8; ++d) {
                        const uint32_t sel = d & 1 ? 0x7632 : 0x5410;
                        mma16816(acc[8 * hh + d], pf, __byte_perm(v[0][d >> 1], v[1][d >> 1], sel),
                                 __byte_perm(v[2][d >> 1], v[3][d >> 1], sel));
                    }
                } else {
#pragma unroll 1
                    for (int c = 0; c < W; ++c) {   // column c alone, with the positions that it sees
                        const int pc = col0 + c < t.s.cols ? t.s.p0 + (col0 + c) / G : pmax;
                        uint32_t pc_f[4];
                        const bool row = gid == (c & 7);
#pragma unroll
                        for (int e = 0; e < 4; ++e) pc_f[e] = row && (Z::split || (e & 1) == c >> 3) ? pf[e] : 0u;
#pragma unroll
                        for (int d = 0; d < 8; ++d) {
                            const uint32_t sel = d & 1 ? 0x7632 : 0x5410;
                            uint32_t u[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                u[e] = kv_sees(pc, j0 + 2 * tig + (e & 1) + 8 * (e >> 1), a.window, a.sinks) ? v[e][d >> 1] : 0u;
                            float o[4] = {acc[8 * hh + d][0], acc[8 * hh + d][1], acc[8 * hh + d][2], acc[8 * hh + d][3]};
                            mma16816(o, pc_f, __byte_perm(u[0], u[1], sel), __byte_perm(u[2], u[3], sel));
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (row && (Z::split || (e >> 1) == c >> 3)) acc[8 * hh + d][e] = o[e];
                        }
                    }
                }
            }
            __syncwarp();
            fetch(stage);
            stage = stage + 1 == kTokStages ? 0 : stage + 1;
        }

        // ---- the warps' parts joined, 8 columns at a time
        const bool whole = t.k == 0 && t.end == t.s.steps;
        float *const dst = slots + (static_cast<size_t>(blockIdx.x) * 2 + (piece > 0)) * W * Z::part;
        if (t.k == 0 && tid == 0 && ends >= 0) {
            // the first of the unit's CTAs says where the others are
            TokCut c{-1, 0u};
            if (!whole) c = {static_cast<int>(blockIdx.x), static_cast<uint32_t>((x + t.s.steps - 1) / share) | (piece == 0 ? 0x80000000u : 0u)};
            cuts[(static_cast<size_t>(t.i) * nkv + g) * max_cb + cb] = c;
        }
        float *const buf = reinterpret_cast<float *>(tok_smem + kTokWarps * Z::ring);
#pragma unroll
        for (int h = 0; h < (Z::split ? 1 : 2); ++h) {
            if (8 * h >= t.s.cols - col0) break;
            float l = sum[h];
            l += __shfl_xor_sync(0xffffffffu, l, 1);
            l += __shfl_xor_sync(0xffffffffu, l, 2);
            if (tig == 0) {
                s_m[warp][gid] = ref[h];
                s_l[warp][gid] = l;
            }
            float *o = buf + (warp * 8 + gid) * Z::part + tig;   // [dimensions in the order of the registers][tig]
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float v = acc[n][Z::split ? e : 2 * h + e];
                    // (an infinite value: the weights' low parts are 0 or of either sign, and would make it NaN)
                    if constexpr (Z::split) v = fabsf(v) == INFINITY ? v : v + acc[n][2 + e];
                    o[(((n >> 3) * 2 + e) * 8 + (n & 7)) * 4] = v;
                }
            __syncthreads();
            const int here = min(8, t.s.cols - col0 - 8 * h);
            for (int n = tid; n < here * HD; n += kTokWarps * 32) {
                const int c = n / HD, d = n % HD;
                const int pos = (((d >> 6) * 2 + (d >> 3 & 1)) * 8 + (d & 7)) * 4 + (d >> 4 & 3);
                float m = -INFINITY;
#pragma unroll
                for (int w = 0; w < kTokWarps; ++w) m = fmaxf(m, s_m[w][c]);
                float lsum = 0.0f, v = 0.0f;
#pragma unroll
                for (int w = 0; w < kTokWarps; ++w) {
                    const float fac = s_m[w][c] == m ? 1.0f : ex2(s_m[w][c] - m);
                    lsum = fmaf(s_l[w][c], fac, lsum);
                    v = fmaf(buf[(w * 8 + c) * Z::part + pos], fac, v);
                }
                const int col = col0 + 8 * h + c;
                if (whole) {
                    T *to = static_cast<T *>(a.out) + (t.s.start + col / G) * a.out_stride + static_cast<size_t>(g * G + col % G) * HD + d;
                    *to = kv_cvt<T>(lsum == 0.0f ? 0.0f : v / lsum);
                } else {
                    float *to = dst + (8 * h + c) * Z::part;
                    to[d] = v;
                    if (d == 0) {
                        to[HD] = m;
                        to[HD + 1] = lsum;
                    }
                }
            }
            __syncthreads();
        }
        x += t.end - t.k + ends;
        tok_next<W>(t, a, G, ends);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (beside) pdl_wait();
}

// One block to `per` columns (all of a unit's, or one) of a unit that was cut: a
// thread to a dimension of a column, or several that share the parts; the parts'
// weights from shared memory.
constexpr int kTokMaxGrid = 256;   // parts that a unit can have
template <typename T, int HD>
__global__ void __launch_bounds__(512) k_paged_tokens_join(const KvPagedAttnArgs a, int G, int max_cb, int grid, int per, int beside) {
    using Z = TokSizes<T, HD>;
    constexpr int W = Z::W;
    __shared__ float s_f[kTokMaxGrid][W], s_sum[W], s_v[512];
    const int cb = blockIdx.x * per / W, c0 = blockIdx.x * per % W, g = blockIdx.y, tid = threadIdx.x;
    pdl_trigger();
    if (!beside) pdl_wait();
    for (int b = blockIdx.z; b < a.b.B; b += gridDim.z) {
        const TokSeq s = tok_seq(a, b, G);
        if (cb * W + c0 >= s.cols) continue;
        const int cols = min(per, s.cols - cb * W - c0);
        const float *slots = static_cast<const float *>(a.ws);
        const TokCut *cuts = reinterpret_cast<const TokCut *>(slots + static_cast<size_t>(grid) * 2 * W * Z::part);
        const TokCut cut = cuts[(static_cast<size_t>(b) * a.c.nkv + g) * max_cb + cb];
        if (cut.first < 0) continue;
        const int n = static_cast<int>(cut.last & 0x7fffffffu) - cut.first + 1;
        auto part = [&](int c) {
            const int slot = c == 0 && !(cut.last & 0x80000000u) ? 1 : 0;
            return slots + ((static_cast<size_t>(cut.first + c) * 2 + slot) * W + c0) * Z::part;
        };
        __syncthreads();
        // a warp to a column: its maximum, each part's factor and the sum
        for (int c = tid >> 5; c < cols; c += 16) {
            const int lane = tid & 31;
            float m = -INFINITY, l = 0.0f;
            for (int k = lane; k < n; k += 32) m = fmaxf(m, part(k)[c * Z::part + HD]);
            m = warp_max(m);
            for (int k = lane; k < n; k += 32) {
                const float mk = part(k)[c * Z::part + HD], f = mk == m ? 1.0f : ex2(mk - m);
                s_f[k][c] = f;
                l = fmaf(part(k)[c * Z::part + HD + 1], f, l);
            }
            l = warp_sum(l);
            if (lane == 0) s_sum[c] = l;
        }
        __syncthreads();
        const int values = cols * HD, shares = max(1, 512 / values);
        for (int i0 = 0; i0 < values; i0 += 512) {
            const int i = i0 + tid % values, share = i0 > 0 || values >= 512 ? 0 : tid / values, at = min(i, values - 1);
            const int c = at / HD, d = at % HD;
            float v = 0.0f;
            if (share < shares) {
#pragma unroll 8
                for (int k = share; k < n; k += shares) v = fmaf(part(k)[c * Z::part + d], s_f[k][c], v);
            }
            if (shares > 1) {
                s_v[tid] = v;
                __syncthreads();
                for (int k = 1; k < shares && share == 0; ++k) v += s_v[k * values + tid];
            }
            if (share == 0 && i < values) {
                const int col = cb * W + c0 + c;
                T *to = static_cast<T *>(a.out) + (s.start + col / G) * a.out_stride + static_cast<size_t>(g * G + col % G) * HD + d;
                *to = kv_cvt<T>(s_sum[c] == 0.0f ? 0.0f : v / s_sum[c]);
            }
        }
    }
    if (beside) pdl_wait();
}

// How the token kernels are launched: the columns that a sequence can have, the
// blocks of them, the CTAs.
struct TokPlan {
    int cols = 0, max_cb = 0, grid = 0, ends = 0, min_share = 0;
    size_t bytes = 0;
};
TokPlan tok_plan(int B, int type, int nh, int nkv, int hd, int max_rows, int max_len, int window, int sinks) {
    TokPlan p;
    const int G = nh / nkv, W = type == QW3_F32 ? 8 : 16;
    p.cols = static_cast<int>(std::min<long long>(static_cast<long long>(max_rows) * G, kTokCols));
    p.max_cb = (p.cols + W - 1) / W;
    long long len = max_len;
    if (window > 0) len = std::min<long long>(len, static_cast<long long>(window) + max_rows + sinks + 3 * kTokKeys);
    const long long units = static_cast<long long>(B) * nkv * p.max_cb;
    const long long most = std::max<long long>(1, (len + kTokKeys - 1) / kTokKeys);   // steps of a unit
    if (units <= num_sms() && most <= kTokWhole) {
        p.ends = -1;
        p.min_share = 1;
        p.grid = static_cast<int>(units);
        return p;
    }
    p.ends = units > num_sms() ? kTokUnit : 0;
    p.min_share = p.ends + kTokWarps;   // a step to a warp: fewer would only be more to join
    const long long work = (p.ends + most) * units;
    p.grid = static_cast<int>(std::max<long long>(1, std::min<long long>(std::min(num_sms(), kTokMaxGrid), (work + p.min_share - 1) / p.min_share)));
    p.bytes = static_cast<size_t>(p.grid) * 2 * W * (hd + 4) * 4 + static_cast<size_t>(B) * nkv * p.max_cb * sizeof(TokCut);
    return p;
}

template <typename T, int HD>
cudaError_t tokens_t(const KvPagedAttnArgs &a, const TokPlan &p, bool join, bool beside, bool pdl, cudaStream_t s) {
    using Z = TokSizes<T, HD>;
    const int G = a.nh / a.c.nkv;
    if (!join)
        return launch_pdl(pdl, k_paged_tokens<T, HD>, dim3(p.grid), kTokWarps * 32, Z::smem, 1, s, a, G, p.max_cb, p.ends, p.min_share,
                          static_cast<int>(beside));
    if (p.grid == 1 || p.ends < 0) return cudaSuccess;
    // few units: a block to a column (1 x 32768, 8 units in 152 parts: 34 us in all where a block to a unit makes it 38)
    const int per = static_cast<long long>(a.b.B) * a.c.nkv * p.max_cb <= 32 ? 1 : Z::W;
    const dim3 grid(per == 1 ? p.cols : p.max_cb, a.c.nkv, std::min(a.b.B, 65535));
    return launch_pdl(pdl, k_paged_tokens_join<T, HD>, grid, 512, 0, 1, s, a, G, p.max_cb, p.grid, per, static_cast<int>(beside));
}
cudaError_t launch_tokens(const KvPagedAttnArgs &a, int type, int hd, const TokPlan &p, bool join, bool beside, bool pdl, cudaStream_t s) {
    if (type == QW3_F32) return hd == 128 ? tokens_t<float, 128>(a, p, join, beside, pdl, s) : tokens_t<float, 64>(a, p, join, beside, pdl, s);
    return hd == 128 ? tokens_t<__half, 128>(a, p, join, beside, pdl, s) : tokens_t<__half, 64>(a, p, join, beside, pdl, s);
}

template <typename T, int HD>
cudaError_t configure_t() {
    return cudaFuncSetAttribute(k_paged_tokens<T, HD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(TokSizes<T, HD>::smem));
}

}  // namespace

cudaError_t configure_kv_paged() {
    cudaError_t e = configure_t<float, 128>();
    if (e == cudaSuccess) e = configure_t<float, 64>();
    if (e == cudaSuccess) e = configure_t<__half, 128>();
    if (e == cudaSuccess) e = configure_t<__half, 64>();
    if (e == cudaSuccess) e = configure_kv_paged_rows();
    return e;
}

cudaError_t launch_kv_paged_append(const KvPagedAppendArgs &a, int type, int hd, bool pdl, cudaStream_t s) {
    if (type == QW3_F32) return hd == 128 ? append_t<float, 128>(a, pdl, s) : append_t<float, 64>(a, pdl, s);
    return hd == 128 ? append_t<__half, 128>(a, pdl, s) : append_t<__half, 64>(a, pdl, s);
}

namespace {

// Which kernels a call needs: sequences of up to kTokCols columns are the token
// kernels', longer ones attn_paged_tc.cu's. One sequence alone goes by max_rows.
struct AttnPlan {
    bool tokens, rows, rows_split;
    TokPlan tok;
    size_t tok_bytes, rows_bytes;
};
AttnPlan attn_plan(int B, int M, int type, int nh, int nkv, int hd, int max_rows, int max_len, int window, int sinks) {
    AttnPlan p{};
    p.rows = static_cast<long long>(max_rows) * (nh / nkv) > kTokCols;
    p.tokens = !p.rows || B > 1;
    if (p.tokens) {
        p.tok = tok_plan(B, type, nh, nkv, hd, max_rows, max_len, window, sinks);
        p.tok_bytes = (p.tok.bytes + 127) / 128 * 128;
    }
    if (p.rows)
        p.rows_bytes = kv_paged_rows_workspace_bytes(B, M, p.tokens ? kTokCols : 0, type, nh, nkv, hd, max_rows, max_len, window, sinks);
    p.rows_split = p.rows_bytes > 0;
    return p;
}

}  // namespace

size_t kv_paged_attn_workspace_bytes(int B, int M, int type, int nh, int nkv, int hd, int max_rows, int max_len,
                                     int window, int sinks) {
    if (B == 0 || M == 0 || max_rows == 0) return 0;
    const AttnPlan p = attn_plan(B, M, type, nh, nkv, hd, max_rows, max_len, window, sinks);
    return p.tok_bytes + p.rows_bytes;
}

cudaError_t launch_kv_paged_attn(const KvPagedAttnArgs &a, int type, int hd, bool pdl, cudaStream_t s) {
    const AttnPlan p = attn_plan(a.b.B, a.b.M, type, a.nh, a.c.nkv, hd, a.b.max_rows, a.b.max_len, a.window, a.sinks);
    // the kernels first, one beside the other where there are both, then what joins their parts
    float *const ws = reinterpret_cast<float *>(static_cast<uint8_t *>(a.ws) + p.tok_bytes);
    for (const bool join : {false, true}) {
        bool before = false;
        if (p.rows) {
            const cudaError_t e = launch_kv_paged_rows(a, type, hd, p.tokens ? kTokCols : 0, ws, join, pdl, s);
            if (e != cudaSuccess) return e;
            before = !join || p.rows_split;
        }
        if (p.tokens) {
            const cudaError_t e = launch_tokens(a, type, hd, p.tok, join, before, pdl, s);
            if (e != cudaSuccess) return e;
        }
    }
    return cudaSuccess;
}

}  // namespace qw3
