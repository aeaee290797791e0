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

// A lane holds 16 bytes of a head: V values, L = HD / V lanes to a head, 32 / L
// heads to a warp at once. The rotation's pair (i, i + hd/2) lies L / 2 lanes
// away.
template <typename T>
struct PgVec {
    static constexpr int V = 16 / sizeof(T);
};

__device__ __forceinline__ void pg_ld(float (&v)[4], const float *p) {
    const float4 t = *reinterpret_cast<const float4 *>(p);
    v[0] = t.x; v[1] = t.y; v[2] = t.z; v[3] = t.w;
}
__device__ __forceinline__ void pg_ld(float (&v)[8], const __half *p) {
    const uint4 t = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}
template <int N>
__device__ __forceinline__ void pg_st_half(__half *p, const float (&v)[N]) {
    uint32_t w[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    if constexpr (N == 8) *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void pg_st(float *p, const float (&v)[4]) {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void pg_st(__half *p, const float (&v)[8]) { pg_st_half(p, v); }

template <int L>
__device__ __forceinline__ float pg_sum(float v) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// 1 / sqrt(mean x^2 + eps) of the lane's head in f64, as a factor that takes x
// in two steps (each a power-of-two-free f32 product could leave f32): x * a * b.
template <int L, int V>
__device__ __noinline__ void pg_norm_f64(const float (&x)[V], float eps, float (&y)[V]) {
    double ss = 0.0;
#pragma unroll
    for (int e = 0; e < V; ++e) ss += static_cast<double>(x[e]) * x[e];
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const double r = 1.0 / sqrt(ss / (L * V) + static_cast<double>(eps));
#pragma unroll
    for (int e = 0; e < V; ++e) y[e] = static_cast<float>(x[e] * r);
}

// One warp takes NP passes (of 32 / L heads) of one row; the passes' loads are
// issued together.
template <typename T, int HD, int NP>
__global__ void __launch_bounds__(128) k_paged_append(const KvPagedAppendArgs a, int passes, int per_row, long long units) {
    constexpr int V = PgVec<T>::V, L = HD / V, H = 32 / L;
    const int lane = threadIdx.x & 31;
    const long long unit = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    pdl_wait();
    if (unit < units) {
        const int row = static_cast<int>(unit / per_row), pass0 = static_cast<int>(unit % per_row) * NP;
        const int i = kv_seq_of(a.b, row, lane);
        if (i >= 0) {
            const int nkv = a.c.nkv, heads = a.nh + 2 * nkv, at = lane % L * V;
            const T *src = static_cast<const T *>(a.qkv) + row * a.qkv_stride;
            float x[NP][V];
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                const int h = (pass0 + k) * H + lane / L;
#pragma unroll
                for (int e = 0; e < V; ++e) x[k][e] = 0.0f;
                if (h < heads) pg_ld(x[k], src + static_cast<size_t>(h) * HD + at);
            }
            // its position: row t of n rows (kv_seq's n may be cut, this one is not)
            const int s0 = min(max(a.b.starts[i], 0), a.b.M), s1 = min(max(a.b.starts[i + 1], 0), a.b.M);
            const int p = row < s1 ? a.b.lens[i] - (s1 - row) : -1;
            const int page = p >= 0 && p < a.rope_len ? kv_page(a.b, a.c, i, p) : -1;
            const bool mine = row >= s0 && row < s1;
            float2 cs[V];
            if (page >= 0) {
                const float4 *r = reinterpret_cast<const float4 *>(a.rope + static_cast<size_t>(p) * (HD / 2) + at % (HD / 2));
#pragma unroll
                for (int e = 0; e < V / 2; ++e) {
                    const float4 t = r[e];
                    cs[2 * e] = make_float2(t.x, t.y);
                    cs[2 * e + 1] = make_float2(t.z, t.w);
                }
            } else {
#pragma unroll
                for (int e = 0; e < V; ++e) cs[e] = make_float2(0.0f, 0.0f);
            }
            const bool first = lane % L < L / 2;   // the lane holds the pairs' first halves
            bool bad = false;
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                const int h = (pass0 + k) * H + lane / L;
                const bool turned = h < a.nh + nkv;
                const float *w = h < a.nh ? a.q_norm : turned ? a.k_norm : nullptr;
                float y[V];
#pragma unroll
                for (int e = 0; e < V; ++e) y[e] = x[k][e];
                float ss = 0.0f;
#pragma unroll
                for (int e = 0; e < V; ++e) ss = fmaf(y[e], y[e], ss);
                const float mean = pg_sum<L>(ss) * (1.0f / HD) + a.eps;
                // where the squares, or their sum, leave f32 the head is normalised in f64
                if (__any_sync(0xffffffffu, w && !(mean > 0x1p-100f && mean < 0x1p120f))) {
                    float z[V];
                    pg_norm_f64<L, V>(y, a.eps, z);
                    if (w) {
#pragma unroll
                        for (int e = 0; e < V; ++e) y[e] = z[e] * w[at + e];
                    }
                } else if (w) {
                    const float r = rsqrtf(mean), r1 = r * fmaf(-0.5f * mean * r, r, 1.5f);   // one Newton step: within a rounding
#pragma unroll
                    for (int e = 0; e < V; ++e) y[e] = y[e] * r1 * w[at + e];
                }
                float z[V];
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float o = __shfl_xor_sync(0xffffffffu, y[e], L / 2);
                    z[e] = !turned ? y[e] : first ? y[e] * cs[e].x - o * cs[e].y : y[e] * cs[e].x + o * cs[e].y;
                }
                // a head of K or V that f16 does not hold
                bool over = false;
#pragma unroll
                for (int e = 0; e < V; ++e) over |= !(fabsf(z[e]) < 65520.0f);
                const unsigned whole = L == 32 ? 0xffffffffu : ((1u << (L & 31)) - 1) << (lane / L * L);
                over = (__ballot_sync(0xffffffffu, over) & whole) != 0;
                if (!mine || h >= heads) continue;
                if (h < a.nh) {
                    if (page < 0) {
#pragma unroll
                        for (int e = 0; e < V; ++e) z[e] = 0.0f;
                    }
                    pg_st(static_cast<T *>(a.q_out) + row * a.q_stride + static_cast<size_t>(h) * HD + at, z);
                } else if (page >= 0) {
                    if (over) {
                        bad = true;
#pragma unroll
                        for (int e = 0; e < V; ++e) z[e] = 0.0f;
                    }
                    const int g = h - a.nh;
                    pg_st_half(kv_paged_row<HD>(a.c, page, g >= nkv, g >= nkv ? g - nkv : g, p) + at, z);
                }
            }
            if (bad) record_status(a.status, QW3_ERR_NONFINITE);
        }
    }
    pdl_trigger();
}

template <typename T, int HD>
cudaError_t append_t(const KvPagedAppendArgs &a, bool pdl, cudaStream_t s) {
    constexpr int V = PgVec<T>::V, H = 32 / (HD / V);
    const int passes = (a.nh + 2 * a.c.nkv + H - 1) / H;
    // few rows: a warp to a pass; many: four passes' loads in flight to a warp
    const bool few = static_cast<long long>(a.b.M) * passes <= 152 * 32;
    const int np = few ? 1 : 4, per_row = (passes + np - 1) / np;
    const long long units = static_cast<long long>(a.b.M) * per_row;
    const dim3 grid(static_cast<unsigned>((units + 3) / 4));
    return few ? launch_pdl(pdl, k_paged_append<T, HD, 1>, grid, 128, 0, 1, s, a, passes, per_row, units)
               : launch_pdl(pdl, k_paged_append<T, HD, 4>, grid, 128, 0, 1, s, a, passes, per_row, units);
}

// ---------------------------------------------------------------- attention

// One warp to a (row, query head): an online softmax over the row's positions.
template <typename T, int HD>
__global__ void __launch_bounds__(128) k_paged_attn(const KvPagedAttnArgs a) {
    constexpr int E = HD / 32;
    const int lane = threadIdx.x & 31;
    const long long unit = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    pdl_wait();
    if (unit >= static_cast<long long>(a.b.M) * a.nh) return;
    const int row = static_cast<int>(unit / a.nh), h = static_cast<int>(unit % a.nh), g = h / (a.nh / a.c.nkv);
    const int i = kv_seq_of(a.b, row, lane);
    if (i < 0) return;
    const KvSeq q = kv_seq(a.b, i);
    if (row < q.start || row >= q.start + q.n) return;
    const int p = q.p0 + row - q.start;
    const T *src = static_cast<const T *>(a.q) + row * a.q_stride + static_cast<size_t>(h) * HD + lane * E;
    float x[E], o[E], m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        x[e] = kv_f32(src[e]);
        o[e] = 0.0f;
    }
    for (int j = 0; j <= p; ++j) {
        if (!kv_sees(p, j, a.window, a.sinks)) continue;
        const int page = kv_page(a.b, a.c, i, j);
        if (page < 0) continue;
        const __half *k = kv_paged_row<HD>(a.c, page, 0, g, j) + lane * E, *v = kv_paged_row<HD>(a.c, page, 1, g, j) + lane * E;
        float d = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) d = fmaf(x[e], kv_f32(k[e]), d);
        d = warp_sum(d) * a.scale;
        const float mn = d > m ? d : m, c = m == -INFINITY ? 0.0f : expf(m - mn), w = expf(d - mn);
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(w, kv_f32(v[e]), o[e] * c);
        l = fmaf(l, c, w);
        m = mn;
    }
    T *dst = static_cast<T *>(a.out) + row * a.out_stride + static_cast<size_t>(h) * HD + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) dst[e] = kv_cvt<T>(l == 0.0f ? 0.0f : o[e] / l);
    pdl_trigger();
}

}  // namespace

cudaError_t configure_kv_paged() { return cudaSuccess; }

cudaError_t launch_kv_paged_append(const KvPagedAppendArgs &a, int type, int hd, bool pdl, cudaStream_t s) {
    if (type == QW3_F32) return hd == 128 ? append_t<float, 128>(a, pdl, s) : append_t<float, 64>(a, pdl, s);
    return hd == 128 ? append_t<__half, 128>(a, pdl, s) : append_t<__half, 64>(a, pdl, s);
}

size_t kv_paged_attn_workspace_bytes(int, int, int, int, int, int, int, int, int, int) { return 0; }

cudaError_t launch_kv_paged_attn(const KvPagedAttnArgs &a, int type, int hd, bool pdl, cudaStream_t s) {
    const long long units = static_cast<long long>(a.b.M) * a.nh;
    const dim3 grid(static_cast<unsigned>((units + 3) / 4));
    if (type == QW3_F32)
        return hd == 128 ? launch_pdl(pdl, k_paged_attn<float, 128>, grid, 128, 0, 1, s, a)
                         : launch_pdl(pdl, k_paged_attn<float, 64>, grid, 128, 0, 1, s, a);
    return hd == 128 ? launch_pdl(pdl, k_paged_attn<__half, 128>, grid, 128, 0, 1, s, a)
                     : launch_pdl(pdl, k_paged_attn<__half, 64>, grid, 128, 0, 1, s, a);
}

}  // namespace qw3
