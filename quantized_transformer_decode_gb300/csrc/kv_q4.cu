// The 4-bit KV cache: rows written (with the per-head Q/K RMSNorm and the
// rotation in the same pass), read back, and attended over.
//
// Layout, in bytes: [slot][K|V][kv head]{codes [capacity][hd / 2], scales
// [capacity][hd / 32] f16}. A row of hd values is nb = hd / 32 blocks of 32
// values; value i of a block is scale * (code_i - 8). A block's codes, taken
// in order with the even value in the low nibble, are 16 bytes; a K row
// interleaves the blocks' 4-byte words ([word][block]), a V row their 2-byte
// halfwords ([halfword][block]), so that a thread of the attention kernel
// finds the codes it multiplies next to each other. Codes and scales lie in
// planes of their own: every code row starts 16-byte aligned (32 bytes at
// hd 64), and 32 positions are whole sectors of both planes.
//
// Encoder: P = max x, N = max -x over the block, m = P if P >= N else -N,
// d = -m / 8, code = clamp(floor(x / d + 8.5), 0, 15) (8 where m = 0), scale
// = f16(d), with x and d taken without rounding. 4.5 bits per value.
#include <algorithm>

#include "qw3_internal.cuh"

namespace qw3 {

namespace {

// ---------------------------------------------------------------- rows in, rows out

// A lane holds values [lane * E, lane * E + E) of a row (E = HD / 32): L = 32 /
// E lanes hold one block.
template <int HD>
struct Q4Row {
    static constexpr int E = HD / 32, L = 32 / E, NB = HD / 32;
};

// Code bytes of a lane's values inside the row: 2 bytes at hd 128, 1 at 64.
template <int HD>
__device__ __forceinline__ int q4_lane_byte(int lane, bool v_row) {
    constexpr int E = Q4Row<HD>::E, L = Q4Row<HD>::L, NB = Q4Row<HD>::NB;
    const int b = lane / L, j = (lane % L) * E / 2;   // block, byte of the block
    return v_row ? 2 * ((j >> 1) * NB + b) + (j & 1) : 4 * ((j >> 2) * NB + b) + (j & 3);
}

__device__ __forceinline__ double shfl_xor_f64(double v, int o) { return __shfl_xor_sync(0xffffffffu, v, o); }

// The row in f64 from its inputs: normalised and rotated (K; w and cs given)
// or as it is (V), then encoded. Called by a whole warp for the few rows whose
// f32 values leave a code or a scale undecided.
template <int HD>
__device__ __noinline__ void q4_encode_f64(const float *raw, const float *w, const float2 *cs, float eps, int lane,
                                           int *code, __half *scale) {
    constexpr int E = Q4Row<HD>::E, L = Q4Row<HD>::L;
    double x[E];
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = raw[e];
    if (w) {
        double ss = 0.0;
#pragma unroll
        for (int e = 0; e < E; ++e) ss += x[e] * x[e];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += shfl_xor_f64(ss, o);
        const double r = 1.0 / sqrt(ss / HD + static_cast<double>(eps));
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = x[e] * r * w[e];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const double o = shfl_xor_f64(x[e], 16);
            const double c = cs[e].x, s = cs[e].y;
            x[e] = lane < 16 ? x[e] * c - o * s : x[e] * c + o * s;
        }
    }
    double P = x[0], N = -x[0];
#pragma unroll
    for (int e = 1; e < E; ++e) {
        P = fmax(P, x[e]);
        N = fmax(N, -x[e]);
    }
#pragma unroll
    for (int o = 1; o < L; o <<= 1) {
        P = fmax(P, shfl_xor_f64(P, o));
        N = fmax(N, shfl_xor_f64(N, o));
    }
    const double m = P >= N ? P : -N;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const double f = floor(-8.0 * x[e] / m + 8.5);
        code[e] = m == 0.0 ? 8 : static_cast<int>(fmin(fmax(f, 0.0), 15.0));
    }
    *scale = m == 0.0 ? __float2half_rn(0.0f) : __double2half(-m / 8.0);
}

// Encode a warp's row x, each value within err of the exact one (0 for a row
// taken as it is). f32 decides every code and scale that lies further from a
// border than err can carry it; where one does not, the whole row goes through
// f64 (about one K row in thirty, hardly ever a V row), so the codes are those
// of the exact values whatever the order of the f32 sums. Returns false for a
// lane whose block holds a value that is not finite or too large for an f16
// scale: it is written as zeros.
template <int HD>
__device__ __forceinline__ bool q4_encode(const float (&x)[HD / 32], float err, const float (&raw)[HD / 32],
                                          const float *w, const float2 *cs, float eps, int lane,
                                          int (&code)[HD / 32], __half &scale) {
    constexpr int E = Q4Row<HD>::E, L = Q4Row<HD>::L;
    float P = x[0], N = -x[0];
    bool bad = false;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        P = fmaxf(P, x[e]);
        N = fmaxf(N, -x[e]);
        bad |= !(fabsf(x[e]) < 524160.0f);   // 8 * 65520, where the scale rounds to infinity
    }
#pragma unroll
    for (int o = 1; o < L; o <<= 1) {
        P = fmaxf(P, __shfl_xor_sync(0xffffffffu, P, o));
        N = fmaxf(N, __shfl_xor_sync(0xffffffffu, N, o));
    }
    const unsigned badmask = __ballot_sync(0xffffffffu, bad);
    const unsigned block = (L == 32 ? 0xffffffffu : ((1u << L) - 1u)) << (lane / L * L);
    const bool fine = (badmask & block) == 0u;
    const float m = P >= N ? P : -N, am = fabsf(m);
    bool near = false;
    if (fine && am > 0.0f) {
        // under 1e-30 the quotient leaves f32's range
        near = am < 1e-30f || (err > 0.0f && fabsf(P - N) <= 2.0f * err);
        const float inv = -8.0f / m, tol = fmaf(16.0f * err, fabsf(inv) * 0.125f, 4e-6f);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float f = fmaf(x[e], inv, 8.5f);
            near |= fabsf(f - rintf(f)) <= tol;
            code[e] = static_cast<int>(fminf(fmaxf(floorf(f), 0.0f), 15.0f));
        }
        const float d = am * 0.125f, de = err * 0.126f;
        scale = __float2half_rn(-m * 0.125f);
        if (err > 0.0f)
            near |= __half_as_ushort(__float2half_rn(d - de)) != __half_as_ushort(__float2half_rn(d + de));
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e) code[e] = 8;
        scale = __float2half_rn(0.0f);
        // an exact value may be tiny where its f32 value is zero
        near = fine && err > 0.0f;
    }
    if (__any_sync(0xffffffffu, near)) {
        int c64[E];
        __half s64;
        q4_encode_f64<HD>(raw, w, cs, eps, lane, c64, &s64);
        if (fine) {
#pragma unroll
            for (int e = 0; e < E; ++e) code[e] = c64[e];
            scale = s64;
        }
    }
    return fine;
}

struct Q4AppendArgs {
    const float *qkv;   // [M][qkv_stride]: nh query heads, nkv key heads, nkv value heads
    int M;
    int64_t qkv_stride;
    const float *q_norm, *k_norm;
    float eps;
    const float2 *rope;   // [capacity][hd / 2]
    KvQ4 c;
    KvQ4Rows rows;
    int nh;
    float *q_out;   // [M][q_stride]; may be qkv itself
    int64_t q_stride;
    int32_t *status;
};

// One warp per (row, head).
template <int HD>
__global__ void __launch_bounds__(128) k_kv_q4_append(Q4AppendArgs a) {
    constexpr int E = Q4Row<HD>::E, L = Q4Row<HD>::L, NB = Q4Row<HD>::NB;
    const int lane = threadIdx.x & 31;
    const int task = blockIdx.y * 4 + (threadIdx.x >> 5), row = blockIdx.x;
    const int nkv = a.c.nkv;
    if (task >= a.nh + 2 * nkv) return;
    int slot, pos;
    if (!kv_q4_row(a.c, a.rows, row, slot, pos)) return;
    const float *src = a.qkv + row * a.qkv_stride + static_cast<int64_t>(task) * HD;
    float raw[E], v[E], w[E];
    float2 cs[E];
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = raw[e] = src[lane * E + e];
    const bool normed = task < a.nh + nkv;
    float err = 0.0f;
    if (normed) {
        const float *wp = task < a.nh ? a.q_norm : a.k_norm;
        const float2 *rr = a.rope + static_cast<size_t>(pos) * (HD / 2) + (lane & 15) * E;
        float ss = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            w[e] = wp[lane * E + e];
            cs[e] = rr[e];
            ss = fmaf(v[e], v[e], ss);
        }
        ss = warp_sum(ss);
        const float r = 1.0f / sqrtf(ss / static_cast<float>(HD) + a.eps);
        float top = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            v[e] = v[e] * r * w[e];
            top = fmaxf(top, fabsf(v[e]));
        }
        // every rotated value is within 20 f32 roundings of the row's largest
        // normalised one: 9 of the sum of squares and its root, 3 products, a
        // sum, times sqrt 2
        err = 20.0f * 5.97e-8f * warp_max(top);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float o = __shfl_xor_sync(0xffffffffu, v[e], 16);
            v[e] = lane < 16 ? v[e] * cs[e].x - o * cs[e].y : o * cs[e].y + v[e] * cs[e].x;
        }
    }
    if (task < a.nh) {
        float *dst = a.q_out + row * a.q_stride + static_cast<int64_t>(task) * HD;
#pragma unroll
        for (int e = 0; e < E; ++e) dst[lane * E + e] = v[e];
        return;
    }
    const int sel = task < a.nh + nkv ? 0 : 1, g = task - a.nh - sel * nkv;
    int code[E];
    __half scale;
    const bool fine = q4_encode<HD>(v, err, raw, normed ? w : nullptr, cs, a.eps, lane, code, scale);
    if (!fine) record_status(a.status, QW3_ERR_NONFINITE);
    uint8_t *codes = kv_q4_codes<HD>(a.c, slot, sel, g) + static_cast<size_t>(pos) * (HD / 2) + q4_lane_byte<HD>(lane, sel);
    if constexpr (E == 4) {
        *reinterpret_cast<uint16_t *>(codes) =
            static_cast<uint16_t>(code[0] | (code[1] << 4) | (code[2] << 8) | (code[3] << 12));
    } else {
        *codes = static_cast<uint8_t>(code[0] | (code[1] << 4));
    }
    if (lane % L == 0) kv_q4_scales<HD>(a.c, slot, sel, g)[static_cast<size_t>(pos) * NB + lane / L] = scale;
}

// Four values of one (row, head) of K and of V per thread.
template <int HD>
__global__ void __launch_bounds__(256) k_kv_q4_read(KvQ4 c, KvQ4Rows rows, int M, float *__restrict__ k_out,
                                                    float *__restrict__ v_out) {
    constexpr int NB = HD / 32, Q = HD / 4;
    const int64_t total = static_cast<int64_t>(M) * c.nkv * Q;
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
        const int j = static_cast<int>(i % Q);
        const int64_t rg = i / Q;
        const int g = static_cast<int>(rg % c.nkv), row = static_cast<int>(rg / c.nkv);
        int slot, pos;
        if (!kv_q4_row(c, rows, row, slot, pos)) continue;
        const int b = j / 8, q = j % 8;   // block, quadruple of the block
#pragma unroll
        for (int sel = 0; sel < 2; ++sel) {
            const int at = sel ? 2 * (q * NB + b) : 4 * ((q >> 1) * NB + b) + 2 * (q & 1);
            const unsigned w = *reinterpret_cast<const uint16_t *>(kv_q4_codes<HD>(c, slot, sel, g) +
                                                                   static_cast<size_t>(pos) * (HD / 2) + at);
            const float s = __half2float(kv_q4_scales<HD>(c, slot, sel, g)[static_cast<size_t>(pos) * NB + b]);
            float4 y;
            y.x = s * static_cast<float>(static_cast<int>(w & 15u) - 8);
            y.y = s * static_cast<float>(static_cast<int>((w >> 4) & 15u) - 8);
            y.z = s * static_cast<float>(static_cast<int>((w >> 8) & 15u) - 8);
            y.w = s * static_cast<float>(static_cast<int>(w >> 12) - 8);
            float *out = (sel ? v_out : k_out) + rg * HD + 4 * j;
            out[0] = y.x; out[1] = y.y; out[2] = y.z; out[3] = y.w;
        }
    }
}

// ---------------------------------------------------------------- attention

// Value d of row pos.
template <int HD>
__device__ __forceinline__ float q4_value(const uint8_t *codes, const __half *scales, int pos, int d, int sel) {
    constexpr int NB = HD / 32;
    const int b = d / 32, j = d % 32 / 2;
    const int at = sel ? 2 * ((j >> 1) * NB + b) + (j & 1) : 4 * ((j >> 2) * NB + b) + (j & 3);
    const int byte = codes[static_cast<size_t>(pos) * (HD / 2) + at];
    const int code = (d & 1) ? byte >> 4 : byte & 15;
    return __half2float(scales[static_cast<size_t>(pos) * NB + b]) * static_cast<float>(code - 8);
}

// One CTA per (query row, head): each warp takes every eighth position.
template <int HD>
__global__ void __launch_bounds__(256) k_kv_q4_attn(KvQ4AttnArgs a) {
    constexpr int E = HD / 32;
    __shared__ float sm[8][HD + 2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int h = blockIdx.x, r = blockIdx.y, b = r / a.rows, t = r % a.rows;
    const int slot = a.slots ? a.slots[b] : b;
    const int len = (slot < 0 || slot >= a.c.slots) ? 0 : min(max(a.lens[b], 0), a.max_len);
    const int n = len - a.rows + t + 1;
    const int g = h / (a.nh / a.c.nkv);
    float q[E], acc[E], m = -INFINITY, l = 0.0f;
    const float *qp = a.q + r * a.q_stride + static_cast<int64_t>(h) * HD;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        q[e] = qp[lane * E + e] * a.scale;
        acc[e] = 0.0f;
    }
    if (n > 0) {
        const uint8_t *kc = kv_q4_codes<HD>(a.c, slot, 0, g), *vc = kv_q4_codes<HD>(a.c, slot, 1, g);
        const __half *ks = kv_q4_scales<HD>(a.c, slot, 0, g), *vs = kv_q4_scales<HD>(a.c, slot, 1, g);
        for (int j = warp; j < n; j += 8) {
            float s = 0.0f;
#pragma unroll
            for (int e = 0; e < E; ++e) s = fmaf(q[e], q4_value<HD>(kc, ks, j, lane * E + e, 0), s);
            s = warp_sum(s);
            const float mn = fmaxf(m, s), f = expf(m - mn), p = expf(s - mn);
            m = mn;
            l = fmaf(l, f, p);
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = fmaf(acc[e], f, p * q4_value<HD>(vc, vs, j, lane * E + e, 1));
        }
    }
#pragma unroll
    for (int e = 0; e < E; ++e) sm[warp][lane * E + e] = acc[e];
    if (lane == 0) {
        sm[warp][HD] = m;
        sm[warp][HD + 1] = l;
    }
    __syncthreads();
    for (int d = threadIdx.x; d < HD; d += 256) {
        float M = -INFINITY, Ls = 0.0f, o = 0.0f;
        for (int w = 0; w < 8; ++w) M = fmaxf(M, sm[w][HD]);
        if (M != -INFINITY)
            for (int w = 0; w < 8; ++w) {
                const float f = expf(sm[w][HD] - M);
                Ls = fmaf(sm[w][HD + 1], f, Ls);
                o = fmaf(sm[w][d], f, o);
            }
        a.out[r * a.out_stride + static_cast<int64_t>(h) * HD + d] = Ls > 0.0f ? o / Ls : 0.0f;
    }
}

}  // namespace

cudaError_t launch_kv_q4_append(const float *qkv, int M, int64_t qkv_stride, const float *q_norm, const float *k_norm,
                                float eps, const float2 *rope, const KvQ4 &c, int hd, const KvQ4Rows &rows, int nh,
                                float *q_out, int64_t q_stride, int32_t *status, cudaStream_t s) {
    if (M <= 0) return cudaSuccess;
    const Q4AppendArgs a{qkv, M, qkv_stride, q_norm, k_norm, eps, rope, c, rows, nh, q_out, q_stride, status};
    const dim3 grid(M, (nh + 2 * c.nkv + 3) / 4);
    if (hd == 128) k_kv_q4_append<128><<<grid, 128, 0, s>>>(a);
    else if (hd == 64) k_kv_q4_append<64><<<grid, 128, 0, s>>>(a);
    else return cudaErrorInvalidValue;
    return cudaGetLastError();
}

cudaError_t launch_kv_q4_read(const KvQ4 &c, int hd, const KvQ4Rows &rows, int M, float *k_out, float *v_out,
                              cudaStream_t s) {
    if (M <= 0) return cudaSuccess;
    const int64_t total = static_cast<int64_t>(M) * c.nkv * (hd / 4);
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>((total + 255) / 256, 152 * 16));
    if (hd == 128) k_kv_q4_read<128><<<grid, 256, 0, s>>>(c, rows, M, k_out, v_out);
    else if (hd == 64) k_kv_q4_read<64><<<grid, 256, 0, s>>>(c, rows, M, k_out, v_out);
    else return cudaErrorInvalidValue;
    return cudaGetLastError();
}

size_t kv_q4_attn_workspace_bytes(int, int, int, int, int, int) { return 0; }

cudaError_t launch_kv_q4_attn(const KvQ4AttnArgs &a, int hd, cudaStream_t s) {
    if (a.B <= 0) return cudaSuccess;
    const dim3 grid(a.nh, a.B * a.rows);
    if (hd == 128) k_kv_q4_attn<128><<<grid, 256, 0, s>>>(a);
    else if (hd == 64) k_kv_q4_attn<64><<<grid, 256, 0, s>>>(a);
    else return cudaErrorInvalidValue;
    return cudaGetLastError();
}

}  // namespace qw3
