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
#include <cstdint>

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
    if (!kv_q4_row(a.c, a.rows, row, slot, pos)) {
        if (task < a.nh) {
            float *dst = a.q_out + row * a.q_stride + static_cast<int64_t>(task) * HD;
            for (int e = 0; e < E; ++e) dst[lane * E + e] = 0.0f;
        }
        return;
    }
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
                                                    float *__restrict__ v_out, size_t out_row, size_t out_head) {
    constexpr int NB = HD / 32, Q = HD / 4;
    const int64_t total = static_cast<int64_t>(M) * c.nkv * Q;
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
        const int j = static_cast<int>(i % Q);
        const int64_t rg = i / Q;
        const int g = static_cast<int>(rg % c.nkv), row = static_cast<int>(rg / c.nkv);
        int slot, pos;
        const bool there = kv_q4_row(c, rows, row, slot, pos);
        const int b = j / 8, q = j % 8;   // block, quadruple of the block
#pragma unroll
        for (int sel = 0; sel < 2; ++sel) {
            const int at = sel ? 2 * (q * NB + b) : 4 * ((q >> 1) * NB + b) + 2 * (q & 1);
            unsigned w = 0x8888u;
            float s = 0.0f;
            if (there) {
                w = *reinterpret_cast<const uint16_t *>(kv_q4_codes<HD>(c, slot, sel, g) +
                                                        static_cast<size_t>(pos) * (HD / 2) + at);
                s = __half2float(kv_q4_scales<HD>(c, slot, sel, g)[static_cast<size_t>(pos) * NB + b]);
            }
            float4 y;
            y.x = s * static_cast<float>(static_cast<int>(w & 15u) - 8);
            y.y = s * static_cast<float>(static_cast<int>((w >> 4) & 15u) - 8);
            y.z = s * static_cast<float>(static_cast<int>((w >> 8) & 15u) - 8);
            y.w = s * static_cast<float>(static_cast<int>(w >> 12) - 8);
            float *out = (sel ? v_out : k_out) + row * out_row + g * out_head + 4 * j;
            out[0] = y.x; out[1] = y.y; out[2] = y.z; out[3] = y.w;
        }
    }
}

// ---------------------------------------------------------------- attention
//
// out = sum_j softmax_j(scale q.K_j) V_j over the 4-bit rows. The columns of
// one kv head (its group's heads times the query rows) share every cached
// byte, so a CTA takes up to 16 columns of one kv head and sequence over a run
// of positions; runs merge in a second small kernel. A warp takes tiles of 32
// positions and multiplies with mma.m16n8k16 (f16 in, f32 out), positions
// along m for S = K Q^T, dimensions along m for O = V^T P^T:
//  - codes are exact in f16 (-8..7): a word of 8 codes becomes 4 half2
//    operands with 9 instructions and no scale. K scales multiply the f32 sums
//    of a 32-value block, V scales the probabilities of their position.
//  - f16 keeps 11 bits, so q and p v_scale go in as two parts, hi + lo (22
//    bits), in columns of their own: of the 8 columns of an operand 4 are hi
//    and 4 lo where that is enough; else hi and lo take an operand each. With
//    2 columns or 1 the spare columns hold P times the scales of other blocks.
//  - q columns are scaled by a power of two (largest value in [2^14, 2^15)),
//    P columns by 2^kf with kf following the largest V scale met so far, so
//    that hi and lo stay clear of f16's subnormals; both undone in f32.
//  - the scores leave the tensor core with positions along rows and enter it
//    again with positions along k: one 8x8 transpose in registers each.
// A chain of products in the tensor core is 2 instructions long; the sums over
// blocks and tiles are f32 with rounding to nearest. mma.sync rather than
// tcgen05: with 8 or 16 columns the product is bound by what the operands
// cost (bytes, then the unpacking), and registers to registers saves writing
// the unpacked codes to shared memory and reading them back.

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

__device__ __forceinline__ float exp2_f32(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// f16 pair, rounded toward zero: low half a, high half b.
__device__ __forceinline__ uint32_t pack_rz(float a, float b) {
    uint32_t r;
    asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}

// Codes less 8 of a word's nibbles as half2: h[p] = (nibble p, nibble p + 4).
// 0x6400 | n is 1024 + n in f16, 0x6400 | n << 4 is 1024 + 16 n.
__device__ __forceinline__ void unpack8(uint32_t w, uint32_t (&h)[4]) {
    const __half2 c1032 = __halves2half2(__ushort_as_half(0x6408), __ushort_as_half(0x6408));
    const __half2 c16 = __halves2half2(__ushort_as_half(0x2C00), __ushort_as_half(0x2C00));     // 1 / 16
    const __half2 c72 = __halves2half2(__ushort_as_half(0xD480), __ushort_as_half(0xD480));     // -72
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t x = i ? w >> 8 : w;
        const uint32_t lo = (x & 0x000F000Fu) | 0x64006400u, hi = (x & 0x00F000F0u) | 0x64006400u;
        const __half2 l = __hsub2(*reinterpret_cast<const __half2 *>(&lo), c1032);
        const __half2 g = __hfma2(*reinterpret_cast<const __half2 *>(&hi), c16, c72);
        h[2 * i] = *reinterpret_cast<const uint32_t *>(&l);
        h[2 * i + 1] = *reinterpret_cast<const uint32_t *>(&g);
    }
}

__device__ __forceinline__ float half_of(uint32_t w, int i) {
    return __half2float(__ushort_as_half(static_cast<unsigned short>(i ? w >> 16 : w)));
}

constexpr int kQ4Warps = 4, kQ4Tile = 32;

// Positions of sequence b, within what the call allows.
__device__ __forceinline__ int q4_len(const KvQ4AttnArgs &a, int b) {
    return min(max(a.lens ? a.lens[b] : 0, -a.len_add) + a.len_add, a.max_len);
}

// Columns that one CTA of width class W takes, and its 8-column operands: W =
// 1, 2, 4 with hi and lo in one operand; 8 and 16 with operands of their own.
__host__ __device__ constexpr int q4_ops(int W) { return W <= 4 ? 1 : W / 4; }

template <int HD>
struct Q4Words {   // words of a thread's share of a row
    static constexpr int K = HD / 32, V = HD / 64, S = HD / 64;
};

template <int N>
__device__ __forceinline__ void ld_words(uint32_t (&d)[N], const void *p) {
    if constexpr (N == 4) {
        const uint4 t = __ldg(static_cast<const uint4 *>(p));
        d[0] = t.x; d[1] = t.y; d[2] = t.z; d[3] = t.w;
    } else if constexpr (N == 2) {
        const uint2 t = __ldg(static_cast<const uint2 *>(p));
        d[0] = t.x; d[1] = t.y;
    } else {
        d[0] = __ldg(static_cast<const uint32_t *>(p));
    }
}

// Partial results of a CTA: per column acc[HD], then log2 of their unit and
// the sum of weights.
template <int HD>
__host__ __device__ constexpr int q4_part() { return HD + 2; }

template <int HD, int W>
__global__ void __launch_bounds__(kQ4Warps * 32, W <= 4 ? 3 : 2) k_kv_q4_attn(KvQ4AttnArgs a, int chunk, int nsplit,
                                                                             int cgroups) {
    constexpr int NB = HD / 32, NT = q4_ops(W), SC = W <= 8 ? 1 : W / 8;
    constexpr int DUP = W <= 4 ? 4 / W : 1;          // blocks that share an operand
    constexpr int NI = (NB + DUP - 1) / DUP;         // P operands per 16 positions
    constexpr int MT = W <= 8 ? 2 : 1;               // 16-position halves held at once
    constexpr int TILE = 16 * MT;
    using Wd = Q4Words<HD>;
    extern __shared__ __align__(16) float q4_smem[];
    // [warp][W][q4_part]: the warps' results; before that the q operands
    uint2 *qfrag = reinterpret_cast<uint2 *>(q4_smem);   // [NB * 2][NT][32]
    __shared__ float s_exp[W];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = lane >> 2, c = lane & 3;
    const int split = blockIdx.x, g = blockIdx.y / cgroups, cg = blockIdx.y % cgroups, b = blockIdx.z;
    const int G = a.nh / a.c.nkv, cols = G * a.rows, col0 = cg * W, ncol = min(W, cols - col0);
    const int slot = a.slots ? a.slots[b] : a.slot0 + b;
    const bool there = slot >= 0 && slot < a.c.slots;
    const int len = there ? q4_len(a, b) : 0;
    // positions that this group's last column sees
    const int seen = len - a.rows + (col0 + ncol - 1) / G + 1;
    const int start = split * chunk, end = min(seen, start + chunk);
    if (start >= end && nsplit > 1) return;   // the merge leaves empty runs out by the same rule

    // ---- q columns: scaled by a power of two, split into hi and lo
    for (int j = warp; j < W; j += kQ4Warps) {
        float amax = 0.0f;
        if (j < ncol) {
            const int cc = col0 + j;
            const float *qp = a.q + (static_cast<int64_t>(b) * a.rows + cc / G) * a.q_stride +
                              static_cast<int64_t>(g * G + cc % G) * HD;
            for (int d = lane; d < HD; d += 32) amax = fmaxf(amax, fabsf(qp[d]));
            amax = warp_max(amax);
        }
        if (lane == 0) s_exp[j] = static_cast<float>(f16_row_exp(amax));
    }
    __syncthreads();
    for (int i = tid; i < NB * 2 * NT * 32; i += kQ4Warps * 32) {
        const int l = i & 31, nt = (i >> 5) % NT, ks = (i >> 5) / NT, blk = ks >> 1, st = ks & 1;
        const int n = l >> 2, cq = l & 3;
        const int j = W <= 4 ? (n & 3) % W : (nt % SC) * 8 + n;
        const bool low = W <= 4 ? n >= 4 : nt >= SC;
        uint32_t o[2] = {0u, 0u};
        if (j < ncol) {
            const int cc = col0 + j;
            const float *qp = a.q + (static_cast<int64_t>(b) * a.rows + cc / G) * a.q_stride +
                              static_cast<int64_t>(g * G + cc % G) * HD + blk * 32 + cq * 8;
            const float f = pow2_f32(static_cast<int>(s_exp[j]));
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float x0 = qp[2 * st + h] * f, x1 = qp[2 * st + h + 4] * f;
                __half2 v = __floats2half2_rn(x0, x1);
                if (low) {
                    const float2 t = __half22float2(v);
                    v = __floats2half2_rn(x0 - t.x, x1 - t.y);
                }
                o[h] = *reinterpret_cast<const uint32_t *>(&v);
            }
        }
        qfrag[i] = make_uint2(o[0], o[1]);
    }
    __syncthreads();
    constexpr bool kQRegs = W <= 8;
    uint32_t qf[kQRegs ? NB * 2 : 1][kQRegs ? NT : 1][2];
    if constexpr (kQRegs) {
#pragma unroll
        for (int ks = 0; ks < NB * 2; ++ks)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const uint2 t = qfrag[(ks * NT + nt) * 32 + lane];
                qf[ks][nt][0] = t.x;
                qf[ks][nt][1] = t.y;
            }
    }
    // this thread's score columns: 2c and 2c + 1 of each set
    float cscale[SC][2];
    int lim[SC][2];
#pragma unroll
    for (int s = 0; s < SC; ++s)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int j = W <= 4 ? (2 * c + e) % 4 % W : 8 * s + 2 * c + e;
            cscale[s][e] = a.scale * 1.4426950408889634f * pow2_f32(-static_cast<int>(s_exp[j]));
            lim[s][e] = j < ncol ? len - a.rows + (col0 + j) / G + 1 : 0;
        }
    int low_lim = len - a.rows + col0 / G + 1;   // positions that every column sees

    const uint8_t *kc = kv_q4_codes<HD>(a.c, there ? slot : 0, 0, g), *vc = kv_q4_codes<HD>(a.c, there ? slot : 0, 1, g);
    const __half *ksc = kv_q4_scales<HD>(a.c, there ? slot : 0, 0, g), *vsc = kv_q4_scales<HD>(a.c, there ? slot : 0, 1, g);

    uint32_t kw[MT][2][Wd::K], kd[MT][2][Wd::S], vw[MT][4][Wd::V], vd[MT][2][Wd::S];
    auto load_k = [&](int k0) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const size_t j = static_cast<size_t>(k0) + 16 * m + 8 * h + r;
                ld_words(kw[m][h], kc + j * (HD / 2) + c * (HD / 8));
                ld_words(kd[m][h], ksc + j * NB);
            }
    };
    auto load_v = [&](int k0) {
#pragma unroll
        for (int m = 0; m < MT; ++m) {
#pragma unroll
            for (int h = 0; h < 4; ++h)
                ld_words(vw[m][h], vc + (static_cast<size_t>(k0) + 16 * m + 2 * c + (h & 1) + 8 * (h >> 1)) * (HD / 2) +
                                       r * (HD / 16));
#pragma unroll
            for (int h = 0; h < 2; ++h) ld_words(vd[m][h], vsc + (static_cast<size_t>(k0) + 16 * m + 8 * h + r) * NB);
        }
    };

    float acc[NB][2][NT][4], mx[SC][2], sum[SC][2];
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][m][n][e] = 0.0f;
#pragma unroll
    for (int s = 0; s < SC; ++s)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            mx[s][e] = -INFINITY;
            sum[s][e] = 0.0f;
        }
    // 2^kf brings P times the largest V scale so far to 2^15 at most; vlim:
    // the largest scale (f16 bits) that the present kf takes
    int kf = 0;
    uint32_t vlim = 0u;
    // hi lanes keep x (cut to f16 below), lo lanes what the cut leaves
    const uint32_t cut = (W <= 4 && c < 2) ? 0u : 0xFFFFE000u;

    int k0 = start + warp * TILE;
    if (k0 < end) {
        load_k(k0);
        load_v(k0);
    }
    for (; k0 < end; k0 += kQ4Warps * TILE) {
        const int kn = k0 + kQ4Warps * TILE;
        // ---- scores
        float s[MT][SC][4];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            float t[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) t[n][e] = 0.0f;
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                uint32_t x0[4], x1[4];
                unpack8(kw[m][0][i], x0);
                unpack8(kw[m][1][i], x1);
                const float d0 = half_of(kd[m][0][i >> 1], i & 1), d1 = half_of(kd[m][1][i >> 1], i & 1);
                const uint32_t a0[4] = {x0[0], x1[0], x0[1], x1[1]}, a1[4] = {x0[2], x1[2], x0[3], x1[3]};
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float u[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    if constexpr (kQRegs) {
                        mma_f16(u, a0, qf[2 * i][n]);
                        mma_f16(u, a1, qf[2 * i + 1][n]);
                    } else {
                        const uint2 q0 = qfrag[(2 * i * NT + n) * 32 + lane], q1 = qfrag[((2 * i + 1) * NT + n) * 32 + lane];
                        const uint32_t b0[2] = {q0.x, q0.y}, b1[2] = {q1.x, q1.y};
                        mma_f16(u, a0, b0);
                        mma_f16(u, a1, b1);
                    }
                    t[n][0] = fmaf(u[0], d0, t[n][0]);
                    t[n][1] = fmaf(u[1], d0, t[n][1]);
                    t[n][2] = fmaf(u[2], d1, t[n][2]);
                    t[n][3] = fmaf(u[3], d1, t[n][3]);
                }
            }
#pragma unroll
            for (int q = 0; q < SC; ++q)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float v = W <= 4 ? t[0][e] + __shfl_xor_sync(0xffffffffu, t[0][e], 2) : t[q][e] + t[q + NT - SC][e];
                    s[m][q][e] = v * cscale[q][e & 1];
                }
        }
        if (kn < end) load_k(kn);
        if (k0 + TILE > low_lim) {
            // the tile that a column's range ends in: what lies past it may be anything
#pragma unroll
            for (int m = 0; m < MT; ++m) {
#pragma unroll
                for (int q = 0; q < SC; ++q)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (k0 + 16 * m + 8 * (e >> 1) + r >= lim[q][e & 1]) s[m][q][e] = -INFINITY;
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (k0 + 16 * m + 8 * h + r >= len)
#pragma unroll
                        for (int w = 0; w < Wd::S; ++w) vd[m][h][w] = 0u;
            }
        }
        // ---- the unit of P: does a V scale pass what kf takes?
        float refit = 1.0f;
        {
            uint32_t big = 0u;
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int w = 0; w < Wd::S; ++w) big = __vmaxu2(big, vd[m][h][w] & 0x7FFF7FFFu);
            const uint32_t top = max(big & 0xFFFFu, big >> 16);
            if (__any_sync(0xffffffffu, top > vlim || vlim == 0u)) {
                const uint32_t t = __reduce_max_sync(0xffffffffu, top);
                // 2^e > the largest scale; two more bits so that a rise is rare
                const int e = t ? static_cast<int>(__float_as_uint(half_of(t, 0)) >> 23) - 126 : -24;
                const int lim2 = min(e + 2, 16), kn2 = 15 - lim2;
                // f16 bits of 2^lim2 (of the largest finite value from 2^16 on)
                vlim = lim2 >= 16 ? 0x7BFFu : __half_as_ushort(__float2half_rn(pow2_f32(lim2)));
                refit = pow2_f32(max(-100, min(100, kn2 - kf)));
                kf = kn2;
            }
        }
        // ---- softmax: running maximum, weights in units of 2^-kf
        float corr[SC][2];
#pragma unroll
        for (int q = 0; q < SC; ++q)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float t = fmaxf(s[0][q][e], s[0][q][e + 2]);
                if constexpr (MT == 2) t = fmaxf(t, fmaxf(s[1][q][e], s[1][q][e + 2]));
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, o));
                const float mn = fmaxf(mx[q][e], t), base = mn == -INFINITY ? 0.0f : mn;
                corr[q][e] = exp2_f32(mx[q][e] - base) * refit;
                mx[q][e] = mn;
                sum[q][e] *= corr[q][e];
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float p = exp2_f32(s[m][q][e + 2 * h] - base) * pow2_f32(kf);
                        s[m][q][e + 2 * h] = p;
                        sum[q][e] += p;
                    }
            }
        // ---- P operands: p times the block's V scale, hi and lo, transposed
        uint32_t pf[NI][MT][NT][2];
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float d0, d1;
                    if constexpr (DUP == 4) {
                        // columns 2c, 2c + 1 take blocks 2 (c & 1), 2 (c & 1) + 1
                        const uint32_t w = Wd::S == 2 ? ((c & 1) ? vd[m][h][Wd::S - 1] : vd[m][h][0]) : ((c & 1) ? 0u : vd[m][h][0]);
                        d0 = half_of(w, 0);
                        d1 = half_of(w, 1);
                    } else if constexpr (DUP == 2) {
                        d0 = d1 = __half2float(__ushort_as_half(static_cast<unsigned short>(vd[m][h][i] >> (16 * (c & 1)))));
                    } else {
                        d0 = d1 = half_of(vd[m][h][i >> 1], i & 1);
                    }
#pragma unroll
                    for (int q = 0; q < SC; ++q) {
                        const float x0 = s[m][q][2 * h] * d0, x1 = s[m][q][2 * h + 1] * d1;
                        const float y0 = x0 - __uint_as_float(__float_as_uint(x0) & cut);
                        const float y1 = x1 - __uint_as_float(__float_as_uint(x1) & cut);
                        if constexpr (W <= 4) {
                            pf[i][m][0][h] = transpose8x8(pack_rz(y0, y1));
                        } else {
                            pf[i][m][q][h] = transpose8x8(pack_rz(x0, x1));
                            pf[i][m][q + SC][h] = transpose8x8(pack_rz(y0, y1));
                        }
                    }
                }
        // ---- O: two positions' halfwords of a block make the pairs along k
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            float u[2][NT][4];
#pragma unroll
            for (int d = 0; d < 2; ++d)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) u[d][n][e] = 0.0f;
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                uint32_t x0[4], x1[4];
                const uint32_t sel = (i & 1) ? 0x7632u : 0x5410u;
                unpack8(__byte_perm(vw[m][0][i >> 1], vw[m][1][i >> 1], sel), x0);
                unpack8(__byte_perm(vw[m][2][i >> 1], vw[m][3][i >> 1], sel), x1);
                const uint32_t a0[4] = {x0[0], x0[1], x1[0], x1[1]}, a1[4] = {x0[2], x0[3], x1[2], x1[3]};
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    mma_f16(u[0][n], a0, pf[i / DUP][m][n]);
                    mma_f16(u[1][n], a1, pf[i / DUP][m][n]);
                }
            }
#pragma unroll
            for (int d = 0; d < 2; ++d)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        acc[i][d][n][e] = fmaf(acc[i][d][n][e], corr[n % SC][e & 1], u[d][n][e]);
        }
        if (kn < end) load_v(kn);
    }

    // ---- the warps' results meet in shared memory
    constexpr int PS = q4_part<HD>();
    __syncthreads();   // the q operands are done with
    float *mine = q4_smem + warp * W * PS;
#pragma unroll
    for (int q = 0; q < SC; ++q)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float t = sum[q][e];
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
            const int n = 2 * c + e, j = W <= 4 ? n : 8 * q + n;
            if (r == 0 && j < W) {
                mine[j * PS + HD] = mx[q][e] - static_cast<float>(kf);
                mine[j * PS + HD + 1] = t;
            }
        }
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int q = 0; q < SC; ++q)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float o[4];   // dimensions 4 r .. 4 r + 3 of the block
#pragma unroll
                for (int d = 0; d < 2; ++d)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        o[2 * d + h] = W <= 4 ? acc[i][d][0][e + 2 * h] + __shfl_xor_sync(0xffffffffu, acc[i][d][0][e + 2 * h], 2)
                                              : acc[i][d][q][e + 2 * h] + acc[i][d][q + NT - SC][e + 2 * h];
                const int n = 2 * c + e, j = W <= 4 ? n % W : 8 * q + n;
                if (W > 4 || (n < 4 && n / W == i % DUP)) {
                    float2 *dst = reinterpret_cast<float2 *>(mine + j * PS + i * 32 + 4 * r);
                    dst[0] = make_float2(o[0], o[1]);
                    dst[1] = make_float2(o[2], o[3]);
                }
            }
    __syncthreads();
    for (int x = tid; x < ncol * HD; x += kQ4Warps * 32) {
        const int j = x / HD, d = x % HD;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kQ4Warps; ++w) M = fmaxf(M, q4_smem[(w * W + j) * PS + HD]);
        float l = 0.0f, o = 0.0f;
        if (M != -INFINITY)
#pragma unroll
            for (int w = 0; w < kQ4Warps; ++w) {
                const float *pw = q4_smem + (w * W + j) * PS;
                const float f = exp2_f32(pw[HD] - M);
                l = fmaf(pw[HD + 1], f, l);
                o = fmaf(pw[d], f, o);
            }
        if (nsplit == 1) {
            const int cc = col0 + j;
            a.out[(static_cast<int64_t>(b) * a.rows + cc / G) * a.out_stride + static_cast<int64_t>(g * G + cc % G) * HD + d] =
                l > 0.0f ? o / l : 0.0f;
        } else {
            float *ws = a.ws + (((static_cast<size_t>(b) * a.c.nkv + g) * cols + col0 + j) * nsplit + split) * PS;
            ws[d] = o;
            if (d == 0) {
                ws[HD] = M;
                ws[HD + 1] = l;
            }
        }
    }
}

// Joins the runs of one column: a warp per (sequence, kv head, column).
template <int HD>
__global__ void __launch_bounds__(128) k_kv_q4_merge(KvQ4AttnArgs a, int chunk, int nsplit, int W) {
    constexpr int E = HD / 32, PS = q4_part<HD>();
    const int lane = threadIdx.x & 31, G = a.nh / a.c.nkv, cols = G * a.rows;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    if (unit >= static_cast<int64_t>(a.B) * a.c.nkv * cols) return;
    const int cc = static_cast<int>(unit % cols), g = static_cast<int>(unit / cols % a.c.nkv);
    const int b = static_cast<int>(unit / cols / a.c.nkv);
    const int slot = a.slots ? a.slots[b] : a.slot0 + b;
    const int len = slot >= 0 && slot < a.c.slots ? q4_len(a, b) : 0;
    const int col0 = cc / W * W, ncol = min(W, cols - col0);
    const int seen = len - a.rows + (col0 + ncol - 1) / G + 1;   // as in the kernel above
    const int runs = seen > 0 ? min(nsplit, (seen + chunk - 1) / chunk) : 0;
    const float *ws = a.ws + static_cast<size_t>(unit) * nsplit * PS;
    float M = -INFINITY;
    for (int i = lane; i < runs; i += 32) M = fmaxf(M, ws[i * PS + HD]);
    M = warp_max(M);
    float l = 0.0f, o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.0f;
    if (M != -INFINITY)
        for (int i = 0; i < runs; ++i) {
            const float f = exp2_f32(ws[i * PS + HD] - M);
            l = fmaf(ws[i * PS + HD + 1], f, l);
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] = fmaf(ws[i * PS + e * 32 + lane], f, o[e]);
        }
    float *out = a.out + (static_cast<int64_t>(b) * a.rows + cc / G) * a.out_stride + static_cast<int64_t>(g * G + cc % G) * HD;
#pragma unroll
    for (int e = 0; e < E; ++e) out[e * 32 + lane] = l > 0.0f ? o[e] / l : 0.0f;
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
                              size_t out_row, size_t out_head, cudaStream_t s) {
    if (M <= 0) return cudaSuccess;
    const int64_t total = static_cast<int64_t>(M) * c.nkv * (hd / 4);
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>((total + 255) / 256, 152 * 16));
    if (hd == 128) k_kv_q4_read<128><<<grid, 256, 0, s>>>(c, rows, M, k_out, v_out, out_row, out_head);
    else if (hd == 64) k_kv_q4_read<64><<<grid, 256, 0, s>>>(c, rows, M, k_out, v_out, out_row, out_head);
    else return cudaErrorInvalidValue;
    return cudaGetLastError();
}

namespace {

// How a call is split: width class of the columns, column groups, and runs of
// `chunk` positions.
struct Q4Plan {
    int W, cgroups, chunk, nsplit;
};

Q4Plan q4_plan(int B, int rows, int nh, int nkv, int max_len) {
    const int cols = nh / nkv * rows;
    Q4Plan p;
    p.W = cols <= 1 ? 1 : cols <= 2 ? 2 : cols <= 4 ? 4 : cols <= 8 ? 8 : 16;
    p.cgroups = (cols + p.W - 1) / p.W;
    const int64_t units = static_cast<int64_t>(B) * nkv * p.cgroups;
    // about four runs for every CTA that fits at once, so that sequences of
    // different lengths even out; no run shorter than one tile per warp
    const int64_t want = (4 * 3 * 152 + units - 1) / std::max<int64_t>(units, 1);
    const int quantum = kQ4Warps * kQ4Tile;
    const int64_t most = std::max<int64_t>(1, (max_len + quantum - 1) / quantum);
    const int64_t n = std::max<int64_t>(1, std::min<int64_t>(want, most));
    p.chunk = static_cast<int>(std::max<int64_t>(1, (max_len + n * quantum - 1) / (n * quantum)) * quantum);
    p.nsplit = std::max(1, (max_len + p.chunk - 1) / p.chunk);
    return p;
}

template <int HD, int W>
cudaError_t launch_q4_attn_w(const KvQ4AttnArgs &a, const Q4Plan &p, cudaStream_t s) {
    constexpr size_t smem = std::max<size_t>(static_cast<size_t>(kQ4Warps) * W * q4_part<HD>() * 4,
                                             static_cast<size_t>(HD / 32) * 2 * q4_ops(W) * 32 * 8);
    static_assert(smem <= 48 * 1024, "fits without an opt-in");
    k_kv_q4_attn<HD, W><<<dim3(p.nsplit, a.c.nkv * p.cgroups, a.B), kQ4Warps * 32, smem, s>>>(a, p.chunk, p.nsplit, p.cgroups);
    return cudaGetLastError();
}

template <int HD>
cudaError_t launch_q4_attn_hd(const KvQ4AttnArgs &a, const Q4Plan &p, cudaStream_t s) {
    cudaError_t e = cudaErrorInvalidValue;
    switch (p.W) {
        case 1: e = launch_q4_attn_w<HD, 1>(a, p, s); break;
        case 2: e = launch_q4_attn_w<HD, 2>(a, p, s); break;
        case 4: e = launch_q4_attn_w<HD, 4>(a, p, s); break;
        case 8: e = launch_q4_attn_w<HD, 8>(a, p, s); break;
        case 16: e = launch_q4_attn_w<HD, 16>(a, p, s); break;
    }
    if (e != cudaSuccess || p.nsplit == 1) return e;
    const int64_t units = static_cast<int64_t>(a.B) * a.nh * a.rows;
    k_kv_q4_merge<HD><<<static_cast<unsigned>((units + 3) / 4), 128, 0, s>>>(a, p.chunk, p.nsplit, p.W);
    return cudaGetLastError();
}

}  // namespace

int kv_q4_attn_launches(int B, int rows, int nh, int nkv, int max_len) {
    return q4_plan(B, rows, nh, nkv, max_len).nsplit > 1 ? 2 : 1;
}

size_t kv_q4_attn_workspace_bytes(int B, int rows, int nh, int nkv, int hd, int max_len) {
    const Q4Plan p = q4_plan(B, rows, nh, nkv, max_len);
    return p.nsplit > 1 ? static_cast<size_t>(B) * nh * rows * p.nsplit * (hd + 2) * 4 : 0;
}

cudaError_t launch_kv_q4_attn(const KvQ4AttnArgs &a, int hd, cudaStream_t s) {
    if (a.B <= 0) return cudaSuccess;
    const Q4Plan p = q4_plan(a.B, a.rows, a.nh, a.c.nkv, a.max_len);
    if (hd == 128) return launch_q4_attn_hd<128>(a, p, s);
    if (hd == 64) return launch_q4_attn_hd<64>(a, p, s);
    return cudaErrorInvalidValue;
}

}  // namespace qw3
