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
#include <type_traits>
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

// Loads and stores of a lane's E values; VEC where everything is aligned for one
// access. CS: what leaves L2 first.
template <int E, bool VEC, bool CS = false>
__device__ __forceinline__ void q4_ld(float (&v)[E], const float *p) {
    if constexpr (VEC && E == 4) {
        const float4 *from = reinterpret_cast<const float4 *>(p);
        const float4 t = CS ? __ldcs(from) : *from;
        v[0] = t.x; v[1] = t.y; v[2] = t.z; v[3] = t.w;
    } else if constexpr (VEC && E == 2) {
        const float2 *from = reinterpret_cast<const float2 *>(p);
        const float2 t = CS ? __ldcs(from) : *from;
        v[0] = t.x; v[1] = t.y;
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = p[e];
    }
}

template <int E, bool VEC, bool CS = false>
__device__ __forceinline__ void q4_st(float *p, const float (&v)[E]) {
    if constexpr (VEC && E == 4) {
        const float4 t = make_float4(v[0], v[1], v[2], v[3]);
        if constexpr (CS) __stcs(reinterpret_cast<float4 *>(p), t);
        else *reinterpret_cast<float4 *>(p) = t;
    } else if constexpr (VEC && E == 2) {
        const float2 t = make_float2(v[0], v[1]);
        if constexpr (CS) __stcs(reinterpret_cast<float2 *>(p), t);
        else *reinterpret_cast<float2 *>(p) = t;
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e) p[e] = v[e];
    }
}

// A number as the unevaluated sum of two floats, |lo| <= ulp(hi) / 2 (about 48
// bits): products by fma, sums by Knuth's two-sum.
struct F2 {
    float hi, lo;
};
__device__ __forceinline__ F2 f2_norm(float h, float l) {
    const float s = __fadd_rn(h, l);
    return {s, __fsub_rn(l, __fsub_rn(s, h))};
}
__device__ __forceinline__ F2 f2_mul(float a, float b) {
    const float h = __fmul_rn(a, b);
    return {h, __fmaf_rn(a, b, -h)};
}
__device__ __forceinline__ F2 f2_mul(F2 a, float b) {
    const float h = __fmul_rn(a.hi, b);
    return f2_norm(h, __fmaf_rn(a.lo, b, __fmaf_rn(a.hi, b, -h)));
}
__device__ __forceinline__ F2 f2_add(F2 a, F2 b) {
    const float s = __fadd_rn(a.hi, b.hi), t = __fsub_rn(s, a.hi);
    const float e = __fadd_rn(__fsub_rn(a.hi, __fsub_rn(s, t)), __fsub_rn(b.hi, t));
    return f2_norm(s, __fadd_rn(e, __fadd_rn(a.lo, b.lo)));
}
__device__ __forceinline__ F2 f2_neg(F2 a) { return {-a.hi, -a.lo}; }
__device__ __forceinline__ bool f2_less(F2 a, F2 b) { return a.hi < b.hi || (a.hi == b.hi && a.lo < b.lo); }
__device__ __forceinline__ F2 f2_shfl(F2 a, int o) {
    return {__shfl_xor_sync(0xffffffffu, a.hi, o), __shfl_xor_sync(0xffffffffu, a.lo, o)};
}

// One row of the cache from a warp: E values to a lane. raw: the inputs; for a
// key its norm weights w and rotation cs too.
template <int HD>
struct Q4Src {
    float raw[HD / 32], w[HD / 32];
    float2 cs[HD / 32];
    bool key;
    float eps;
};

// Whether a head's mean square (with eps) may be had in f32: beyond these the
// squares, or their sum, leave its range, and f64 takes the head (so 1e30 in an
// input is as good as 1).
__device__ __forceinline__ bool q4_norm_fits(float mean) { return mean > 0x1p-100f && mean < 0x1p120f; }

// A query head normalised and rotated in f64: for those whose squares leave f32.
template <int HD>
__device__ __noinline__ void q4_query_f64(const Q4Src<HD> &in, int lane, float *y) {
    constexpr int E = Q4Row<HD>::E;
    double ss = 0.0;
#pragma unroll
    for (int e = 0; e < E; ++e) ss += static_cast<double>(in.raw[e]) * in.raw[e];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const double r = 1.0 / sqrt(ss / HD + static_cast<double>(in.eps));
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const double x = static_cast<double>(in.raw[e]) * in.w[e] * r;
        const double o = __shfl_xor_sync(0xffffffffu, x, 16), c = in.cs[e].x, s = in.cs[e].y;
        y[e] = static_cast<float>(lane < 16 ? x * c - o * s : o * s + x * c);
    }
}

// The row encoded in f64: for the values that two floats do not hold or decide
// (outside their range, or on a border to the last bit). Returns whether one of
// the lane's values cannot be held.
template <int HD>
__device__ __noinline__ bool q4_encode_f64(const Q4Src<HD> &in, int lane, int *code, __half *scale) {
    constexpr int E = Q4Row<HD>::E, L = Q4Row<HD>::L;
    double x[E], r = 1.0;
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = in.raw[e];
    if (in.key) {
        double ss = 0.0;
#pragma unroll
        for (int e = 0; e < E; ++e) ss += x[e] * x[e];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        r = 1.0 / sqrt(ss / HD + static_cast<double>(in.eps));
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] *= in.w[e];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const double o = __shfl_xor_sync(0xffffffffu, x[e], 16), c = in.cs[e].x, s = in.cs[e].y;
            x[e] = lane < 16 ? x[e] * c - o * s : x[e] * c + o * s;
        }
    }
    double P = x[0], N = -x[0];
    bool bad = false;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        P = fmax(P, x[e]);
        N = fmax(N, -x[e]);
        bad |= !(fabs(x[e] * r) < 524160.0);
    }
#pragma unroll
    for (int o = 1; o < L; o <<= 1) {
        P = fmax(P, __shfl_xor_sync(0xffffffffu, P, o));
        N = fmax(N, __shfl_xor_sync(0xffffffffu, N, o));
    }
    const double m = P >= N ? P : -N;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const double f = floor(-8.0 * x[e] / m + 8.5);
        code[e] = m == 0.0 ? 8 : static_cast<int>(fmin(fmax(f, 0.0), 15.0));
    }
    *scale = m == 0.0 ? __float2half_rn(0.0f) : __double2half(-m * r / 8.0);
    return bad || __hisinf(*scale);   // a value at the limit to the last bit goes by its scale
}

// The row encoded with two floats to a number. The norm's factor r > 0 is
// common to the row, so codes come from the rotated values without it: code k
// or k - 1 by the sign of -8 y / m - (k - 8.5). The scale's rounding compares
// squares, (m / 8)^2 against (midpoint)^2 (mean + eps), without a root. Returns
// false (for the whole warp) where that decides nothing.
template <int HD>
__device__ __noinline__ bool q4_encode_f2(const Q4Src<HD> &in, int lane, int *code, __half *scale) {
    constexpr int E = Q4Row<HD>::E, L = Q4Row<HD>::L;
    constexpr float kSure = 0x1p-42f;
    F2 y[E], S{0.0f, 0.0f};
    if (in.key) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            S = f2_add(S, f2_mul(in.raw[e], in.raw[e]));
            y[e] = f2_mul(in.raw[e], in.w[e]);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) S = f2_add(S, f2_shfl(S, o));
        S = f2_add({S.hi / HD, S.lo / HD}, {in.eps, 0.0f});
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const F2 o = f2_shfl(y[e], 16);
            y[e] = f2_add(f2_mul(y[e], in.cs[e].x), f2_mul(o, lane < 16 ? -in.cs[e].y : in.cs[e].y));
        }
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e) y[e] = {in.raw[e], 0.0f};
    }
    F2 P = y[0], N = f2_neg(y[0]);
#pragma unroll
    for (int e = 1; e < E; ++e) {
        if (f2_less(P, y[e])) P = y[e];
        if (f2_less(N, f2_neg(y[e]))) N = f2_neg(y[e]);
    }
#pragma unroll
    for (int o = 1; o < L; o <<= 1) {
        const F2 p = f2_shfl(P, o), n = f2_shfl(N, o);
        if (f2_less(P, p)) P = p;
        if (f2_less(N, n)) N = n;
    }
    const F2 m = f2_less(P, N) ? f2_neg(N) : P;
    const float am = fabsf(m.hi);
    // products' low parts stay normal in this range
    bool sure = am == 0.0f || (am > 0x1p-30f && am < 0x1p30f);
    if (am == 0.0f) {
        // exactly zero where the inputs are; a key's sum may have lost what f64 keeps
        sure = !in.key || S.hi == in.eps;
#pragma unroll
        for (int e = 0; e < E; ++e) code[e] = 8;
        *scale = __float2half_rn(0.0f);
    } else {
        const float inv = -8.0f / m.hi;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float k = rintf(fmaf(y[e].hi, inv, 8.5f));
            // sign of -8 y - (k - 8.5) m, for m > 0
            const F2 d = f2_add({-8.0f * y[e].hi, -8.0f * y[e].lo}, f2_neg(f2_mul(m, k - 8.5f)));
            const float side = m.hi > 0.0f ? d.hi : -d.hi;
            // a value's two floats are exact for V, and a tie goes up; a key's are not
            if (in.key && fabsf(side) < kSure * am) sure = false;
            code[e] = static_cast<int>(fminf(fmaxf(side >= 0.0f ? k : k - 1.0f, 0.0f), 15.0f));
        }
        if (!in.key) {
            *scale = __float2half_rn(m.hi * -0.125f);   // m is exact
        } else {
            const float a32 = am * 0.125f, d32 = a32 / sqrtf(S.hi);
            const __half h = __float2half_rn(d32);
            const unsigned bits = __half_as_ushort(h);
            const float hf = __half2float(h);
            // midpoints to the f16 neighbours: 12 bits, their squares exact
            const float up = 0.5f * (hf + __half2float(__ushort_as_half(static_cast<unsigned short>(bits + 1))));
            const float dn = 0.5f * (hf + __half2float(__ushort_as_half(static_cast<unsigned short>(bits - 1))));
            const F2 a{a32, (m.hi > 0.0f ? m.lo : -m.lo) * 0.125f};
            const F2 aa = f2_add(f2_mul(a, a.hi), f2_mul(a, a.lo));
            const F2 over = f2_add(aa, f2_neg(f2_mul(S, up * up))), under = f2_add(aa, f2_neg(f2_mul(S, dn * dn)));
            if (!(d32 > 0x1p-13f && d32 < 65000.0f) || fabsf(over.hi) < kSure * aa.hi || fabsf(under.hi) < kSure * aa.hi) sure = false;
            const unsigned c = over.hi > 0.0f ? bits + 1 : (under.hi < 0.0f ? bits - 1 : bits);
            *scale = __ushort_as_half(static_cast<unsigned short>(c | (m.hi > 0.0f ? 0x8000u : 0u)));
        }
    }
    return __all_sync(0xffffffffu, sure);
}

// Encode a warp's row: y are its values in f32 (a key's rotated, without the
// norm's factor r), each within err of the exact one. f32 decides every code
// and scale that lies further from a border than err can carry it; where one
// does not, the whole row goes through two floats to a number (about one key
// row in eighty, hardly ever a value row), so the codes are those of the exact
// values whatever the order of the f32 sums. far: a key whose norm f32 does not
// hold, for f64 from the start. Returns false for a lane whose block holds a value
// that is not finite or too large for an f16 scale: it is written as zeros.
template <int HD>
__device__ __forceinline__ bool q4_encode(const float (&y)[HD / 32], float err, float r, bool far, const Q4Src<HD> &in,
                                          int lane, int (&code)[HD / 32], __half &scale) {
    constexpr int E = Q4Row<HD>::E, L = Q4Row<HD>::L;
    float P = y[0], N = -y[0];
    bool bad = false;
    // 8 * 65520, where the scale rounds to infinity; a key's value is within `room` of the exact one there
    constexpr float kLimit = 524160.0f;
    const float room = in.key ? fmaf(err * 1.01f, r, kLimit * 12.0f * 5.97e-8f) : 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        P = fmaxf(P, y[e]);
        N = fmaxf(N, -y[e]);
        bad |= !(fabsf(y[e] * r) < kLimit + room);
    }
#pragma unroll
    for (int o = 1; o < L; o <<= 1) {
        P = fmaxf(P, __shfl_xor_sync(0xffffffffu, P, o));
        N = fmaxf(N, __shfl_xor_sync(0xffffffffu, N, o));
    }
    const unsigned badmask = __ballot_sync(0xffffffffu, bad);
    const unsigned block = (L == 32 ? 0xffffffffu : ((1u << L) - 1u)) << (lane / L * L);
    bool fine = (badmask & block) == 0u;
    const float m = P >= N ? P : -N, am = fabsf(m);
    bool near = far;
    if (fine && am > 0.0f) {
        // under 1e-30 the quotient leaves f32's range
        near |= am < 1e-30f || (err > 0.0f && (fabsf(P - N) <= 2.0f * err || am * r >= kLimit - room));
        const float inv = -8.0f / m, tol = fmaf(2.0f * err, fabsf(inv), 2e-6f);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float f = fmaf(y[e], inv, 8.5f);
            near |= fabsf(f - rintf(f)) <= tol;
            code[e] = static_cast<int>(fminf(fmaxf(floorf(f), 0.0f), 15.0f));
        }
        const float d = am * 0.125f * r;
        scale = __float2half_rn(m > 0.0f ? -d : d);
        if (err > 0.0f) {
            // r is within 9 roundings (4.5 for half of a sum of 9, the mean, 4 for the
            // root), d within one more and m's err
            const float de = fmaf(d, 10.0f * 5.97e-8f, err * 0.126f * r);
            near |= __half_as_ushort(__float2half_rn(d - de)) != __half_as_ushort(__float2half_rn(d + de));
        }
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e) code[e] = 8;
        scale = __float2half_rn(0.0f);
        // an exact value may be tiny where its f32 value is zero
        near |= fine && err > 0.0f;
    }
    if (__any_sync(0xffffffffu, near)) {
        int c2[E];
        __half s2;
        // (a value at the limit is beyond the scales that two floats decide)
        if (far || !q4_encode_f2<HD>(in, lane, c2, &s2))
            fine = (__ballot_sync(0xffffffffu, q4_encode_f64<HD>(in, lane, c2, &s2)) & block) == 0u;
#pragma unroll
        for (int e = 0; e < E; ++e) code[e] = fine ? c2[e] : 8;
        scale = fine ? s2 : __float2half_rn(0.0f);
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

// A warp takes TPW heads of a row, one after another, their loads first: one
// for a few rows (every warp of the GPU has something to do), four for many
// (four loads in flight for each warp). A row is read once and its queries
// written once: 4096 rows of 48 heads of 128 (172 MB, a floor of 25 us) take 47
// us, 0.54 of the measured copy rate. What bounds it there: waiting for loads (the
// rotation's depends on the position's) at 32 warps to an SM, a third of the
// issue slots; more warps in fewer registers (40 to 56 a thread) or two heads to
// a warp are no faster. Few rows: the launch and two loads in a row.
template <int HD, int TPW, bool VEC>
__global__ void __launch_bounds__(128, 8) k_kv_q4_append(Q4AppendArgs a) {
    constexpr int E = Q4Row<HD>::E, L = Q4Row<HD>::L, NB = Q4Row<HD>::NB;
    // many rows pass through L2 once and leave it first (with the rows' reading back
    // 55.5 us against 58.6 with plain accesses)
    constexpr bool kMany = TPW > 1;
    const int lane = threadIdx.x & 31;
    const int task0 = (blockIdx.y * 4 + (threadIdx.x >> 5)) * TPW, row = blockIdx.x;
    const int nkv = a.c.nkv, tasks = a.nh + 2 * nkv;
    if (task0 >= tasks) return;
    const float *src = a.qkv + row * a.qkv_stride + lane * E;
    Q4Src<HD> in;
    float raw[TPW][E];
    in.eps = a.eps;
    pdl_wait();
    // every load that waits for no other first
#pragma unroll
    for (int t = 0; t < TPW; ++t)
        if (task0 + t < tasks) q4_ld<E, VEC, kMany>(raw[t], src + static_cast<int64_t>(task0 + t) * HD);
    if (TPW == 1) q4_ld<E, VEC>(in.w, (task0 < a.nh ? a.q_norm : a.k_norm) + lane * E);
    int slot, pos;
    const bool there = kv_q4_row(a.c, a.rows, row, slot, pos);
    if (there && task0 < a.nh + nkv) {
        float cs[2 * E];
        q4_ld<E, VEC>(*reinterpret_cast<float(*)[E]>(&cs[0]), reinterpret_cast<const float *>(a.rope + static_cast<size_t>(pos) * (HD / 2) + (lane & 15) * E));
        q4_ld<E, VEC>(*reinterpret_cast<float(*)[E]>(&cs[E]), reinterpret_cast<const float *>(a.rope + static_cast<size_t>(pos) * (HD / 2) + (lane & 15) * E) + E);
#pragma unroll
        for (int e = 0; e < E; ++e) in.cs[e] = make_float2(cs[2 * e], cs[2 * e + 1]);
    }
    if (TPW > 1 && there && task0 + TPW <= a.nh) {
        // queries only, as most heads are: side by side, their shuffles in flight together
        float w[E], ss[TPW];
        q4_ld<E, VEC>(w, a.q_norm + lane * E);
#pragma unroll
        for (int t = 0; t < TPW; ++t) {
            ss[t] = 0.0f;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                ss[t] = fmaf(raw[t][e], raw[t][e], ss[t]);
                raw[t][e] *= w[e];
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
            for (int t = 0; t < TPW; ++t) ss[t] += __shfl_xor_sync(0xffffffffu, ss[t], o);
        bool fits = true;
#pragma unroll
        for (int t = 0; t < TPW; ++t) {
            ss[t] = ss[t] / static_cast<float>(HD) + a.eps;
            fits &= q4_norm_fits(ss[t]);
        }
        if (fits) {
#pragma unroll
            for (int t = 0; t < TPW; ++t) {
                const float r = rsqrtf(ss[t]);   // within 2 roundings: queries are f32 sums anyway
                float y[E];
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const float o = __shfl_xor_sync(0xffffffffu, raw[t][e], 16);
                    y[e] = r * (lane < 16 ? raw[t][e] * in.cs[e].x - o * in.cs[e].y : o * in.cs[e].y + raw[t][e] * in.cs[e].x);
                }
                q4_st<E, VEC, kMany>(a.q_out + row * a.q_stride + static_cast<int64_t>(task0 + t) * HD + lane * E, y);
            }
            return;
        }
        // one by one below, from the inputs again
#pragma unroll
        for (int t = 0; t < TPW; ++t) q4_ld<E, VEC, kMany>(raw[t], src + static_cast<int64_t>(task0 + t) * HD);
    }
#pragma unroll
    for (int t = 0; t < TPW; ++t) {
        const int task = task0 + t;
        if (task >= tasks) return;
        const bool query = task < a.nh;
        if (!there) {
            const float zero[E] = {};
            if (query) q4_st<E, VEC, kMany>(a.q_out + row * a.q_stride + static_cast<int64_t>(task) * HD + lane * E, zero);
            continue;
        }
        in.key = task < a.nh + nkv;
        float y[E], err = 0.0f, r = 1.0f;
        bool far = false;
#pragma unroll
        for (int e = 0; e < E; ++e) y[e] = in.raw[e] = raw[t][e];
        if (in.key) {
            if (TPW > 1) q4_ld<E, VEC>(in.w, (query ? a.q_norm : a.k_norm) + lane * E);
            float ss = 0.0f, top = 0.0f;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                ss = fmaf(y[e], y[e], ss);
                y[e] *= in.w[e];
                top = fmaxf(top, fabsf(y[e]));
            }
            const float mean = warp_sum(ss) / static_cast<float>(HD) + a.eps;
            far = !q4_norm_fits(mean);
            r = rsqrtf(mean);
            // a rotated value is within 4 roundings of sqrt 2 times the row's
            // largest: one for each product with w, with cos and with sin, one sum
            if (!query) err = 6.0f * 5.97e-8f * __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float o = __shfl_xor_sync(0xffffffffu, y[e], 16);
                y[e] = lane < 16 ? y[e] * in.cs[e].x - o * in.cs[e].y : o * in.cs[e].y + y[e] * in.cs[e].x;
            }
        }
        if (query) {
#pragma unroll
            for (int e = 0; e < E; ++e) y[e] *= r;
            if (far) q4_query_f64<HD>(in, lane, y);
            q4_st<E, VEC, kMany>(a.q_out + row * a.q_stride + static_cast<int64_t>(task) * HD + lane * E, y);
            continue;
        }
        const int sel = in.key ? 0 : 1, g = task - a.nh - sel * nkv;
        int code[E];
        __half scale;
        const bool fine = q4_encode<HD>(y, err, r, far, in, lane, code, scale);
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
}

// A block per row, four values of one head of K and of V to a thread: a warp
// writes whole rows. Bound by the f32 values written, which leave L2 first
// (8192 rows of 8 heads, 67 MB: 17.2 us a call, 22.2 with plain stores).
template <int HD, bool VEC>
__global__ void __launch_bounds__(256) k_kv_q4_read(KvQ4 c, KvQ4Rows rows, int M, float *__restrict__ k_out,
                                                    float *__restrict__ v_out, size_t out_row, size_t out_head) {
    constexpr int NB = HD / 32, Q = HD / 4;
    const int row = blockIdx.x;
    int slot, pos;
    pdl_wait();
    const bool there = kv_q4_row(c, rows, row, slot, pos);
    for (int i = threadIdx.x; i < c.nkv * Q; i += blockDim.x) {
        const int j = i % Q, g = i / Q;
        const int b = j / 8, q = j % 8;   // block, quadruple of the block
        unsigned w[2] = {0x8888u, 0x8888u};
        float s[2] = {0.0f, 0.0f};
        if (there) {
#pragma unroll
            for (int sel = 0; sel < 2; ++sel) {
                const int at = sel ? 2 * (q * NB + b) : 4 * ((q >> 1) * NB + b) + 2 * (q & 1);
                w[sel] = *reinterpret_cast<const uint16_t *>(kv_q4_codes<HD>(c, slot, sel, g) +
                                                             static_cast<size_t>(pos) * (HD / 2) + at);
                s[sel] = __half2float(kv_q4_scales<HD>(c, slot, sel, g)[static_cast<size_t>(pos) * NB + b]);
            }
        }
#pragma unroll
        for (int sel = 0; sel < 2; ++sel) {
            float y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = s[sel] * static_cast<float>(static_cast<int>((w[sel] >> (4 * e)) & 15u) - 8);
            float *to = (sel ? v_out : k_out) + row * out_row + g * out_head + 4 * j;
            q4_st<4, VEC, true>(to, y);
        }
    }
}

// ---------------------------------------------------------------- attention
//
// out = sum_j softmax_j(scale q.K_j) V_j over the 4-bit rows. The columns of
// one kv head (its group's heads times the query rows) share every cached
// byte: a unit of work is up to 8 columns of one kv head and sequence, a block
// of it 128 positions. Few units: a cluster of CTAs takes each and joins its
// results through distributed shared memory, in one launch. Many: the blocks of
// all units in one row are dealt to the CTAs in equal contiguous shares (the
// lengths are on the device: each CTA sums them), so that sequences of any
// lengths keep every SM busy to the end; a unit that a share's end cuts leaves
// partial results, which a second small kernel joins. A warp takes tiles of 32
// positions and multiplies with mma.m16n8k16 (f16 in, f32 out), positions along
// m for S = K Q^T, dimensions along m for O = V^T P^T:
//  - codes are exact in f16 (-8..7): a word of 8 codes becomes 4 half2
//    operands with 9 instructions and no scale. K scales multiply the f32 sums
//    of a 32-value block, V scales the probabilities of their position.
//  - f16 keeps 11 bits, so q and p v_scale go in as two parts, hi + lo (22
//    bits: less than f32, and below its sums' own error), in columns of their own: of the 8 columns of an operand 4 are hi
//    and 4 lo where that is enough; else hi and lo take an operand each. With
//    2 columns or 1 the spare columns hold P times the scales of other blocks.
//  - q columns are scaled by a power of two (largest value in [2^14, 2^15)),
//    P columns by 2^kf with kf following the largest V scale met so far, so
//    that hi and lo stay clear of f16's subnormals; both undone in f32.
//  - the scores leave the tensor core with positions along rows and enter it
//    again with positions along k: one 8x8 transpose in registers each.
// A chain of products in the tensor core is 2 instructions long (4 where hi and
// lo take an operand each: the small lo products first, so that they add no
// rounding to speak of); the sums over blocks and tiles are f32 with rounding to
// nearest. mma.sync rather than
// tcgen05: with at most 8 columns the product is bound by what the codes cost
// (bytes, then the unpacking), and registers to registers saves writing the
// unpacked codes to shared memory and reading them back.
// What bounds it: instructions, and the register file's ports, for which mma and
// FMA compete (8 mma and 64 FMA take the sum of their times, not the longer). A
// warp's tile of 4.6 KB takes some 750 instructions (830 at 8 columns: unpacking,
// the split of P, the softmax); the copies alone would take 29 of the 43 us of 64
// sequences of 2048 positions (47 with a graph's launch, as all times below; 32/8
// heads, 151 MB; 3.5 TB/s, 0.52 of the measured copy rate), the instructions alone 38.

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// The first of a chain: d = a b.
__device__ __forceinline__ void mma_f16_first(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]), "f"(0.0f));
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

// Codes less 8 of a word's nibbles as half2: h[p] = (nibble p, nibble p + 4), by the
// widely published way to turn nibbles into halves: under the exponent of 1024.
// 0x6400 | n is 1024 + n in f16, 0x6400 | n << 4 is 1024 + 16 n.
// `magic` is 0x64006400 in a register (q4_magic), so that mask and or are one
// three-operand instruction.
__device__ __forceinline__ uint32_t q4_magic() {
    uint32_t r;
    asm volatile("mov.b32 %0, 0x64006400;" : "=r"(r));
    return r;
}
template <uint32_t MASK>
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t y) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(x), "n"(MASK), "r"(y));
    return r;
}
__device__ __forceinline__ void unpack8(uint32_t w, uint32_t magic, uint32_t (&h)[4]) {
    const __half2 c1032 = __halves2half2(__ushort_as_half(0x6408), __ushort_as_half(0x6408));
    const __half2 c16 = __halves2half2(__ushort_as_half(0x2C00), __ushort_as_half(0x2C00));     // 1 / 16
    const __half2 c72 = __halves2half2(__ushort_as_half(0xD480), __ushort_as_half(0xD480));     // -72
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t x = i ? w >> 8 : w;
        const uint32_t lo = and_or<0x000F000Fu>(x, magic), hi = and_or<0x00F000F0u>(x, magic);
        const __half2 l = __hsub2(*reinterpret_cast<const __half2 *>(&lo), c1032);
        const __half2 g = __hfma2(*reinterpret_cast<const __half2 *>(&hi), c16, c72);
        h[2 * i] = *reinterpret_cast<const uint32_t *>(&l);
        h[2 * i + 1] = *reinterpret_cast<const uint32_t *>(&g);
    }
}

__device__ __forceinline__ float half_of(uint32_t w, int i) {
    const __half2 h = *reinterpret_cast<const __half2 *>(&w);
    return i ? __high2float(h) : __low2float(h);
}

// Warps of a CTA: kQ4Warps where units are dealt out in blocks, kQ4ClusterWarps
// where a cluster takes a unit.
constexpr int kQ4Warps = 4, kQ4ClusterWarps = 8, kQ4Tile = 32, kQ4Block = kQ4Warps * kQ4Tile, kQ4MaxCluster = 16;

// Positions of sequence b, within what the call allows.
__device__ __forceinline__ int q4_len(const KvQ4AttnArgs &a, int b) {
    return min(max(a.lens ? a.lens[b] : 0, -a.len_add) + a.len_add, a.max_len);
}

// A CTA of width class W takes W columns in q4_ops(W) operands of 8: W = 1, 2,
// 4 with hi and lo in one operand, 8 with one for each.
__host__ __device__ constexpr int q4_ops(int W) { return W <= 4 ? 1 : 2; }

// CTAs of kQ4Warps warps that share an SM: three in 168 registers, two where 8
// columns of 128 dimensions want 254 (three spill: 4 x 5000 with 16 rows and 32/8
// heads 68 us against 64; at 64 dimensions three are faster, 30 x 4000 with 4 rows
// 57 against 64). Four in 128 spill too: 64 x 2048 with 32/8 heads 51 us against 47.
__host__ __device__ constexpr int q4_per_sm(int hd, int W) { return W <= 4 || hd <= 64 ? 3 : 2; }

template <int HD>
struct Q4Words {   // words of a thread's share of a row
    static constexpr int K = HD / 32, V = HD / 64, S = HD / 64;
};

template <int N>
__device__ __forceinline__ void ld_words(uint32_t (&d)[N], const uint8_t *p) {
    if constexpr (N == 4) {
        const uint4 t = *reinterpret_cast<const uint4 *>(p);
        d[0] = t.x; d[1] = t.y; d[2] = t.z; d[3] = t.w;
    } else if constexpr (N == 2) {
        const uint2 t = *reinterpret_cast<const uint2 *>(p);
        d[0] = t.x; d[1] = t.y;
    } else {
        d[0] = *reinterpret_cast<const uint32_t *>(p);
    }
}

// The power of two that brings a query's largest magnitude into [2^14, 2^15), over
// all of f32 (f16_row_exp stops at 2^100, short of the largest and smallest
// queries): both it and its inverse are normal. 0, NaN and infinities as they are.
__device__ __forceinline__ int q4_query_exp(float amax) {
    if (!(amax > 0.0f && amax < INFINITY)) return 0;
    return min(126, 14 + 127 - static_cast<int>(__float_as_uint(amax) >> 23));
}

// How far (log2) a score may pass the highest at the last change of the
// weights' unit. P is cut at 2^-24 where its largest product lies in [2^12,
// 2^15]: these 2 bits and one of the V scale's rounding up to a power of two.
// More room costs precision beside tokens with far larger values and gains
// little: 24 x 8192 with 5 rows 197 us with none, 192 with 2 bits, 190 with 6.
constexpr float kRoom = 2.0f;

// A warp's tile in shared memory: codes of K, of V, scales of K, of V. Each
// warp has a ring of kQ4Stages of them, filled by bulk copies.
constexpr int kQ4Stages = 2;
template <int HD>
struct Q4Stage {
    static constexpr int kCodes = kQ4Tile * HD / 2, kScales = kQ4Tile * HD / 16;
    static constexpr int V = kCodes, KS = 2 * kCodes, VS = KS + kScales, bytes = VS + kScales;
};

// Partial results: per column acc[HD], then log2 of their unit and the sum of
// weights.
template <int HD>
__host__ __device__ constexpr int q4_part() { return HD + 2; }

// What a unit costs besides its blocks (its queries, the joining of its warps),
// in blocks (64 sequences of 1 to 4101 positions, 16/8 heads: 45 us at 2, 51 at
// 1, 62 at 0).
constexpr int kQ4UnitCost = 2;

// Blocks of sequence b (one at least: a sequence without positions still has
// outputs to write) and, if asked, its length and slot.
__device__ __forceinline__ int q4_blocks(const KvQ4AttnArgs &a, int b, int *len_out = nullptr, int *slot_out = nullptr) {
    const int slot = a.slots ? a.slots[b] : a.slot0 + b;
    const bool there = slot >= 0 && slot < a.c.slots;
    const int len = there ? q4_len(a, b) : 0;
    if (len_out) *len_out = len;
    if (slot_out) *slot_out = there ? slot : 0;
    return max(1, (len + kQ4Block - 1) / kQ4Block);
}

// a / b for a >= 0, in 32 bits where that is enough.
__device__ __forceinline__ int64_t q4_div(int64_t a, unsigned b) {
    return a >> 32 ? a / b : static_cast<int64_t>(static_cast<unsigned>(a) / b);
}

// A warp's part of one column, plainly in f32, for far scores: from kFar on (log2
// units) the reference of the weights, the highest score less the unit's power of
// two, is rounded in one f32 number by 2^-3 and more, soon by more than P's spare
// bits, to weights of several times f16's largest or next to nothing. Here the
// reference is the highest score. The positions are first .. first + 31 and every
// step-th tile from there, below lim; k: the head's K codes, its scales `plane`
// bytes on, V to_v bytes on; a lane to a position for the scores, to HD / 32
// dimensions for the output. (Inside the tiles the same cost every call 1 to 3
// percent; what such scores cost here does not matter.)
constexpr float kFar = 2097152.0f;
template <int HD>
__device__ __noinline__ void q4_far_column(const float *q, float scale, const uint8_t *k, size_t plane, size_t to_v,
                                           int first, int step, int lim, float *res) {
    constexpr int E = HD / 32, NB = HD / 32;
    const int lane = threadIdx.x & 31;
    float amax = 0.0f;
    for (int d = lane; d < HD; d += 32) amax = fmaxf(amax, fabsf(q[d]));
    const int t = q4_query_exp(warp_max(amax));
    const float f = pow2_f32(t), c = scale * 1.4426950408889634f * pow2_f32(-t);
    float mx = -INFINITY, sum = 0.0f, o[E] = {};
    for (int k0 = first; k0 < lim; k0 += step) {
        const int n = min(32, lim - k0);
        float s = -INFINITY;
        if (lane < n) {
            const uint8_t *row = k + static_cast<size_t>(k0 + lane) * (HD / 2);
            const __half *sc = reinterpret_cast<const __half *>(k + plane) + static_cast<size_t>(k0 + lane) * NB;
            s = 0.0f;
            for (int b = 0; b < NB; ++b) {
                float x = 0.0f;
                for (int j = 0; j < 16; ++j) {
                    const int w = row[4 * ((j >> 2) * NB + b) + (j & 3)];
                    x = fmaf(q[32 * b + 2 * j] * f, static_cast<float>((w & 15) - 8), x);
                    x = fmaf(q[32 * b + 2 * j + 1] * f, static_cast<float>((w >> 4) - 8), x);
                }
                s = fmaf(x, __half2float(sc[b]), s);
            }
            s *= c;
        }
        const float top = fmaxf(mx, warp_max(s)), now = top == -INFINITY ? 0.0f : top;
        const float corr = exp2_f32(mx - now), p = exp2_f32(s - now);
        mx = top;
        sum = fmaf(sum, corr, warp_sum(p));
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] *= corr;
        const uint8_t *v = k + to_v + static_cast<size_t>(k0) * (HD / 2);
        const __half *sv = reinterpret_cast<const __half *>(k + to_v + plane) + static_cast<size_t>(k0) * NB;
        for (int i = 0; i < n; ++i) {
            const float w = __shfl_sync(0xffffffffu, p, i) * __half2float(sv[i * NB + lane * E / 32]);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int code = v[i * (HD / 2) + q4_lane_byte<HD>(lane, true) + e / 2] >> (4 * (e & 1)) & 15;
                o[e] = fmaf(w, static_cast<float>(code - 8), o[e]);
            }
        }
    }
#pragma unroll
    for (int e = 0; e < E; ++e) res[lane * E + e] = o[e];
    if (lane == 0) {
        res[HD] = sum != sum ? 0.0f : mx;
        res[HD + 1] = sum;
    }
}

// Workspace: two partial results of W columns for each CTA (of the unit that
// its share begins inside, and of the one that it ends inside), then the first
// and the last CTA of each unit.
// CL: clusters of CTAs, CL to an SM (0: blocks dealt out); no workspace; grid
// (csize, units), clusters along x.
template <int HD, int W, int CL>
__global__ void __launch_bounds__((CL ? kQ4ClusterWarps : kQ4Warps) * 32, CL ? CL : q4_per_sm(HD, W))
    k_kv_q4_attn(KvQ4AttnArgs a, int cgroups, int2 *owners) {
    constexpr bool CLUSTER = CL > 0;
    constexpr int NW = CLUSTER ? kQ4ClusterWarps : kQ4Warps, kStep = NW * kQ4Tile;
    constexpr int NB = HD / 32, NT = q4_ops(W);
    constexpr int DUP = W <= 4 ? 4 / W : 1;          // blocks that share an operand
    constexpr int NI = (NB + DUP - 1) / DUP;         // P operands per 16 positions
    constexpr int MT = kQ4Tile / 16;
    constexpr int PS = q4_part<HD>();
    constexpr int QS = HD + 8;                       // a q row in shared memory, padded
    using Wd = Q4Words<HD>;
    using St = Q4Stage<HD>;
    static_assert(W * PS * 4 <= kQ4Stages * St::bytes, "a warp's results fit its ring");
    extern __shared__ __align__(128) uint8_t q4_ring[];   // [warp][kQ4Stages] tiles; a piece's results after it
    __shared__ uint64_t s_bar[NW][kQ4Stages];
    __shared__ float s_joined[CLUSTER ? W * PS : 1];   // this CTA's result, for its cluster
    __shared__ __align__(16) __half s_q[W][2][QS];      // hi and lo; see below for the order of a row
    __shared__ float s_exp[W];
    __shared__ int64_t s_red[NW];
    __shared__ int s_from[NW];      // each warp's first position of the piece

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = lane >> 2, c = lane & 3;
    const int G = a.nh / a.c.nkv, cols = G * a.rows, U = a.c.nkv * cgroups;
    uint8_t *ring = q4_ring + warp * kQ4Stages * St::bytes;
    const auto results = [&](int w) { return reinterpret_cast<float *>(q4_ring + w * kQ4Stages * St::bytes); };
    if (lane == 0) {
        for (int i = 0; i < kQ4Stages; ++i) mbar_init(&s_bar[warp][i], 1);
        fence_mbar_init();
    }
    const uint32_t magic = q4_magic();
    uint32_t taken = 0;     // tiles this warp has taken from its ring
    bool lost = false;      // a copy did not arrive in time, the lost_at-th tile's
    uint32_t lost_at = 0;
    const uint64_t policy = policy_evict_first();
    pdl_wait();

    // ---- this CTA's share [at, stop) of the blocks, its first sequence b and the
    // cost (of one unit) of the sequences below that
    int64_t at = 0, stop = 1, before = 0;
    int b = CLUSTER ? static_cast<int>(blockIdx.y) / U : 0;
    if constexpr (!CLUSTER) {
        // costs of kQ4Warps * 32 sequences from b0 on: this thread's, their sum up to
        // and with it, and all of them
        int64_t n = 0, run = 0, sum = 0;
        const auto scan = [&](int b0) {
            n = b0 + tid < a.B ? q4_blocks(a, b0 + tid) + kQ4UnitCost : 0;
            run = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t x = __shfl_up_sync(0xffffffffu, run, o);
                if (lane >= o) run += x;
            }
            __syncthreads();
            if (lane == 31) s_red[warp] = run;
            __syncthreads();
            sum = 0;
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                if (w < warp) run += s_red[w];
                sum += s_red[w];
            }
        };
        constexpr int kAtOnce = NW * 32;
        int64_t all = 0;
        for (int b0 = 0; b0 < a.B; b0 += kAtOnce) {
            scan(b0);
            all += sum;
        }
        // no share is empty: the join counts on every CTA between a unit's first and last
        const int64_t total = all * U;
        const unsigned P = static_cast<unsigned>(min(static_cast<int64_t>(gridDim.x), total));
        if (blockIdx.x >= P) return;
        const int64_t each = q4_div(total, P), more = total - each * P;
        at = each * blockIdx.x + min(static_cast<int64_t>(blockIdx.x), more);
        stop = at + each + (blockIdx.x < more ? 1 : 0);
        const int64_t want = q4_div(at, static_cast<unsigned>(U));
        for (int b0 = 0; b0 < a.B; b0 += kAtOnce) {
            if (a.B > kAtOnce) scan(b0);
            if (want < before + sum) {
                __syncthreads();
                if (n > 0 && before + run - n <= want && want < before + run) {
                    s_red[0] = b0 + tid;
                    s_red[1] = before + run - n;
                }
                __syncthreads();
                b = static_cast<int>(s_red[0]);
                before = s_red[1];
                break;
            }
            before += sum;
        }
    }

    for (; at < stop; ) {
    // ---- the next piece: blocks [blk0, blk1) of unit (b, g, cg)
    int len, slot;
    const int blocks = q4_blocks(a, b, &len, &slot);
    int unit, blk0 = 0, blk1 = 1, start, end, cost = 0;
    if constexpr (CLUSTER) {
        unit = static_cast<int>(blockIdx.y) % U;
    } else {
        // a unit's cost: kQ4UnitCost, then its blocks
        const int64_t in_b = at - before * U;
        cost = blocks + kQ4UnitCost;
        unit = static_cast<int>(q4_div(in_b, static_cast<unsigned>(cost)));
        const int off0 = static_cast<int>(in_b - static_cast<int64_t>(unit) * cost);
        const int off1 = static_cast<int>(min(static_cast<int64_t>(cost), off0 + (stop - at)));
        blk0 = max(0, off0 - kQ4UnitCost);
        blk1 = max(0, off1 - kQ4UnitCost);
        at += off1 - off0;
        if (blk0 == blk1) continue;   // the share ends before the unit's first block
    }
    const int g = unit / cgroups, cg = unit % cgroups;
    const int col0 = cg * W, ncol = min(W, cols - col0);
    // positions that this group's last column sees
    const int seen = len - a.rows + (col0 + ncol - 1) / G + 1;
    if constexpr (CLUSTER) {
        // an even share of the unit's tiles
        const int64_t tiles = max(0, (seen + kQ4Tile - 1) / kQ4Tile);
        start = static_cast<int>(tiles * blockIdx.x / gridDim.x) * kQ4Tile;
        end = min(seen, static_cast<int>(tiles * (blockIdx.x + 1) / gridDim.x) * kQ4Tile);
        at = stop;
    } else {
        start = blk0 * kQ4Block;
        end = min(seen, blk1 * kQ4Block);
    }

    // ---- tiles of this warp: every NW-th of the piece, the first ones on
    // their way before anything else
    int k0 = start + warp * kQ4Tile;
    if (lane == 0) s_from[warp] = k0;   // read again for far scores: a register for it costs every tile
    // (lane 0's) next tile: codes and scales of K; V's lie a fixed distance behind
    const uint8_t *codes = kv_q4_codes<HD>(a.c, slot, 0, g) + static_cast<size_t>(k0) * (HD / 2);
    const uint8_t *scales = reinterpret_cast<const uint8_t *>(kv_q4_scales<HD>(a.c, slot, 0, g)) + static_cast<size_t>(k0) * (HD / 16);
    const size_t to_v = static_cast<size_t>(a.c.nkv) * kv_q4_head_bytes(a.c.cap, HD);
    const auto fetch = [&](uint32_t n) {   // the tile that is the warp's n-th
        uint8_t *to = ring + n % kQ4Stages * St::bytes;
        uint64_t *bar = &s_bar[warp][n % kQ4Stages];
        mbar_arrive_expect_tx(bar, St::bytes);
        bulk_g2s(to, codes, St::kCodes, bar, policy);
        bulk_g2s(to + St::KS, scales, St::kScales, bar, policy);
        bulk_g2s(to + St::V, codes + to_v, St::kCodes, bar, policy);
        bulk_g2s(to + St::VS, scales + to_v, St::kScales, bar, policy);
        codes += kStep * (HD / 2);
        scales += kStep * (HD / 16);
    };
    if (lane == 0 && !lost) {
        // the last piece's results lay in the ring
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
#pragma unroll
        for (int i = 0; i < kQ4Stages; ++i)
            if (k0 + i * kStep < end) fetch(taken + i);
    }
    // Rows i of an operand along m hold positions of its eight in this order, so
    // that the four positions of one load of V lie together and no load of K
    // meets a bank twice.
    const int pr = (r & 1) ? 4 + ((r >> 1) ^ 1) : r >> 1;

    // ---- q columns, while the first rows are on their way: scaled by a power
    // of two, split into hi and lo. Value 8 i + p of a row lies at 8 i + 2 (p &
    // 3) + (p >> 2), so that the pairs (p, p + 4) of an operand lie together.
    for (int j = warp; j < W; j += NW) {
        constexpr int E = HD / 32;
        float x[E], amax = 0.0f;
        const int cc = col0 + j;
        const float *qp = a.q + (static_cast<int64_t>(b) * a.rows + cc / G) * a.q_stride +
                          static_cast<int64_t>(g * G + cc % G) * HD;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            x[e] = j < ncol ? qp[lane + 32 * e] : 0.0f;
            amax = fmaxf(amax, fabsf(x[e]));
        }
        const int t = q4_query_exp(warp_max(amax));
        const float f = pow2_f32(t);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int d = lane + 32 * e, to = (d & ~7) | 2 * (d & 3) | ((d >> 2) & 1);
            const float v = x[e] * f;
            const __half hi = __float2half_rn(v);
            s_q[j][0][to] = hi;
            s_q[j][1][to] = __float2half_rn(v - __half2float(hi));
        }
        if (lane == 0) s_exp[j] = static_cast<float>(t);
    }
    __syncthreads();
    uint32_t qf[NB * 2][NT][2];
#pragma unroll
    for (int ks = 0; ks < NB * 2; ++ks)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            // column r of operand nt, words c of block ks / 2
            const __half *row = W <= 4 ? s_q[(r & 3) % W][r >> 2] : s_q[r % W][nt];
            const uint2 t = *reinterpret_cast<const uint2 *>(row + (ks >> 1) * 32 + c * 8 + (ks & 1) * 4);
            qf[ks][nt][0] = t.x;
            qf[ks][nt][1] = t.y;
        }
    // this thread's score columns: 2c and 2c + 1
    float cscale[2];
    int lim[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int j = W <= 4 ? (2 * c + e) % 4 % W : 2 * c + e;
        cscale[e] = a.scale * 1.4426950408889634f * pow2_f32(-static_cast<int>(s_exp[j]));
        lim[e] = j < ncol ? len - a.rows + (col0 + j) / G + 1 : 0;
    }
    const int low_lim = len - a.rows + col0 / G + 1;   // positions that every column sees

    float acc[NB][2][4], mx[2], ref[2], sum[2];
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int m = 0; m < 2; ++m)
            for (int e = 0; e < 4; ++e) acc[i][m][e] = 0.0f;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        mx[e] = -INFINITY;
        ref[e] = -INFINITY;
        sum[e] = 0.0f;
    }
    // 2^(kf + kRoom) brings P times the largest V scale so far to 2^15 at most; vlim:
    // the largest scale that the present kf takes
    float kf = 37.0f;
    __half2 vlim = __float2half2_rn(0.0f);
    // hi lanes keep x (cut to f16 below), lo lanes what the cut leaves
    const uint32_t cut = (W <= 4 && c < 2) ? 0u : 0xFFFFE000u;

    // one tile; tail: a column's range ends in it, and what lies past that may be anything
    const auto tile = [&](auto tail) {
        const uint8_t *st = ring + taken % kQ4Stages * St::bytes;
        if (!lost && !mbar_wait_bounded(&s_bar[warp][taken % kQ4Stages], (taken / kQ4Stages) & 1u)) {
            lost = true;   // no further copy is started
            lost_at = taken;
            record_status(a.status, QW3_ERR_TIMEOUT);
        }
        // ---- scores
        float s[MT][4];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            float t[4];
            uint32_t kw[2][Wd::K], kd[2][Wd::S];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                ld_words(kw[h], st + (16 * m + 8 * h + pr) * (HD / 2) + c * (HD / 8));
                ld_words(kd[h], st + St::KS + (16 * m + 8 * h + pr) * (HD / 16));
            }
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                uint32_t x0[4], x1[4];
                unpack8(kw[0][i], magic, x0);
                unpack8(kw[1][i], magic, x1);
                const float d0 = half_of(kd[0][i >> 1], i & 1), d1 = half_of(kd[1][i >> 1], i & 1);
                const uint32_t a0[4] = {x0[0], x1[0], x0[1], x1[1]}, a1[4] = {x0[2], x1[2], x0[3], x1[3]};
                float u[4];
                mma_f16_first(u, a0, qf[2 * i][NT - 1]);
                mma_f16(u, a1, qf[2 * i + 1][NT - 1]);
                if constexpr (NT == 2) {
                    mma_f16(u, a0, qf[2 * i][0]);
                    mma_f16(u, a1, qf[2 * i + 1][0]);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) t[e] = i ? fmaf(u[e], e < 2 ? d0 : d1, t[e]) : u[e] * (e < 2 ? d0 : d1);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float v = W <= 4 ? t[e] + __shfl_xor_sync(0xffffffffu, t[e], 2) : t[e];
                s[m][e] = v * cscale[e & 1];
            }
        }
        uint32_t vd[MT][2][Wd::S];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) ld_words(vd[m][h], st + St::VS + (16 * m + 8 * h + pr) * (HD / 16));
        if constexpr (decltype(tail)::value) {
#pragma unroll
            for (int m = 0; m < MT; ++m) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (k0 + 16 * m + 8 * (e >> 1) + pr >= lim[e & 1]) s[m][e] = -INFINITY;
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (k0 + 16 * m + 8 * h + pr >= len)
#pragma unroll
                        for (int w = 0; w < Wd::S; ++w) vd[m][h][w] = 0u;
            }
        }
        // ---- weights 2^(s - ref) (any reference serves as long as one is used
        // throughout): a new one where a score passes the highest so far by more
        // than kRoom, or a V scale what kf takes
        __half2 big = __float2half2_rn(0.0f);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int w = 0; w < Wd::S; ++w) big = __hmax2(big, __habs2(*reinterpret_cast<const __half2 *>(&vd[m][h][w])));
        bool stays = __hble2(big, vlim);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) stays &= s[m][e] <= mx[e & 1] + kRoom;
        if (!__all_sync(0xffffffffu, stays)) {
            const uint32_t top = __reduce_max_sync(0xffffffffu, max(static_cast<uint32_t>(__half_as_ushort(__low2half(big))),
                                                                    static_cast<uint32_t>(__half_as_ushort(__high2half(big)))));
            if (half_of(top, 0) > __low2float(vlim)) {
                // 2^e > the largest scale
                const int e = min(static_cast<int>(__float_as_uint(half_of(top, 0)) >> 23) - 126, 16);
                vlim = e >= 16 ? __half2half2(__ushort_as_half(0x7BFF)) : __float2half2_rn(pow2_f32(e));
                kf = 15.0f - kRoom - static_cast<float>(e);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float t = fmaxf(fmaxf(s[0][e], s[0][e + 2]), fmaxf(s[1][e], s[1][e + 2]));
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, o));
                mx[e] = fmaxf(mx[e], t);
                const float to = mx[e] - kf, now = to == -INFINITY ? 0.0f : to, corr = exp2_f32(ref[e] - now);
                ref[e] = to;
                sum[e] *= corr;
#pragma unroll
                for (int i = 0; i < NB; ++i)
#pragma unroll
                    for (int d = 0; d < 2; ++d)
#pragma unroll
                        for (int h = 0; h < 2; ++h) acc[i][d][e + 2 * h] *= corr;
            }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float now = ref[e] == -INFINITY ? 0.0f : ref[e];
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float p = exp2_f32(s[m][e + 2 * h] - now);
                    s[m][e + 2 * h] = p;
                    sum[e] += p;
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
                    const float x0 = s[m][2 * h] * d0, x1 = s[m][2 * h + 1] * d1;
                    const float y0 = x0 - __uint_as_float(__float_as_uint(x0) & cut);
                    const float y1 = x1 - __uint_as_float(__float_as_uint(x1) & cut);
                    if constexpr (W > 4) pf[i][m][0][h] = transpose8x8(pack_rz(x0, x1));
                    pf[i][m][NT - 1][h] = transpose8x8(pack_rz(y0, y1));
                }
        // ---- O: two positions' halfwords of a block make the pairs along k
        uint32_t vw[MT][4][Wd::V];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 4; ++h)
                ld_words(vw[m][h], st + St::V + (16 * m + 8 * (h >> 1) + ((h & 1) ? 4 + (c ^ 1) : c)) * (HD / 2) + r * (HD / 16));
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            float u[2][4];
            uint32_t a0[MT][4], a1[MT][4];
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                uint32_t x0[4], x1[4];
                const uint32_t sel = (i & 1) ? 0x7632u : 0x5410u;
                unpack8(__byte_perm(vw[m][0][i >> 1], vw[m][1][i >> 1], sel), magic, x0);
                unpack8(__byte_perm(vw[m][2][i >> 1], vw[m][3][i >> 1], sel), magic, x1);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    a0[m][e] = x0[e];
                    a0[m][2 + e] = x1[e];
                    a1[m][e] = x0[2 + e];
                    a1[m][2 + e] = x1[2 + e];
                }
            }
#pragma unroll
            for (int n = NT - 1; n >= 0; --n)
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    if (m == 0 && n == NT - 1) {
                        mma_f16_first(u[0], a0[m], pf[i / DUP][m][n]);
                        mma_f16_first(u[1], a1[m], pf[i / DUP][m][n]);
                    } else {
                        mma_f16(u[0], a0[m], pf[i / DUP][m][n]);
                        mma_f16(u[1], a1[m], pf[i / DUP][m][n]);
                    }
                }
#pragma unroll
            for (int d = 0; d < 2; ++d)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][d][e] += u[d][e];
        }
        ++taken;
        __syncwarp();   // the tile is in registers: its place may be filled again
        if (lane == 0 && !lost && k0 + kQ4Stages * kStep < end) fetch(taken + kQ4Stages - 1);
    };
    for (; k0 < end; k0 += kStep) {
        if (k0 + kQ4Tile <= low_lim) tile(std::false_type{});
        else tile(std::true_type{});
    }

    const auto far = [](float v) { return fabsf(v) >= kFar && fabsf(v) < INFINITY; };
    const bool any_far = __any_sync(0xffffffffu, !lost && (far(mx[0]) || far(mx[1])));
    // ---- the warps' results meet in shared memory
    float *res = results(warp);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        float t = sum[e];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
        const int j = 2 * c + e;
        if (r == 0 && j < W) {
            res[j * PS + HD] = t != t ? 0.0f : ref[e];   // a NaN is not taken for an empty range
            res[j * PS + HD + 1] = t;
        }
    }
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float o[4];   // dimensions 4 r .. 4 r + 3 of the block
#pragma unroll
            for (int d = 0; d < 2; ++d)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    o[2 * d + h] = W <= 4 ? acc[i][d][e + 2 * h] + __shfl_xor_sync(0xffffffffu, acc[i][d][e + 2 * h], 2)
                                          : acc[i][d][e + 2 * h];
            const int n = 2 * c + e, j = W <= 4 ? n % W : n;
            if (W > 4 || (n < 4 && n / W == i % DUP)) {
                float2 *dst = reinterpret_cast<float2 *>(res + j * PS + i * 32 + 4 * r);
                dst[0] = make_float2(o[0], o[1]);
                dst[1] = make_float2(o[2], o[3]);
            }
        }
    if (__builtin_expect(any_far, 0)) {
        __syncwarp();   // over what the lanes have just written
        int n, sl;
        q4_blocks(a, b, &n, &sl);
        const int from = s_from[warp];
        for (int j = 0; j < ncol; ++j) {
            const int cc = col0 + j;
            q4_far_column<HD>(a.q + (static_cast<int64_t>(b) * a.rows + cc / G) * a.q_stride +
                                  static_cast<int64_t>(g * G + cc % G) * HD,
                              a.scale, kv_q4_codes<HD>(a.c, sl, 0, g), static_cast<size_t>(a.c.cap) * (HD / 2),
                              static_cast<size_t>(a.c.nkv) * kv_q4_head_bytes(a.c.cap, HD),
                              from, kStep, min(end, n - a.rows + cc / G + 1), res + j * PS);
        }
    }
    __syncthreads();
    const bool begins = blk0 == 0, ends = blk1 == blocks;
    float *ws = a.ws + (static_cast<size_t>(blockIdx.x) * 2 + (begins ? 1 : 0)) * W * PS;
    for (int x = tid; x < ncol * HD; x += NW * 32) {
        const int j = x / HD, d = x % HD;
        float M = -INFINITY, l = 0.0f, o = 0.0f;
#pragma unroll
        for (int w = 0; w < NW; ++w) M = fmaxf(M, results(w)[j * PS + HD]);
        if (M != -INFINITY)
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const float *p = results(w) + j * PS;
                const float f = exp2_f32(p[HD] - M);
                l = fmaf(p[HD + 1], f, l);
                o = fmaf(p[d], f, o);
            }
        if constexpr (CLUSTER) {
            s_joined[j * PS + d] = o;
            if (d == 0) {
                s_joined[j * PS + HD] = M;
                s_joined[j * PS + HD + 1] = l;
            }
        } else if (begins && ends) {
            const int cc = col0 + j;
            a.out[(static_cast<int64_t>(b) * a.rows + cc / G) * a.out_stride + static_cast<int64_t>(g * G + cc % G) * HD + d] =
                l == 0.0f ? 0.0f : o / l;
        } else {
            ws[j * PS + d] = o;
            if (d == 0) {
                ws[j * PS + HD] = M;
                ws[j * PS + HD + 1] = l;
            }
        }
    }
    if constexpr (CLUSTER) {
        // each CTA joins its share of the outputs over the cluster
        const int peers = static_cast<int>(gridDim.x);
        __syncwarp();
        hw_cluster_sync();
        for (int x = static_cast<int>(blockIdx.x) * NW * 32 + tid; x < ncol * HD; x += peers * NW * 32) {
            const int j = x / HD, d = x % HD;
            float M = -INFINITY, l = 0.0f, o = 0.0f;
#pragma unroll 4
            for (int p = 0; p < peers; ++p) M = fmaxf(M, dsmem_ld(dsmem_map(&s_joined[j * PS + HD], p)));
            if (M != -INFINITY)
#pragma unroll 4
                for (int p = 0; p < peers; ++p) {
                    const float f = exp2_f32(dsmem_ld(dsmem_map(&s_joined[j * PS + HD], p)) - M);
                    l = fmaf(dsmem_ld(dsmem_map(&s_joined[j * PS + HD + 1], p)), f, l);
                    o = fmaf(dsmem_ld(dsmem_map(&s_joined[j * PS + d], p)), f, o);
                }
            const int cc = col0 + j;
            a.out[(static_cast<int64_t>(b) * a.rows + cc / G) * a.out_stride + static_cast<int64_t>(g * G + cc % G) * HD + d] =
                l == 0.0f ? 0.0f : o / l;
        }
        __syncwarp();
        hw_cluster_sync();   // nobody leaves while its result is read
    }
    if (!CLUSTER && tid == 0 && owners) {
        int2 *own = owners + static_cast<size_t>(b) * U + unit;
        if (begins) own->x = static_cast<int>(blockIdx.x);
        if (ends) own->y = static_cast<int>(blockIdx.x);
    }
    __syncthreads();   // results and q rows are read: the next piece may write its own
    if (!CLUSTER && ends && unit == U - 1) {
        before += cost;
        ++b;
    }
    }
    // a warp that gave up leaves no copy in flight behind it
    if (lost)
        for (uint32_t n = lost_at; n < lost_at + kQ4Stages; ++n)
            (void)mbar_wait_bounded(&s_bar[warp][n % kQ4Stages], (n / kQ4Stages) & 1u);
}

// Joins the partial results of the columns whose unit more than one CTA worked
// on: a CTA per (sequence, kv head, column), a thread per dimension; Y rows of
// threads where a unit's results are many, each taking every Y-th.
template <int HD, int Y>
__global__ void __launch_bounds__(HD * Y) k_kv_q4_join(KvQ4AttnArgs a, int cgroups, int W, const int2 *owners) {
    constexpr int PS = q4_part<HD>();
    __shared__ float s_part[Y][PS];
    pdl_wait();
    const int G = a.nh / a.c.nkv, cols = G * a.rows, U = a.c.nkv * cgroups;
    const int cc = blockIdx.x % cols, g = blockIdx.x / cols % a.c.nkv, b = blockIdx.x / (cols * a.c.nkv);
    const int d = threadIdx.x % HD, y = threadIdx.x / HD;
    const int2 own = owners[static_cast<size_t>(b) * U + g * cgroups + cc / W];
    if (own.x == own.y) return;
    // the first CTA ended inside the unit (its second result), the others began inside it
    const auto part = [&](int i) { return a.ws + (static_cast<size_t>(i) * 2 + (i == own.x ? 1 : 0)) * W * PS + cc % W * PS; };
    float M = -INFINITY, l = 0.0f, o = 0.0f;
#pragma unroll 8
    for (int i = own.x + y; i <= own.y; i += Y) M = fmaxf(M, part(i)[HD]);
    if (M != -INFINITY)
#pragma unroll 8
        for (int i = own.x + y; i <= own.y; i += Y) {
            const float *p = part(i);
            const float f = exp2_f32(p[HD] - M);
            l = fmaf(p[HD + 1], f, l);
            o = fmaf(p[d], f, o);
        }
    if constexpr (Y > 1) {
        s_part[y][d] = o;
        if (d == 0) {
            s_part[y][HD] = M;
            s_part[y][HD + 1] = l;
        }
        __syncthreads();
        if (y > 0) return;
#pragma unroll
        for (int k = 1; k < Y; ++k) M = fmaxf(M, s_part[k][HD]);
        l = o = 0.0f;
        if (M != -INFINITY)
#pragma unroll
            for (int k = 0; k < Y; ++k) {
                const float f = exp2_f32(s_part[k][HD] - M);
                l = fmaf(s_part[k][HD + 1], f, l);
                o = fmaf(s_part[k][d], f, o);
            }
    }
    a.out[(static_cast<int64_t>(b) * a.rows + cc / G) * a.out_stride + static_cast<int64_t>(g * G + cc % G) * HD + d] =
        l == 0.0f ? 0.0f : o / l;
}

}  // namespace

namespace {
bool aligned16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }
}  // namespace

cudaError_t launch_kv_q4_append(const float *qkv, int M, int64_t qkv_stride, const float *q_norm, const float *k_norm,
                                float eps, const float2 *rope, const KvQ4 &c, int hd, const KvQ4Rows &rows, int nh,
                                float *q_out, int64_t q_stride, int32_t *status, bool pdl, cudaStream_t s) {
    if (M <= 0) return cudaSuccess;
    const Q4AppendArgs a{qkv, M, qkv_stride, q_norm, k_norm, eps, rope, c, rows, nh, q_out, q_stride, status};
    const int tasks = nh + 2 * c.nkv;
    const bool vec = aligned16(qkv) && aligned16(q_norm) && aligned16(k_norm) && aligned16(rope) && aligned16(q_out) &&
                     qkv_stride % 4 == 0 && q_stride % 4 == 0;
    // four heads to a warp once one to a warp would fill the GPU's 64 warps per
    // SM four times (a call with the rows' reading back: 4096 rows of 48 heads 56
    // us against 100, 2048 of 20 of 64 16.1 against 20.5; 128 of 32 10.3 against 8.9)
    const bool four = static_cast<int64_t>(M) * tasks >= 4ll * 64 * 152;
    const auto go = [&](auto hd_, auto tpw_, auto vec_) {
        constexpr int T = decltype(tpw_)::value;
        const dim3 grid(M, (tasks + 4 * T - 1) / (4 * T));
        return launch_pdl(pdl, k_kv_q4_append<decltype(hd_)::value, T, decltype(vec_)::value>, grid, 128, 0, 1, s, a);
    };
    const auto pick = [&](auto hd_) {
        if (four && vec) return go(hd_, std::integral_constant<int, 4>{}, std::true_type{});
        if (four) return go(hd_, std::integral_constant<int, 4>{}, std::false_type{});
        if (vec) return go(hd_, std::integral_constant<int, 1>{}, std::true_type{});
        return go(hd_, std::integral_constant<int, 1>{}, std::false_type{});
    };
    if (hd == 128) return pick(std::integral_constant<int, 128>{});
    if (hd == 64) return pick(std::integral_constant<int, 64>{});
    return cudaErrorInvalidValue;
}

cudaError_t launch_kv_q4_read(const KvQ4 &c, int hd, const KvQ4Rows &rows, int M, float *k_out, float *v_out,
                              size_t out_row, size_t out_head, bool pdl, cudaStream_t s) {
    if (M <= 0) return cudaSuccess;
    const unsigned threads = static_cast<unsigned>(std::min(256, (c.nkv * (hd / 4) + 31) / 32 * 32));
    const bool vec = aligned16(k_out) && aligned16(v_out) && out_row % 4 == 0 && out_head % 4 == 0;
    const auto kernel = hd == 128 ? (vec ? k_kv_q4_read<128, true> : k_kv_q4_read<128, false>)
                                  : (vec ? k_kv_q4_read<64, true> : k_kv_q4_read<64, false>);
    if (hd != 128 && hd != 64) return cudaErrorInvalidValue;
    return launch_pdl(pdl, kernel, dim3(M), threads, 0, 1, s, c, rows, M, k_out, v_out, out_row, out_head);
}

namespace {

// How a call is split: width class of the columns, column groups; CTAs to a
// unit's cluster and to an SM, or (0) CTAs to deal the blocks to.
struct Q4Plan {
    int W, cgroups, csize = 0, per_sm = 0, ctas;
    bool whole;   // no unit is cut: no workspace, no second kernel
};

Q4Plan q4_plan(int B, int rows, int nh, int nkv, int hd, int max_len) {
    const int cols = nh / nkv * rows;
    Q4Plan p;
    p.W = cols <= 1 ? 1 : cols <= 2 ? 2 : cols <= 4 ? 4 : 8;
    p.cgroups = (cols + p.W - 1) / p.W;
    const int64_t units = static_cast<int64_t>(std::max(B, 1)) * nkv * p.cgroups;
    const int64_t most = std::max<int64_t>(1, (static_cast<int64_t>(max_len) + kQ4Block - 1) / kQ4Block);
    // Clusters while all of them fit at once (against dealing out blocks, with its
    // second kernel: 1 x 517 with 16/8 heads 8.3 us and 13.7, 4 x 8000 with 32/8 19.2
    // and 21.3): with an SM to each CTA, whose threads then have 255 registers (16 x
    // 2000 with 16/8 16.5 us, 18.5 in two CTAs to an SM), else two CTAs to an SM in 128
    // (24 x 500 with 16/8 12.3 us, dealt out 16.4; 36 x 1000 with 32/8 18.9 and 24.4). A
    // warp takes eight tiles at most, five where the clusters leave room for more CTAs
    // (1 x 8317 with 32/8 14.4 us, dealt out 16.4; but 1 x 32000 with 16/8 26.8 in
    // clusters, 22.6 dealt out). The sizes are powers of two; a GPC of 18 or 20 SMs
    // holds one or two clusters of 8 and one of 16 at most.
    constexpr int kFit[2][5] = {{152, 76, 36, 15, 0}, {304, 152, 74, 36, 14}};
    const int64_t need = std::max<int64_t>(1, (static_cast<int64_t>(max_len) + kQ4ClusterWarps * kQ4Tile - 1) / (kQ4ClusterWarps * kQ4Tile));
    for (int per_sm = 1; per_sm <= (p.W <= 4 ? 2 : 1) && !p.csize; ++per_sm) {
        int log2 = 0;
        while (log2 < 4 && (1 << log2) < need && units <= kFit[per_sm - 1][log2 + 1]) ++log2;
        const int64_t tiles = units << log2 >= (per_sm == 1 ? 96 : 240) ? 8 : 5;
        if (units <= kFit[per_sm - 1][log2] && need <= tiles << log2) {
            p.csize = 1 << log2;
            p.per_sm = per_sm;
        }
    }
    // the CTAs that fit at once; for little work two blocks to each
    const int fit = 152 * q4_per_sm(hd, p.W);
    p.ctas = static_cast<int>(std::min<int64_t>(fit, std::max(units, units * ((most + 1) / 2))));
    p.whole = p.csize > 0 || most == 1;
    return p;
}

size_t q4_parts_bytes(const Q4Plan &p, int hd) {
    return (static_cast<size_t>(p.ctas) * 2 * p.W * (hd + 2) * 4 + 15) / 16 * 16;
}

template <int HD, int W>
constexpr size_t q4_attn_smem(int warps) { return static_cast<size_t>(warps) * kQ4Stages * Q4Stage<HD>::bytes; }

template <int HD, int W, int CL>
cudaError_t configure_q4_clusters() {
    cudaError_t e = cudaFuncSetAttribute(k_kv_q4_attn<HD, W, CL>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(q4_attn_smem<HD, W>(kQ4ClusterWarps)));
    if (e == cudaSuccess) e = cudaFuncSetAttribute(k_kv_q4_attn<HD, W, CL>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    return e;
}

template <int HD, int W>
cudaError_t configure_q4_attn() {
    cudaError_t e = configure_q4_clusters<HD, W, 1>();
    if constexpr (W <= 4)
        if (e == cudaSuccess) e = configure_q4_clusters<HD, W, 2>();
    return e;
}

template <int HD, int W, int CL>
cudaError_t launch_q4_clusters(const KvQ4AttnArgs &a, const Q4Plan &p, bool pdl, cudaStream_t s) {
    return launch_pdl(pdl, k_kv_q4_attn<HD, W, CL>, dim3(p.csize, static_cast<unsigned>(a.B) * a.c.nkv * p.cgroups),
                      kQ4ClusterWarps * 32, q4_attn_smem<HD, W>(kQ4ClusterWarps), p.csize, s, a, p.cgroups,
                      static_cast<int2 *>(nullptr));
}

template <int HD, int W>
cudaError_t launch_q4_attn_w(const KvQ4AttnArgs &a, const Q4Plan &p, int2 *owners, bool pdl, cudaStream_t s) {
    static_assert(q4_attn_smem<HD, W>(kQ4Warps) <= 40 * 1024, "fits without an opt-in");
    if (p.per_sm == 1) return launch_q4_clusters<HD, W, 1>(a, p, pdl, s);
    if constexpr (W <= 4)
        if (p.per_sm == 2) return launch_q4_clusters<HD, W, 2>(a, p, pdl, s);
    return launch_pdl(pdl, k_kv_q4_attn<HD, W, 0>, dim3(p.ctas), kQ4Warps * 32, q4_attn_smem<HD, W>(kQ4Warps), 1, s, a,
                      p.cgroups, owners);
}

template <int HD>
cudaError_t launch_q4_attn_hd(const KvQ4AttnArgs &a, const Q4Plan &p, bool pdl, cudaStream_t s) {
    int2 *owners = p.whole ? nullptr : reinterpret_cast<int2 *>(reinterpret_cast<uint8_t *>(a.ws) + q4_parts_bytes(p, HD));
    cudaError_t e = cudaErrorInvalidValue;
    switch (p.W) {
        case 1: e = launch_q4_attn_w<HD, 1>(a, p, owners, pdl, s); break;
        case 2: e = launch_q4_attn_w<HD, 2>(a, p, owners, pdl, s); break;
        case 4: e = launch_q4_attn_w<HD, 4>(a, p, owners, pdl, s); break;
        case 8: e = launch_q4_attn_w<HD, 8>(a, p, owners, pdl, s); break;
    }
    if (e != cudaSuccess || p.whole) return e;
    // a unit's results, eight at a time where there are many: 1 x 100000 with 8/1
    // heads 31 us against 90, 4 x 20000 with 32/8 (14 results) 33 against 36, but 1 x
    // 8000 with 16 rows (5 results) 37 against 35
    const unsigned joins = static_cast<unsigned>(a.nh) * a.rows * a.B;
    const bool many = p.ctas >= 8ll * a.B * a.c.nkv * p.cgroups;
    return launch_pdl(pdl, many ? k_kv_q4_join<HD, 8> : k_kv_q4_join<HD, 1>, dim3(joins), many ? HD * 8 : HD, 0, 1, s, a,
                      p.cgroups, p.W, static_cast<const int2 *>(owners));
}

}  // namespace

cudaError_t configure_kv_q4() {
    cudaError_t e = configure_q4_attn<128, 1>();
    if (e == cudaSuccess) e = configure_q4_attn<128, 2>();
    if (e == cudaSuccess) e = configure_q4_attn<128, 4>();
    if (e == cudaSuccess) e = configure_q4_attn<128, 8>();
    if (e == cudaSuccess) e = configure_q4_attn<64, 1>();
    if (e == cudaSuccess) e = configure_q4_attn<64, 2>();
    if (e == cudaSuccess) e = configure_q4_attn<64, 4>();
    if (e == cudaSuccess) e = configure_q4_attn<64, 8>();
    return e;
}

int kv_q4_attn_launches(int B, int rows, int nh, int nkv, int hd, int max_len) {
    return q4_plan(B, rows, nh, nkv, hd, max_len).whole ? 1 : 2;
}

size_t kv_q4_attn_workspace_bytes(int B, int rows, int nh, int nkv, int hd, int max_len) {
    const Q4Plan p = q4_plan(B, rows, nh, nkv, hd, max_len);
    return p.whole ? 0 : q4_parts_bytes(p, hd) + static_cast<size_t>(B) * nkv * p.cgroups * sizeof(int2);
}

cudaError_t launch_kv_q4_attn(const KvQ4AttnArgs &a, int hd, bool pdl, cudaStream_t s) {
    if (a.B <= 0) return cudaSuccess;
    const Q4Plan p = q4_plan(a.B, a.rows, a.nh, a.c.nkv, hd, a.max_len);
    if (hd == 128) return launch_q4_attn_hd<128>(a, p, pdl, s);
    if (hd == 64) return launch_q4_attn_hd<64>(a, p, pdl, s);
    return cudaErrorInvalidValue;
}

}  // namespace qw3
