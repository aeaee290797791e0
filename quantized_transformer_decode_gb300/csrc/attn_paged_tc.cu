// Attention of many rows over the paged cache on the 5th-generation tensor
// cores: prompts, and chunks of prompts behind a cached context.
//
// Rows are packed: the G query heads that read one kv head and consecutive
// tokens of one sequence fill a tile of 128 rows (row r: token r / G, head
// r % G), so that each K and V tile is used by all of them. A CTA takes a unit
// (one kv head and f16: two row tiles, f32: one) and walks the key tiles of 128
// positions that some row sees.
//
//   S = Q K^T   tcgen05.mma, both operands from shared memory (128-byte swizzle)
//   P = 2^(S c - ref)   a thread to a row: S from tensor memory, P back over it
//   O += P V    tcgen05.mma, P from tensor memory, V as it lies (MN-major)
//
// Roles: three warps load K and V tiles by TMA (a box to a page) into a ring, a warp
// issues the products, two warpgroups do the softmax, so that one is at work
// while the tensor cores serve the other.
//  * f16 activations: the warpgroups have a row tile each and share the key
//    tiles. O stays in tensor memory; a row's reference maximum moves only when
//    it is passed by 2^8, and the row is then rescaled in place. P is rounded to
//    f16, once (an operand of the product with V has V's type; what it adds, 2^-11
//    of a weight at most, is less than what the output's own rounding to f16 does:
//    2.6e-4 of 64 bits in all, 2.0e-4 with P in 32 bits). Sums of P are of the
//    weights before it.
//  * f32 activations: Q and P in two f16 parts (hi + lo), two products each. The
//    warpgroups take alternate key tiles of the same rows, and each adds its
//    tile's O to a master in registers (f32, round to nearest): the tensor core
//    truncates its sums, a relative 1.6e-8 for every step of a chain, and a chain
//    of one tile has 16. The low parts' products come first, while the sum is small
//    (the other way round outputs are twice as far from 64 bits: 1.2e-6 instead of
//    0.57e-6 for 3 x 946 rows with a window of 1208). The two masters are joined at
//    the end.
//
// What a row does not see must not reach it, and 0 * NaN would: in a tile that
// is not seen whole, V rows that no row of the unit sees are set to zero, and if
// one that only some rows see is not finite the unit is done again without
// matrix products (rw_slow); in f32 also where one that is seen has made a NaN of
// two infinite parts.
//
// CTAs stay and take the units to and fro, longest first; the next unit's Q comes
// by TMA while the last one's rows go out by TMA. Few units are split along the
// keys and joined by a second kernel.
//
// Bound by the tensor cores, and nearly as much by shared memory, which holds both
// operands of the first product and one of the second: a 128 x 128 x 16 product
// takes 83 cycles (plain library products 79, the peak rate 64). A prompt of 4096
// tokens with 32 query and 8 kv heads of 128, f16: 105 us, 1.31 PFLOP/s; f32 (twice
// the products): 222 us. 509 rows behind 7680 positions, f32 (128 units on 152 SMs):
// 99 us.
#include <algorithm>
#include <cstdint>

#include <cuda.h>

#include "qw3_internal.cuh"

namespace qw3 {

namespace {

constexpr int kRwThreads = 384;
constexpr int kRwKeys = 128, kRwRows = 128;
constexpr float kRwOff16 = 6.0f, kRwLazy = 8.0f, kRwOff32 = 14.0f;

template <typename T, int HD>
struct RwSizes {
    static constexpr bool split = sizeof(T) == 4;
    static constexpr int QT = split ? 1 : 2;                       // row tiles of a unit
    static constexpr uint32_t tile = kRwRows * HD * 2;             // bytes of a row tile, a K tile, a V tile
    // f16: rows go out through a place of their own (per warpgroup 128 bytes of each row), so that the next unit's Q
    // comes while this one ends; f32: through Q's
    static constexpr int stages = HD == 128 ? (split ? 5 : 4) : 8;
    static constexpr uint32_t out = split ? 0 : kRwRows * 128;
    static constexpr uint32_t smem = 2 * tile + stages * tile + 2 * out + 1024;
    // a warpgroup's part in the workspace: [HD outputs, maximum, sum][128 rows] floats, so that a warp's rows are written
    // and read side by side; two of them to a unit's part (f16: of its row tiles, f32: of its warpgroups)
    static constexpr int part = (HD + 2) * kRwRows;
    // P goes to the products in parts, so that these begin before the last exponentials are there
    static constexpr int parts = 2, part_keys = kRwKeys / parts;
};

struct RwUnit {
    int seq, start, tok0, n, p0;   // token tok0 + k of the sequence's n rows is at p0 + tok0 + k
};

// What the join needs of a unit.
struct RwCut {
    int start, tokens, parts, unused;
};

struct RwArgs {
    KvPagedAttnArgs a;
    int G, TT;          // query heads of a kv head, tokens of a row tile
    int g_inv;          // ceil(2^16 / G): x / G = x g_inv >> 16 for x < 128 (G <= 16: the error x (g_inv - 2^16 / G) 2^-16 is below 1 / G)
    int min_cols;       // sequences with as many columns, or fewer, are others'
    int split_tiles;    // key tiles of a part
    int splits, units;  // parts of a unit, and units, at most
    float *ws;
};

__device__ __forceinline__ float rw_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t rw_pack(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float2 rw_unpack(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2 *>(&v)); }

__device__ __forceinline__ void rw_ld32(uint32_t at, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(at)
        : "memory");
}
__device__ __forceinline__ void rw_st32(uint32_t at, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
        ::"r"(at), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
          "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
          "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
          "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void rw_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void rw_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void rw_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void rw_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void rw_commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// One lane of the warp, the same each time.
__device__ __forceinline__ bool rw_elect() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// Shared-memory operand with a 128-byte swizzle: K-major (rows of 128 bytes, 8-row
// groups 1024 bytes apart) or MN-major (8-row groups along K 1024 bytes apart, 64
// columns of N `lbo` bytes apart). at16: the address in 16-byte words.
__device__ __forceinline__ uint64_t rw_desc(uint32_t at16, uint32_t lbo) {
    constexpr uint32_t hi = (1024u >> 4) | (1u << 14) | (2u << 29);
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(at16 | (lbo >> 4) << 16), "r"(hi));
    return d;
}
// kind::f16, f16 operands, f32 sums; B K-major or MN-major.
__host__ __device__ constexpr uint32_t rw_idesc(int N, bool b_mn) {
    return (1u << 4) | (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(kRwRows >> 4) << 24);
}
__device__ __forceinline__ void rw_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                 ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(add)) : "memory");
}
__device__ __forceinline__ void rw_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
                 ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(add)) : "memory");
}
__device__ __forceinline__ void rw_tma(uint32_t to, const CUtensorMap *map, int x, int y, uint64_t *bar) {
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
                 ::"r"(to), "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar)) : "memory");
}
// A bounded wait that gives up with the others: *err is set by the first that ran
// out, and looked at by those that have to wait. A warpgroup that does its rows
// without matrix products may be long about it: the limit counts from the last time
// that it wrote to *beat (Beat: where the wait may be for such a warpgroup).
template <bool Beat>
__device__ __forceinline__ void rw_wait(uint64_t *bar, int parity, volatile int *err, volatile int64_t *beat) {
    if (mbar_try_wait(bar, static_cast<uint32_t>(parity & 1))) return;
    const int64_t t0 = static_cast<int64_t>(globaltimer_ns());
    while (!mbar_try_wait(bar, static_cast<uint32_t>(parity & 1))) {
        if (*err) return;
        const int64_t since = Beat ? max(t0, *beat) : t0;
        if (static_cast<int64_t>(globaltimer_ns()) - since > static_cast<int64_t>(kWaitLimitNs)) *err = 1;
    }
}
__device__ __forceinline__ void rw_tma3(uint32_t to, const CUtensorMap *map, int x, int y, int z, uint64_t *bar) {
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
                 ::"r"(to), "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void rw_tma3_out(const CUtensorMap *map, int x, int y, int z, uint32_t from) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];"
                 ::"l"(map), "r"(x), "r"(y), "r"(z), "r"(from) : "memory");
}
__device__ __forceinline__ void rw_out_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void rw_out_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }   // its source may change
__device__ __forceinline__ void rw_out_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void rw_bar(int id) { asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(N) : "memory"); }

// The key tiles of rows at pmin .. pmax: tile i is key tile i < sink ? i : i - sink + first.
struct RwTiles {
    int sink, first, n;
    __device__ __forceinline__ int key(int i) const { return (i < sink ? i : i - sink + first) * kRwKeys; }
};
__device__ __forceinline__ RwTiles rw_tiles(int pmin, int pmax, int window, int sinks) {
    RwTiles t;
    const int lo = window > 0 ? max(0, pmin - window + 1) : 0;
    t.first = lo / kRwKeys;
    t.sink = window > 0 ? min((min(sinks, lo) + kRwKeys - 1) / kRwKeys, t.first) : 0;
    t.n = pmax < 0 ? 0 : t.sink + pmax / kRwKeys - t.first + 1;
    return t;
}

// Rows row0 .. row1 - 1 of the unit without matrix products, for the tiles i0 .. i1
// - 1: warp `warp` of `warps`, a row at a time. Scores: a lane to a position, which
// reads its K row whole, 32 at once; outputs: a lane to E dimensions, 16 V rows on
// their way. dst: the part, or null for the output. *beat is the time of the last tile
// of a row (the other roles' waits count from it). Bound by the latency of its loads:
// 509 rows behind 7680 positions, 32/8 heads, f32, every unit: 23 ms; 256 rows x 98
// thousand positions 0.37 s (a position at a time, a lane to E dimensions for the
// scores too: 4.5 times as long).
template <typename T, int HD>
__device__ __noinline__ void rw_slow(const RwArgs &r, const RwUnit &u, const RwTiles &t, int i0, int i1, int g, int row0, int row1,
                                     int warp, int warps, float off, float *dst, volatile int64_t *beat) {
    constexpr int E = HD / 32;
    const int lane = threadIdx.x & 31;
    const KvPagedAttnArgs &a = r.a;
    for (int row = row0 + warp; row < row1; row += warps) {
        const int tok = row / kRwRows * r.TT + row % kRwRows / r.G, h = g * r.G + row % kRwRows % r.G;
        if (row % kRwRows >= r.TT * r.G || u.tok0 + tok >= u.n) continue;
        const int p = u.p0 + u.tok0 + tok;
        const size_t at = static_cast<size_t>(u.start + u.tok0 + tok);
        const T *q = static_cast<const T *>(a.q) + at * a.q_stride + static_cast<size_t>(h) * HD + lane * E;
        float x[E], o[E], m = -INFINITY, l = 0.0f;   // (l: of this lane's positions)
#pragma unroll
        for (int e = 0; e < E; ++e) {
            x[e] = kv_f32(q[e]) * (a.scale * 1.4426950408889634f);   // (before the sum, which large queries would take out of f32)
            o[e] = 0.0f;
        }
        for (int i = i0; i < i1; ++i) {
            if (lane == 0) *beat = static_cast<int64_t>(globaltimer_ns());
            const int end = min(t.key(i) + kRwKeys - 1, p);
#pragma unroll 1
            for (int j0 = t.key(i); j0 <= end; j0 += 32) {
                const int j = j0 + lane, page = j <= end ? kv_page(a.b, a.c, u.seq, j) : -1;
                const bool sees = page >= 0 && kv_sees(p, j, a.window, a.sinks);
                const uint32_t seen = __ballot_sync(0xffffffffu, sees);
                if (seen == 0) continue;
                const __half *k = kv_paged_row<HD>(a.c, max(page, 0), 0, g, j);
                float d = 0.0f;
#pragma unroll 4
                for (int c = 0; c < HD; c += 8) {
                    const uint4 y = sees ? *reinterpret_cast<const uint4 *>(k + c) : make_uint4(0, 0, 0, 0);
                    const uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 f = rw_unpack(w[e]);
                        d = fmaf(__shfl_sync(0xffffffffu, x[2 * e % E], (c + 2 * e) / E), f.x, d);
                        d = fmaf(__shfl_sync(0xffffffffu, x[(2 * e + 1) % E], (c + 2 * e + 1) / E), f.y, d);
                    }
                }
                const float mn = fmaxf(m, warp_max(sees ? d : -INFINITY)), c = m == mn ? 1.0f : rw_ex2(m - mn);
                const float w = sees ? rw_ex2(d - mn + off) : 0.0f;
                m = mn;
                l = fmaf(l, c, w);
#pragma unroll
                for (int e = 0; e < E; ++e) o[e] *= c;
#pragma unroll 1
                for (int n0 = 0; n0 < 32; n0 += 16) {   // (16 positions lie in one page)
                    const int pg = __shfl_sync(0xffffffffu, page, n0);
                    if ((seen >> n0 & 0xffffu) == 0) continue;
                    const __half *v = kv_paged_row<HD>(a.c, max(pg, 0), 1, g, j0 + n0) + lane * E;
#pragma unroll
                    for (int n = 0; n < 16; ++n) {
                        float y[E];
                        if constexpr (E == 4) {
                            const uint2 b = *reinterpret_cast<const uint2 *>(v + n * HD);
                            const float2 f = rw_unpack(b.x), s = rw_unpack(b.y);
                            y[0] = f.x; y[1] = f.y; y[2] = s.x; y[3] = s.y;
                        } else {
                            const float2 f = rw_unpack(*reinterpret_cast<const uint32_t *>(v + n * HD));
                            y[0] = f.x; y[1] = f.y;
                        }
                        const float wn = __shfl_sync(0xffffffffu, w, n0 + n);
#pragma unroll
                        for (int e = 0; e < E; ++e) o[e] = seen >> (n0 + n) & 1 ? fmaf(wn, y[e], o[e]) : o[e];   // (whatever y is)
                    }
                }
            }
        }
        l = warp_sum(l);
        if (dst) {
            float *to = dst + row % kRwRows;
#pragma unroll
            for (int e = 0; e < E; ++e) to[(lane * E + e) * kRwRows] = o[e];
            if (lane == 0) {
                to[HD * kRwRows] = m;
                to[(HD + 1) * kRwRows] = l;
            }
        } else {
            T *to = static_cast<T *>(a.out) + at * a.out_stride + static_cast<size_t>(h) * HD + lane * E;
#pragma unroll
            for (int e = 0; e < E; ++e) to[e] = kv_cvt<T>(l == 0.0f ? 0.0f : o[e] / l);
        }
    }
}

// The units in order: numbers that grow from call to call, so the sequences are
// walked through once. A warp's lanes look at 32 of them; all lanes call it.
struct RwFind {
    int b0 = 0, before = 0;
};
template <typename T, int HD>
__device__ __forceinline__ bool rw_find(const RwArgs &r, int pair, RwFind &f, RwUnit &u) {
    const int lane = threadIdx.x & 31, UT = r.TT * RwSizes<T, HD>::QT;
    for (; f.b0 < r.a.b.B; f.b0 += 32) {
        const int b = f.b0 + lane;
        KvSeq q{0, 0, 0};
        int mine = 0;
        if (b < r.a.b.B) {
            q = kv_seq(r.a.b, b);
            if (q.n * r.G > r.min_cols) mine = (q.n + UT - 1) / UT;
        }
        int upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += v;
        }
        const int at = f.before + upto - mine, all = __shfl_sync(0xffffffffu, upto, 31);
        if (pair < f.before + all) {
            const int who = __ffs(__ballot_sync(0xffffffffu, pair >= at && pair < at + mine)) - 1;
            // a sequence's last (longest) unit first
            const int tok0 = (mine - 1 - (pair - at)) * UT;
            u = RwUnit{f.b0 + who, __shfl_sync(0xffffffffu, q.start, who), __shfl_sync(0xffffffffu, tok0, who),
                       __shfl_sync(0xffffffffu, q.n, who), __shfl_sync(0xffffffffu, q.p0, who)};
            return true;
        }
        f.before += all;
    }
    return false;
}

// A part of a unit, as every role of a CTA sees it.
struct RwItem {
    RwUnit u;
    RwTiles tiles;
    int g, tokens, pmin, pmax, i0, NT, parts, part, unit;
};

template <typename T, int HD>
__global__ void __launch_bounds__(kRwThreads, 1)
    k_paged_rows(const RwArgs r, const __grid_constant__ CUtensorMap map, const __grid_constant__ CUtensorMap qmap,
                 const __grid_constant__ CUtensorMap omap) {
    using Z = RwSizes<T, HD>;
    constexpr int ST = Z::stages, QT = Z::QT;
    extern __shared__ uint8_t rw_smem[];
    __shared__ uint64_t b_full[ST], b_empty[ST], b_s[2], b_p[2][Z::parts], b_o[2], b_q, b_q_free, b_end;
    __shared__ uint32_t s_tmem;
    __shared__ int64_t s_beat;
    __shared__ int s_err, s_bad[2][3];
    __shared__ float s_c[kRwRows];
    const KvPagedAttnArgs &a = r.a;
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);   // (known to be the warp's own: uniform branches)
    const uint32_t base = (smem_u32(rw_smem) + 1023) & ~1023u;
    uint8_t *const smem = rw_smem + (base - smem_u32(rw_smem));
    if (tid == 0) {
        for (int i = 0; i < ST; ++i) {
            mbar_init(&b_full[i], 1);
            mbar_init(&b_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&b_s[i], 1);
            for (int k = 0; k < Z::parts; ++k) mbar_init(&b_p[i][k], 128);
            mbar_init(&b_o[i], 1);
            for (int k = 0; k < 3; ++k) s_bad[i][k] = 0;
        }
        mbar_init(&b_q, Z::split ? 256 : 1);
        mbar_init(&b_q_free, 1);
        mbar_init(&b_end, 1);
        fence_mbar_init();
        s_err = 0;
        s_beat = 0;
    }
    if (warp == 9) {   // (nothing else holds tensor memory here: no two of these CTAs fit an SM)
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)), "r"(512) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        rw_before();
    }
    __syncthreads();
    rw_after();
    const uint32_t tmem = s_tmem;
    pdl_wait();
    pdl_trigger();   // (after the wait: what is launched next may begin beside this kernel, and needs what came before it)

    // a negative scale is taken into the scores' sign, so that they are scaled by c > 0
    const float sign = a.scale < 0.0f ? -1.0f : a.scale == 0.0f ? 0.0f : 1.0f;
    const float c0 = a.scale == 0.0f ? 1.0f : fabsf(a.scale) * 1.4426950408889634f;
    const uint32_t ring = base + 2 * Z::tile;
    volatile int *err = &s_err;
    auto wait = [&](uint64_t *bar, int parity) { rw_wait<false>(bar, parity, err, &s_beat); };
    // for what a warpgroup without matrix products may hold up: in f16 its P, and with it the other one; in f32, where both go
    // that way together, the next Q; the ring's places
    auto wait_long = [&](uint64_t *bar, int parity) { rw_wait<true>(bar, parity, err, &s_beat); };
    RwCut *const cuts = reinterpret_cast<RwCut *>(r.ws);
    // Item k of this CTA: the items (parts of units, long ones first) go to the CTAs to and fro, so that the lengths
    // add up to about the same. Every role walks through them by itself; false behind the last one.
    const int items = r.units * r.splits;
    auto number = [&](int k) { return k * static_cast<int>(gridDim.x) + (k & 1 ? static_cast<int>(gridDim.x - 1 - blockIdx.x) : static_cast<int>(blockIdx.x)); };
    auto item = [&](int k, RwFind &f, RwItem &it) {
        const int w = number(k);
        if (w >= items) return false;
        it.unit = w / r.splits;
        it.part = w % r.splits;
        it.g = it.unit % a.c.nkv;
        if (!rw_find<T, HD>(r, it.unit / a.c.nkv, f, it.u)) return false;
        it.tokens = min(r.TT * QT, it.u.n - it.u.tok0);
        it.pmin = it.u.p0 + it.u.tok0;
        it.pmax = it.pmin + it.tokens - 1;
        it.tiles = rw_tiles(it.pmin, it.pmax, a.window, a.sinks);
        it.parts = max(1, (it.tiles.n + r.split_tiles - 1) / r.split_tiles);
        it.i0 = it.part * r.split_tiles;
        it.NT = max(0, min(it.tiles.n, it.i0 + r.split_tiles) - it.i0);
        return true;
    };
    // fill n of an item's in the ring: its key tile, and whether it is V
    auto fill = [](int n, int NT, int &i, bool &v) {
        if constexpr (!Z::split) {   // K0 V0 K1 V1 ..
            v = n & 1;
            i = n >> 1;
        } else {                     // K0 K1 V0 K2 V1 .. (the order of the products)
            v = n == 2 * NT - 1 || (n >= 2 && !(n & 1));
            i = n == 2 * NT - 1 ? NT - 1 : v ? (n - 2) >> 1 : (n + 1) >> 1;
        }
    };
    auto fill_of_k = [](int i) { return Z::split ? max(0, 2 * i - 1) : 2 * i; };
    auto fill_of_v = [](int i, int NT) { return Z::split ? min(2 * i + 2, 2 * NT - 1) : 2 * i + 1; };

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        RwFind f;
        RwItem it;
        if (warp != 9) {
            // ---- loads: three warps take turns, a lane to a page of the tile; the first one sees to Q, and at last to the cuts
            const int turn = warp == 8 ? 0 : warp - 9;
            const int shift = min(a.c.shift, 7), boxes = kRwKeys >> shift;
            const uint32_t bytes = static_cast<uint32_t>(HD * 2) << shift;
            int done = 0, nq = 0;   // fills, and Qs, of the items before
            bool ok = true;
            for (int k = 0; ok && item(k, f, it); ++k) {
                if (it.NT == 0) continue;
                if (!Z::split && turn == 0) {
                    if (nq > 0) wait_long(&b_q_free, nq - 1);
                    if (__any_sync(0xffffffffu, *err != 0)) {
                        ok = false;
                        break;
                    }
                    if (lane == 0) {
                        const int two = it.tokens > r.TT ? 2 : 1;
                        mbar_arrive_expect_tx(&b_q, two * (HD * 2) * r.G * r.TT);
                        for (int s = 0; s < two; ++s)
#pragma unroll
                            for (int h = 0; h < HD / 64; ++h)
                                rw_tma3(base + s * Z::tile + h * (kRwRows * 128), &qmap, h * 64, it.g * r.G,
                                        it.u.start + it.u.tok0 + s * r.TT, &b_q);
                    }
                    __syncwarp();
                    ++nq;
                }
                // the fills of this item that are this warp's: those whose number among all is `turn` modulo 3
                for (int n = (turn + 3 - done % 3) % 3; n < 2 * it.NT; n += 3) {
                    const int all = done + n, st = all % ST;
                    int i;
                    bool v;
                    fill(n, it.NT, i, v);
                    const int j = it.tiles.key(it.i0 + i) + (lane << shift);
                    const int page = lane < boxes && j <= it.pmax ? kv_page(a.b, a.c, it.u.seq, j) : -1;
                    if (all >= ST) wait_long(&b_empty[st], all / ST - 1);
                    if (__any_sync(0xffffffffu, *err != 0)) {
                        ok = false;
                        break;
                    }
                    const int held = __popc(__ballot_sync(0xffffffffu, page >= 0));
                    if (lane == 0) mbar_arrive_expect_tx(&b_full[st], held * bytes);
                    __syncwarp();
                    if (page >= 0) {
                        const int y = (((page * 2 + v) * a.c.nkv + it.g) << a.c.shift) + (j & ((1 << a.c.shift) - 1));
                        const uint32_t to = ring + st * Z::tile + (static_cast<uint32_t>(lane) << shift) * 128;
#pragma unroll
                        for (int h = 0; h < HD / 64; ++h) rw_tma(to + h * (kRwKeys * 128), &map, h * 64, y, &b_full[st]);
                    }
                }
                if (ok) done += 2 * it.NT;
            }
            // the cuts, of units that are not there too: all of them, whatever has become of the loads, because the join
            // goes by them
            if (turn == 0 && r.splits > 1) {
                RwFind all;
                int k = 0;
                for (; item(k, all, it); ++k)
                    if (lane == 0 && it.part == 0) cuts[it.unit] = RwCut{it.u.start + it.u.tok0, it.tokens, it.parts, 0};
                for (; number(k) < items; ++k)
                    if (lane == 0 && number(k) % r.splits == 0) cuts[number(k) / r.splits] = RwCut{0, 0, 0, 0};
            }
            // the CTA may end when every copy has landed, and every stage has been released
            if (ok) {
                for (int n = max(0, done - ST); n < done; ++n)
                    if (n % 3 == turn) wait_long(&b_empty[n % ST], n / ST);
            }
        } else {
            // ---- products: the whole warp walks along, one lane issues
            const uint32_t ring16 = (ring & 0x3FFFFu) >> 4, base16 = (base & 0x3FFFFu) >> 4;
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            const bool one = rw_elect();
            int done = 0, nq = 0, np[2] = {0, 0};   // fills, Qs, and tiles of P, of the items before
            auto release = [&](int n) {
                if (one) rw_commit(&b_empty[(done + n) % ST]);
            };
            auto qk = [&](int s, int i) {
                const int n = done + fill_of_k(i), st = n % ST;
                wait(&b_full[st], n / ST);
                rw_after();
                const uint32_t k = ring16 + st * (Z::tile >> 4), q = base16 + (QT == 2 ? s * (Z::tile >> 4) : 0);
                if (one) {
                    // f32: the low parts first
                    constexpr int parts = Z::split ? 2 : 1;
#pragma unroll
                    for (int h = parts - 1; h >= 0; --h)
#pragma unroll
                        for (int e = 0; e < HD / 16; ++e) {
                            const uint32_t at = (e >> 2) * (kRwRows * 128 >> 4) + (e & 3) * 2;
                            rw_mma_ss(tm + s * 128, rw_desc(q + h * (Z::tile >> 4) + at, 16), rw_desc(k + at, 16),
                                      rw_idesc(kRwKeys, false), e > 0 || h < parts - 1);
                        }
                    rw_commit(&b_s[s]);
                }
            };
            auto pv = [&](int s, int i, bool add) {
                const int n = done + fill_of_v(i, it.NT), st = n % ST;
                wait(&b_full[st], n / ST);
                const uint32_t v = ring16 + st * (Z::tile >> 4), p = tm + s * 128;
#pragma unroll
                for (int k = 0; k < Z::parts; ++k) {   // as the parts of P come
                    rw_wait<!Z::split>(&b_p[s][k], np[s], err, &s_beat);
                    rw_after();
                    if (one) {
#pragma unroll
                        for (int lo = Z::split ? 1 : 0; lo >= 0; --lo)
#pragma unroll
                            for (int ee = 0; ee < Z::part_keys / 16; ++ee) {
                                const int e = k * (Z::part_keys / 16) + ee;
                                // P: f16 [64 columns]; f32: hi and lo of 32 keys next to each other, 16 columns each (low parts first here too)
                                const uint32_t at = p + (Z::split ? (e >> 1) * 32 + (e & 1) * 8 + lo * 16 : e * 8);
                                rw_mma_ts(tm + 256 + s * HD, at, rw_desc(v + e * (2048 >> 4), kRwKeys * 128), rw_idesc(HD, true),
                                          add || e > 0 || (Z::split && lo == 0));
                            }
                    }
                }
                ++np[s];
            };
            auto commit = [&](uint64_t *bar) {
                if (one) rw_commit(bar);
            };
            for (int k = 0; item(k, f, it); ++k) {
                const int NT = it.NT;
                if (NT == 0) continue;
                if (*err) break;
                rw_wait<Z::split>(&b_q, nq++, err, &s_beat);
                if constexpr (!Z::split) {
                    const int two = it.tokens > r.TT ? 2 : 1;
                    for (int s = 0; s < two; ++s) qk(s, 0);
                    if (NT == 1) commit(&b_q_free);
                    release(0);
                    for (int i = 0; i < NT; ++i) {
                        for (int s = 0; s < two; ++s) {
                            pv(s, i, i > 0);
                            if (i + 1 < NT) qk(s, i + 1);
                            else commit(&b_o[s]);
                        }
                        if (i + 2 == NT) commit(&b_q_free);   // (its last scores)
                        release(fill_of_v(i, NT));
                        if (i + 1 < NT) release(fill_of_k(i + 1));
                    }
                } else {
                    for (int i = 0; i < min(2, NT); ++i) {
                        qk(i, i);
                        release(fill_of_k(i));
                    }
                    for (int i = 0; i < NT; ++i) {
                        pv(i & 1, i, false);
                        release(fill_of_v(i, NT));
                        if (i + 2 < NT) {
                            qk(i & 1, i + 2);
                            release(fill_of_k(i + 2));
                        } else {
                            commit(&b_o[i & 1]);
                        }
                    }
                }
                done += 2 * NT;
            }
        }
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        // ---- softmax: warpgroup s, a thread to a row
        const int s = warp >> 2, rr = tid & 127;
        const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
        const uint32_t tS = tmem + lanes + s * 128, tO = tmem + lanes + 256 + s * HD;
        constexpr float kOff = Z::split ? kRwOff32 : kRwOff16;
        constexpr int kStep = Z::split ? 2 : 1;
        auto wait = [&](uint64_t *bar, int parity) { rw_wait<!Z::split>(bar, parity, err, &s_beat); };
        RwFind f;
        RwItem it;
        int done = 0, ns = 0, no = 0;   // fills, tiles of S, outputs, of the items before
        int turn = 0;                   // this item's flag
        int k = 0;
        auto next = [&](RwItem &to) {   // the next item that has a part of its unit
            while (item(k++, f, to))
                if (to.part < to.parts) return true;
            return false;
        };
        RwItem ahead;
        bool more = next(ahead);
        while (more) {
            it = ahead;
            const int NT = it.NT, tokens = it.tokens, pmin = it.pmin, pmax = it.pmax;
            // (an error ends the waits, not this loop: the barriers below need every thread)
            int *const bad_flag = &s_bad[Z::split ? 0 : s][turn];
            const int turn_next = turn == 2 ? 0 : turn + 1;
            turn = turn_next;
            float *const dst = it.parts == 1 ? nullptr
                                             : r.ws + static_cast<size_t>(r.units) * 4 +
                                                   ((static_cast<size_t>(it.unit) * r.splits + it.part) * 2 + s) * Z::part;
            // the output of row x of a row tile, or null
            const size_t out_row = static_cast<size_t>(a.out_stride);
            T *const out0 = static_cast<T *>(a.out) + static_cast<size_t>(it.u.start + it.u.tok0) * out_row + static_cast<size_t>(it.g * r.G) * HD;
            auto row_of = [&](int x, int tile) {
                const int tx = x * r.g_inv >> 16, tk = (QT == 2 ? tile * r.TT : 0) + tx;
                return x < r.TT * r.G && tk < tokens ? out0 + tk * out_row + (x - tx * r.G) * HD : nullptr;
            };
            if constexpr (Z::split) {
                // ---- Q to shared memory: L lanes to a row, PW rows to a warp at once, all loads before the stores
                constexpr int L = HD / 8, PW = 32 / L, NB = kRwRows / (8 * PW);
                const int ch = lane % L, row0 = warp * PW + lane / L;
                uint4 x[NB], y[NB];
#pragma unroll
                for (int n = 0; n < NB; ++n) {
                    const int row = row0 + n * 8 * PW, tk = row * r.g_inv >> 16;
                    const bool real = row < r.TT * r.G && tk < tokens;
                    const T *q = static_cast<const T *>(a.q) + static_cast<size_t>(it.u.start + it.u.tok0 + (real ? tk : 0)) * a.q_stride +
                                 static_cast<size_t>(it.g * r.G + (real ? row - tk * r.G : 0)) * HD + ch * 8;
                    x[n] = real ? *reinterpret_cast<const uint4 *>(q) : make_uint4(0, 0, 0, 0);
                    y[n] = real ? *reinterpret_cast<const uint4 *>(q + 4) : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int n = 0; n < NB; ++n) {
                    const int row = row0 + n * 8 * PW;
                    uint8_t *to = smem + (ch >> 3) * (kRwRows * 128) + row * 128 + (((ch & 7) ^ (row & 7)) << 4);
                    float v[8] = {__uint_as_float(x[n].x), __uint_as_float(x[n].y), __uint_as_float(x[n].z), __uint_as_float(x[n].w),
                                  __uint_as_float(y[n].x), __uint_as_float(y[n].y), __uint_as_float(y[n].z), __uint_as_float(y[n].w)};
                    float amax = 0.0f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(v[e]));
#pragma unroll
                    for (int o = L / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                    // the power of two that takes the row's largest into [2^14, 2^15)
                    const int ex = min(126, 14 + 127 - static_cast<int>(__float_as_uint(amax) >> 23 & 0xffu));
                    const float up = pow2_f32(ex) * sign;
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] *= up;
                    uint4 hi, lo;
                    split8_f16(v, hi, lo);
                    *reinterpret_cast<uint4 *>(to) = hi;
                    *reinterpret_cast<uint4 *>(to + Z::tile) = lo;
                    // (never 0: -inf times it has to stay -inf. At 2^-126 every score is 0 to the last bit: they are below 2^38.)
                    if (ch == 0) s_c[row] = fmaxf(pow2_f32(-ex) * c0, 0x1p-126f);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                if (NT > 0) mbar_arrive(&b_q);
                rw_bar<256>(1);   // (s_c)
            }
            const int tok = (QT == 2 ? s * r.TT : 0) + (rr * r.g_inv >> 16);
            const int p = pmin + min(tok, tokens - 1);
            // the rows of this warpgroup's tile
            const int smin = QT == 2 ? min(pmin + s * r.TT, pmax) : pmin, smax = QT == 2 ? min(smin + r.TT - 1, pmax) : pmax;
            const float c = Z::split ? s_c[rr] : c0;
            float m = -INFINITY, l = 0.0f;   // reference (a score before c), sum of weights
            float master[Z::split ? HD : 1];
            if constexpr (Z::split) {
#pragma unroll
                for (int d = 0; d < HD; ++d) master[d] = 0.0f;
            }
            const bool active = QT == 1 || s == 0 || tokens > r.TT;
            // which 16 positions of a tile have a page (lanes 0..7 look, a tile ahead)
            auto look = [&](int i) {
                const int j = it.tiles.key(it.i0 + i) + 16 * (lane & 7);
                return j > pmax || kv_page(a.b, a.c, it.u.seq, j) >= 0;
            };
            const int first = Z::split ? s : 0;
            bool there = active && NT > first && look(first);
            int own = 0;   // tiles taken
            for (int i = first; active && i < NT; i += kStep, ++own) {
                const int j0 = it.tiles.key(it.i0 + i);
                const uint32_t pages = __ballot_sync(0xffffffffu, there) & 0xffu;
                const bool holes = pages != 0xffu;
                if (i + kStep < NT) there = look(i + kStep);
                // does every row of the tile see every position?
                const bool open = !holes && j0 + kRwKeys - 1 <= smin && (a.window == 0 || smax - j0 < a.window || j0 + kRwKeys <= a.sinks);
                wait(&b_s[s], ns + own);
                rw_after();
                if (!open) {
                    // V: this thread's position. (Behind the wait for the scores: they say that every fill before their K
                    // has come, and only then does the parity of V's barrier tell this fill from the one before the last.)
                    const int n = done + fill_of_v(i, NT), st = n % ST, j = j0 + rr;
                    const bool page = pages >> (rr >> 4) & 1;
                    const bool any = page && j <= pmax && kv_sees(max(j, pmin), j, a.window, a.sinks);
                    const bool all = page && j <= smin && kv_sees(smax, j, a.window, a.sinks);
                    wait(&b_full[st], n / ST);
                    uint8_t *v = smem + (2 + st) * Z::tile + rr * 128;
                    bool bad = false;
                    if (!all) {
#pragma unroll
                        for (int h = 0; h < HD / 64; ++h)
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                uint4 *at = reinterpret_cast<uint4 *>(v + h * (kRwKeys * 128) + ((e ^ (lane & 7)) << 4));
                                if (!any) {
                                    *at = make_uint4(0, 0, 0, 0);
                                } else {
                                    const uint4 x = *at;
                                    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                                    for (int q = 0; q < 4; ++q) bad |= (w[q] & 0x7c00u) == 0x7c00u || (w[q] & 0x7c000000u) == 0x7c000000u;
                                }
                            }
                    }
                    if (bad) *bad_flag = 1;
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                }
                // the row's positions j0 + k, k in [k_lo, k_hi) or [0, k_sink), of pages that are there: bits of 32 positions
                const int k_hi = p - j0 + 1, k_lo = a.window > 0 ? p - a.window + 1 - j0 : 0, k_sink = a.window > 0 ? a.sinks - j0 : 0;
                auto below = [](int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1; };
                auto sees = [&](int k0) {
                    const uint32_t held = (pages >> (k0 >> 4) & 1 ? 0xffffu : 0u) | (pages >> ((k0 >> 4) + 1) & 1 ? 0xffff0000u : 0u);
                    return held & below(k_hi - k0) & (~below(k_lo - k0) | below(k_sink - k0));
                };
                if constexpr (!Z::split) {
                    uint32_t v[128];
#pragma unroll
                    for (int q = 0; q < 4; ++q) rw_ld32(tS + 32 * q, v + 32 * q);
                    rw_wait_ld();
                    if (sign != 1.0f) {
#pragma unroll
                        for (int q = 0; q < 128; ++q) v[q] = __float_as_uint(__uint_as_float(v[q]) * sign);
                    }
                    if (!open) {
#pragma unroll
                        for (int k0 = 0; k0 < 128; k0 += 32) {
                            const uint32_t bits = sees(k0);
#pragma unroll
                            for (int q = 0; q < 32; ++q) v[k0 + q] = bits >> q & 1 ? v[k0 + q] : 0xff800000u;
                        }
                    }
                    float mx8[8];   // (chains of their own)
#pragma unroll
                    for (int q = 0; q < 8; ++q) mx8[q] = __uint_as_float(v[q]);
#pragma unroll
                    for (int q = 8; q < 128; ++q) mx8[q & 7] = fmaxf(mx8[q & 7], __uint_as_float(v[q]));
                    const float mx = fmaxf(fmaxf(fmaxf(mx8[0], mx8[1]), fmaxf(mx8[2], mx8[3])), fmaxf(fmaxf(mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7])));
                    const bool far = m == -INFINITY ? mx > -INFINITY : (mx - m) * c > kRwLazy;
                    if (__any_sync(0xffffffffu, far)) {
                        const float mn = far ? mx : m, fac = m == mn ? 1.0f : m == -INFINITY ? 0.0f : rw_ex2((m - mn) * c);
                        m = mn;
                        l *= fac;
                        if (own > 0) {
#pragma unroll 1
                            for (int d = 0; d < HD; d += 32) {
                                uint32_t o[32];
                                rw_ld32(tO + d, o);
                                rw_wait_ld();
#pragma unroll
                                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * fac);
                                rw_st32(tO + d, o);
                            }
                        }
                    }
                    const float b = (m == -INFINITY ? 0.0f : m * c) - kOff;
                    float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int h = 0; h < Z::parts; ++h) {
#pragma unroll
                        for (int kk = 0; kk < Z::part_keys; kk += 2) {
                            const int q = h * Z::part_keys + kk;
                            const float x = rw_ex2(fmaf(__uint_as_float(v[q]), c, -b)), y = rw_ex2(fmaf(__uint_as_float(v[q + 1]), c, -b));
                            sum[q >> 1 & 1] += x;
                            sum[2 + (q >> 1 & 1)] += y;
                            v[q >> 1] = rw_pack(x, y);
                        }
                        rw_st32(tS + 32 * h, v + 32 * h);
                        rw_wait_st();
                        rw_before();
                        mbar_arrive(&b_p[s][h]);
                    }
                    l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                } else {
                    float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int k0 = 0; k0 < 128; k0 += 64) {
                        uint32_t v[64];
                        rw_ld32(tS + k0, v);
                        rw_ld32(tS + k0 + 32, v + 32);
                        rw_wait_ld();
                        if (!open) {   // what the row does not see is -inf from here on
#pragma unroll
                            for (int h = 0; h < 64; h += 32) {
                                const uint32_t bits = sees(k0 + h);
#pragma unroll
                                for (int q = 0; q < 32; ++q) v[h + q] = bits >> q & 1 ? v[h + q] : 0xff800000u;
                                rw_st32(tS + k0 + h, v + h);
                            }
                        }
#pragma unroll
                        for (int q = 0; q < 64; ++q) mx4[q & 3] = fmaxf(mx4[q & 3], __uint_as_float(v[q]));
                    }
                    if (!open) rw_wait_st();
                    const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
                    const float mn = fmaxf(m, mx), fac = m == mn ? 1.0f : rw_ex2((m - mn) * c);
                    // the O of this warpgroup's last tile, beside the old reference
                    if (own > 0) {
#pragma unroll
                        for (int d = 0; d < HD; d += 32) {
                            uint32_t o[32];
                            rw_ld32(tO + d, o);
                            rw_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e) master[d + e] = (master[d + e] + __uint_as_float(o[e])) * fac;
                        }
                    }
                    m = mn;
                    l *= fac;
                    const float b = (m == -INFINITY ? 0.0f : m * c) - kOff;
                    float sum[2] = {0.0f, 0.0f};
#pragma unroll
                    for (int k0 = 0; k0 < 128; k0 += 32) {
                        uint32_t v[32], w[32];
                        rw_ld32(tS + k0, v);
                        rw_wait_ld();
#pragma unroll
                        for (int q = 0; q < 32; q += 2) {
                            const float x = rw_ex2(fmaf(__uint_as_float(v[q]), c, -b)), y = rw_ex2(fmaf(__uint_as_float(v[q + 1]), c, -b));
                            sum[0] += x;
                            sum[1] += y;
                            const uint32_t hi = rw_pack(x, y);
                            const float2 h = rw_unpack(hi);
                            w[q >> 1] = hi;
                            w[16 + (q >> 1)] = rw_pack(x - h.x, y - h.y);
                        }
                        rw_st32(tS + k0, w);
                        if ((k0 + 32) % Z::part_keys == 0) {
                            rw_wait_st();
                            rw_before();
                            mbar_arrive(&b_p[s][k0 / Z::part_keys]);
                        }
                    }
                    l += sum[0] + sum[1];
                }
            }
            more = next(ahead);   // (while the last products are made)
            if (own > 0) {
                wait(&b_o[s], no++);
                rw_after();
            }
            ns += own;
            done += 2 * NT;
            const float m2 = m == -INFINITY ? -INFINITY : m * c;   // the reference in base 2
            // Rows go out through shared memory, 128 bytes of each at a time (chunk c of 16 bytes of row x at c ^ (x & 7),
            // the tensor maps' swizzle): by TMA where the row tile is full, else by the threads. Parts go to the workspace
            // as they are.
            auto copy_out = [&](const uint8_t *place, int tile, int d0, int thread, int threads) {
#pragma unroll 2
                for (int q = thread; q < kRwRows * 8; q += threads) {
                    const int x = q >> 3, ch = q & 7;
                    T *to = row_of(x, tile);
                    if (to)
                        *reinterpret_cast<uint4 *>(reinterpret_cast<uint8_t *>(to + d0) + ch * 16) =
                            *reinterpret_cast<const uint4 *>(place + x * 128 + ((ch ^ (x & 7)) << 4));
                }
            };
            if constexpr (!Z::split) {
                // (three flags by turns: the one that is set to 0 here was read two items ago, and is next used after the barrier)
                if (rr == 0) {
                    s_bad[s][turn_next] = 0;
                    rw_out_read();   // (the last item's rows have left)
                }
                rw_bar<128>(2 + s);
                const bool bad = *bad_flag;
                if (!bad && active && dst) {
#pragma unroll 1
                    for (int d = 0; d < HD; d += 32) {
                        uint32_t o[32];
                        rw_ld32(tO + d, o);
                        rw_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) dst[(d + e) * kRwRows + rr] = own > 0 ? __uint_as_float(o[e]) : 0.0f;
                    }
                    dst[HD * kRwRows + rr] = m2;
                    dst[(HD + 1) * kRwRows + rr] = l;
                } else if (!bad && active) {
                    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
                    const bool full = tokens >= (s + 1) * r.TT;
                    uint8_t *const place = smem + (2 + ST) * Z::tile + s * Z::out;
#pragma unroll 1
                    for (int d0 = 0; d0 < HD; d0 += 64) {
                        if (d0 > 0) {
                            if (rr == 0) rw_out_read();
                            rw_bar<128>(2 + s);
                        }
#pragma unroll
                        for (int d = 0; d < 64; d += 32) {
                            uint32_t o[32];
                            rw_ld32(tO + d0 + d, o);
                            rw_wait_ld();
                            if (own == 0) {
#pragma unroll
                                for (int e = 0; e < 32; ++e) o[e] = 0;
                            }
#pragma unroll
                            for (int e = 0; e < 32; e += 8) {
                                uint32_t w[4];
#pragma unroll
                                for (int q = 0; q < 4; ++q)
                                    w[q] = rw_pack(__uint_as_float(o[e + 2 * q]) * inv, __uint_as_float(o[e + 2 * q + 1]) * inv);
                                *reinterpret_cast<uint4 *>(place + rr * 128 + ((((d + e) / 8) ^ (rr & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
                            }
                        }
                        if (full) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        rw_bar<128>(2 + s);
                        if (!full) {
                            copy_out(place, s, d0, rr, 128);
                        } else if (rr == 0) {
                            rw_tma3_out(&omap, d0, it.g * r.G, it.u.start + it.u.tok0 + s * r.TT, smem_u32(place));
                            rw_out_commit();
                        }
                    }
                }
                if (bad) rw_slow<T, HD>(r, it.u, it.tiles, it.i0, it.i0 + NT, it.g, s * kRwRows, (s + 1) * kRwRows, warp & 3, 4, kOff, dst, &s_beat);
            } else {
                if (own > 0) {
#pragma unroll
                    for (int d = 0; d < HD; d += 32) {
                        uint32_t o[32];
                        rw_ld32(tO + d, o);
                        rw_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) master[d + e] += __uint_as_float(o[e]);
                    }
                    // an infinite value times a weight's low part, which is 0 or of either sign, is NaN: the unit is done again
                    bool nan = false;
#pragma unroll
                    for (int d = 0; d < HD; ++d) nan |= master[d] != master[d];
                    if (nan && l == l) *bad_flag = 1;
                }
                // The warpgroups' parts join in Q's place: each leaves half of its dimensions to the other, and adds its
                // other half to what it finds. (Behind the barrier: with one tile the second has waited for nothing, and
                // Q may still be read before.)
                if (tid == 0) s_bad[0][turn_next] = 0;
                rw_bar<256>(1);
                const bool bad = *bad_flag;
                if (!bad && dst) {
#pragma unroll
                    for (int d = 0; d < HD; ++d) dst[d * kRwRows + rr] = master[d];
                    dst[HD * kRwRows + rr] = m2;
                    dst[(HD + 1) * kRwRows + rr] = l;
                } else if (!bad) {
                    float2 *const ml = reinterpret_cast<float2 *>(smem);
                    ml[s * kRwRows + rr] = make_float2(m2, l);
                    rw_bar<256>(1);
                    const float2 other = ml[(s ^ 1) * kRwRows + rr];
                    rw_bar<256>(1);
                    const float top = fmaxf(m2, other.x);
                    const float f0 = m2 == top ? 1.0f : rw_ex2(m2 - top), f1 = other.x == top ? 1.0f : rw_ex2(other.x - top);
                    const float sum = l * f0 + other.y * f1, fac = sum == 0.0f ? 0.0f : f0 / sum;
                    auto at = [&](int d) {
                        return reinterpret_cast<float4 *>(smem + (d >> 5) * (kRwRows * 128) + rr * 128 + (((d >> 2 & 7) ^ (rr & 7)) << 4));
                    };
                    auto leave = [&](int d) { *at(d) = make_float4(master[d] * fac, master[d + 1] * fac, master[d + 2] * fac, master[d + 3] * fac); };
                    auto join = [&](int d) {
                        const float4 x = *at(d);
                        *at(d) = make_float4(fmaf(master[d], fac, x.x), fmaf(master[d + 1], fac, x.y), fmaf(master[d + 2], fac, x.z), fmaf(master[d + 3], fac, x.w));
                    };
                    if (s == 0) {
#pragma unroll
                        for (int d = HD / 2; d < HD; d += 4) leave(d);
                        rw_bar<256>(1);
#pragma unroll
                        for (int d = 0; d < HD / 2; d += 4) join(d);
                    } else {
#pragma unroll
                        for (int d = 0; d < HD / 2; d += 4) leave(d);
                        rw_bar<256>(1);
#pragma unroll
                        for (int d = HD / 2; d < HD; d += 4) join(d);
                    }
                    const bool full = tokens >= r.TT;
                    if (full) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    rw_bar<256>(1);
                    if (!full) {
#pragma unroll 1
                        for (int d0 = 0; d0 < HD; d0 += 32) copy_out(smem + (d0 >> 5) * (kRwRows * 128), 0, d0, tid, 256);
                    } else if (tid == 0) {
#pragma unroll
                        for (int d0 = 0; d0 < HD; d0 += 32)
                            rw_tma3_out(&omap, d0, it.g * r.G, it.u.start + it.u.tok0, base + (d0 >> 5) * (kRwRows * 128));
                        rw_out_commit();
                        rw_out_read();
                    }
                } else {
                    if (dst && s == 1) {   // the first warpgroup's part is the whole, this one is nothing
#pragma unroll 1
                        for (int d = 0; d < HD + 2; ++d) dst[d * kRwRows + rr] = d == HD ? -INFINITY : 0.0f;
                    }
                    rw_slow<T, HD>(r, it.u, it.tiles, it.i0, it.i0 + NT, it.g, 0, kRwRows, warp, 8, kOff, dst ? dst - s * Z::part : nullptr, &s_beat);
                }
                rw_bar<256>(1);   // (the next item's Q comes to this place)
            }
        }
        rw_out_done();
        rw_before();
    }
    __syncthreads();
    if (tid == 0 && s_err) record_status(a.status, QW3_ERR_TIMEOUT);
    if (s_err) {   // given up: copies and products that nobody has waited for end first (both parities: no phase is open then, or a second is over)
        if (warp == 9 && rw_elect()) rw_commit(&b_end);
        if (tid < ST + 2) {
            uint64_t *const bar = tid < ST ? &b_full[tid] : tid == ST ? &b_q : &b_end;
            (void)mbar_wait_bounded(bar, 0);
            if (tid <= ST) (void)mbar_wait_bounded(bar, 1);
        }
        __syncthreads();
    }
    rw_after();
    if (warp == 9) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
}

// 32 rows and 32 dimensions of a unit that was split to a block: a lane to a row, a
// warp to a fourth of the parts.
template <typename T, int HD>
__global__ void __launch_bounds__(128) k_paged_rows_join(const RwArgs r) {
    using Z = RwSizes<T, HD>;
    __shared__ float s_o[4][33][32];   // the warps' outputs, and sums
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row = blockIdx.y * 32 + lane, d0 = blockIdx.z * 32, unit = blockIdx.x;
    pdl_wait();
    pdl_trigger();
    const RwCut cut = reinterpret_cast<const RwCut *>(r.ws)[unit];
    if (cut.parts < 2) return;
    const int rr = row % kRwRows, tk = rr * r.g_inv >> 16, tok = row / kRwRows * r.TT + tk;
    const bool real = rr < r.TT * r.G && tok < cut.tokens;
    if (__all_sync(0xffffffffu, !real)) return;   // (the same in every warp)
    const float *src = r.ws + static_cast<size_t>(r.units) * 4 + (static_cast<size_t>(unit) * r.splits * 2 + row / kRwRows) * Z::part + rr;
    auto part = [&](int k) { return src + static_cast<size_t>(Z::split ? k : 2 * k) * Z::part; };
    const int n = cut.parts * (Z::split ? 2 : 1);
    float m = -INFINITY, l = 0.0f, o[32];
    if (real) {
#pragma unroll 8
        for (int k = 0; k < n; ++k) m = fmaxf(m, part(k)[HD * kRwRows]);
    }
#pragma unroll
    for (int e = 0; e < 32; ++e) o[e] = 0.0f;
    if (real) {
#pragma unroll 2
        for (int k = warp; k < n; k += 4) {
            const float *q = part(k);
            const float mk = q[HD * kRwRows], f = mk == m ? 1.0f : rw_ex2(mk - m);
            l = fmaf(q[(HD + 1) * kRwRows], f, l);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = fmaf(q[(d0 + e) * kRwRows], f, o[e]);
        }
    }
#pragma unroll
    for (int e = 0; e < 32; ++e) s_o[warp][e][lane] = o[e];
    s_o[warp][32][lane] = l;
    __syncthreads();
    if (!real) return;
    l = (s_o[0][32][lane] + s_o[1][32][lane]) + (s_o[2][32][lane] + s_o[3][32][lane]);
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    float v[8];   // a warp to 8 dimensions
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int d = warp * 8 + e;
        v[e] = ((s_o[0][d][lane] + s_o[1][d][lane]) + (s_o[2][d][lane] + s_o[3][d][lane])) * inv;
    }
    T *to = static_cast<T *>(r.a.out) + static_cast<size_t>(cut.start + tok) * r.a.out_stride +
            static_cast<size_t>(unit % r.a.c.nkv * r.G + rr - tk * r.G) * HD + d0 + warp * 8;
    if constexpr (Z::split) {
        *reinterpret_cast<float4 *>(to) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4 *>(to + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        *reinterpret_cast<uint4 *>(to) = make_uint4(rw_pack(v[0], v[1]), rw_pack(v[2], v[3]), rw_pack(v[4], v[5]), rw_pack(v[6], v[7]));
    }
}

// How the units are launched and split: `units` (an upper bound: starts are on the
// device) in `splits` parts each at most, which up to one CTA to an SM take in turn.
struct RwPlan {
    int TT = 0, units = 0, splits = 1, split_tiles = 0;
    size_t bytes = 0;
};
RwPlan rw_plan(int B, int M, int min_cols, int type, int nh, int nkv, int hd, int max_rows, int max_len, int window, int sinks) {
    RwPlan p;
    const int G = nh / nkv, QT = type == QW3_F32 ? 1 : 2;
    p.TT = kRwRows / G;
    const int UT = p.TT * QT;
    // at most so many: each sequence has more than min_cols columns, and all of them M rows
    const long long least = min_cols / G + 1, seqs = std::min<long long>(B, M / least);
    const long long pairs = std::max<long long>(1, std::min(seqs * ((max_rows + UT - 1) / UT), (M - seqs) / UT + seqs));
    p.units = static_cast<int>(pairs * nkv);
    // and likely so many: beside sequences of one row (min_cols: others' are there too) the rest is in few sequences
    const long long likely = min_cols ? std::min(pairs, (M - std::min(B, M)) / UT + 1ll) * nkv : p.units;
    long long len = max_len;
    if (window > 0) len = std::min<long long>(len, static_cast<long long>(window) + UT + 2 * kRwKeys + sinks);
    const int tiles = static_cast<int>(std::max<long long>(1, (len + kRwKeys - 1) / kRwKeys));
    // the parts that take the fewest rounds of tiles, with three tiles' time for a part's ends and four for the join
    const int sms = num_sms();
    double best = 0.0;
    for (int s = 1; s <= std::min(tiles, 32) && (s == 1 || static_cast<long long>(p.units) * s <= 6 * sms); ++s) {
        const int per = (tiles + s - 1) / s;
        const double cost = static_cast<double>((likely * s + sms - 1) / sms) * (per + 3) + (s > 1 ? 4 : 0);
        if (s == 1 || cost < best) {
            best = cost;
            p.splits = s;
            p.split_tiles = per;
        }
    }
    if (p.splits > 1)
        p.bytes = static_cast<size_t>(p.units) * sizeof(RwCut) +
                  static_cast<size_t>(p.units) * p.splits * 2 * (hd + 2) * kRwRows * sizeof(float);
    return p;
}

// cuTensorMapEncodeTiled, found at run time: the library loads without a driver too.
using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                                 const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled encode_tiled() {
    static const EncodeTiled f = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return f;
}

template <typename T, int HD>
cudaError_t rows_t(const KvPagedAttnArgs &a, int min_cols, const RwPlan &p, float *ws, bool join, bool pdl, cudaStream_t s) {
    using Z = RwSizes<T, HD>;
    const int G = a.nh / a.c.nkv;
    const RwArgs r{a, G, p.TT, (65536 + G - 1) / G, min_cols, p.split_tiles, p.splits, p.units, ws};
    if (join)
        return p.splits == 1 ? cudaSuccess
                             : launch_pdl(pdl, k_paged_rows_join<T, HD>, dim3(p.units, Z::QT * kRwRows / 32, HD / 32), 128, 0, 1, s, r);
    const EncodeTiled encode = encode_tiled();
    if (!encode) return cudaErrorNotSupported;
    // the pool as rows of HD values; a box is 64 values of the rows of a page that lie in one key tile
    CUtensorMap map;
    const cuuint64_t dims[2] = {HD, (static_cast<cuuint64_t>(a.c.pages) * 2 * a.c.nkv) << a.c.shift}, strides[1] = {HD * 2};
    const cuuint32_t box[2] = {64, std::min<cuuint32_t>(1u << a.c.shift, kRwKeys)}, step[2] = {1, 1};
    if (encode(&map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, a.c.data, dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    // rows of queries (f16) and outputs: a box is 128 bytes of G heads of TT tokens, a row tile
    constexpr cuuint32_t size = sizeof(T);
    const auto rows_map = [&](CUtensorMap *to, const void *from, int64_t stride) {
        const cuuint64_t rdims[3] = {HD, static_cast<cuuint64_t>(a.nh), static_cast<cuuint64_t>(a.b.M)};
        const cuuint64_t rstrides[2] = {HD * size, static_cast<cuuint64_t>(stride) * size};
        const cuuint32_t rbox[3] = {128 / size, static_cast<cuuint32_t>(r.G), static_cast<cuuint32_t>(p.TT)}, rstep[3] = {1, 1, 1};
        return encode(to, Z::split ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void *>(from), rdims,
                      rstrides, rbox, rstep, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    };
    CUtensorMap qmap, omap;
    if (rows_map(&qmap, a.q, a.q_stride) != CUDA_SUCCESS || rows_map(&omap, a.out, a.out_stride) != CUDA_SUCCESS) return cudaErrorInvalidValue;
    const int grid = static_cast<int>(std::min<long long>(num_sms(), static_cast<long long>(p.units) * p.splits));
    return launch_pdl(pdl, k_paged_rows<T, HD>, dim3(grid), kRwThreads, Z::smem, 1, s, r, map, qmap, omap);
}

template <typename T, int HD>
cudaError_t configure_rows_t() {
    return cudaFuncSetAttribute(k_paged_rows<T, HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(RwSizes<T, HD>::smem));
}

}  // namespace

cudaError_t configure_kv_paged_rows() {
    cudaError_t e = configure_rows_t<float, 128>();
    if (e == cudaSuccess) e = configure_rows_t<float, 64>();
    if (e == cudaSuccess) e = configure_rows_t<__half, 128>();
    if (e == cudaSuccess) e = configure_rows_t<__half, 64>();
    return e;
}

size_t kv_paged_rows_workspace_bytes(int B, int M, int min_cols, int type, int nh, int nkv, int hd, int max_rows, int max_len, int window,
                                     int sinks) {
    return rw_plan(B, M, min_cols, type, nh, nkv, hd, max_rows, max_len, window, sinks).bytes;
}

cudaError_t launch_kv_paged_rows(const KvPagedAttnArgs &a, int type, int hd, int min_cols, float *ws, bool join, bool pdl, cudaStream_t s) {
    const RwPlan p = rw_plan(a.b.B, a.b.M, min_cols, type, a.nh, a.c.nkv, hd, a.b.max_rows, a.b.max_len, a.window, a.sinks);
    if (type == QW3_F32) return hd == 128 ? rows_t<float, 128>(a, min_cols, p, ws, join, pdl, s) : rows_t<float, 64>(a, min_cols, p, ws, join, pdl, s);
    return hd == 128 ? rows_t<__half, 128>(a, min_cols, p, ws, join, pdl, s) : rows_t<__half, 64>(a, min_cols, p, ws, join, pdl, s);
}

}  // namespace qw3
