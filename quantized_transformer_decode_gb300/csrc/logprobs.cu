// Log probabilities of given tokens, the entropy of a row of logits and its
// most likely tokens.
//
// With M = max l, R = the sum of exp(l_i - M) over all i but one that holds the
// maximum, and W = sum exp(l_i - M) (l_i - M):
//     log Z = M + log1p(R),   log p_t = (l_t - M) - log1p(R),
//     entropy = log1p(R) - W / (1 + R).
// The maximum's own term is kept apart because log1p(R) is then as exact for a
// row that is almost certain (R ~ 1e-9) as for a flat one; both terms of the
// entropy are >= 0, so nothing cancels. A thread sums all terms, S, beside its own
// maximum, without a branch; a CTA takes the 1 from its sum, or, where that would
// cancel (S < 1.25), reads the logits of the one thread that holds the maximum
// again and adds them without it. CTAs' results (M, R, W) join by a shift of the
// reference; one that has seen nothing has R = -1, so that 1 + R counts as 0.
//
// One pass over the logits, a cluster of CTAs to a row. The largest tokens are
// found on the way: when each thread has seen its first 16 logits, and again after
// 2, 4, 8 .. times as many, every warp names its largest of the threads' own
// maxima (4 to 16), and the n-th largest of all named is a bound that the n
// largest cannot lie below. What passes it (some n for every doubling, for logits in any usual
// order) goes to a list in shared memory; what of the list passes the last bound
// is put in order by counting for each how many are before it. A list that
// overflows is read from the slice again, with the last bound.
//
// Bound by HBM for many rows (512 x 151936 is 311 MB, 46 us of copying: 50 us
// without alternatives, 54 with one, 62 with 20), by latency for one (4.6 us
// without, 11 with five, 14.4 with 20).
#include <algorithm>
#include <cstdint>

#include "qw3_internal.cuh"

namespace qw3 {

namespace {

constexpr int kLpThreads = 256, kLpWarps = kLpThreads / 32;
constexpr int kLpChunk = 4;        // 16-byte loads of a thread in flight
constexpr int kLpList = 2048;
constexpr int kLpNamed = 16;       // maxima that a warp names at most: in all twice the alternatives and more
constexpr int kLpMaxCluster = 8;   // (16 to a row: 16 rows take 23 us where 8 take 16)
constexpr float kLog2e = 1.4426950408889634f;

struct LpPart {
    float m, r, w;
};

__device__ __forceinline__ float lp_exp(float d) { return exp2f(d * kLog2e); }

// a += b: both parts of one row.
__device__ __forceinline__ void lp_join(LpPart &a, LpPart b) {
    if (b.m > a.m) {
        const LpPart t = a;
        a = b;
        b = t;
    }
    // (a difference of -1000 is as good as any below: exp is 0, and 0 * d is not NaN)
    const float t = 1.0f + b.r, d = fmaxf(b.m - a.m, -1000.0f), s = lp_exp(d);
    a.r += t * s;
    a.w += s * (b.w + d * t);
}

// The same for parts whose r is the sum of all terms, the maximum's among them.
__device__ __forceinline__ void lp_join_all(LpPart &a, float m, float r, float w) {
    const float top = fmaxf(a.m, m);
    const float d0 = fmaxf(a.m - top, -1000.0f), d1 = fmaxf(m - top, -1000.0f), f0 = lp_exp(d0), f1 = lp_exp(d1);
    a.w = f0 * (a.w + d0 * a.r) + f1 * (w + d1 * r);
    a.r = a.r * f0 + r * f1;
    a.m = top;
}

__device__ __forceinline__ float lp_ex2(float x) {   // (2^-126 and less is 0)
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A logit above -inf as a key: larger value first, the lower index among equal
// ones (-0 is 0); no key is 0.
__device__ __forceinline__ unsigned long long lp_key(float v, int i) { return argmax_pack(v + 0.0f, i); }
__device__ __forceinline__ float lp_value(unsigned long long k) { return float_from_order_key(static_cast<uint32_t>(k >> 32)); }
__device__ __forceinline__ int lp_index(unsigned long long k) { return static_cast<int>(0xffffffffu - static_cast<uint32_t>(k)); }

struct __align__(16) LpShared {
    unsigned long long list[kLpList], some[kLpList + 2];
    unsigned long long best[kLogprobMaxTop];
    unsigned long long top[kLpMaxCluster][kLogprobMaxTop];   // rank 0's: every CTA's best
    unsigned long long named[kLpWarps * kLpNamed];
    unsigned long long bound[2];   // by turns: one is reset while the other may still be read
    LpPart warp[kLpWarps];
    float rest[kLpWarps];
    LpPart cta[kLpMaxCluster];   // rank 0's: every CTA's part
    int count, kept;
};

__device__ __forceinline__ void st_cluster(uint32_t addr, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

__device__ __forceinline__ void st_cluster64(uint32_t addr, unsigned long long v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

// The n best of the list's `count` keys, in order, to s.best; 0 past their end.
// Only those from `least` on need be looked at: the n best are among them.
// Between barriers.
__device__ __forceinline__ void lp_rank(LpShared &s, int count, int n, float least) {
    if (threadIdx.x == 0) s.kept = 0;
    for (int i = threadIdx.x; i < n; i += kLpThreads) s.best[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < count; i += kLpThreads) {
        const unsigned long long k = s.list[i];
        if (lp_value(k) >= least) s.some[atomicAdd(&s.kept, 1)] = k;
    }
    __syncthreads();
    const int kept = s.kept;
    if (threadIdx.x == 0 && (kept & 1)) s.some[kept] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < kept; i += kLpThreads) {
        const unsigned long long k = s.some[i];
        int before = 0;
#pragma unroll 4
        for (int j = 0; j < kept; j += 2) {
            const ulonglong2 t = *reinterpret_cast<const ulonglong2 *>(&s.some[j]);
            before += (t.x > k) + (t.y > k);
        }
        if (before < n) s.best[before] = k;
    }
    __syncthreads();
}

// The key that n - 1 of the warps' named keys come before; 0 where fewer are
// named. key: the thread's best, 0 for none. turn: 0, 1, 0, .. from call to call.
__device__ __forceinline__ unsigned long long lp_bound(LpShared &s, int n, unsigned long long key, int turn) {
    const int tid = threadIdx.x, lane = tid & 31;
    uint32_t high = static_cast<uint32_t>(key >> 32);
    const int rounds = n <= 16 ? 4 : n <= 32 ? 8 : kLpNamed;
    for (int i = 0; i < rounds; ++i) {
        const uint32_t m = __reduce_max_sync(0xffffffffu, high);
        const int who = __ffs(__ballot_sync(0xffffffffu, high == m)) - 1;
        if (lane == who) {
            s.named[(tid >> 5) * rounds + i] = m ? key : 0;
            high = 0;
        }
    }
    if (tid == 0) s.bound[turn] = 0;
    __syncthreads();
    if (tid < kLpWarps * rounds) {
        const unsigned long long k = s.named[tid];
        int before = 0;
#pragma unroll 8
        for (int j = 0; j < kLpWarps * rounds; j += 2) {
            const ulonglong2 t = *reinterpret_cast<const ulonglong2 *>(&s.named[j]);
            before += (t.x > k) + (t.y > k);
        }
        if (k && before == n - 1) s.bound[turn] = k;
    }
    __syncthreads();
    return s.bound[turn];
}

__device__ __forceinline__ void lp_push(LpShared &s, float x, int i) {
    const int at = atomicAdd(&s.count, 1);
    if (at < kLpList) s.list[at] = lp_key(x, i);
}

// Row blockIdx.x / C in C slices. Slices begin at whole 16-byte words of the
// row's memory; the up to 3 logits before the first and after the last word are
// taken one by one by rank 0, behind its slice: no bound for the slice may come
// from them. (A logit that equals the bound is left out because what set the bound
// has lower indices, and the row's last ones have the highest.)
__global__ void __launch_bounds__(kLpThreads, 4) k_logprobs(const LogprobArgs a, int C) {
    __shared__ LpShared s;
    const int tid = threadIdx.x, lane = tid & 31;
    const long long row = blockIdx.x / C;
    const int rank = blockIdx.x % C;
    const bool one = C == 1;
    if (!one) cluster_arrive_release();   // (completed below: peers' shared memory is there)
    pdl_trigger();
    pdl_wait();
    const float *x = a.logits + row * a.stride;
    const int head = min(a.V, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(x) & 15)) / 4 & 3));
    const int words = (a.V - head) / 4, tail = head + words * 4;
    const float4 *xv = reinterpret_cast<const float4 *>(x + head);
    const int per = (words + C - 1) / C, w0 = min(words, rank * per), w1 = min(words, w0 + per);

    LpPart part{-3.402823466e38f, 0.0f, 0.0f};   // r: all terms, until the CTA's are joined
    // a thread's lone logit
    int lone = -1;
    if (rank == 0) lone = tid < head ? tid : tid - head < a.V - tail && tid >= head ? tail + tid - head : -1;
    const float lone_x = lone >= 0 ? x[lone] : -INFINITY;
    // the first given token of this thread, early
    int given = -1;
    float given_x = -INFINITY;
    if (rank == 0 && tid < a.T) {
        given = a.tokens[row * a.T + tid];
        if (given >= 0 && given < a.V) given_x = x[given];
    }
    float bound = INFINITY;   // what passes it goes to the list
    constexpr int N = 4 * kLpChunk;
    auto load = [&](float (&v)[N], int base) {
#pragma unroll
        for (int k = 0; k < kLpChunk; ++k) {
            const int at = base + k * kLpThreads + tid;
            const float4 t = at < w1 ? __ldcs(xv + at) : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
            v[4 * k] = t.x; v[4 * k + 1] = t.y; v[4 * k + 2] = t.z; v[4 * k + 3] = t.w;
        }
    };
    if (tid == 0) s.count = 0;   // (a barrier follows before the first is pushed)
    int chunk = 0, turn = 0;
    auto raise = [&]() {   // the bound that the threads' maxima so far give (each of them a logit, were there two alike)
        const unsigned long long k = lp_bound(s, a.top, part.r > 0.0f ? lp_key(part.m, tid) : 0, turn);
        turn ^= 1;
        if (k) bound = fmaxf(bound, lp_value(k));
    };
    float next[N];
    load(next, w0);
    for (int base = w0; base < w1 || base == w0; base += kLpThreads * kLpChunk) {
        float v[N];
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = next[k];
        load(next, base + kLpThreads * kLpChunk);
        const bool begin = base == w0;
        float mx = -INFINITY;
#pragma unroll
        for (int k = 0; k < N; ++k) mx = fmaxf(mx, v[k]);
        {
            const float m = fmaxf(part.m, mx), d = fmaxf(part.m - m, -1000.0f), f = lp_ex2(d * kLog2e);
            float w[2] = {f * (part.w + d * part.r), 0.0f}, r[2] = {part.r * f, 0.0f};
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const float dk = v[k] - m, e = lp_ex2(dk * kLog2e);
                r[k & 1] += e;
                w[k & 1] = fmaf(e, fmaxf(dk, -1000.0f), w[k & 1]);   // (0 * -inf is no part of the sum; NaN: e keeps it)
            }
            part = {m, r[0] + r[1], w[0] + w[1]};
        }
        if (a.top > 0) {
            if (begin) {
                int id = 0x7fffffff;
#pragma unroll
                for (int k = N - 1; k >= 0; --k)
                    if (v[k] == mx) id = min(id, head + 4 * (base + (k >> 2) * kLpThreads + tid) + (k & 3));
                const unsigned long long least = lp_bound(s, a.top, mx > -INFINITY ? lp_key(mx, id) : 0, turn);
                turn ^= 1;
                bound = least ? lp_value(least) : -INFINITY;
                if (mx >= bound) {
#pragma unroll
                    for (int k = 0; k < N; ++k) {
                        const int i = head + 4 * (base + (k >> 2) * kLpThreads + tid) + (k & 3);
                        if (v[k] > -INFINITY && lp_key(v[k], i) >= least) lp_push(s, v[k], i);
                    }
                }
            } else {
                if (mx > bound) {   // (one that equals the bound comes after it)
#pragma unroll
                    for (int k = 0; k < N; ++k)
                        if (v[k] > bound) lp_push(s, v[k], head + 4 * (base + (k >> 2) * kLpThreads + tid) + (k & 3));
                }
                if ((chunk & (chunk + 1)) == 0) raise();
            }
            ++chunk;
        }
    }

    if (lone >= 0) {
        const float m = fmaxf(part.m, lone_x), d = fmaxf(part.m - m, -1000.0f), f = lp_ex2(d * kLog2e);
        const float dk = lone_x - m, e = lp_ex2(dk * kLog2e);
        part = {m, fmaf(part.r, f, e), fmaf(e, fmaxf(dk, -1000.0f), f * (part.w + d * part.r))};
        if (a.top > 0 && lone_x > -INFINITY && lone_x >= bound) lp_push(s, lone_x, lone);
    }
    if (!one) cluster_wait_acquire();
    if (a.top > 0) {
        if (chunk > 1) raise();
        __syncthreads();
        // a list that overflowed (a row that rises): the slice is read again, for what reaches the last bound and the best
        // keys that the list holds. (By those alone a rising row of 151936 takes some 70 readings: 512 of them 25 ms.)
        while (s.count > kLpList) {
            lp_rank(s, kLpList, a.top, -INFINITY);
            const unsigned long long least = max(s.best[a.top - 1], lp_key(bound, 0x7fffffff));
            if (tid == 0) s.count = 0;
            __syncthreads();
            if (lone_x > -INFINITY && lp_key(lone_x, lone) >= least) lp_push(s, lone_x, lone);
            for (int at = w0 + tid; at < w1; at += kLpThreads) {
                const float4 t = xv[at];
                const float u[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (u[k] > -INFINITY && lp_key(u[k], head + 4 * at + k) >= least) lp_push(s, u[k], head + 4 * at + k);
            }
            __syncthreads();
        }
        if (!one) {
            lp_rank(s, s.count, a.top, bound);
            const uint32_t home = dsmem_map(s.top[rank], 0);
            for (int i = tid; i < a.top; i += kLpThreads) st_cluster64(home + 8 * i, s.best[i]);
        }
    }
    // ---- the CTA's part
    const LpPart own = part;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        lp_join_all(part, __shfl_xor_sync(0xffffffffu, part.m, o), __shfl_xor_sync(0xffffffffu, part.r, o),
                    __shfl_xor_sync(0xffffffffu, part.w, o));
    if (lane == 0) s.warp[tid >> 5] = part;
    __syncthreads();
    part = s.warp[0];
    for (int i = 1; i < kLpWarps; ++i) lp_join_all(part, s.warp[i].m, s.warp[i].r, s.warp[i].w);
    // (every thread has joined the same parts in the same order: to the last bit all of them go the same way)
    if (part.r < 1.25f && part.r > 0.0f) {
        float rest = own.m == part.m ? 0.0f : own.r * lp_exp(own.m - part.m);
        if (__any_sync(0xffffffffu, own.m == part.m)) {
            // the thread with the maximum (there is one: a second would make the sum 2): its logits, a lane to a word
            const int who = __ffs(__ballot_sync(0xffffffffu, own.m == part.m)) - 1, t = (tid & ~31) + who;
            bool taken = false;
            auto add = [&](float u) {
                if (u == part.m && !taken) taken = true;
                else rest += lp_exp(u - part.m);
            };
            for (int at = w0 + t + lane * kLpThreads; at < w1; at += 32 * kLpThreads) {
                const float4 u = xv[at];
                add(u.x);
                add(u.y);
                add(u.z);
                add(u.w);
            }
            if (lane == who && lone >= 0) add(lone_x);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) rest += __shfl_xor_sync(0xffffffffu, rest, o);
        if (lane == 0) s.rest[tid >> 5] = rest;
        __syncthreads();
        rest = s.rest[lane % kLpWarps];
#pragma unroll
        for (int o = kLpWarps / 2; o > 0; o >>= 1) rest += __shfl_xor_sync(0xffffffffu, rest, o);
        part.r = rest;
    } else {
        part.r -= 1.0f;
    }
    if (tid == 0) {
        if (one) {
            s.cta[0] = part;
        } else {
            const uint32_t to = dsmem_map(&s.cta[rank], 0);
            st_cluster(to, __float_as_uint(part.m));
            st_cluster(to + 4, __float_as_uint(part.r));
            st_cluster(to + 8, __float_as_uint(part.w));
        }
    }
    if (one) __syncthreads();
    else hw_cluster_sync();
    if (rank != 0) return;

    part = s.cta[0];
    for (int i = 1; i < C; ++i) lp_join(part, s.cta[i]);
    const float total = 1.0f + part.r, log_r = log1pf(part.r);
    const bool bad = !(total > 0.0f) || part.m == INFINITY || !(total < INFINITY);
    for (int i = tid; i < a.T; i += kLpThreads) {
        if (i != tid) {
            given = a.tokens[row * a.T + i];
            given_x = given >= 0 && given < a.V ? x[given] : -INFINITY;
        }
        const float lp = (given_x - part.m) - log_r;
        a.logprob[row * a.T + i] = bad ? NAN : lp;
    }
    if (tid == 0) {
        if (a.entropy) a.entropy[row] = bad ? NAN : log_r - part.w / total;
        if (bad) record_status(a.status, QW3_ERR_NONFINITE);
    }
    if (a.top > 0) {
        if (!one) {   // the CTAs' best, as the list
            __syncthreads();
            if (tid == 0) s.count = 0;
            __syncthreads();
            for (int i = tid; i < C * a.top; i += kLpThreads) {
                const unsigned long long k = s.top[i / a.top][i % a.top];
                if (k) s.list[atomicAdd(&s.count, 1)] = k;
            }
            __syncthreads();
        }
        lp_rank(s, s.count, a.top, one ? bound : -INFINITY);
        for (int i = tid; i < a.top; i += kLpThreads) {
            const unsigned long long k = s.best[i];
            a.top_id[row * a.top + i] = bad || !k ? -1 : lp_index(k);
            a.top_lp[row * a.top + i] = bad ? NAN : !k ? -INFINITY : (lp_value(k) - part.m) - log_r;
        }
    }
}

}  // namespace

cudaError_t launch_logprobs(const LogprobArgs &a, int B, bool pdl, cudaStream_t s) {
    // a row's CTAs: as many as give each SM two, while a slice is worth a CTA. 512 rows of 151936 with 20
    // alternatives take 61 us with one CTA to a row, 78 with two, 152 rows 36 and 29, 64 rows 28 with four, 23 with
    // eight (what a row's end costs against SMs without work)
    int C = 1;
    while (C < kLpMaxCluster && static_cast<long long>(B) * C < 300 && a.V / C > 4 * kLpThreads * kLpChunk) C *= 2;
    for (long long r = 0; r < B; r += 1 << 26) {   // the grid's limit
        LogprobArgs p = a;
        p.logits += r * a.stride;
        p.tokens += r * a.T;
        p.logprob += r * a.T;
        if (p.entropy) p.entropy += r;
        p.top_id += r * a.top;
        p.top_lp += r * a.top;
        const int n = static_cast<int>(std::min<long long>(B - r, 1 << 26));
        const cudaError_t e = launch_pdl(pdl, k_logprobs, dim3(static_cast<unsigned>(n) * C), kLpThreads, 0, C, s, p, C);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace qw3
