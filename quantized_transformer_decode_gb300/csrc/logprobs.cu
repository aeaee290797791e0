// Log probabilities of given tokens, the entropy of a row of logits and its
// most likely tokens.
//
// With M = max l, R = the sum of exp(l_i - M) over all i but one that holds the
// maximum, and W = sum exp(l_i - M) (l_i - M):
//     log Z = M + log1p(R),   log p_t = (l_t - M) - log1p(R),
//     entropy = log1p(R) - W / (1 + R).
// The maximum's own term is kept apart because log1p(R) is then as exact for a
// row that is almost certain (R ~ 1e-9) as for a flat one; both terms of the
// entropy are >= 0, so nothing cancels. Partial results (M, R, W) of threads,
// warps and CTAs join by the same shift of the reference; a part that has seen
// nothing has R = -1, so that 1 + R = 0 counts it as nothing.
//
// One pass over the logits, a cluster of CTAs to a row. The largest tokens are
// found on the way: when each thread has seen its first 16 logits, the n-th
// largest of the threads' own maxima is a bound that the n largest cannot lie
// below, and what passes it (a few times n for logits in any usual order) goes
// to a list in shared memory. A list that overflows raises the bound and the
// slice is read again.
//
// Bound by HBM for many rows (512 x 151936 is 311 MB), by latency for one.
#include <algorithm>
#include <cstdint>

#include "qw3_internal.cuh"

namespace qw3 {

namespace {

constexpr int kLpThreads = 512, kLpWarps = kLpThreads / 32;
constexpr int kLpChunk = 4;        // 16-byte loads of a thread in flight
constexpr int kLpList = 2048;      // more than kLpThreads * 4 * kLpChunk / kLpThreads * kLogprobMaxTop, see collect()
constexpr int kLpMaxCluster = 16;
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

__device__ __forceinline__ void lp_add(LpPart &a, float x) {
    const float d = x - a.m, e = lp_exp(d);
    a.r += e;
    a.w = fmaf(e, fmaxf(d, -1000.0f), a.w);   // (NaN: e keeps it)
}

// (value, index) pairs: larger value first, the lower index among equal ones.
__device__ __forceinline__ bool lp_before(float v, int i, float u, int j) { return v > u || (v == u && i < j); }

struct LpShared {
    LpPart warp[kLpWarps];
    LpPart cta[kLpMaxCluster];               // rank 0's: every CTA's part
    float top_v[kLpMaxCluster][kLogprobMaxTop];   // rank 0's: every CTA's largest
    int top_i[kLpMaxCluster][kLogprobMaxTop];
    float list_v[kLpList];
    int list_i[kLpList];
    float max_v[kLpThreads];
    int max_i[kLpThreads];
    float bound_v;
    int bound_i;
    int count;
};

__device__ __forceinline__ void st_cluster(uint32_t addr, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// The n best of a list's `count` pairs, in order, by counting for each how many
// come before it (a few hundred pairs; equal pairs do not occur). Places past
// the list's end get -inf and -1. Barrier first: all pairs are written.
__device__ __forceinline__ void lp_rank(const float *v, const int *id, int count, int n, float *to_v, int *to_i) {
    for (int i = threadIdx.x; i < count; i += kLpThreads) {
        const float x = v[i];
        const int k = id[i];
        int before = 0;
        for (int j = 0; j < count; ++j) before += lp_before(v[j], id[j], x, k);
        if (before < n) {
            to_v[before] = x;
            to_i[before] = k;
        }
    }
    for (int i = count + threadIdx.x; i < n; i += kLpThreads) {
        to_v[i] = -INFINITY;
        to_i[i] = -1;
    }
}

// The pair that `n - 1` of the threads' best pairs come before, as the bound;
// where fewer than n threads have one, anything above -inf passes.
__device__ __forceinline__ void lp_bound(LpShared &s, int n, float v, int id) {
    s.max_v[threadIdx.x] = v;
    s.max_i[threadIdx.x] = id;
    if (threadIdx.x == 0) {
        s.bound_v = -INFINITY;
        s.bound_i = -1;
        s.count = 0;
    }
    __syncthreads();
    if (v > -INFINITY) {
        int before = 0;
        for (int j = 0; j < kLpThreads; ++j) before += lp_before(s.max_v[j], s.max_i[j], v, id);
        if (before == n - 1) {
            s.bound_v = v;
            s.bound_i = id;
        }
    }
    __syncthreads();
}

__device__ __forceinline__ void lp_push(LpShared &s, float x, int i) {
    const int at = atomicAdd(&s.count, 1);
    if (at < kLpList) {
        s.list_v[at] = x;
        s.list_i[at] = i;
    }
}

// Row blockIdx.x / C in C slices. Slices begin at whole 16-byte words of the
// row's memory; the up to 3 logits before the first and after the last word are
// taken one by one by rank 0.
__global__ void __launch_bounds__(kLpThreads) k_logprobs(const LogprobArgs a, int C) {
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

    LpPart part{-3.402823466e38f, -1.0f, 0.0f};
    // a thread's lone logit
    int lone = -1;
    if (rank == 0) lone = tid < head ? tid : tid - head < a.V - tail && tid >= head ? tail + tid - head : -1;
    const float lone_x = lone >= 0 ? x[lone] : -INFINITY;
    float bound = INFINITY;
    for (int base = w0; base < w1 || base == w0; base += kLpThreads * kLpChunk) {
        float v[4 * kLpChunk];
#pragma unroll
        for (int k = 0; k < kLpChunk; ++k) {
            const int at = base + k * kLpThreads + tid;
            const float4 t = at < w1 ? __ldcs(xv + at) : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
            v[4 * k] = t.x; v[4 * k + 1] = t.y; v[4 * k + 2] = t.z; v[4 * k + 3] = t.w;
        }
        const bool begin = base == w0;
        float mx = begin ? lone_x : -INFINITY;
#pragma unroll
        for (int k = 0; k < 4 * kLpChunk; ++k) mx = fmaxf(mx, v[k]);
        if (mx > part.m) {
            const float t = 1.0f + part.r, d = fmaxf(part.m - mx, -1000.0f), e = lp_exp(d);
            part.w = e * (part.w + d * t);
            part.r = t * e;
            part.m = mx;
            // the new maximum's own term stays apart
            bool taken = begin && lone_x == mx;
            if (begin && !taken) lp_add(part, lone_x);
#pragma unroll
            for (int k = 0; k < 4 * kLpChunk; ++k) {
                if (!taken && v[k] == mx) taken = true;
                else lp_add(part, v[k]);
            }
        } else {
            if (begin) lp_add(part, lone_x);
#pragma unroll
            for (int k = 0; k < 4 * kLpChunk; ++k) lp_add(part, v[k]);
        }
        if (a.top > 0) {
            if (begin) {
                int id = lone_x == mx && lone >= 0 ? lone : 0x7fffffff;
#pragma unroll
                for (int k = 4 * kLpChunk - 1; k >= 0; --k)
                    if (v[k] == mx) id = min(id, head + 4 * (base + (k >> 2) * kLpThreads + tid) + (k & 3));
                lp_bound(s, a.top, mx, id);
                bound = s.bound_v;
                const int bi = s.bound_i;
                if (lone >= 0 && lone_x > -INFINITY && !lp_before(bound, bi, lone_x, lone)) lp_push(s, lone_x, lone);
                if (mx >= bound && mx > -INFINITY) {
#pragma unroll
                    for (int k = 0; k < 4 * kLpChunk; ++k) {
                        const int i = head + 4 * (base + (k >> 2) * kLpThreads + tid) + (k & 3);
                        if (v[k] > -INFINITY && !lp_before(bound, bi, v[k], i)) lp_push(s, v[k], i);
                    }
                }
            } else if (mx > bound) {   // (equal ones come after the bound's index)
#pragma unroll
                for (int k = 0; k < 4 * kLpChunk; ++k)
                    if (v[k] > bound) lp_push(s, v[k], head + 4 * (base + (k >> 2) * kLpThreads + tid) + (k & 3));
            }
        }
    }

    if (!one) cluster_wait_acquire();
    const uint32_t home_v = one ? 0 : dsmem_map(s.top_v[rank], 0), home_i = one ? 0 : dsmem_map(s.top_i[rank], 0);
    if (a.top > 0) {
        __syncthreads();
        // a list that overflowed: the best pairs that it holds give a higher bound, and the slice is read again
        while (s.count > kLpList) {
            lp_rank(s.list_v, s.list_i, kLpList, a.top, s.max_v, s.max_i);
            __syncthreads();
            const float bv = s.max_v[a.top - 1];
            const int bi = s.max_i[a.top - 1];
            if (tid == 0) s.count = 0;
            __syncthreads();
            if (lone >= 0 && lone_x > -INFINITY && !lp_before(bv, bi, lone_x, lone)) lp_push(s, lone_x, lone);
            for (int at = w0 + tid; at < w1; at += kLpThreads) {
                const float4 t = xv[at];
                const float u[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (u[k] > -INFINITY && !lp_before(bv, bi, u[k], head + 4 * at + k)) lp_push(s, u[k], head + 4 * at + k);
            }
            __syncthreads();
        }
        lp_rank(s.list_v, s.list_i, s.count, a.top, s.max_v, s.max_i);
        __syncthreads();
        for (int i = tid; i < a.top; i += kLpThreads) {
            if (one) {
                s.top_v[0][i] = s.max_v[i];
                s.top_i[0][i] = s.max_i[i];
            } else {
                st_cluster(home_v + 4 * i, __float_as_uint(s.max_v[i]));
                st_cluster(home_i + 4 * i, static_cast<uint32_t>(s.max_i[i]));
            }
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const LpPart t{__shfl_xor_sync(0xffffffffu, part.m, o), __shfl_xor_sync(0xffffffffu, part.r, o),
                       __shfl_xor_sync(0xffffffffu, part.w, o)};
        lp_join(part, t);
    }
    if (lane == 0) s.warp[tid >> 5] = part;
    __syncthreads();
    if (tid == 0) {
        part = s.warp[0];
        for (int i = 1; i < kLpWarps; ++i) lp_join(part, s.warp[i]);
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
        const int t = a.tokens[row * a.T + i];
        const float lp = t < 0 || t >= a.V ? -INFINITY : (x[t] - part.m) - log_r;
        a.logprob[row * a.T + i] = bad ? NAN : lp;
    }
    if (tid == 0) {
        if (a.entropy) a.entropy[row] = bad ? NAN : log_r - part.w / total;
        if (bad) record_status(a.status, QW3_ERR_NONFINITE);
    }
    if (a.top > 0) {
        // the CTAs' pairs above -inf, gathered into the list
        if (tid == 0) s.count = 0;
        __syncthreads();
        for (int i = tid; i < C * a.top; i += kLpThreads) {
            const int c = i / a.top, k = i - c * a.top;
            if (s.top_i[c][k] >= 0) lp_push(s, s.top_v[c][k], s.top_i[c][k]);
        }
        __syncthreads();
        lp_rank(s.list_v, s.list_i, s.count, a.top, s.max_v, s.max_i);
        __syncthreads();
        for (int i = tid; i < a.top; i += kLpThreads) {
            const int id = s.max_i[i];
            a.top_id[row * a.top + i] = bad ? -1 : id;
            a.top_lp[row * a.top + i] = bad ? NAN : id < 0 ? -INFINITY : (s.max_v[i] - part.m) - log_r;
        }
    }
}

}  // namespace

cudaError_t configure_logprobs() {
    return cudaFuncSetAttribute(k_logprobs, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
}

cudaError_t launch_logprobs(const LogprobArgs &a, int B, bool pdl, cudaStream_t s) {
    // a row's CTAs: as many as keep the GPU's 608 places for them filled, while a slice is worth a CTA
    int C = 1;
    while (C < kLpMaxCluster && static_cast<long long>(B) * C < 1216 && a.V / C > 4 * kLpThreads * kLpChunk) C *= 2;
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
