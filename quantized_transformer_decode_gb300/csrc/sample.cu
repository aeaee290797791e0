// Sampling a token from each row of logits: temperature, top-k, top-p, min-p
// and a draw from a given uniform number.
//
// w_i = exp((l_i - max l) / T), tokens ordered by (l descending, i ascending).
// top-k keeps the first k; top-p the shortest prefix whose sum reaches p times
// the top-k sum; min-p the tokens with w >= min_p (the largest w is 1). The
// token is the first i, in vocabulary order, whose running sum of kept weights
// passes u times their total. Both cuts are prefixes of one order, so the set
// that they leave is (key of the last kept logit, how many of its equals).
//
// Sums are taken in 64-bit fixed point (2^40 for the largest weight): they are
// the same whatever the order of the additions, so one input gives one token.
#include "qw3_internal.cuh"

namespace qw3 {

namespace {

constexpr int kThreads = 1024;
using u64 = unsigned long long;

// Order of logits as unsigned keys; the two zeros are one value.
__device__ __forceinline__ uint32_t logit_key(float v) { return float_order_key(v + 0.0f); }

__device__ __forceinline__ u64 fixed_weight(float l, float top, float inv_t) {
    return static_cast<u64>(__float2ull_rn(expf((l - top) * inv_t) * 1099511627776.0f));
}

// Sum over the block, known to every thread; s: 33 words.
__device__ u64 block_sum(u64 v, u64 *s) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if (lane == 0) s[warp] = v;
    __syncthreads();
    if (warp == 0) {
        u64 t = s[lane];
        for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
        if (lane == 0) s[32] = t;
    }
    __syncthreads();
    return s[32];
}

// Exclusive sum over the threads below this one.
__device__ u64 block_before(u64 v, u64 *s) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    u64 t = v;
    for (int o = 1; o < 32; o <<= 1) {
        const u64 x = __shfl_up_sync(0xffffffffu, t, o);
        if (lane >= o) t += x;
    }
    __syncthreads();
    if (lane == 31) s[warp] = t;
    __syncthreads();
    if (warp == 0) {
        const u64 mine = s[lane];
        u64 x = mine;
        for (int o = 1; o < 32; o <<= 1) {
            const u64 y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        s[lane] = x - mine;
    }
    __syncthreads();
    return s[warp] + t - v;
}

// The largest key whose elements, with all larger ones, reach `target` (of
// counts, or of weights where `weigh`), among keys >= floor; *above: the sum
// over larger keys.
__device__ uint32_t select_key(const float *l, int V, float top, float inv_t, bool weigh, u64 target, uint32_t floor_key,
                               u64 *hist, u64 *above) {
    __shared__ uint32_t s_key;
    __shared__ u64 s_above;
    uint32_t prefix = 0;
    u64 sum = 0;
    for (int shift = 24; shift >= 0; shift -= 8) {
        for (int i = threadIdx.x; i < 256; i += kThreads) hist[i] = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < V; i += kThreads) {
            const uint32_t k = logit_key(l[i]);
            if (k < floor_key || (shift < 24 && (k >> (shift + 8)) != prefix)) continue;
            atomicAdd(&hist[(k >> shift) & 255u], weigh ? fixed_weight(l[i], top, inv_t) : 1ull);
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            u64 t = sum;
            int b = 255;
            while (b > 0 && t + hist[b] < target) t += hist[b--];
            s_key = (prefix << 8) | static_cast<uint32_t>(b);
            s_above = t;
        }
        __syncthreads();
        prefix = s_key;
        sum = s_above;
        __syncthreads();
    }
    *above = sum;
    return prefix;
}

__global__ void __launch_bounds__(kThreads) k_sample(SampleArgs a) {
    __shared__ u64 hist[256], red[33];
    __shared__ float s_top;
    __shared__ int s_idx, s_bad;
    const int b = blockIdx.x, tid = threadIdx.x, V = a.V;
    const float *l = a.logits + b * a.stride;
    if (tid == 0) {
        s_bad = 0;
        s_idx = 0x7fffffff;
        hist[0] = 0;
    }
    __syncthreads();
    bool bad = false;
    u64 best = 0;
    for (int i = tid; i < V; i += kThreads) {
        const float v = l[i];
        bad |= v != v;
        const u64 k = argmax_pack(v + 0.0f, i);
        best = k > best ? k : best;
    }
    atomicMax(&hist[0], best);
    if (bad) s_bad = 1;
    __syncthreads();
    const float top = float_from_order_key(static_cast<uint32_t>(hist[0] >> 32));
    const int arg = static_cast<int>(0xffffffffu - static_cast<uint32_t>(hist[0]));
    const float T = a.temperature ? a.temperature[b] : 1.0f;
    const bool greedy = T <= 0.0f;
    __syncthreads();
    if (s_bad || top == -INFINITY || !(T < INFINITY) || (!greedy && top == INFINITY)) {
        if (tid == 0) {
            record_status(a.status, QW3_ERR_NONFINITE);
            a.token[b] = -1;
            if (a.prob) a.prob[b] = 0.0f;
        }
        return;
    }
    if (greedy) {
        if (tid == 0) {
            a.token[b] = arg;
            if (a.prob) a.prob[b] = 1.0f;
        }
        return;
    }
    const float inv_t = 1.0f / fmaxf(T, 1e-30f);
    const int k = a.top_k ? a.top_k[b] : 0;
    const float p = a.top_p ? a.top_p[b] : 1.0f, mp = a.min_p ? a.min_p[b] : 0.0f;
    uint32_t cut = 0;         // kept: key > cut, and the first `ties` of those equal to it
    u64 ties = ~0ull;
    if (k > 0 && k < V) {
        u64 above;
        cut = select_key(l, V, top, inv_t, false, static_cast<u64>(k), 0u, hist, &above);
        ties = static_cast<u64>(k) - above;
    }
    if (p < 1.0f) {
        u64 w = 0, n = 0;
        for (int i = tid; i < V; i += kThreads) {
            const uint32_t key = logit_key(l[i]);
            if (key > cut) w += fixed_weight(l[i], top, inv_t);
            n += key == cut;
        }
        w = block_sum(w, red);
        n = block_sum(n, red);
        const u64 have = n < ties ? n : ties;
        if (have) w += have * fixed_weight(float_from_order_key(cut), top, inv_t);
        u64 target = static_cast<u64>(ceil(static_cast<double>(fmaxf(p, 0.0f)) * static_cast<double>(w)));
        if (target < 1) target = 1;
        u64 above;
        const uint32_t key = select_key(l, V, top, inv_t, true, target, cut, hist, &above);
        const u64 one = fixed_weight(float_from_order_key(key), top, inv_t);
        u64 m = one ? (target - above + one - 1) / one : 1;
        if (key == cut && m > ties) m = ties;
        cut = key;
        ties = m;
    }
    // the kept tokens in vocabulary order: a thread takes a run of them
    const int run = (V + kThreads - 1) / kThreads, i0 = min(V, tid * run), i1 = min(V, i0 + run);
    u64 n = 0;
    for (int i = i0; i < i1; ++i) n += logit_key(l[i]) == cut;
    const u64 n0 = block_before(n, red);
    auto weight = [&](int i, u64 &seen) -> u64 {
        const uint32_t key = logit_key(l[i]);
        const bool in = key > cut || (key == cut && seen++ < ties);
        return in && (expf((l[i] - top) * inv_t) >= mp || l[i] == top) ? fixed_weight(l[i], top, inv_t) : 0ull;
    };
    u64 w = 0, seen = n0;
    for (int i = i0; i < i1; ++i) w += weight(i, seen);
    const u64 w0 = block_before(w, red);
    const u64 total = block_sum(w, red);
    const float u = a.u[b];
    u64 at = static_cast<u64>(static_cast<double>(u > 0.0f ? u : 0.0f) * static_cast<double>(total));
    if (at >= total) at = total - 1;
    if (w0 <= at && at < w0 + w) {
        u64 c = w0;
        seen = n0;
        for (int i = i0; i < i1; ++i) {
            c += weight(i, seen);
            if (c > at) {
                a.token[b] = i;
                if (a.prob)
                    a.prob[b] = static_cast<float>(exp((static_cast<double>(l[i]) - top) / fmaxf(T, 1e-30f)) *
                                                   1099511627776.0 / static_cast<double>(total));
                break;
            }
        }
    }
}

}  // namespace

cudaError_t launch_sample(const SampleArgs &a, int B, cudaStream_t s) {
    if (B <= 0) return cudaSuccess;
    k_sample<<<B, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace qw3
