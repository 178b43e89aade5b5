// Log probabilities of given tokens, the entropy, and the top alternatives of
// rows of float32 logits (the values a serving step reports beside its tokens).
//
// With M = max z, S = sum exp(z_i - M) over the row:
//   logp_i = (z_i - M) - log S,  entropy = log S - (sum (z_i - M) exp(z_i - M)) / S
// (nats).  NaN and -inf logits take no part.  A +inf logit is the maximum: the
// +inf tokens share the mass.  The top alternatives are the k highest logits,
// equal ones by index.
//
// Bound by HBM: the logits are read once.  One cluster of up to 8 CTAs per row,
// each CTA a contiguous slice.  Each thread keeps a running maximum with its
// index, and sums rescaled when the maximum moves (float32).  The top k need no
// second pass over the slice: the k-th highest of the maxima of 128 groups of
// four threads is a lower bound of the slice's k-th highest logit, and only the
// k groups whose maximum reaches it can hold one.  Their elements (k / 128 of the
// slice, still in L2) are looked at again, those that reach the bound are ranked
// by counting, and the cluster's first CTA ranks the lists of all.
#include <math.h>

#include "common.cuh"
#include "kernels.h"

namespace bloom {

constexpr int kLpThreads = 512;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kLpMaxCluster = 8;
constexpr int kLpGroups = kLpThreads / 4;    // of four threads: 16 neighbouring logits a step
constexpr int kLpStep = 4 * kLpThreads;      // logits of a CTA's step
constexpr int kLpUnroll = 4;                 // steps whose loads are in flight together
constexpr int kLpCand = 1024;                // candidates ranked in shared memory
constexpr float kLpFar = -1e4f;              // stands for any difference whose exponential is 0

typedef unsigned long long lp_u64;

// (logit, index) as one number: a larger logit is larger, then a lower index; 0:
// a logit that takes no part.  -0 orders as +0.
__device__ __forceinline__ lp_u64 lp_key(float z, uint32_t i) {
    if (!(z > -INFINITY)) return 0ull;
    return pack_argmax(z == 0.f ? 0.f : z, i);
}
__device__ __forceinline__ float lp_logit(lp_u64 key) {   // key > 0
    const uint32_t k = (uint32_t)(key >> 32);
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}
__device__ __forceinline__ lp_u64 lp_max(lp_u64 a, lp_u64 b) { return a > b ? a : b; }
// a - b for a <= b; 0 for equal ones (infinities too), kLpFar at least (a NaN too)
__device__ __forceinline__ float lp_diff(float a, float b) { return a == b ? 0.f : fmaxf(a - b, kLpFar); }
__device__ __forceinline__ float lp_exp(float d) {
    float r;
    asm("ex2.approx.f32 %0, %1;" : "=f"(r) : "f"(d * 1.4426950408889634f));
    return r;
}

struct LpStat {   // maximum, sum exp(z - m), sum (z - m) exp(z - m)
    float m, s, t;
    __device__ __forceinline__ void shift(float to) {   // to >= m
        const float d = lp_diff(m, to), c = lp_exp(d);
        t = c * (t + d * s);
        s *= c;
        m = to;
    }
    __device__ __forceinline__ void join(LpStat o) {
        const float to = fmaxf(m, o.m);
        shift(to);
        o.shift(to);
        s += o.s;
        t += o.t;
    }
};

struct LpSmem {
    lp_u64 group[kLpGroups];
    lp_u64 cand[kLpCand];
    lp_u64 list[kLpMaxTop];                       // this slice's top, highest first
    lp_u64 lists[kLpMaxCluster][kLpMaxTop];       // first CTA: every slice's
    lp_u64 top[kLpMaxTop];
    LpStat stats[kLpMaxCluster];
    LpStat warp[kLpWarps];
    lp_u64 wmax[kLpWarps];
    lp_u64 bound;
    int hot[kLpMaxTop];
    int nhot, ncand;
};

__device__ __forceinline__ uint32_t lp_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t lp_first(const void *p) {   // address in the cluster's first CTA
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"((uint32_t)__cvta_generic_to_shared(p)));
    return r;
}

__global__ void __launch_bounds__(kLpThreads) logprobs_kernel(const LogprobsArgs a) {
    __shared__ LpSmem sm;
    const int b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const uint32_t rank = lp_rank(), cluster = gridDim.x;
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");   // waited for before the first push
    if (tid == 0) sm.nhot = sm.ncand = 0;
    griddep_launch();
    griddep_wait();
    const float *z = a.logits + (long long)b * a.ld;
    // 16-byte aligned body of the row in slices of whole float4s, the ragged ends apart
    const int head = min(a.V, (int)((0u - (uint32_t)(uintptr_t)z >> 2) & 3u));
    const int quads = (a.V - head) >> 2, tail = head + 4 * quads;
    const int per = (quads + (int)cluster - 1) / (int)cluster;
    const int q0 = min(quads, (int)rank * per), nq = min(quads, q0 + per) - q0;
    const float4 *zq = reinterpret_cast<const float4 *>(z + head) + q0;
    const int at0 = head + 4 * q0;                          // index of the slice's first logit
    const int ends = rank == 0 ? head + (a.V - tail) : 0;   // at most 6, the first CTA's
    auto end_at = [&](int i) { return i < head ? i : tail + i - head; };

    LpStat st = {-INFINITY, 0.f, 0.f};
    lp_u64 best = 0;
    auto take = [&](const float *v, int n, auto index) {   // n logits, index(i) of each ascending
        float mx = st.m;
#pragma unroll
        for (int i = 0; i < n; ++i) mx = fmaxf(mx, v[i]);
        if (mx > st.m) {   // rare after the first steps
            st.shift(mx);
#pragma unroll
            for (int i = n - 1; i >= 0; --i)
                if (v[i] == mx) best = lp_key(mx, index(i));
        }
#pragma unroll
        for (int i = 0; i < n; ++i) {
            // below the maximum; kLpFar for NaN, -inf and in a row of nothing so far
            float d = fmaxf(v[i] - st.m, kLpFar);
            if (st.m == INFINITY) d = v[i] == INFINITY ? 0.f : kLpFar;
            const float e = lp_exp(d);
            st.s += e;
            st.t += e * d;
        }
    };
    for (int i0 = tid; i0 < nq; i0 += kLpUnroll * kLpThreads) {
        float v[4 * kLpUnroll];
#pragma unroll
        for (int k = 0; k < kLpUnroll; ++k) {
            const int i = i0 + k * kLpThreads;
            float4 f = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
            if (i < nq) f = __ldg(zq + i);
            v[4 * k] = f.x;
            v[4 * k + 1] = f.y;
            v[4 * k + 2] = f.z;
            v[4 * k + 3] = f.w;
        }
        take(v, 4 * kLpUnroll, [&](int j) { return (uint32_t)(at0 + 4 * (i0 + (j >> 2) * kLpThreads) + (j & 3)); });
    }
    if (tid < ends) {   // a lower index than the body's, or a higher one
        const int i = end_at(tid);
        const float v[1] = {z[i]};
        const lp_u64 before = best;
        const float m0 = st.m;
        take(v, 1, [&](int) { return (uint32_t)i; });
        if (v[0] == m0) best = lp_max(before, lp_key(v[0], i));
    }

    // ---- sums of the slice
    {
        LpStat r = st;
        const float mw = warp_max(r.m);
        r.shift(mw);
        r.s = warp_sum(r.s);
        r.t = warp_sum(r.t);
        if (lane == 0) sm.warp[w] = r;
    }
    if (a.top > 0) {
        lp_u64 g = lp_max(best, __shfl_xor_sync(0xffffffffu, best, 1));
        g = lp_max(g, __shfl_xor_sync(0xffffffffu, g, 2));
        if ((tid & 3) == 0) sm.group[tid >> 2] = g;
    }
    __syncthreads();
    if (a.top > 0) {
        // ---- the bound: the top-th highest of the group maxima (0: fewer groups hold logits)
        if (tid < kLpGroups) {
            const lp_u64 mine = sm.group[tid];
            int above = 0;
#pragma unroll 16
            for (int i = 0; i < kLpGroups; ++i) above += sm.group[i] > mine;
            if (mine && above < a.top) {
                sm.hot[atomicAdd(&sm.nhot, 1)] = tid;
                if (above == a.top - 1) sm.bound = mine;
            }
        }
        if (tid < kLpMaxTop) sm.list[tid] = 0ull;
        __syncthreads();
        const int nhot = sm.nhot;
        const lp_u64 bound = nhot < a.top ? 1ull : sm.bound;
        // ---- the logits of those groups (and the ends) that reach it
        auto offer = [&](float v, int i) {
            const lp_u64 k = lp_key(v, (uint32_t)i);
            if (k >= bound) {
                const int at = atomicAdd(&sm.ncand, 1);
                if (at < kLpCand) sm.cand[at] = k;
            }
        };
        const int steps = (nq + kLpThreads - 1) / kLpThreads;
        auto each_hot = [&](auto f) {   // every logit of the hot groups, once, by all threads
            for (long long j = tid; j < (long long)nhot * 4 * steps; j += kLpThreads) {
                const int i = sm.hot[(int)(j >> 2) % nhot] * 4 + (int)(j & 3) + (int)((j >> 2) / nhot) * kLpThreads;
                if (i < nq) {
                    const float4 v = __ldg(zq + i);
                    f(v.x, at0 + 4 * i);
                    f(v.y, at0 + 4 * i + 1);
                    f(v.z, at0 + 4 * i + 2);
                    f(v.w, at0 + 4 * i + 3);
                }
            }
            if (tid < ends) f(z[end_at(tid)], end_at(tid));
        };
        each_hot(offer);
        __syncthreads();
        const int n = sm.ncand;
        if (n <= kLpCand) {
            for (int i = tid; i < n; i += kLpThreads) {
                const lp_u64 k = sm.cand[i];
                int above = 0;
                for (int j = 0; j < n; ++j) above += sm.cand[j] > k;
                if (above < a.top) sm.list[above] = k;
            }
        } else {
            // more logits crowd into the hot groups than are ranked (large ones at
            // regular places): the next highest, one at a time
            lp_u64 last = ~0ull;
            for (int r = 0; r < a.top; ++r) {
                lp_u64 next = 0;
                each_hot([&](float v, int i) {
                    const lp_u64 k = lp_key(v, (uint32_t)i);
                    if (k < last && k > next) next = k;
                });
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) next = lp_max(next, __shfl_xor_sync(0xffffffffu, next, o));
                if (lane == 0) sm.wmax[w] = next;
                __syncthreads();
#pragma unroll
                for (int i = 0; i < kLpWarps; ++i) next = lp_max(next, sm.wmax[i]);
                if (tid == 0) sm.list[r] = next;
                last = next;
                __syncthreads();
            }
        }
        __syncthreads();
    }

    // ---- to the cluster's first CTA
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");   // it runs
    if (tid < a.top)
        asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(lp_first(&sm.lists[rank][tid])), "l"(sm.list[tid]) : "memory");
    if (tid == 0) {
        LpStat r = sm.warp[0];
#pragma unroll
        for (int i = 1; i < kLpWarps; ++i) r.join(sm.warp[i]);
        const uint32_t p = lp_first(&sm.stats[rank]);
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(p), "f"(r.m) : "memory");
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(p + 4), "f"(r.s) : "memory");
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(p + 8), "f"(r.t) : "memory");
    }
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (rank != 0) return;

    LpStat r = sm.stats[0];
    for (uint32_t i = 1; i < cluster; ++i) r.join(sm.stats[i]);
    const bool any = r.m > -INFINITY;
    const float ls = logf(r.s);
    if (tid == 0 && a.entropy) a.entropy[b] = any ? ls - r.t / r.s : 0.f;
    for (int j = tid; j < a.J; j += kLpThreads) {
        const int tok = a.tokens[(long long)b * a.J + j];
        float p = 0.f;   // no token
        if (tok < -1 || tok >= a.V) p = __uint_as_float(0x7fc00000u);
        else if (tok >= 0) p = any && z[tok] > -INFINITY ? (z[tok] == r.m ? 0.f : z[tok] - r.m) - ls : -INFINITY;
        a.logp[(long long)b * a.J + j] = p;
    }
    if (a.top > 0) {
        if (tid < a.top) sm.top[tid] = 0ull;
        __syncthreads();
        const int n = (int)cluster * a.top;
        if (tid < n) {
            const lp_u64 k = sm.lists[tid / a.top][tid % a.top];
            int above = 0;
            for (int i = 0; i < (int)cluster; ++i)
                for (int j = 0; j < a.top; ++j) above += sm.lists[i][j] > k;
            if (k && above < a.top) sm.top[above] = k;
        }
        __syncthreads();
        if (tid < a.top) {
            const lp_u64 k = sm.top[tid];
            const float v = k ? lp_logit(k) : 0.f;
            a.top_ids[(long long)b * a.top + tid] = k ? (int)unpack_index(k) : -1;
            a.top_logp[(long long)b * a.top + tid] = k ? (v == r.m ? 0.f : v - r.m) - ls : -INFINITY;
        }
    }
}

cudaError_t launch_logprobs(const LogprobsArgs &a, cudaStream_t s) {
    // slices of 8192 logits (one round of a CTA's loads) at least, eight of them at most
    int cluster = 1;
    while (cluster < kLpMaxCluster && a.V / (2 * cluster) >= kLpUnroll * kLpStep) cluster *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)cluster, (unsigned)a.B);
    cfg.blockDim = dim3(kLpThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = g_pdl ? 1 : 0;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, logprobs_kernel, a);
}

}  // namespace bloom
