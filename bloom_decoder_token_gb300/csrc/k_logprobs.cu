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
// each CTA a contiguous slice, in rounds of 16 logits a thread.  Each thread keeps a
// running maximum and sums rescaled when it moves (float32), the next round's
// loads in flight meanwhile.  The top k come out of the same pass: after the
// first round (and, for a large k and many rounds, after the 5th, 25th, 125th)
// the k-th highest of the maxima of its groups of four threads is a lower bound
// of the slice's k-th highest logit; from then on a logit that reaches the bound becomes
// a candidate.  The candidates are ranked by counting, and the cluster's first
// CTA ranks the lists of all.  Measured (rows of 250880): 509 rows, top 1, 85 us =
// 6.0 TB/s (top 0: 78 us); 32 rows, top 20, 17 us (top 0: 9); one row, top 5, 8 us,
// most of it the chain of loads, bound, ranking and the cluster's barriers.
#include <float.h>
#include <math.h>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace bloom {

constexpr int kLpMaxCluster = 8;
constexpr int kLpUnroll = 4;                 // float4s of a thread's round
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
// Pairs of floats in one register pair, one instruction for both.
typedef unsigned long long lp_f2;
__device__ __forceinline__ lp_f2 lp_pack(float a, float b) {
    lp_f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void lp_unpack(lp_f2 v, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ lp_f2 lp_add2(lp_f2 a, lp_f2 b) {
    lp_f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ lp_f2 lp_mul2(lp_f2 a, lp_f2 b) {
    lp_f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ lp_f2 lp_fma2(lp_f2 a, lp_f2 b, lp_f2 c) {
    lp_f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ float lp_ex2(float x) {   // 2^x, relative error 2^-22
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float lp_exp(float d) { return lp_ex2(d * 1.4426950408889634f); }

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

// How many of p[0, n) are above k; p 16-byte aligned, in shared memory.
__device__ __forceinline__ int lp_above(const lp_u64 *p, int n, lp_u64 k) {
    int above = 0;
#pragma unroll 8
    for (int j = 0; j + 1 < n; j += 2) {
        const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(p + j);
        above += (v.x > k) + (v.y > k);
    }
    return above + ((n & 1) && p[n - 1] > k);
}

template <int THREADS>
struct LpSmem {
    static constexpr int kWarps = THREADS / 32, kGroups = THREADS / 4;
    alignas(16) uint32_t group[kGroups];          // order-preserving keys of the groups' maxima
    int index[kLpCand];                           // candidates
    alignas(16) lp_u64 cand[kLpCand];
    lp_u64 list[kLpMaxTop];                       // this slice's top, highest first
    alignas(16) lp_u64 lists[kLpMaxCluster * kLpMaxTop];   // first CTA: every slice's, [cluster][top]
    lp_u64 top[kLpMaxTop];
    LpStat stats[kLpMaxCluster];
    LpStat warp[kWarps];
    lp_u64 wmax[kWarps];
    uint32_t bound[2];                            // of alternate calls of rebound()
    lp_u64 key_bound;
    int ncand;
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

template <int THREADS>
__global__ void __launch_bounds__(THREADS) logprobs_kernel(const LogprobsArgs a) {
    // groups of four threads; float4s of a CTA's round
    constexpr int kWarps = THREADS / 32, kGroups = THREADS / 4, kRound = kLpUnroll * THREADS;
    static_assert(kGroups >= kLpMaxTop && THREADS >= kLpMaxTop, "a bound and a list for every top");
    __shared__ LpSmem<THREADS> sm;
    const int b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const uint32_t rank = lp_rank(), cluster = gridDim.x;
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");   // waited for before the first push
    if (tid == 0) sm.ncand = 0;
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
    float bound = __uint_as_float(0x7fc00000u);   // NaN: no logit reaches it
    auto offer = [&](int i) {
        const int at = atomicAdd(&sm.ncand, 1);
        if (at < kLpCand) sm.index[at] = i;
    };
    auto offer_all = [&](const float *v, int i0) {   // a round's logits that reach the bound
        uint32_t reach = 0;
#pragma unroll
        for (int j = 0; j < 4 * kLpUnroll; ++j) reach |= v[j] >= bound ? 1u << j : 0u;
        for (; reach; reach &= reach - 1) {
            const int j = __ffs(reach) - 1;
            offer(at0 + 4 * (i0 + (j >> 2) * THREADS) + (j & 3));
        }
    };
    auto take = [&](const float *v, int n) {   // into the sums; returns the maximum
        float mx = v[0];
#pragma unroll
        for (int i = 1; i < n; ++i) mx = fmaxf(mx, v[i]);
        if (mx > st.m) st.shift(mx);
        if (st.m == INFINITY) {
            for (int i = 0; i < n; ++i)
                if (v[i] == INFINITY) st.s += 1.f;
            return mx;
        }
        lp_f2 s = lp_pack(st.s, 0.f), t = lp_pack(st.t, 0.f);
        const lp_f2 minus = lp_pack(-st.m, -st.m), log2e = lp_pack(1.4426950408889634f, 1.4426950408889634f);
#pragma unroll
        for (int i = 0; i + 1 < n; i += 2) {
            float d0, d1, x0, x1;
            lp_unpack(lp_add2(lp_pack(v[i], v[i + 1]), minus), d0, d1);
            const lp_f2 d = lp_pack(fmaxf(d0, kLpFar), fmaxf(d1, kLpFar));   // kLpFar for NaN and -inf
            lp_unpack(lp_mul2(d, log2e), x0, x1);
            const lp_f2 e = lp_pack(lp_ex2(x0), lp_ex2(x1));
            s = lp_add2(s, e);
            t = lp_fma2(e, d, t);
        }
        float s0, s1, t0, t1;
        lp_unpack(s, s0, s1);
        lp_unpack(t, t0, t1);
        st.s = s0 + s1;
        st.t = t0 + t1;
        if (n & 1) {
            const float d = fmaxf(v[n - 1] - st.m, kLpFar), e = lp_exp(d);
            st.s += e;
            st.t += e * d;
        }
        return mx;
    };
    auto load_if = [&](int i0, float *v, auto all) {
        constexpr bool inside = decltype(all)::value;
#pragma unroll
        for (int k = 0; k < kLpUnroll; ++k) {
            const int i = i0 + k * THREADS;
            float4 f = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
            if (inside || i < nq) f = __ldg(zq + i);
            v[4 * k] = f.x;
            v[4 * k + 1] = f.y;
            v[4 * k + 2] = f.z;
            v[4 * k + 3] = f.w;
        }
    };
    auto load = [&](int r, float *v) {   // round r
        if ((r + 1) * kRound <= nq) load_if(r * kRound + tid, v, std::true_type{});
        else load_if(r * kRound + tid, v, std::false_type{});
    };
    int turn = 0;
    auto rebound = [&]() {   // from the maxima so far; by the whole CTA
        turn ^= 1;
        const float g = fmaxf(fmaxf(st.m, __shfl_xor_sync(0xffffffffu, st.m, 1)),
                              fmaxf(__shfl_xor_sync(0xffffffffu, st.m, 2), __shfl_xor_sync(0xffffffffu, st.m, 3)));
        if ((tid & 3) == 0) sm.group[tid >> 2] = (uint32_t)(lp_key(g, 0u) >> 32);   // 0: nothing
        if (tid == 0) sm.bound[turn] = 0u;
        __syncthreads();
        if (tid < kGroups) {
            const uint32_t mine = sm.group[tid];
            int above = 0, upto = 0;   // groups above this one; and equal ones too
#pragma unroll 8
            for (int i = 0; i < kGroups; i += 4) {
                const uint4 o = *reinterpret_cast<const uint4 *>(&sm.group[i]);
                above += (o.x > mine) + (o.y > mine) + (o.z > mine) + (o.w > mine);
                upto += (o.x >= mine) + (o.y >= mine) + (o.z >= mine) + (o.w >= mine);
            }
            if (above < a.top && a.top <= upto) sm.bound[turn] = mine;
        }
        __syncthreads();
        // no bound while fewer groups hold logits: all that take part
        const uint32_t found = sm.bound[turn];
        bound = found ? lp_logit((lp_u64)found << 32) : -FLT_MAX;
        return found != 0u;
    };
    const int rounds = (nq + kRound - 1) / kRound;
    const float end = tid < ends ? z[end_at(tid)] : -INFINITY;
    {
        int next = 0;   // the round after which the bound is found (again, where the first leaves many)
        auto round = [&](int r, const float *v) {
            const float mx = take(v, 4 * kLpUnroll);
            const int i0 = r * kRound + tid;
            if (a.top > 0 && r == next) {
                const float before = bound;
                // once more after the next round while there is none (logits ruled out in bulk)
                next = !rebound() ? r + 1 : a.top * rounds > kLpCand / 4 ? 5 * r + 4 : rounds;
                if (!(before == before)) {   // the first
                    offer_all(v, i0);
                    if (end >= bound) offer(end_at(tid));
                    return;
                }
            }
            if (mx >= bound && *(volatile int *)&sm.ncand <= kLpCand) offer_all(v, i0);   // more are not ranked
        };
        float v[2][4 * kLpUnroll];
        load(0, v[0]);
        if (tid < ends) take(&end, 1);
        for (int r = 0; r < max(rounds, 1); r += 2) {
            load(r + 1, v[1]);
            round(r, v[0]);
            load(r + 2, v[0]);
            if (r + 1 < rounds) round(r + 1, v[1]);
        }
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
    if (a.top > 0 && tid < kLpMaxTop) sm.list[tid] = 0ull;
    __syncthreads();
    if (a.top > 0) {
        int n = sm.ncand;
        auto each = [&](auto see) {   // the slice's logits and their indexes
            for (int i = tid; i < nq; i += THREADS) {
                const float4 v = __ldg(zq + i);
                see(v.x, at0 + 4 * i);
                see(v.y, at0 + 4 * i + 1);
                see(v.z, at0 + 4 * i + 2);
                see(v.w, at0 + 4 * i + 3);
            }
            if (tid < ends) see(end, end_at(tid));
        };
        if (n > kLpCand) {
            // More logits reached the bounds than are ranked (equal ones, a finite value for
            // ruled-out tokens, ascending ones).  No two (logit, index) keys are equal: the
            // k-th highest of the groups' highest keys leaves few however many logits are
            // equal, for two more passes over the slice (32 rows of 250880, all but three one
            // value, top 20: 38 us; a pass for each alternative: 175).
            lp_u64 best = 0;
            each([&](float v, int i) { best = lp_max(best, lp_key(v, (uint32_t)i)); });
            best = lp_max(best, __shfl_xor_sync(0xffffffffu, best, 1));
            best = lp_max(best, __shfl_xor_sync(0xffffffffu, best, 2));
            if ((tid & 3) == 0) sm.cand[tid >> 2] = best;
            if (tid == 0) sm.key_bound = 0ull;
            __syncthreads();
            if (tid < kGroups) {
                const lp_u64 mine = sm.cand[tid];
                if (mine && lp_above(sm.cand, kGroups, mine) == a.top - 1) sm.key_bound = mine;
            }
            if (tid == 0) sm.ncand = 0;
            __syncthreads();
            const lp_u64 kb = lp_max(sm.key_bound, 1ull);   // 0, fewer groups than top: all that take part
            each([&](float v, int i) {
                if (lp_key(v, (uint32_t)i) >= kb) offer(i);
            });
            __syncthreads();
            n = sm.ncand;
        }
        if (n <= kLpCand) {
            for (int i = tid; i < n; i += THREADS) sm.cand[i] = lp_key(z[sm.index[i]], (uint32_t)sm.index[i]);
            __syncthreads();
            for (int i = tid; i < n; i += THREADS) {
                const lp_u64 k = sm.cand[i];
                const int above = lp_above(sm.cand, n, k);
                if (above < a.top) sm.list[above] = k;
            }
        } else {
            // still more (a few groups hold them all): the next highest, one at a time
            lp_u64 last = ~0ull;
            for (int r = 0; r < a.top; ++r) {
                lp_u64 next = 0;
                each([&](float v, int i) {
                    const lp_u64 k = lp_key(v, (uint32_t)i);
                    if (k < last && k > next) next = k;
                });
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) next = lp_max(next, __shfl_xor_sync(0xffffffffu, next, o));
                if (lane == 0) sm.wmax[w] = next;
                __syncthreads();
#pragma unroll
                for (int i = 0; i < kWarps; ++i) next = lp_max(next, sm.wmax[i]);
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
        asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(lp_first(&sm.lists[rank * a.top + tid])), "l"(sm.list[tid]) : "memory");
    if (tid == 0) {
        LpStat r = sm.warp[0];
#pragma unroll
        for (int i = 1; i < kWarps; ++i) r.join(sm.warp[i]);
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
    for (int j = tid; j < a.J; j += THREADS) {
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
        for (int i = tid; i < n; i += THREADS) {
            const lp_u64 k = sm.lists[i];
            const int above = lp_above(sm.lists, n, k);
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

template <int THREADS>
static cudaError_t lp_launch(const LogprobsArgs &a, int cluster, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)cluster, (unsigned)a.B);
    cfg.blockDim = dim3(THREADS);
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
    return cudaLaunchKernelEx(&cfg, logprobs_kernel<THREADS>, a);
}

cudaError_t launch_logprobs(const LogprobsArgs &a, cudaStream_t s) {
    // Many short rows: CTAs of 128 threads, eight of which fit an SM, hide one another's
    // phases (512 against 128 threads, top 5: 5000 rows of 2000 103, 27 us; 512 of 8000 13.9,
    // 9.3; 2000 of 30000 66, 52; but 300 of 16000 8.9, 10.7; 500 of 30000 21, 24; 64 of 12000,
    // top 20, 7.0, 12.4).  The bound of 32 groups is low for a top near 32: normal logits
    // then give hundreds of candidates, or more than are ranked (512 against 128 threads, 700 rows of
    // 16000, top 20, 24, 32: 28, 28, 28 against 34, 44, 120 us; 2000 of 6000: 50, 52, 52
    // against 28, 32, 100; but top 32 of 2000 rows of 3000: 50 against 40; of 1000 of 4096: 30, 40)
    const int sms = bloom_device_sms();
    const bool many = a.V < 65536 && a.B > (a.V <= 8192 ? 2 : 4) * sms;
    if (a.V <= 2048 || (many && (a.V <= 4096 || a.top <= 24))) return lp_launch<128>(a, 1, s);
    // Two CTAs of 512 fit an SM.  Slices of a round (8192 logits) at least, eight at most,
    // and no more of them than fill the GPU twice: what a slice costs beside its loads
    // (its bound, its list) is then shared by more logits (509 rows of 250880, top 1:
    // 87 us in whole rows, 94 in halves, 111 in quarters, 157 in eighths; 32 rows,
    // top 20, in eighths: 17 us)
    int cluster = 1;
    while (cluster < kLpMaxCluster && a.V / (2 * cluster) >= 4 * kLpUnroll * 512 &&
           2ll * a.B * cluster <= 4ll * sms)
        cluster *= 2;
    return lp_launch<512>(a, cluster, s);
}

}  // namespace bloom
