// Log probabilities of given tokens, the entropy, and the top alternatives of
// rows of float32 logits (the values a serving step reports beside its tokens).
//
// With M = max z, S = sum exp(z_i - M) over the row:
//   logp_i = (z_i - M) - log S,  entropy = log S - (sum (z_i - M) exp(z_i - M)) / S
// (nats).  NaN and -inf logits take no part.  A +inf logit is the maximum: the
// +inf tokens share the mass.  The top alternatives are the k highest logits,
// equal ones by index.
#include <math.h>

#include "common.cuh"
#include "kernels.h"

namespace bloom {

constexpr int kLpThreads = 512;
constexpr int kLpWarps = kLpThreads / 32;

// (logit, index) as one number: a larger logit is larger, then a lower index; 0:
// a logit that takes no part.  -0 orders as +0.
__device__ __forceinline__ unsigned long long lp_key(float z, uint32_t i) {
    if (!(z > -INFINITY)) return 0ull;
    return pack_argmax(z == 0.f ? 0.f : z, i);
}
__device__ __forceinline__ float lp_logit(unsigned long long key) {
    const uint32_t k = (uint32_t)(key >> 32);
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

__global__ void __launch_bounds__(kLpThreads) logprobs_kernel(const LogprobsArgs a) {
    __shared__ unsigned long long sm_k[kLpWarps];
    __shared__ float sm_s[kLpWarps];
    griddep_launch();
    griddep_wait();
    const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const float *z = a.logits + (long long)b * a.ld;
    auto block_max = [&](unsigned long long v) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const unsigned long long y = __shfl_xor_sync(0xffffffffu, v, o);
            v = y > v ? y : v;
        }
        __syncthreads();
        if (lane == 0) sm_k[w] = v;
        __syncthreads();
        v = 0;
#pragma unroll
        for (int i = 0; i < kLpWarps; ++i) v = sm_k[i] > v ? sm_k[i] : v;
        return v;
    };
    unsigned long long best = 0;
    for (int i = tid; i < a.V; i += kLpThreads) {
        const unsigned long long k = lp_key(z[i], i);
        best = k > best ? k : best;
    }
    best = block_max(best);
    const float mx = lp_logit(best);
    const bool any = best != 0;
    float s = 0.f, t = 0.f;
    for (int i = tid; i < a.V; i += kLpThreads) {
        const float d = z[i] == mx ? 0.f : z[i] - mx, e = any && d <= 0.f ? expf(d) : 0.f;
        s += e;
        t += e > 0.f ? e * d : 0.f;
    }
    s = block_sum<kLpWarps>(s, sm_s);
    t = block_sum<kLpWarps>(t, sm_s);
    const float ls = logf(s);
    if (tid == 0 && a.entropy) a.entropy[b] = any ? ls - t / s : 0.f;
    for (int j = tid; j < a.J; j += kLpThreads) {
        const int tok = a.tokens[(long long)b * a.J + j];
        float r = 0.f;   // no token
        if (tok < -1 || tok >= a.V) r = __uint_as_float(0x7fc00000u);
        else if (tok >= 0) r = any && z[tok] > -INFINITY ? (z[tok] == mx ? 0.f : z[tok] - mx) - ls : -INFINITY;
        a.logp[(long long)b * a.J + j] = r;
    }
    for (int i = 0; i < a.top; ++i) {
        if (tid == 0) {
            const long long at = (long long)b * a.top + i;
            a.top_ids[at] = best ? (int)unpack_index(best) : -1;
            a.top_logp[at] = best ? (lp_logit(best) == mx ? 0.f : lp_logit(best) - mx) - ls : -INFINITY;
        }
        if (i + 1 == a.top) break;
        unsigned long long next = 0;
        for (int v = tid; v < a.V; v += kLpThreads) {
            const unsigned long long k = lp_key(z[v], v);
            if (k < best && k > next) next = k;
        }
        best = block_max(next);
    }
}

cudaError_t launch_logprobs(const LogprobsArgs &a, cudaStream_t s) {
    return launch_pdl(logprobs_kernel, dim3(a.B), dim3(kLpThreads), s, a);
}

}  // namespace bloom
