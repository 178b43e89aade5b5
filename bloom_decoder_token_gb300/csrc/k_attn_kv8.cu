// ALiBi decode attention over the 8-bit KV cache, for the last T tokens of every
// sequence (T = 1: a decode step; more: drafted tokens checked at once).
//
// Query token t of sequence b, t = 0 .. T-1, sits at slot lens[b] - T + t and
// sees the slots up to its own whose position is not -1:
//   s_k = (q . K_k) / sqrt(d) + slope_j * pos_k,  o = sum_k softmax(s)_k V_k,
// K and V being code * scale.  Scores, maxima, sums and the accumulators are
// float32.  A query that sees nothing gets 0.  Positions enter as pos_k - pos_ref
// (the softmax does not change), pos_ref the highest position among the last
// slots, so that a far position costs no bits of a near key's score.
#include <math.h>

#include "common.cuh"
#include "kernels.h"
#include "kv8_ops.cuh"

namespace bloom {

// One block per (query head, token, sequence); the warps take keys in turn, each
// with its own running maximum, sum and accumulator, merged in shared memory.
constexpr int kAk8Threads = 128;

template <int D, bool E4M3>
__global__ void __launch_bounds__(kAk8Threads) attn_kv8_kernel(const AttnKv8Args a) {
    constexpr int EPL = D / 32, NW = kAk8Threads / 32;   // elements per lane (2 or 4)
    __shared__ float sm_m[NW], sm_l[NW], sm_o[NW][D];
    griddep_launch();
    griddep_wait();
    const int j = blockIdx.x % a.n, t = blockIdx.x / a.n, b = blockIdx.y;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    int len = a.lens[b];
    if (len > a.max_seq) {
        if (a.err && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(a.err, kErrSlot);
        len = a.max_seq;
    }
    const int seen = len <= 0 ? 0 : len - a.T + t + 1;   // slots [0, seen)
    const int *pos = a.pos + (long long)b * a.max_seq;
    int ref = -1;
    for (int k0 = len; k0 > 0 && ref < 0; k0 -= 32)
        ref = __reduce_max_sync(0xffffffffu, k0 - 1 - lane >= 0 ? pos[k0 - 1 - lane] : -1);
    const long long bh = (long long)b * a.kv + j / (a.n / a.kv);
    const uint8_t *kc = a.kc + bh * a.max_seq * D + lane * EPL;
    const uint8_t *vc = a.vc + bh * a.max_seq * D + lane * EPL;
    const float *ks = a.ks + bh * a.blocks, *vs = a.vs + bh * a.blocks;
    const uint16_t *q = a.q + (((long long)b * a.T + t) * a.n + j) * D + lane * EPL;
    const float slope = a.slopes ? a.slopes[j] : 0.f;
    float qf[4], acc[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) qf[e] = e < EPL ? bf2f(q[e]) * a.scale : 0.f;
    auto load = [&](const uint8_t *p, float *f) {
        kv8_widen<E4M3>(EPL == 4 ? *reinterpret_cast<const uint32_t *>(p) : *reinterpret_cast<const uint16_t *>(p), f);
    };
    for (int k = w; k < seen; k += NW) {
        const int pk = pos[k];
        if (pk < 0) continue;
        float f[4], s = 0.f;
        load(kc + (long long)k * D, f);
#pragma unroll
        for (int e = 0; e < EPL; ++e) s += qf[e] * f[e];
        s = warp_sum(s) * ks[k / kKv8Block] + slope * (float)(pk - ref);
        const float mn = fmaxf(m, s), c = m == mn ? 1.f : expf(m - mn), p = expf(s - mn);
        load(vc + (long long)k * D, f);
        const float pv = p * vs[k / kKv8Block];
        l = l * c + p;
#pragma unroll
        for (int e = 0; e < EPL; ++e) acc[e] = acc[e] * c + pv * f[e];
        m = mn;
    }
    if (lane == 0) {
        sm_m[w] = m;
        sm_l[w] = l;
    }
#pragma unroll
    for (int e = 0; e < EPL; ++e) sm_o[w][lane * EPL + e] = acc[e];
    __syncthreads();
    if (threadIdx.x < D) {
        float mx = -INFINITY, lt = 0.f, o = 0.f;
#pragma unroll
        for (int i = 0; i < NW; ++i) mx = fmaxf(mx, sm_m[i]);
#pragma unroll
        for (int i = 0; i < NW; ++i) {
            const float c = sm_m[i] == -INFINITY && sm_l[i] == 0.f ? 0.f : expf(sm_m[i] - mx);
            if (c == 0.f) continue;
            lt += sm_l[i] * c;
            o += sm_o[i][threadIdx.x] * c;
        }
        a.o[(((long long)b * a.T + t) * a.n + j) * D + threadIdx.x] = f2bf(lt == 0.f ? 0.f : o / lt);
    }
}

cudaError_t launch_attn_kv8(const AttnKv8Args &a, int d, int e4m3, cudaStream_t s) {
    dim3 grid(a.n * a.T, a.B);
    if (d == 64)
        return launch_pdl(e4m3 ? attn_kv8_kernel<64, true> : attn_kv8_kernel<64, false>, grid, dim3(kAk8Threads), s, a);
    return launch_pdl(e4m3 ? attn_kv8_kernel<128, true> : attn_kv8_kernel<128, false>, grid, dim3(kAk8Threads), s, a);
}

}  // namespace bloom
