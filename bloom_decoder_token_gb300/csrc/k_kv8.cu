// Writing and reading back the 8-bit KV cache (kv8_ops.cuh has its arithmetic).
//
// Both kernels give one warp to one tile of up to 32 tokens of one (sequence,
// head), K or V: 32 x d values, all of whose loads (16 per lane at d = 128) are
// in flight at once.  Both are bound by HBM: 3 bytes a value (2 + 1).
// Neighbouring warps take K and V, then neighbouring heads, which lie side by
// side in a fused QKV row.  Measured (int8, 8 x 2048 tokens, 32 x 128, 403 MB
// each): write 59.5 us, read-back 61.8 us = 6.8, 6.5 TB/s (a copy: 6.7); one
// token for each of 32 rows 3.4 us, 7 us where every block's scale grows.
#include "common.cuh"
#include "kernels.h"
#include "kv8_ops.cuh"

namespace bloom {

constexpr int kKv8Threads = 128;

// Rows idle in this call: start < 0.  Tokens t in [0, count) go to slots start + t.
struct Kv8Range {
    long long lo, hi;   // slots [lo, hi) of the row
};
__device__ __forceinline__ Kv8Range kv8_range(const int *start, const int *count, int b, int T,
                                              int max_seq, int *err, bool report) {
    const int s = start[b];
    const int c = count ? max(0, min(count[b], T)) : T;
    Kv8Range r;
    r.lo = s;
    r.hi = s < 0 ? s : (long long)s + c;
    if (r.hi > max_seq) {
        if (report && err) atomicOr(err, kErrSlot);
        r.hi = max_seq;
    }
    return r;
}

// One warp: the tokens of one call that fall into one block of kKv8Block slots
// of a (sequence, head), K or V.  The block's scale covers what the block held
// before (slots below the row's start) and the new tokens; where it grows, the
// codes held before are rounded again.  A masked token is stored as zeros.
template <int D, bool E4M3>
__global__ void __launch_bounds__(kKv8Threads) kv8_write_kernel(const Kv8WriteArgs a) {
    constexpr int LPR = D / 16, RPP = 32 / LPR, NP = kKv8Block / RPP;   // lanes a row, rows a pass, passes
    griddep_launch();
    griddep_wait();
    const long long wid = (long long)blockIdx.x * (kKv8Threads / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const int kv = (int)(wid & 1);
    const uint32_t rest = (uint32_t)(wid >> 1), tile = rest / (uint32_t)a.n;
    const int h = (int)(rest - tile * (uint32_t)a.n), b = (int)(tile / (uint32_t)a.tiles);
    const int i = (int)(tile - (uint32_t)b * (uint32_t)a.tiles);
    if (b >= a.B) return;
    const Kv8Range row = kv8_range(a.start, a.count, b, a.T, a.max_seq, a.err, i == 0 && h == 0 && lane == 0);
    if (row.lo >= row.hi) return;
    const int blk = (int)(row.lo / kKv8Block) + i, base = blk * kKv8Block;
    const int lo = max((int)row.lo, base), hi = (int)min(row.hi, (long long)base + kKv8Block);
    if (lo >= hi) return;

    const uint16_t *src = (kv ? a.v : a.k) + b * a.stride[kv][0] + h * a.stride[kv][2];
    const long long ts = a.stride[kv][1];
    const int r0 = lane / LPR, c0 = (lane % LPR) * 16;
    uint4 x[NP][2];
    uint32_t m2 = 0;   // two running maxima of |bf16| bits
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        const int slot = base + p * RPP + r0, t = slot - (int)row.lo;
        const bool on = slot >= lo && slot < hi && (!a.mask || a.mask[(long long)b * a.T + t]);
        x[p][0] = x[p][1] = make_uint4(0u, 0u, 0u, 0u);
        if (on) {
            const uint4 *q = reinterpret_cast<const uint4 *>(src + t * ts + c0);
            x[p][0] = q[0];
            x[p][1] = q[1];
        }
    }
#pragma unroll
    for (int p = 0; p < NP; ++p)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            m2 = __vmaxu2(m2, x[p][u].x & 0x7fff7fffu);
            m2 = __vmaxu2(m2, x[p][u].y & 0x7fff7fffu);
            m2 = __vmaxu2(m2, x[p][u].z & 0x7fff7fffu);
            m2 = __vmaxu2(m2, x[p][u].w & 0x7fff7fffu);
        }
    const uint32_t amax = __reduce_max_sync(0xffffffffu, max(m2 & 0xffffu, m2 >> 16));
    float s = kv8_scale<E4M3>(amax);

    const long long bh = (long long)b * a.n + h;
    uint8_t *codes = (kv ? a.vc : a.kc) + (bh * a.max_seq + base) * D;
    float *scale = (kv ? a.vs : a.ks) + bh * a.blocks + blk;
    if (lo > base) {   // the block held tokens before
        const float old = *scale;
        s = old > s || old != old ? old : s;   // NaN, once there, stays
        __syncwarp();
        if (s > old) {
            const float shift = old / s;
#pragma unroll 1
            for (int r = r0; r < lo - base; r += RPP) {
                uint4 *p = reinterpret_cast<uint4 *>(codes + r * D + c0);
                if (old == 0.f) {   // whatever the codes, they stood for 0
                    *p = make_uint4(0u, 0u, 0u, 0u);
                    continue;
                }
                uint4 w = *p;
                uint32_t *wp = &w.x;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float f[4];
                    kv8_widen<E4M3>(wp[e], f);
                    wp[e] = kv8_narrow<E4M3>(f[0] * shift, f[1] * shift, f[2] * shift, f[3] * shift);
                }
                *p = w;
            }
        }
    }
    if (lane == 0) *scale = s;
    const float inv = s > 0.f ? 1.f / s : 0.f;   // s NaN: zero codes
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        const int r = p * RPP + r0;
        if (base + r < lo || base + r >= hi) continue;
        uint4 w;
        uint32_t *wp = &w.x;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            float f[8];
            unpack8(x[p][u], f);
            if (!(inv > 0.f)) {
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = 0.f;
            }
            wp[2 * u] = kv8_narrow<E4M3>(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv);
            wp[2 * u + 1] = kv8_narrow<E4M3>(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv);
        }
        *reinterpret_cast<uint4 *>(codes + r * D + c0) = w;
    }
}

// One warp: 32 tokens of one (sequence, head), K or V, widened to bf16.  Tokens
// that the call does not read (idle row, t >= count, beyond the cache) are 0.
// A lane takes 8 codes of a row, so that its 16-byte store lies beside its
// neighbours' (16 codes a lane, two 16-byte stores 32 bytes apart: 5.4 TB/s).
template <int D, bool E4M3>
__global__ void __launch_bounds__(kKv8Threads) kv8_read_kernel(const Kv8ReadArgs a) {
    constexpr int LPR = D / 8, RPP = 32 / LPR, NP = 32 / RPP;
    griddep_launch();
    griddep_wait();
    const long long wid = (long long)blockIdx.x * (kKv8Threads / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const int kv = (int)(wid & 1);
    const uint32_t rest = (uint32_t)(wid >> 1), tile = rest / (uint32_t)a.n;
    const int h = (int)(rest - tile * (uint32_t)a.n), b = (int)(tile / (uint32_t)a.tiles);
    const int i = (int)(tile - (uint32_t)b * (uint32_t)a.tiles);
    if (b >= a.B) return;
    const Kv8Range row = kv8_range(a.start, a.count, b, a.T, a.max_seq, a.err, i == 0 && h == 0 && lane == 0);
    const long long bh = (long long)b * a.n + h;
    const int r0 = lane / LPR, c0 = (lane % LPR) * 8;
    const long long first = row.lo + i * 32;   // the tile's first slot; `here` of its slots are read
    const int here = row.lo < 0 ? 0 : (int)max(0ll, min(32ll, row.hi - first));
    const uint8_t *codes = (kv ? a.vc : a.kc) + (bh * a.max_seq + first + r0) * D + c0;
    const float *scale = (kv ? a.vs : a.ks) + bh * a.blocks;
    uint2 w[NP];
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        w[p] = make_uint2(0u, 0u);
        if (p * RPP + r0 < here) w[p] = *reinterpret_cast<const uint2 *>(codes + p * RPP * D);
    }
    // a tile lies in two blocks at most: slots below `turn` in the first
    const int blk = (int)(first / kKv8Block), turn = kKv8Block - (int)(first - (long long)blk * kKv8Block);
    const float s0 = here > 0 ? scale[blk] : 0.f, s1 = here > turn ? scale[blk + 1] : 0.f;
    uint16_t *dst = (kv ? a.v : a.k) + b * a.stride[kv][0] + h * a.stride[kv][2] + (i * 32 + r0) * a.stride[kv][1] + c0;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        const int r = p * RPP + r0;
        if (i * 32 + r >= a.T) continue;
        const float s = r < turn ? s0 : s1;
        float f[8];
        kv8_widen<E4M3>(w[p].x, f);
        kv8_widen<E4M3>(w[p].y, f + 4);
        uint4 o = make_uint4(kv8_bf16x2(f[0] * s, f[1] * s), kv8_bf16x2(f[2] * s, f[3] * s),
                             kv8_bf16x2(f[4] * s, f[5] * s), kv8_bf16x2(f[6] * s, f[7] * s));
        if (r >= here) o = make_uint4(0u, 0u, 0u, 0u);
        *reinterpret_cast<uint4 *>(dst + p * RPP * a.stride[kv][1]) = o;
    }
}

template <typename A, typename K>
static cudaError_t kv8_launch(K k64i, K k64e, K k128i, K k128e, const A &a, int d, int e4m3,
                              cudaStream_t s) {
    const long long warps = (long long)a.B * a.tiles * a.n * 2;
    const long long ctas = (warps + kKv8Threads / 32 - 1) / (kKv8Threads / 32);
    if (ctas > 0x7fffffffll) return cudaErrorInvalidValue;
    return launch_pdl(d == 64 ? (e4m3 ? k64e : k64i) : (e4m3 ? k128e : k128i), dim3((unsigned)ctas),
                      dim3(kKv8Threads), s, a);
}

cudaError_t launch_kv8_write(Kv8WriteArgs a, int d, int e4m3, cudaStream_t s) {
    a.tiles = (a.T + 2 * kKv8Block - 2) / kKv8Block;   // blocks that T slots touch at most
    return kv8_launch(kv8_write_kernel<64, false>, kv8_write_kernel<64, true>,
                      kv8_write_kernel<128, false>, kv8_write_kernel<128, true>, a, d, e4m3, s);
}

cudaError_t launch_kv8_read(Kv8ReadArgs a, int d, int e4m3, cudaStream_t s) {
    a.tiles = (a.T + 31) / 32;
    return kv8_launch(kv8_read_kernel<64, false>, kv8_read_kernel<64, true>,
                      kv8_read_kernel<128, false>, kv8_read_kernel<128, true>, a, d, e4m3, s);
}

}  // namespace bloom
