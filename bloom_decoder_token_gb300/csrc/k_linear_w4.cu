// Linear layer over 4-bit weights with group scales, for the few tokens of a decode
// step: y[m][n] = epilogue(sum_k code[n][k] scale[n][k / group] x[m][k] + bias[n]).
//
// At so few tokens the time is the time to read the weights once, 4.25 bits each at
// groups of 64, and the arithmetic has to stay out of the way of 46 codes a clock and SM:
//  * The codes go into mma.sync m16n8k32 as e4m3 numbers, which they are but for two
//    masks and a turn a word (w4_ops.cuh): 3 instructions for 8 codes, where f16 took
//    9.  Measured here (2070 MHz, one SM): m16n8k32 of e4m3 1.2 clocks, m16n8k16 of f16
//    2.1, so the same product costs 3.6 times less; its sums keep 24 bits.
//  * An activation is two e4m3 numbers in neighbouring columns: x = hi + lo / 16, after a
//    power of two that brings the largest of the token's 256 values to [2^7, 2^8).  bf16 has 8
//    significant bits, an e4m3 4: nothing is lost down to 2^-14 of that largest value;
//    smaller ones are off by 2^-22 of it at most.  So four tokens fill the eight columns.
//    A token with an infinity or NaN gives NaN.
//  * A group's products are summed apart, then times the scale into the float32 sums.
//  * A warp owns 256 columns, whose activations stay in its registers, and goes down the
//    matrix: tile after tile of 16 rows, by bulk copies into a ring of its own.  The
//    warps of a CTA that share the rows hold the CTA's columns together; their sums
//    meet in shared memory, in the warps' order, once a row of tiles.
//  * Longer rows are split over the CTAs of a cluster, whose sums meet through distributed
//    shared memory, in rank order; still longer ones are taken in passes.
#include <atomic>
#include <math.h>

#include "common.cuh"
#include "kernels.h"
#include "tc_ops.cuh"
#include "w4_ops.cuh"

namespace bloom {

constexpr int kLw4Partial = 16384;               // bytes of a buffer of sums that wait for the cluster
constexpr int kLw4Stride = 24;                   // floats of a token's 16 rows in a warp's sums: no bank twice
constexpr int lw4_warps(int NT) { return NT == 8 ? 8 : 16; }

template <int NT, int G>
struct Lw4Smem {
    static constexpr int kWarps = lw4_warps(NT), kStages = 64 / kWarps, kTile = w4_tile_bytes(G);
    static constexpr int kSums = kWarps * 4 * NT * kLw4Stride * 4;   // one of the two buffers
    static constexpr int kRing = kWarps * kStages * kTile;
    static constexpr int kBytes = kRing + 2 * kSums + 2 * kLw4Partial + kWarps * kStages * 8;
};

__device__ __forceinline__ void lw4_mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint16_t lw4_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ void lw4_widen(uint16_t v, float &lo, float &hi) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(v));
    asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.f32.f16 %0, l;\n cvt.f32.f16 %1, h;\n}\n" : "=f"(lo), "=f"(hi) : "r"(h));
}
__device__ __forceinline__ void lw4_bulk(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(tc_smem(dst)),
                 "l"(src), "r"(bytes), "r"(tc_smem(bar))
                 : "memory");
}
__device__ __forceinline__ void lw4_cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ void lw4_store(const LinearW4Args &a, int m, int row, float v) {
    if (row >= a.N) return;
    if (a.bias) v += bf2f(a.bias[row]);
    if (a.epi == EPI_GELU) v = gelu_tanh(v);
    const long long at = m * a.ldy + row;
    if (a.f32) {
        float *y = static_cast<float *>(a.y) + at;
        *y = a.epi == EPI_RESID ? *y + v : v;
    } else {
        uint16_t *y = static_cast<uint16_t *>(a.y) + at;
        *y = f2bf(a.epi == EPI_RESID ? bf2f(*y) + v : v);
    }
}

// Where a warp is: its rows of tiles in chunks (whose sums wait for the cluster
// together), the passes over the columns within a chunk, the steps within a pass.
struct Lw4Place {
    int cb, pass, rb;
};

// NT: column tiles, four tokens each.
template <int NT, int G>
__global__ void __launch_bounds__(32 * lw4_warps(NT), 1) linear_w4_kernel(const LinearW4Args a) {
    using Smem = Lw4Smem<NT, G>;
    constexpr int NW = Smem::kWarps, ST = Smem::kStages, TB = Smem::kTile, THREADS = 32 * NW;
    extern __shared__ __align__(128) unsigned char lw4_smem[];
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, g = lane >> 2, q = lane & 3;
    unsigned char *ring = lw4_smem + w * ST * TB;
    float *sums = reinterpret_cast<float *>(lw4_smem + Smem::kRing);              // [2][NW][4 NT][kLw4Stride]
    float *part = sums + 2 * (Smem::kSums / 4);                                   // [2][rows of tiles][tokens][16]
    uint64_t *bar = reinterpret_cast<uint64_t *>(part + 2 * (kLw4Partial / 4)) + w * ST;
    if (lane == 0) {
        for (int i = 0; i < ST; ++i) tc_mbar_init(&bar[i], 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncwarp();
    griddep_wait();
    griddep_launch();

    const int P = a.cluster, cl = (int)blockIdx.x / P, rank = (int)blockIdx.x - cl * P, clusters = (int)gridDim.x / P;
    const int rb0 = (int)((long long)a.row_tiles * cl / clusters), rb1 = (int)((long long)a.row_tiles * (cl + 1) / clusters);
    const int m0 = (int)blockIdx.y * 4 * NT, Mt = min(a.M - m0, 4 * NT);
    const int KW = a.k_warps, RW = a.row_warps, slot = w / KW, kw = w - slot * KW;
    const bool direct = P == 1 && a.passes == 1;

    // the place's column tile, and whether this warp has work there
    auto kt_of = [&](int pass) { return (pass * P + rank) * KW + kw; };
    auto has = [&](const Lw4Place &at) {
        return slot < RW && at.rb + slot < min(at.cb + a.chunk, rb1) && kt_of(at.pass) < a.k_tiles;
    };
    auto next = [&](Lw4Place &at) {
        at.rb += RW;
        if (at.rb < min(at.cb + a.chunk, rb1)) return;
        at.rb = at.cb;
        if (++at.pass < a.passes) return;
        at.pass = 0;
        at.cb += a.chunk;
        at.rb = at.cb;
    };
    Lw4Place ahead = {rb0, 0, rb0};
    int issued = 0;
    auto issue = [&](int st) {
        while (ahead.cb < rb1 && !has(ahead)) next(ahead);
        if (ahead.cb >= rb1) return;
        if (lane == 0) {
            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(tc_smem(&bar[st])), "r"(TB) : "memory");
            lw4_bulk(ring + st * TB, a.tiles + ((long long)(ahead.rb + slot) * a.k_tiles + kt_of(ahead.pass)) * TB, TB, &bar[st]);
        }
        ++issued;
        next(ahead);
    };
    for (int i = 0; i < ST; ++i) issue(i);

    uint32_t b[NT][8][2];   // activations: column g (token g / 2, part g % 2), elements 32 j + 8 q + (0..3 | 4..7)
    float inv[NT];          // 2^-up of token q of the tile
    auto load_x = [&](int kt) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int token = 4 * nt + (g >> 1), piece = g & 1;   // both parts of half the elements; the rest by the neighbour
            const uint16_t *x = a.x + (m0 + token) * a.ldx + kt * kW4Cols + 8 * q + 4 * piece;
            uint2 raw[8];
            uint32_t m2 = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                raw[j] = make_uint2(0u, 0u);
                if (token < Mt && kt * kW4Cols + 32 * j + 8 * q < a.K) raw[j] = __ldg(reinterpret_cast<const uint2 *>(x + 32 * j));
                m2 = __vmaxu2(m2, raw[j].x & 0x7fff7fffu);
                m2 = __vmaxu2(m2, raw[j].y & 0x7fff7fffu);
            }
            uint32_t amax = max(m2 & 0xffffu, m2 >> 16);
            amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 4));
            // 2^up brings the largest element to [2^7, 2^8)
            const int up = min(120, 7 + 127 - (int)(amax >> 7));
            const float mul = __uint_as_float((uint32_t)(127 + up) << 23);
            inv[nt] = __shfl_sync(0xffffffffu, __uint_as_float((uint32_t)(127 - up) << 23), 8 * q);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float f[4] = {bf_lo(raw[j].x) * mul, bf_hi(raw[j].x) * mul, bf_lo(raw[j].y) * mul, bf_hi(raw[j].y) * mul};
                const uint16_t h0 = lw4_e4m3x2(f[0], f[1]), h1 = lw4_e4m3x2(f[2], f[3]);
                float r[4];
                lw4_widen(h0, r[0], r[1]);
                lw4_widen(h1, r[2], r[3]);
                const uint16_t l0 = lw4_e4m3x2((f[0] - r[0]) * 16.f, (f[1] - r[1]) * 16.f);
                const uint16_t l1 = lw4_e4m3x2((f[2] - r[2]) * 16.f, (f[3] - r[3]) * 16.f);
                uint32_t hi = (uint32_t)h0 | (uint32_t)h1 << 16, lo = (uint32_t)l0 | (uint32_t)l1 << 16;
                if (amax >= 0x7f80u) hi = lo = 0x7f7f7f7fu;   // NaN
                // piece 0 (elements 0..3) keeps its hi and gets the neighbour's, piece 1 the lo's
                const uint32_t other = __shfl_xor_sync(0xffffffffu, piece ? hi : lo, 4);
                b[nt][j][0] = piece ? other : hi;
                b[nt][j][1] = piece ? lo : other;
            }
        }
    };

    int st = 0, used = 0, turn = 0, fill = 0;   // turn: buffer of sums; fill: of partial sums
    uint32_t parity = 0;
    bool lost = false;                          // a wait expired
    for (int cb = rb0; cb < rb1; cb += a.chunk, fill ^= 1) {
        const int ce = min(cb + a.chunk, rb1);
        float *mine = part + fill * (kLw4Partial / 4);
        for (int pass = 0; pass < a.passes; ++pass) {
            const int kt = kt_of(pass);
            if (slot < RW && kt < a.k_tiles && (a.passes > 1 || cb == rb0)) load_x(kt);
            const int nk = min(KW, a.k_tiles - (pass * P + rank) * KW);   // warps with columns, of those that share rows
            for (int rb = cb; rb < ce; rb += RW, turn ^= 1) {
                float *sum = sums + turn * (Smem::kSums / 4);
                if (has(Lw4Place{cb, pass, rb})) {
                    if (!lost && !__all_sync(0xffffffffu, tc_mbar_wait_within(&bar[st], parity, a.wait_ns))) {
                        lost = true;
                        if (a.err && lane == 0) atomicOr(a.err, kErrTimeout);
                    }
                    float acc[NT][2];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) acc[nt][0] = acc[nt][1] = lost ? __uint_as_float(0x7fc00000u) : 0.f;
                    if (!lost) {
                        const unsigned char *tile = ring + st * TB;
                        uint4 v[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const uint4 *>(tile + i * 512 + lane * 16);
#pragma unroll
                        for (int gr = 0; gr < kW4Cols / G; ++gr) {
                            const uint32_t sc = *reinterpret_cast<const uint32_t *>(tile + 2048 + gr * 32 + g * 4);
                            float c[NT][4];
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int e = 0; e < 4; ++e) c[nt][e] = 0.f;
#pragma unroll
                            for (int j = gr * (G / 32); j < (gr + 1) * (G / 32); ++j) {
                                const uint32_t w0 = (&v[j / 2].x)[2 * (j & 1)], w1 = (&v[j / 2].x)[2 * (j & 1) + 1];
                                const uint32_t a0 = w4_low(w0), a1 = w4_low(w1), a2 = w4_high(w0), a3 = w4_high(w1);
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) lw4_mma(c[nt], a0, a1, a2, a3, b[nt][j][0], b[nt][j][1]);
                            }
                            const float s0 = bf_lo(sc), s1 = bf_hi(sc);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                acc[nt][0] += s0 * (c[nt][0] + c[nt][1] * 0.0625f);
                                acc[nt][1] += s1 * (c[nt][2] + c[nt][3] * 0.0625f);
                            }
                        }
                        __syncwarp();   // the tile has been read
                        ++used;
                        issue(st);
                        if (++st == ST) {
                            st = 0;
                            parity ^= 1u;
                        }
                    }
                    float *to = sum + w * (4 * NT * kLw4Stride) + q * kLw4Stride + g;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {   // the codes' 2^-9 back, then the activations' power of two
                        to[4 * nt * kLw4Stride] = acc[nt][0] * 512.f * inv[nt];
                        to[4 * nt * kLw4Stride + 8] = acc[nt][1] * 512.f * inv[nt];
                    }
                }
                __syncthreads();
                // the warps' sums; each step other warps begin
                const int rows = min(RW, ce - rb);
                for (int i = (tid - 32 * (rb - cb)) & (THREADS - 1); i < rows * Mt * 16; i += THREADS) {
                    const int r = i & 15, mt = i >> 4, s = mt / Mt, m = mt - s * Mt;
                    const float *from = sum + s * KW * (4 * NT * kLw4Stride) + m * kLw4Stride + r;
                    float v = 0.f;
                    for (int k = 0; k < nk; ++k) v += from[k * (4 * NT * kLw4Stride)];
                    if (direct) {
                        lw4_store(a, m0 + m, (rb + s) * kW4Rows + r, v);
                    } else {
                        float *p = mine + ((rb - cb + s) * 4 * NT + m) * 16 + r;
                        *p = pass == 0 ? v : *p + v;
                    }
                }
            }
        }
        if (direct) continue;
        // the ranks' sums.  A buffer is written again after the next one's barrier, which
        // every rank reaches when it has read this one.
        lw4_cluster_sync();
        for (int i = rank * THREADS + tid; i < (ce - cb) * Mt * 16; i += P * THREADS) {
            const int r = i & 15, mt = i >> 4, s = mt / Mt, m = mt - s * Mt;
            const uint32_t at = tc_smem(mine + (s * 4 * NT + m) * 16 + r);
            float v = 0.f;
#pragma unroll 8
            for (int k = 0; k < P; ++k) {
                uint32_t there;
                float f;
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(at), "r"(k));
                asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(f) : "r"(there) : "memory");
                v += f;
            }
            lw4_store(a, m0 + m, (cb + s) * kW4Rows + r, v);
        }
    }
    if (!direct) lw4_cluster_sync();   // a rank's shared memory lives until all have read it
    // copies in flight behind an expired wait land before the CTA ends
    for (; lost && used < issued; ++used) {
        tc_mbar_wait(&bar[st], parity, kTcWaitNs);
        if (++st == ST) {
            st = 0;
            parity ^= 1u;
        }
    }
}

template <int NT, int G>
static cudaError_t lw4_launch(LinearW4Args a, int sms, cudaStream_t s) {
    using Smem = Lw4Smem<NT, G>;
    constexpr int kDevices = 64, kMaxCluster = 8, NW = Smem::kWarps;
    static std::atomic<int> known[kDevices][kMaxCluster + 1];   // clusters that are resident at once
    const auto kern = linear_w4_kernel<NT, G>;
    const int per = (a.k_tiles + NW - 1) / NW;
    a.cluster = per < kMaxCluster ? per : kMaxCluster;
    a.passes = (a.k_tiles + a.cluster * NW - 1) / (a.cluster * NW);
    a.k_warps = (a.k_tiles + a.cluster * a.passes - 1) / (a.cluster * a.passes);

    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(32 * NW);
    cfg.dynamicSmemBytes = Smem::kBytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)a.cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = g_pdl ? 1 : 0;
    cfg.attrs = attr;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    int clusters = dev < kDevices ? known[dev][a.cluster].load(std::memory_order_relaxed) : 0;
    if (clusters == 0) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem::kBytes);
        if (e != cudaSuccess) return e;
        clusters = sms / a.cluster;
        if (a.cluster > 1) {   // fewer where the SMs of a GPC are no multiple of the cluster
            int most = 0;
            cfg.gridDim = dim3((unsigned)(sms / a.cluster * a.cluster));
            cfg.numAttrs = 1;
            e = cudaOccupancyMaxActiveClusters(&most, kern, &cfg);
            if (e != cudaSuccess) return e;
            if (most > 0 && most < clusters) clusters = most;
        }
        if (clusters < 1) clusters = 1;
        if (dev < kDevices) known[dev][a.cluster].store(clusters, std::memory_order_relaxed);
    }
    if (clusters > a.row_tiles) clusters = a.row_tiles;
    const int rows = (a.row_tiles + clusters - 1) / clusters;   // of tiles, at most, of a cluster
    a.row_warps = NW / a.k_warps < rows ? NW / a.k_warps : rows;
    const int fit = kLw4Partial / (4 * NT * 16 * 4);
    a.chunk = a.cluster == 1 && a.passes == 1 ? rows : (fit < a.row_warps ? a.row_warps : fit / a.row_warps * a.row_warps);
    cfg.gridDim = dim3((unsigned)(clusters * a.cluster), (unsigned)((a.M + 4 * NT - 1) / (4 * NT)));
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

template <int G>
static cudaError_t lw4_launch_tokens(const LinearW4Args &a, int sms, cudaStream_t s) {
    if (a.M <= 4) return lw4_launch<1, G>(a, sms, s);
    if (a.M <= 8) return lw4_launch<2, G>(a, sms, s);
    if (a.M <= 16) return lw4_launch<4, G>(a, sms, s);
    return lw4_launch<8, G>(a, sms, s);
}

cudaError_t launch_linear_w4(LinearW4Args a, int sms, cudaStream_t s) {
    a.row_tiles = (a.N + kW4Rows - 1) / kW4Rows;
    a.k_tiles = (a.K + kW4Cols - 1) / kW4Cols;
    return a.group == 32 ? lw4_launch_tokens<32>(a, sms, s)
                         : a.group == 64 ? lw4_launch_tokens<64>(a, sms, s) : lw4_launch_tokens<128>(a, sms, s);
}

}  // namespace bloom
