// Linear layer over 4-bit weights with group scales, for the few tokens of a decode
// step: y[m][n] = epilogue(sum_k code[n][k] scale[n][k / group] x[m][k] + bias[n]).
//
// At so few tokens the time is the time to read the weights once, 4.25 bits each at
// groups of 64, and the arithmetic has to stay out of the way of 46 codes a clock and SM:
//  * The products run on mma.sync m16n8k16 with 16 rows of weights as one operand and 8
//    tokens as the other.  The codes are f16 numbers but for a turn and a mask a pair
//    (w4_ops.cuh): 7 instructions for 8 codes, exact.  (e4m3 numbers and m16n8k32 would take 3,
//    but that instruction takes 5.1 clocks of an SM against 2.5 of the f16 one, and bf16
//    activations need two e4m3 columns.  12288 x 4096, one token: 11.1 us with them.)
//  * An activation goes in as f16 after a power of two that brings the largest of the
//    token's 256 values to [2^14, 2^15): exact down to 2^-31 of that largest value; smaller
//    ones are off by 2^-39 of it at most.  Sums are float32.
//  * A group's products are summed apart, then times the scale into the float32 sums.
//  * A warp owns 256 columns, whose activations stay in its registers, and goes down the
//    matrix: tile after tile of 16 rows, by bulk copies into a ring of its own.  The
//    warps of a CTA that share the rows hold the CTA's columns together; their sums
//    meet in shared memory, in the warps' order, every 32 rows.
//  * Longer rows are split over the CTAs of a cluster, whose sums meet through distributed
//    shared memory, in rank order; still longer ones are taken in passes.
// Before the wait for the kernel before, which may be what writes the tiles, the first of them are only brought to
// L2 (behind a layer norm 12288 x 4096, one token: 12.0 -> 11.4 us, 4096 x 16384 17.0 -> 16.0).
// One token, from HBM: 4096 x 1024 3.6 us, 12288 x 4096 10.1 (4.0 to read the weights), 4096 x 16384
// 12.1 (5.2, groups of 128), 57344 x 14336 94 (65), 14336 x 57344 111 (65); 8 tokens, 250880 x 4096: 107
// (83).  Long matrices: bound by instructions as much as by HBM (a step of 32 rows takes the 16 warps
// about as long as its tiles take to come); short ones by the start, 3 us, and the last tiles' way.
#include <atomic>
#include <math.h>

#include "common.cuh"
#include "kernels.h"
#include "tc_ops.cuh"
#include "w4_ops.cuh"

namespace bloom {

constexpr int kLw4Warps = 16;
constexpr int kLw4Unit = 2;                      // tiles of a step: 32 rows
constexpr int kLw4Partial = 16384;               // bytes of a buffer of sums that wait for the cluster
constexpr int kLw4Stride = 20;                   // floats of a token's 16 rows in a warp's sums: no bank twice
constexpr int kLw4MaxCluster = 8;
// Tiles of a warp from 2 up to which its first ones are asked for ahead of the wait (one token, columns 4096, with
// and without: 5 tiles 10.1 and 10.8 us, 11 15.6 and 16.0, 14 19.3 and 19.3, 27 33.7 and 32.7; 1 tile, 4096 x 1024,
// 3.8 and 3.6).
constexpr int kLw4Short = 16;

template <int G>
struct Lw4Smem {
    static constexpr int kStages = 4, kTile = w4_tile_bytes(G);
    static constexpr int kSum = kLw4MaxM * kLw4Stride;                 // floats of a row of tiles' sums
    static constexpr int kSums = kLw4Warps * kLw4Unit * kSum;          // of one of the two buffers
    static constexpr int kRing = kLw4Warps * kStages * kTile;
    static constexpr int kBytes = kRing + 8 * kSums + 2 * kLw4Partial + 8 * kLw4Warps * kStages;
    static_assert(kBytes <= 227 * 1024, "shared memory of an SM");
};

__device__ __forceinline__ void lw4_mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t lw4_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ void lw4_bulk(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(tc_smem(dst)),
                 "l"(src), "r"(bytes), "r"(tc_smem(bar))
                 : "memory");
}
__device__ __forceinline__ void lw4_prefetch(const void *src, uint32_t bytes) {   // both multiples of 16
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void lw4_cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float4 lw4_peer(const float *p, int rank) {   // the same place in a rank's shared memory
    uint32_t there;
    float4 f;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(tc_smem(p)), "r"(rank));
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(f.x), "=f"(f.y), "=f"(f.z), "=f"(f.w) : "r"(there) : "memory");
    return f;
}
__device__ __forceinline__ void lw4_add(float4 &a, float4 b) {
    a.x += b.x; a.y += b.y; a.z += b.z; a.w += b.w;
}

// Rows row .. row + 3 of token m.
__device__ __forceinline__ void lw4_store(const LinearW4Args &a, int m, int row, float4 v4) {
    const float v[4] = {v4.x, v4.y, v4.z, v4.w};
    const long long at = m * a.ldy + row;
    float o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        o[e] = v[e];
        if (row + e >= a.N) continue;
        if (a.bias) o[e] += bf2f(a.bias[row + e]);
        if (a.epi == EPI_GELU) o[e] = gelu_tanh(o[e]);
        if (a.epi == EPI_RESID) o[e] += a.f32 ? static_cast<float *>(a.y)[at + e] : bf2f(static_cast<uint16_t *>(a.y)[at + e]);
    }
    if (a.wide && row + 3 < a.N) {
        if (a.f32) *reinterpret_cast<float4 *>(static_cast<float *>(a.y) + at) = make_float4(o[0], o[1], o[2], o[3]);
        else *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.y) + at) = make_uint2(pack_bf2(o[0], o[1]), pack_bf2(o[2], o[3]));
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (row + e >= a.N) continue;
        if (a.f32) static_cast<float *>(a.y)[at + e] = o[e];
        else static_cast<uint16_t *>(a.y)[at + e] = f2bf(o[e]);
    }
}

// AHEAD: a form of its own, for with these lines in it the kernel took 109 us instead of 107 (8 tokens, 250880
// x 4096) even where they were passed over.
template <int G, bool AHEAD>
__global__ void __launch_bounds__(32 * kLw4Warps, 1) linear_w4_kernel(const LinearW4Args a) {
    using Smem = Lw4Smem<G>;
    constexpr int NW = kLw4Warps, ST = Smem::kStages, TB = Smem::kTile, THREADS = 32 * NW, UT = kLw4Unit, SG = kW4Cols / G;
    extern __shared__ __align__(128) unsigned char lw4_smem[];
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, g = lane >> 2, q = lane & 3;
    unsigned char *ring = lw4_smem + w * ST * TB;
    float *sums = reinterpret_cast<float *>(lw4_smem + Smem::kRing);              // [2][NW][UT][kLw4MaxM][kLw4Stride]
    float *part = sums + 2 * Smem::kSums;                                         // [2][tiles][M][16]
    uint64_t *bar = reinterpret_cast<uint64_t *>(part + 2 * (kLw4Partial / 4)) + w * ST;
    if (lane == 0) {
        for (int i = 0; i < ST; ++i) tc_mbar_init(&bar[i], 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncwarp();
    const int P = a.cluster, cl = (int)blockIdx.x / P, rank = (int)blockIdx.x - cl * P, clusters = (int)gridDim.x / P;
    const int KW = a.k_warps, RW = a.row_warps, slot = w / KW, kw = w - slot * KW, M = a.M;
    const int items = RW * UT * M * 4, NR = (items + 31) / 32;   // a step's sums, four rows a lane; warps for them
    griddep_launch();

    // The cluster's tiles of rows, [r0, r0 + n), in RW runs of at most `run`, one for each KW
    // warps side by side; a warp's own: len from `row` on.
    const int r0 = (int)((long long)a.row_tiles * cl / clusters), n = (int)((long long)a.row_tiles * (cl + 1) / clusters) - r0;
    const int each = n / RW, more = n - each * RW;
    auto first_of = [&](int s) { return s * each + min(s, more); };
    // i / M for the products of tiles and tokens that come up, less than 2^20 / M
    const uint32_t per_token = (1u << 20) / (uint32_t)M + 1u;
    auto by_tokens = [&](int i) { return (int)((uint32_t)i * per_token >> 20); };
    const int run = (n + RW - 1) / RW, row = r0 + first_of(slot), len = slot < RW ? r0 + first_of(slot + 1) - row : 0;
    const bool direct = P == 1 && a.passes == 1;
    auto kt_of = [&](int pass) { return (pass * P + rank) * KW + kw; };   // the column tile

    // The warp's stream: for every chunk of its rows, in every pass, the chunk's tiles.
    int ahead = 0, ahead_pass = -1, left = 0;   // chunk's first tile; tiles left in it
    const unsigned char *src = nullptr;
    auto issue = [&](int st) {
        while (left == 0) {
            if (++ahead_pass == a.passes) {
                ahead_pass = 0;
                ahead += a.chunk;
            }
            if (ahead >= len) {                 // the end
                ahead_pass = -1;
                return false;
            }
            const int kt = kt_of(ahead_pass);
            if (kt >= a.k_tiles) continue;
            left = min(a.chunk, len - ahead);
            src = a.tiles + ((long long)kt * a.row_tiles + row + ahead) * TB;
        }
        if (lane == 0) {
            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(tc_smem(&bar[st])), "r"(TB) : "memory");
            lw4_bulk(ring + st * TB, src, TB, &bar[st]);
        }
        src += TB;
        --left;
        return true;
    };
    // The first tiles go to L2 while the kernel before still runs; read they are behind the wait, for it may be
    // what writes them.
    if (AHEAD && lane == 0 && len > 0 && kt_of(0) < a.k_tiles)
        lw4_prefetch(a.tiles + ((long long)kt_of(0) * a.row_tiles + row) * TB, (uint32_t)(min(min(ST, a.chunk), len) * TB));
    griddep_wait();   // the tiles, the activations and y
    int flying = 0;
    for (int i = 0; i < ST; ++i) flying += issue(i);

    uint32_t b[8][4];       // activations: token g, elements 32 j + 8 q + (0, 1 | 2, 3 | 4, 5 | 6, 7)
    float inv[2];           // 2^-up of tokens 2 q and 2 q + 1
    auto load_x = [&](int k0) {
        const uint16_t *x = a.x + g * a.ldx + k0 + 8 * q;
        uint32_t m2 = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            uint4 raw = make_uint4(0u, 0u, 0u, 0u);
            if (g < M && k0 + 32 * j + 8 * q < a.K) raw = ld_act(x + 32 * j);
            b[j][0] = raw.x; b[j][1] = raw.y; b[j][2] = raw.z; b[j][3] = raw.w;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) m2 = __vmaxu2(m2, b[j][e] & 0x7fff7fffu);
        uint32_t amax = max(m2 & 0xffffu, m2 >> 16);
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        // 2^up brings the largest element to [2^14, 2^15); an infinity or NaN makes the token NaN
        const int up = min(120, 14 + 127 - (int)(amax >> 7));
        const float mul = __uint_as_float((uint32_t)(127 + up) << 23);
        const float back = amax >= 0x7f80u ? __uint_as_float(0x7fc00000u) : __uint_as_float((uint32_t)(127 - up) << 23);
        inv[0] = __shfl_sync(0xffffffffu, back, 8 * q);
        inv[1] = __shfl_sync(0xffffffffu, back, 8 * q + 4);
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) b[j][e] = lw4_f16x2(bf_lo(b[j][e]) * mul, bf_hi(b[j][e]) * mul);
    };

    int st = 0, turn = 0, fill = 0;   // turn: buffer of the warps' sums; fill: of those that wait for the cluster
    int first_warp = 0;               // of those that add a step's sums: they take turns
    uint32_t parity = 0;              // of the ring
    bool lost = false;                // a wait expired
    for (int c0 = 0; c0 < run; c0 += a.chunk, fill ^= 1) {
        const int c1 = min(c0 + a.chunk, run);
        float *mine = part + fill * (kLw4Partial / 4);
        for (int pass = 0; pass < a.passes; ++pass) {
            const int kt = kt_of(pass);
            const int own = kt < a.k_tiles ? min(c1, len) : 0;   // this warp's tiles of the chunk end here
            if (own > 0 && (a.passes > 1 || c0 == 0)) load_x(kt * kW4Cols);
            const int nk = min(KW, a.k_tiles - (pass * P + rank) * KW);   // warps side by side that have columns
            for (int t0 = c0; t0 < c1; t0 += UT) {
                float *sum = sums + turn * Smem::kSums;
                float *to = sum + w * (UT * Smem::kSum) + 2 * q * kLw4Stride + g;
#pragma unroll 1
                for (int t = t0; t < min(t0 + UT, own); ++t, to += Smem::kSum) {
                    lost = lost || !tc_mbar_wait_within(&bar[st], parity, a.wait_ns);
                    lost = __any_sync(0xffffffffu, lost);
                    float acc[4];   // row g, tokens 2 q and 2 q + 1; row g + 8
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[e] = lost ? __uint_as_float(0x7fc00000u) : 0.f;
                    if (!lost) {
                        const unsigned char *tile = ring + st * TB;
                        uint4 v[4];
                        uint32_t sc[SG];
#pragma unroll
                        for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const uint4 *>(tile + i * 512 + lane * 16);
#pragma unroll
                        for (int i = 0; i < SG; ++i) sc[i] = *reinterpret_cast<const uint32_t *>(tile + 2048 + i * 32 + g * 4);
                        __syncwarp();   // the tile has been read
                        if (!issue(st)) --flying;
                        if (++st == ST) {
                            st = 0;
                            parity ^= 1u;
                        }
#pragma unroll
                        for (int gr = 0; gr < SG; ++gr) {
                            float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                            for (int j = gr * (G / 32); j < (gr + 1) * (G / 32); ++j) {
                                const uint32_t w0 = (&v[j / 2].x)[2 * (j & 1)], w1 = (&v[j / 2].x)[2 * (j & 1) + 1];
#pragma unroll
                                for (int h = 0; h < 2; ++h)
                                    lw4_mma(c, w4_pair(w0, 2 * h), w4_pair(w1, 2 * h), w4_pair(w0, 2 * h + 1), w4_pair(w1, 2 * h + 1),
                                            b[j][2 * h], b[j][2 * h + 1]);
                            }
                            const float s0 = bf_lo(sc[gr]), s1 = bf_hi(sc[gr]);
#pragma unroll
                            for (int e = 0; e < 4; ++e) acc[e] += (e < 2 ? s0 : s1) * c[e];
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e)   // the codes' 2^-16 back, then the activations' power of two
                        to[(e & 1) * kLw4Stride + 8 * (e >> 1)] = acc[e] * 0x1p16f * inv[e & 1];
                }
                __syncthreads();
                // the warps' sums, in their order; each step other warps begin
                {
                    for (int i = (tid - 32 * first_warp) & (THREADS - 1); i < items; i += THREADS) {
                        const int r = 4 * (i & 3), um = i >> 2, u = by_tokens(um), m = um - u * M, s = u / UT, t = t0 + u - s * UT;
                        const int first = first_of(s);
                        if (t >= min(c1, first_of(s + 1) - first)) continue;
                        const float *from = sum + (s * KW * UT + u - s * UT) * Smem::kSum + m * kLw4Stride + r;
                        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
                        for (int k = 0; k < nk; ++k) lw4_add(v, *reinterpret_cast<const float4 *>(from + k * (UT * Smem::kSum)));
                        if (direct) {
                            lw4_store(a, m, (r0 + first + t) * kW4Rows + r, v);
                        } else {
                            float4 *p = reinterpret_cast<float4 *>(mine + ((s * a.chunk + t - c0) * M + m) * 16 + r);
                            if (pass > 0) lw4_add(v, *p);
                            *p = v;
                        }
                    }
                }
                first_warp = (first_warp + NR) & (NW - 1);
                turn ^= 1;
            }
        }
        if (direct) continue;
        // the ranks' sums.  A buffer is written again after the next one's barrier, which
        // every rank reaches when it has read this one.
        lw4_cluster_sync();
        for (int i = rank * THREADS + tid; i < RW * (c1 - c0) * M * 4; i += P * THREADS) {
            const int r = 4 * (i & 3), um = i >> 2, u = by_tokens(um), m = um - u * M, s = u / (c1 - c0), t = c0 + u - s * (c1 - c0);
            const int first = first_of(s);
            if (t >= first_of(s + 1) - first) continue;
            const float *p = mine + ((s * a.chunk + t - c0) * M + m) * 16 + r;
            float4 f[kLw4MaxCluster], v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < kLw4MaxCluster; ++k) f[k] = k < P ? lw4_peer(p, k) : v;
#pragma unroll
            for (int k = 0; k < kLw4MaxCluster; ++k)
                if (k < P) lw4_add(v, f[k]);
            lw4_store(a, m, (r0 + first + t) * kW4Rows + r, v);
        }
    }
    if (lost && a.err && lane == 0) atomicOr(a.err, kErrTimeout);
    if (!direct) lw4_cluster_sync();   // a rank's shared memory lives until all have read it
    // copies in flight behind an expired wait land before the CTA ends
    for (; lost && flying > 0; --flying) {
        tc_mbar_wait(&bar[st], parity, kTcWaitNs);
        if (++st == ST) {
            st = 0;
            parity ^= 1u;
        }
    }
}

template <int G>
static cudaError_t lw4_launch(LinearW4Args a, int sms, cudaStream_t s) {
    using Smem = Lw4Smem<G>;
    constexpr int kDevices = 64, NW = kLw4Warps;
    static std::atomic<int> known[kDevices][kLw4MaxCluster + 1];   // clusters that are resident at once
    const auto kern = linear_w4_kernel<G, false>, ahead = linear_w4_kernel<G, true>;   // alike in what they need
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(32 * kLw4Warps);
    cfg.dynamicSmemBytes = Smem::kBytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = g_pdl ? 1 : 0;
    cfg.attrs = attr;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= kDevices) return cudaErrorInvalidDevice;
    if (known[dev][1].load(std::memory_order_acquire) == 0) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem::kBytes);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(ahead, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem::kBytes);
        if (e != cudaSuccess) return e;
        for (int P = kLw4MaxCluster; P >= 1; --P) {   // fewer than sms / P where a GPC's SMs are no multiple of P
            int most = sms / P;
            if (P > 1) {
                attr[0].val.clusterDim.x = (unsigned)P;
                cfg.gridDim = dim3((unsigned)(sms / P * P));
                cfg.numAttrs = 1;
                e = cudaOccupancyMaxActiveClusters(&most, kern, &cfg);
                if (e != cudaSuccess) return e;
            }
            known[dev][P].store(most < 1 ? 1 : most < sms / P ? most : sms / P, std::memory_order_release);
        }
    }
    // The cluster that keeps most warps busy; of equals the smallest.  One pass if eight CTAs' warps
    // hold the columns.
    long long best = -1;
    for (int P = 1; P <= kLw4MaxCluster; ++P) {
        const int passes = (a.k_tiles + P * NW - 1) / (P * NW), kw = (a.k_tiles + P * passes - 1) / (P * passes);
        if (passes > 1 && P < kLw4MaxCluster) continue;
        const long long busy = (long long)known[dev][P].load(std::memory_order_relaxed) * (NW / kw) * a.k_tiles / passes;
        if (busy <= best) continue;
        best = busy;
        a.cluster = P;
        a.passes = passes;
        a.k_warps = kw;
    }
    int clusters = known[dev][a.cluster].load(std::memory_order_relaxed);
    if (clusters > a.row_tiles) clusters = a.row_tiles;
    const int rows = (a.row_tiles + clusters - 1) / clusters;   // of tiles, at most, of a cluster
    const bool direct = a.cluster == 1 && a.passes == 1;
    const int fit = kLw4Partial / (a.M * kW4Rows * 4);   // tiles of sums that wait for the cluster
    static_assert(kLw4Partial >= NW * kLw4Unit * kLw4MaxM * kW4Rows * 4, "a step's");
    a.row_warps = NW / a.k_warps < rows ? NW / a.k_warps : rows;
    const int run = (rows + a.row_warps - 1) / a.row_warps;
    a.chunk = direct ? run : fit / a.row_warps / kLw4Unit * kLw4Unit;
    a.wide = a.ldy % 4 == 0 && ((uintptr_t)a.y & (a.f32 ? 15u : 7u)) == 0;
    attr[0].val.clusterDim.x = (unsigned)a.cluster;
    cfg.gridDim = dim3((unsigned)(clusters * a.cluster));
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, run > 1 && run <= kLw4Short ? ahead : kern, a);
}

cudaError_t launch_linear_w4(LinearW4Args a, int sms, cudaStream_t s) {
    a.row_tiles = (a.N + kW4Rows - 1) / kW4Rows;
    a.k_tiles = (a.K + kW4Cols - 1) / kW4Cols;
    return a.group == 32 ? lw4_launch<32>(a, sms, s) : a.group == 64 ? lw4_launch<64>(a, sms, s) : lw4_launch<128>(a, sms, s);
}

}  // namespace bloom
