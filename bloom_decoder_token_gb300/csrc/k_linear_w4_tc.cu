// Linear layer over 4-bit weights for more tokens than k_linear_w4.cu takes, on the
// 5th-generation tensor cores: y[m][n] = epilogue(sum_k code[n][k] scale[n][k / group] x[m][k] +
// bias[n]).
//
// mma.sync has 957 multiply-adds a clock and SM here, so from about 10 tokens on it, and
// not the weights, would be what the time is made of (32 tokens, 16384 x 4096: 31 us with it, 5.4
// for the weights).  tcgen05.mma has 8192:
//  * W is the 128-row A operand, taken from TMEM: the tiles come by bulk copies, and warps
//    turn a word of eight codes into f16 pairs (w4_ops.cuh, 7 instructions) that tcgen05.st of
//    16x256b shape stores as they lie, for its registers are dealt to rows and columns as
//    those of an mma.sync fragment.
//  * The tokens are the N operand: f16 after a power of two for each token, in the order and
//    swizzle of the shared-memory operand, so that a block of 256 columns is one bulk copy.
//    A small kernel before this one lays them out (done here, every tile of rows would repeat
//    the conversion).
//  * A group's products make an accumulator of their own; four warps, a thread a row, add them times
//    the rows' scales to float32 sums in registers, as many groups a wait as half of the accumulators hold.
//  * Few tiles of rows: the columns are split over a cluster, whose sums meet through
//    distributed shared memory, in rank order.  Many: a CTA goes from tile to tile, and copies and
//    products of the next one go on while the sums of the last are stored (250880 x 4096, 64 tokens, groups of
//    128: some 310 -> 262 us, 12 tokens, of 64: 143 -> 139).
// Weights are loaded before the wait for the kernel before: that is the one that lays out
// the tokens, and it starts its successors only after its own wait, when all work before it is done.
// (Started at once, as the layer norms' successors are, this kernel's CTAs found the SMs partly taken: 12288
// x 4096, 16 tokens, 15 -> 21 us.)
//
// 16 tokens, 12288 x 4096: 14.3 us (4.1 to read the weights); 32, 16384 x 4096, groups of 128 17.6 (5.4), of
// 32 21; 64 25.8 (5.6); 12, 250880 x 4096 137 (83); 64 in groups of 128 262 (84), of 64 346 (86).  Bound by instructions: a block of 128 x
// 256 takes about 3000 warp instructions, 900 of them the codes', a third the scales' and most others waits
// and their polling; and at 64 tokens by L2, which gives a block's tokens, 32 KB, beside 17 KB of weights.  Four
// widening warps, two tiles each, against eight: 12 tokens, 250880 x 4096 154 -> 151; scales by two groups a
// wait: 151 -> 143, and 32 tokens in groups of 32 24.8 -> 20.6.
#include <atomic>
#include <math.h>

#include "common.cuh"
#include "kernels.h"
#include "tc_ops.cuh"
#include "w4_ops.cuh"

namespace bloom {

constexpr int kLtRows = 128, kLtTiles = kLtRows / kW4Rows;
constexpr int kLtThreads = 320;      // producer, MMA issuer, 4 scaling warps, 4 widening warps
constexpr int kLtMaxSplits = 8;
constexpr int kLtSteps = kW4Cols / 16;

template <int NT, int G>
struct LtCfg {
    static constexpr int kTile = w4_tile_bytes(G), kX = NT * kW4Cols * 2, kW = (kLtTiles * kTile + 1023) / 1024 * 1024;
    static constexpr int kStage = kX + kW, kPerSm = NT == 64 ? 1 : 2;
    static constexpr int kStages = (kPerSm == 1 ? 216 : 104) * 1024 / kStage;
    static constexpr size_t kSmem = (size_t)kStages * kStage + 1024;
    static constexpr int kA = NT == 16 ? 3 : 2, kDB = NT == 64 ? 2 : 4;   // buffers; A's of 128 columns of weights, 64 of TMEM
    static constexpr uint32_t kD = 64 * kA;                  // then two of sums
    static_assert(kD + kDB * NT <= 256, "TMEM");
    static_assert((NT / 4 + kLtMaxSplits) * kLtRows * 16 <= kStages * kStage, "room for the cluster's sums");
};

// Where a token's elements lie in a block of 256 columns: four boxes of 64 columns, rows of 128
// bytes (a token each), 16-byte pieces swizzled by the row.  A product of 16 columns takes, as the weights'
// fragments have it, place 4 q + i of product 2 j + o from column 32 j + 8 q + 4 o + i: half of eight columns goes
// to the left or right half of piece 4 (j & 1) + 2 o + q / 2.
// One CTA a token; up to 8192 columns are read once (behind a layer norm 12 tokens, 4096 x 16384: 23.0 -> 22.1 us
// against two readings of all).  With 512 threads it took so much of its SMs that the next kernel's clusters found
// no room until it had ended: 16 tokens, 12288 x 4096, 14.3 -> 15.5.
constexpr int kLtTokenThreads = 256;
__global__ void __launch_bounds__(kLtTokenThreads) w4_tokens_kernel(const uint16_t *x, long long ldx, int M, int K, int NT, int k_tiles,
                                                                    unsigned char *image, float *inv) {
    constexpr int T = kLtTokenThreads, R = 4;
    __shared__ uint32_t red[T / 32];
    griddep_wait();
    griddep_launch();
    const int n = blockIdx.x, m = blockIdx.y * NT + n, tid = threadIdx.x, chunks = k_tiles * 32;   // of eight columns
    const uint16_t *row = x + (long long)m * ldx;
    uint4 v[R];
    auto load = [&](int c0) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int c = c0 + i * T + tid;
            v[i] = make_uint4(0u, 0u, 0u, 0u);
            if (m < M && 8 * c < K) v[i] = ld_act(row + 8 * c);
        }
    };
    uint32_t m2 = 0;
    for (int c0 = 0; c0 < chunks; c0 += R * T) {
        load(c0);
#pragma unroll
        for (int i = 0; i < R; ++i)
            m2 = __vmaxu2(m2, __vmaxu2(__vmaxu2(v[i].x & 0x7fff7fffu, v[i].y & 0x7fff7fffu), __vmaxu2(v[i].z & 0x7fff7fffu, v[i].w & 0x7fff7fffu)));
    }
    uint32_t amax = __reduce_max_sync(0xffffffffu, max(m2 & 0xffffu, m2 >> 16));
    if ((tid & 31) == 0) red[tid >> 5] = amax;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < T / 32; ++i) amax = max(amax, red[i]);
    // 2^up brings the largest element to [2^14, 2^15); an infinity or NaN makes the token NaN
    const int up = min(120, 14 + 127 - (int)(amax >> 7));
    const float mul = __uint_as_float((uint32_t)(127 + up) << 23);
    if (tid == 0)
        inv[m] = amax >= 0x7f80u ? __uint_as_float(0x7fc00000u) : __uint_as_float((uint32_t)(127 - up) << 23);
    image += (size_t)blockIdx.y * k_tiles * NT * 512 + n * 128;
    for (int c0 = 0; c0 < chunks; c0 += R * T) {
        if (chunks > R * T) load(c0);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int c = c0 + i * T + tid;
            if (c >= chunks) break;
            const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
            uint32_t o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(o[e]) : "f"(bf_hi(w[e]) * mul), "f"(bf_lo(w[e]) * mul));
            const int piece = (c & 4) | (c >> 1 & 1);
            unsigned char *box = image + (size_t)(c >> 3) * NT * 128 + 8 * (c & 1);
            *reinterpret_cast<uint2 *>(box + ((piece ^ (n & 7)) << 4)) = make_uint2(o[0], o[1]);
            *reinterpret_cast<uint2 *>(box + (((piece | 2) ^ (n & 7)) << 4)) = make_uint2(o[2], o[3]);
        }
    }
}

__device__ __forceinline__ void lt_bulk(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(tc_smem(dst)),
                 "l"(src), "r"(bytes), "r"(tc_smem(bar))
                 : "memory");
}
__device__ __forceinline__ void lt_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(tc_smem(bar)) : "memory");
}
__device__ __forceinline__ void lt_cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// 16 rows x 64 32-bit columns; registers as fragments of 16 x 8: lane (g, q) holds of rows g and g + 8
// columns 2 q and 2 q + 1.
__device__ __forceinline__ void lt_store_a(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x256b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
        "%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]),
        "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]),
        "r"(r[31])
        : "memory");
}
// 32 columns of this thread's TMEM lane, on their way until tc_wait_ld().
__device__ __forceinline__ void lt_load32(uint32_t taddr, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,"
        "%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
          "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
          "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
__device__ __forceinline__ void lt_load16(uint32_t taddr, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
// Orders the loaded registers' uses behind the wait.
template <int N>
__device__ __forceinline__ void lt_wait_ld(uint32_t (&r)[N]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}
__device__ __forceinline__ bool lt_elect() {
    uint32_t r;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
    return r != 0;
}
// Waits for three phases at once: three tests in flight together where all have come to pass.
__device__ __forceinline__ bool lt_wait3(uint64_t *b0, uint32_t p0, uint64_t *b1, uint32_t p1, uint64_t *b2, uint32_t p2,
                                         unsigned long long limit_ns) {
    uint32_t r;
    asm volatile(
        "{\n .reg .pred p, q, r;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        " mbarrier.test_wait.parity.shared::cta.b64 q, [%3], %4;\n mbarrier.test_wait.parity.shared::cta.b64 r, [%5], %6;\n"
        " and.pred p, p, q;\n and.pred p, p, r;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(r)
        : "r"(tc_smem(b0)), "r"(p0), "r"(tc_smem(b1)), "r"(p1), "r"(tc_smem(b2)), "r"(p2)
        : "memory");
    return r || (tc_mbar_wait_within(b0, p0, limit_ns) && tc_mbar_wait_within(b1, p1, limit_ns) && tc_mbar_wait_within(b2, p2, limit_ns));
}
// tc_mma_tmem_a with the operand's descriptor (tc_desc) by its first 14 bits.
__device__ __forceinline__ void lt_mma(uint32_t d, uint32_t ta, uint32_t desc, uint32_t idesc, bool accumulate) {
    constexpr uint32_t kLow = 1u << 16, kHigh = (1024u >> 4) | 1u << 14 | 2u << 29;
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 b;\n setp.ne.b32 p, %5, 0;\n mov.b64 b, {%2, %3};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n}\n" ::"r"(d),
        "r"(ta), "r"(desc | kLow), "r"(kHigh), "r"(idesc), "r"((uint32_t)accumulate));
}
__device__ __forceinline__ void lt_store(const LinearW4Args &a, int m, int n, float bias, float v) {
    v += bias;
    if (a.epi == EPI_GELU) v = gelu_tanh(v);
    const long long at = m * a.ldy + n;
    if (a.f32) {
        float *y = static_cast<float *>(a.y) + at;
        *y = a.epi == EPI_RESID ? *y + v : v;
    } else {
        uint16_t *y = static_cast<uint16_t *>(a.y) + at;
        *y = f2bf(a.epi == EPI_RESID ? bf2f(*y) + v : v);
    }
}

template <int NT, int G>
__global__ void __launch_bounds__(kLtThreads, LtCfg<NT, G>::kPerSm) linear_w4_tc_kernel(const LinearW4Args a) {
    using C = LtCfg<NT, G>;
    constexpr int TB = C::kTile, ST = C::kStages, SG = kW4Cols / G, GS = G / 16;   // groups of a block, products of a group
    extern __shared__ unsigned char lt_raw[];
    unsigned char *smem = lt_raw + ((0u - tc_smem(lt_raw)) & 1023u);
    constexpr int NA = C::kA, ND = C::kDB;
    // groups at a time: a half block's, of half of the accumulators at most
    constexpr int BG = SG / 2 < ND / 2 ? SG / 2 : ND / 2;
    static_assert(ND % BG == 0 && SG / 2 % BG == 0, "groups at a time");
    __shared__ uint64_t full[ST], empty[ST], a_full[NA], a_empty[NA], d_full[ND], d_empty[ND], done;
    __shared__ uint32_t tmem_base;
    __shared__ float s_inv[NT];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int split = blockIdx.y, S = (int)gridDim.y, m0 = (int)blockIdx.z * NT;
    const int kb0 = (int)((long long)a.k_tiles * split / S), my_kb = (int)((long long)a.k_tiles * (split + 1) / S) - kb0;
    // this CTA's blocks: 128 rows at a time (every gridDim.x-th; with S > 1 one), their columns from kb0 on
    const int of_rows = (a.row_tiles + kLtTiles - 1) / kLtTiles, mine_rows = (of_rows - (int)blockIdx.x - 1) / (int)gridDim.x + 1;
    const int total = mine_rows * my_kb;   // fits: a block has 17 KB of weights

    if (tid == 0) {
        for (int s = 0; s < ST; ++s) {
            tc_mbar_init(&full[s], 1);
            tc_mbar_init(&empty[s], 4 + 4 + 1);   // widening warps, scaling warps, the products' commit
        }
        for (int b = 0; b < NA; ++b) {
            tc_mbar_init(&a_full[b], 4);
            tc_mbar_init(&a_empty[b], 1);
        }
        for (int b = 0; b < ND; ++b) {
            tc_mbar_init(&d_full[b], 1);
            tc_mbar_init(&d_empty[b], 4);
        }
        tc_mbar_init(&done, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 256;" ::"r"(tc_smem(&tmem_base)));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = tmem_base;
    griddep_launch();

    const int quarter = warp & 3;
    const uint32_t tquarter = tmem + ((uint32_t)(quarter * 32) << 16);
    float acc[NT];                   // scaling warps: this thread's row
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[i] = 0.f;
    bool ok = true;

    if (warp == 0) {
        if (lane == 0) {
            // ---- copies: the weights of the first stages before the wait for the tokens
            int tile = blockIdx.x, kb = 0;   // the next block of weights
            auto weights = [&](int s) {
                const uint32_t bytes = (uint32_t)(min(kLtTiles, a.row_tiles - tile * kLtTiles) * TB);
                asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(tc_smem(&full[s])), "r"(bytes + C::kX) : "memory");
                lt_bulk(smem + (size_t)s * C::kStage + C::kX, a.tiles + ((long long)(kb0 + kb) * a.row_tiles + tile * kLtTiles) * TB, bytes,
                        &full[s]);
                if (++kb == my_kb) {
                    kb = 0;
                    tile += (int)gridDim.x;
                }
            };
            const unsigned char *xsrc = a.image + ((size_t)blockIdx.z * a.k_tiles + kb0) * C::kX;
            int xb = 0;                      // and of tokens
            auto tokens = [&](int s) {
                lt_bulk(smem + (size_t)s * C::kStage, xsrc + (size_t)xb * C::kX, C::kX, &full[s]);
                if (++xb == my_kb) xb = 0;
            };
            const int pre = min(total, ST);
            for (int i = 0; i < pre; ++i) weights(i);
            griddep_wait();
            for (int i = 0; i < pre; ++i) tokens(i);
            int s = 0;
            uint32_t parity = 0;
            for (int i = pre; i < total; ++i) {
                ok = tc_mbar_wait_within(&empty[s], parity, a.wait_ns);
                if (!ok) break;
                weights(s);
                tokens(s);
                if (++s == ST) {
                    s = 0;
                    parity ^= 1u;
                }
            }
            // no copy lands after the CTA has ended: the stages' last fills, oldest first
            for (int j = 0; j < pre; ++j) {
                ok &= tc_mbar_wait(&full[s], parity, kTcWaitNs);
                if (++s == pre) {
                    s = 0;
                    parity ^= 1u;
                }
            }
        }
    } else if (warp == 1) {
        // ---- products: the warp goes along together, so that addresses stay in uniform registers (one
        // thread alone took 130 clocks a product), and one lane issues
        constexpr uint32_t idesc = tc_idesc(kLtRows, NT, true);
        const uint32_t tbase = __shfl_sync(0xffffffffu, tmem, 0), sbase = __shfl_sync(0xffffffffu, tc_smem(smem), 0);
        const bool lead = lt_elect();
        griddep_wait();
        int s = 0, ab = 0, db = 0;
        uint32_t sp = 0, ap = 0, dp = 1;   // the buffers' parities
        for (int i = 0; i < total && ok; ++i) {
            const uint32_t desc0 = (sbase + (uint32_t)s * C::kStage) >> 4 & 0x3fffu;
#pragma unroll
            for (int hb = 0; hb < 2; ++hb) {
#pragma unroll
                for (int g0 = 0; g0 < SG / 2; g0 += BG) {
                    // what the next groups need, in one round trip; the accumulators come free in order
                    uint64_t *const last = &d_empty[db];
                    ok = ok && lt_wait3(hb == 0 && g0 == 0 ? &full[s] : last, hb == 0 && g0 == 0 ? sp : dp, g0 == 0 ? &a_full[ab] : last,
                                        g0 == 0 ? ap : dp, last, dp, a.wait_ns);
                    ok = __all_sync(0xffffffffu, ok);
                    if (ok) {
                        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                        if (lead) {
#pragma unroll
                            for (int gr = g0; gr < g0 + BG; ++gr) {
                                const uint32_t td = tbase + C::kD + (uint32_t)((db + gr - g0) * NT), ta = tbase + (uint32_t)(ab * 64);
#pragma unroll
                                for (int k = 0; k < GS; ++k) {
                                    const int step = gr * GS + k, at = hb * (kLtSteps / 2) + step;
                                    lt_mma(td, ta + (uint32_t)(8 * step), desc0 + (uint32_t)(at / 4 * NT * 8 + 2 * (at % 4)), idesc, k > 0);
                                }
                            }
                            tc_commit(&d_full[db]);
                        }
                    }
                    if ((db += BG) == ND) {
                        db = 0;
                        dp ^= 1u;
                    }
                }
                if (ok && lead) tc_commit(&a_empty[ab]);
                if (++ab == NA) {
                    ab = 0;
                    ap ^= 1u;
                }
            }
            if (ok && lead) tc_commit(&empty[s]);
            if (++s == ST) {
                s = 0;
                sp ^= 1u;
            }
        }
        if (lead) tc_commit(&done);        // all have finished before TMEM is freed, on every path
        __syncwarp();
        ok &= tc_mbar_wait(&done, 0, kTcWaitNs);
    } else if (warp < 6) {
        // ---- sums: a thread a row
        const int r = quarter * 32 + lane, rr = r & 15;
        griddep_wait();
        const float inv = r < NT ? a.inv[m0 + r] : 0.f;
        int block = 0;
        for (int tile = blockIdx.x; tile < of_rows; tile += (int)gridDim.x) {
            const int n = tile * kLtRows + r;
            const float bias = S == 1 && a.bias && n < a.N ? bf2f(a.bias[n]) : 0.f;
#pragma unroll
            for (int i = 0; i < NT; ++i) acc[i] = 0.f;
            for (int kb = 0; kb < my_kb && ok; ++kb, ++block) {
                const int s = block % ST;
                ok = __all_sync(0xffffffffu, tc_mbar_wait_within(&full[s], (uint32_t)(block / ST & 1), a.wait_ns));
                if (!ok) break;
                const unsigned char *sc = smem + (size_t)s * C::kStage + C::kX + (r >> 4) * TB + 2048 + (rr & 7) * 4 + (rr >> 3) * 2;
                float scale[SG];
#pragma unroll
                for (int gr = 0; gr < SG; ++gr) scale[gr] = bf2f(*reinterpret_cast<const uint16_t *>(sc + gr * 32));
                __syncwarp();
                if (lane == 0) lt_arrive(&empty[s]);
#pragma unroll
                for (int g0 = 0; g0 < SG; g0 += BG) {
                    const int d = block * SG + g0, db = d % ND;
                    ok = ok && __all_sync(0xffffffffu, tc_mbar_wait_within(&d_full[db], (uint32_t)(d / ND & 1), a.wait_ns));
                    if (!ok) break;
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    constexpr int COLS = BG * NT, AT = COLS < 32 || NT == 64 ? COLS : 32;   // columns; those of one wait
#pragma unroll
                    for (int c0 = 0; c0 < COLS; c0 += AT) {
                        uint32_t v[AT];
                        const uint32_t from = tquarter + C::kD + (uint32_t)(db * NT + c0);
                        if constexpr (AT == 16) lt_load16(from, v);
                        else
#pragma unroll
                            for (int c = 0; c < AT; c += 32) lt_load32(from + (uint32_t)c, v + c);
                        lt_wait_ld(v);
#pragma unroll
                        for (int j = 0; j < AT; ++j)
                            acc[(c0 + j) % NT] = fmaf(scale[g0 + (c0 + j) / NT], __uint_as_float(v[j]), acc[(c0 + j) % NT]);
                    }
                    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) lt_arrive(&d_empty[db]);
                }
            }
            // the activations' power of two
            if (tile == (int)blockIdx.x) {
                if (r < NT) s_inv[r] = inv;
                asm volatile("bar.sync 1, 128;" ::: "memory");   // these four warps
            }
#pragma unroll
            for (int i = 0; i < NT; ++i)                     // and the codes' 2^-16 back
                acc[i] = ok ? acc[i] * 0x1p16f * s_inv[i] : __uint_as_float(0x7fc00000u);
            if (S == 1 && n < a.N) {
                const int mmax = min(a.M - m0, NT);
#pragma unroll
                for (int i = 0; i < NT; ++i)
                    if (i < mmax) lt_store(a, m0 + i, n, bias, acc[i]);
            }
        }
    } else {
        // ---- codes to f16 in TMEM, 128 columns at a time: a warp two tiles of rows
        for (int i = 0; i < total && ok; ++i) {
            const int s = i % ST;
            ok = __all_sync(0xffffffffu, tc_mbar_wait_within(&full[s], (uint32_t)(i / ST & 1), a.wait_ns));
            if (!ok) break;
            const unsigned char *tile = smem + (size_t)s * C::kStage + C::kX + 2 * quarter * TB + lane * 16;
#pragma unroll
            for (int hb = 0; hb < 2; ++hb) {
                uint4 v[2][2];
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int c = 0; c < 2; ++c) v[t][c] = *reinterpret_cast<const uint4 *>(tile + t * TB + (2 * hb + c) * 512);
                if (hb == 1) {
                    __syncwarp();
                    if (lane == 0) lt_arrive(&empty[s]);
                }
                const int h = 2 * i + hb;
                if (h >= NA) ok = ok && __all_sync(0xffffffffu, tc_mbar_wait_within(&a_empty[h % NA], (uint32_t)((h / NA - 1) & 1), a.wait_ns));
                if (!ok) break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    uint32_t r[32];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint4 &c = v[t][j >> 1];
                        const uint32_t w0 = j & 1 ? c.z : c.x, w1 = j & 1 ? c.w : c.y;
#pragma unroll
                        for (int o = 0; o < 2; ++o) {
                            r[8 * j + 4 * o] = w4_pair(w0, 2 * o);
                            r[8 * j + 4 * o + 1] = w4_pair(w0, 2 * o + 1);
                            r[8 * j + 4 * o + 2] = w4_pair(w1, 2 * o);
                            r[8 * j + 4 * o + 3] = w4_pair(w1, 2 * o + 1);
                        }
                    }
                    lt_store_a(tquarter + ((uint32_t)(16 * t) << 16) + (uint32_t)(h % NA * 64), r);
                }
                tc_wait_st();
                asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                __syncwarp();
                if (lane == 0) lt_arrive(&a_full[h % NA]);
            }
        }
    }
    if (!ok && a.err) atomicOr(a.err, kErrTimeout);
    __syncwarp();

    if (S > 1) {
        // ---- the splits' sums
        griddep_wait();              // every thread's own, for the bias and y
        const bool sums = warp >= 2 && warp < 6;
        const int r = quarter * 32 + lane, mmax = min(a.M - m0, NT);
        // Four tokens at a time to the rank that finishes them, into its ring: [split][row][its groups]
        const int groups = (mmax + 3) / 4, each = (groups + S - 1) / S;
        float4 *recv = reinterpret_cast<float4 *>(smem);
        lt_cluster_sync();           // every rank's ring is idle
        if (sums) {
#pragma unroll
            for (int q = 0; q < NT / 4; ++q) {
                if (q >= groups) break;
                uint32_t there;
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                             : "=r"(there)
                             : "r"(tc_smem(recv + (split * kLtRows + r) * each + q / S)), "r"(q % S));
                asm volatile("st.shared::cluster.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(there), "f"(acc[4 * q]), "f"(acc[4 * q + 1]),
                             "f"(acc[4 * q + 2]), "f"(acc[4 * q + 3])
                             : "memory");
            }
        }
        lt_cluster_sync();
        for (int i = tid; i < each * kLtRows; i += kLtThreads) {   // all warps: a row's four tokens each
            const int l = i / kLtRows, row = i % kLtRows, q = l * S + split, n = (int)blockIdx.x * kLtRows + row;
            if (q >= groups || n >= a.N) continue;
            const float bias = a.bias ? bf2f(a.bias[n]) : 0.f;
            float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int p = 0; p < S; ++p) {
                const float4 v = recv[(p * kLtRows + row) * each + l];
                t.x += v.x;
                t.y += v.y;
                t.z += v.z;
                t.w += v.w;
            }
            const float f[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (4 * q + j < mmax) lt_store(a, m0 + 4 * q + j, n, bias, f[j]);
        }
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    if (warp == 0) {
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 256;" ::"r"(tmem));
    }
}

static int lt_tokens(int M) { return M <= 16 ? 16 : M <= 32 ? 32 : 64; }

size_t linear_w4_tc_workspace(int M, int K) {
    const int NT = lt_tokens(M), blocks = (M + NT - 1) / NT, k_tiles = (K + kW4Cols - 1) / kW4Cols;
    return (size_t)blocks * NT * ((size_t)k_tiles * kW4Cols * 2 + 4);
}

template <int NT, int G>
static cudaError_t lt_launch(LinearW4Args a, void *workspace, int sms, cudaStream_t s) {
    using C = LtCfg<NT, G>;
    constexpr int kDevices = 64;
    static std::atomic<bool> ready[kDevices];
    const auto kern = linear_w4_tc_kernel<NT, G>;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= kDevices) return cudaErrorInvalidDevice;
    if (!ready[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
        if (e != cudaSuccess) return e;
        ready[dev].store(true, std::memory_order_release);
    }
    const int tiles = (a.row_tiles + kLtTiles - 1) / kLtTiles, blocks = (a.M + NT - 1) / NT;
    unsigned char *image = static_cast<unsigned char *>(workspace);
    float *inv = reinterpret_cast<float *>(image + (size_t)blocks * a.k_tiles * C::kX);
    a.image = image;
    a.inv = inv;
    e = launch_pdl(w4_tokens_kernel, dim3(NT, (unsigned)blocks), dim3(kLtTokenThreads), s, a.x, a.ldx, a.M, a.K, NT, a.k_tiles, image, inv);
    if (e != cudaSuccess) return e;
    // As many splits as leave the CTAs of one block of tokens resident at once, however many blocks there are: a
    // token's sums are the same beside any number of others (of more than 32).  That costs many tokens on a matrix of few
    // rows: 1024 x 2048, 65 tokens 11.5 us, 300 24, 4096 271, where fewer splits as blocks fill the GPU take 11.5, 12.4
    // and 76; 4096 x 4096, 300 57 (55), 4096 633 (435).  (Read the weights back and use the GEMM there.)
    int S = 1;
    while (S < kLtMaxSplits && (long long)tiles * (S + 1) <= (long long)sms * C::kPerSm && S + 1 <= a.k_tiles) ++S;
    // more tiles than that: each CTA takes several, as many as the others
    const int slots = sms * C::kPerSm, wide = blocks < slots ? slots / blocks : 1;
    const int each = S > 1 || tiles < wide ? 1 : (tiles + wide - 1) / wide;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((tiles + each - 1) / each), (unsigned)S, (unsigned)blocks);
    cfg.blockDim = dim3(kLtThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = g_pdl ? 1 : 0;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 1;
    attr[1].val.clusterDim.y = (unsigned)S;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

template <int G>
static cudaError_t lt_launch_tokens(const LinearW4Args &a, void *workspace, int sms, cudaStream_t s) {
    if (a.M <= 16) return lt_launch<16, G>(a, workspace, sms, s);
    if (a.M <= 32) return lt_launch<32, G>(a, workspace, sms, s);
    return lt_launch<64, G>(a, workspace, sms, s);
}

cudaError_t launch_linear_w4_tc(LinearW4Args a, void *workspace, int sms, cudaStream_t s) {
    a.row_tiles = (a.N + kW4Rows - 1) / kW4Rows;
    a.k_tiles = (a.K + kW4Cols - 1) / kW4Cols;
    return a.group == 32 ? lt_launch_tokens<32>(a, workspace, sms, s)
                         : a.group == 64 ? lt_launch_tokens<64>(a, workspace, sms, s) : lt_launch_tokens<128>(a, workspace, sms, s);
}

}  // namespace bloom
