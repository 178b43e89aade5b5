// ALiBi decode attention over the 8-bit KV cache, for the last T tokens of every
// sequence (T = 1: a decode step; more: drafted tokens checked at once).
//
// Query token t of sequence b, t = 0 .. T-1, sits at slot lens[b] - T + t and
// sees the slots up to its own whose position is not -1:
//   s_k = (q . K_k) / sqrt(d) + slope_j * pos_k,  o = sum_k softmax(s)_k V_k,
// K and V being code * scale.  A query that sees nothing gets 0.  Positions enter
// as pos_k - pos_ref (the softmax does not change), pos_ref the highest position
// among the last slots, so that a far position costs no bits of a near key's score.
//
// Bound by HBM (the codes are read once); the arithmetic has to stay out of the
// way, 23 codes per clock and SM.  So:
//  * The products run on mma.sync m16n8k16 with the keys (for V: the elements d)
//    as the 16-row operand and the queries of one key head as the 8 columns: 8
//    queries cost what one costs, and a code costs half a conversion to f16
//    (exact for both code types) and, in V, half a byte permutation that pairs
//    two keys.  tcgen05 would want the codes in f16 in shared memory first.
//  * q is multiplied by a power of two that brings its largest element to
//    [2^14, 2^15), where bf16 -> f16 is exact over 2^-28 of that element; the
//    scores are float32 sums of exact products.
//  * The softmax is one pass: running maxima and sums in float32, in powers of
//    two.  The weight of V_k carries the block's V scale: exp2(s_k + log2 scale -
//    M + 14) with a running maximum M of its own, so that scales far apart cost
//    nothing, rounded to f16 (relative 2^-11; the bf16 result rounds at 2^-8)
//    and multiplied with exact codes into float32 accumulators.
//  * Work is cut evenly whatever the lengths: the scale blocks (32 slots) of all
//    rows and key heads are numbered in one sequence, and each resident warp takes
//    an equal run of it.  A (row, key head) of at most kAk8Short blocks is left
//    whole; a longer one that falls into several runs leaves partial results,
//    which a second kernel joins in order.
//  * A warp keeps its own ring of stages ahead of it, one block each: two bulk copies
//    (K, V), completing on an mbarrier, and by cp.async positions, scales and, at
//    the first block of a (row, key head), its queries.  Warps never wait for
//    one another.
#include <atomic>
#include <math.h>

#include "common.cuh"
#include "kernels.h"
#include "kv8_ops.cuh"
#include "tc_ops.cuh"

namespace bloom {

constexpr int kAk8Warps = 4, kAk8Threads = 32 * kAk8Warps;
constexpr int kAk8Short = 8;      // blocks of a (row, key head) that is never cut
constexpr int kAk8MinRun = 4;     // blocks a warp takes at least, while there are warps to spare
constexpr int kAk8Part = 4;       // floats beside a partial's accumulator: m, M, l

// ---- conversions of codes to f16 pairs
__device__ __forceinline__ uint32_t ak8_s8x2(uint32_t biased, uint32_t sel) {
    // bytes u = code + 128 -> f16 1024 + u -> code, exact
    uint32_t r;
    asm("sub.f16x2 %0, %1, %2;" : "=r"(r) : "r"(__byte_perm(biased, 0x64646464u, sel)), "r"(0x64806480u));
    return r;
}
template <bool E4M3>
__device__ __forceinline__ void ak8_widen(uint32_t w, uint32_t &lo, uint32_t &hi) {   // bytes 0,1 | 2,3
    if (E4M3) {
        lo = kv8_e4m3x2_f16x2((uint16_t)w);
        hi = kv8_e4m3x2_f16x2((uint16_t)(w >> 16));
    } else {
        lo = ak8_s8x2(w, 0x4140);
        hi = ak8_s8x2(w, 0x4342);
    }
}
template <bool E4M3>
__device__ __forceinline__ uint32_t ak8_bias(uint32_t w) { return E4M3 ? w : w ^ 0x80808080u; }

__device__ __forceinline__ void ak8_mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t ak8_pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t ak8_transpose(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ float ak8_exp2(float x) {
    float r;
    asm("ex2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));   // relative error 2^-22
    return r;
}
__device__ __forceinline__ float ak8_finite(float m) { return m == -INFINITY ? 0.f : m; }

// ---- where a block number lies
struct Ak8Rows {
    const int *lens;
    int B, max_seq, heads;   // heads: (key head, column chunk) pairs of a row
    __device__ __forceinline__ int len(int b) const { return max(0, min(lens[b], max_seq)); }
    // blocks of one head of row b; at least one, so that every output is written
    __device__ __forceinline__ int blocks(int b) const { return max(1, (len(b) + kKv8Block - 1) / kKv8Block); }
};
__device__ __forceinline__ long long ak8_total(const Ak8Rows &r) {   // by the whole warp
    const int lane = threadIdx.x & 31;
    int t = 0;
    for (int b = lane; b < r.B; b += 32) t += r.blocks(b);
    return (long long)__reduce_add_sync(0xffffffffu, t) * r.heads;
}
struct Ak8Cursor {   // a block: its row, head, place in that head; the row's length and blocks a head
    int b, head, blk, len, blocks;
    // block number x < total, by the whole warp
    __device__ __forceinline__ void at(const Ak8Rows &r, long long x) {
        const int lane = threadIdx.x & 31;
        long long before = 0;
        for (int b0 = 0;; b0 += 32) {
            const int mine = b0 + lane < r.B ? r.blocks(b0 + lane) : 0;
            int sum = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += y;
            }
            const unsigned past = __ballot_sync(0xffffffffu, before + (long long)sum * r.heads > x);
            if (past || b0 + 32 >= r.B) {
                const int src = past ? __ffs(past) - 1 : 31;
                b = b0 + src;
                x -= before + (long long)__shfl_sync(0xffffffffu, sum - mine, src) * r.heads;
                break;
            }
            before += (long long)__shfl_sync(0xffffffffu, sum, 31) * r.heads;
        }
        row(r);
        head = (int)(x / blocks);
        blk = (int)(x - (long long)head * blocks);
    }
    __device__ __forceinline__ void row(const Ak8Rows &r) {
        len = b < r.B ? r.len(b) : 0;
        blocks = b < r.B ? r.blocks(b) : 1;
    }
    __device__ __forceinline__ void next(const Ak8Rows &r) {
        if (++blk < blocks) return;
        blk = 0;
        if (++head < r.heads) return;
        head = 0;
        ++b;
        row(r);
    }
};
// Run k of R: blocks [ak8_cut(k), ak8_cut(k + 1)), equal shares, but that a short
// (row, head) belongs to the run that its last block falls into.
__device__ __forceinline__ long long ak8_cut(const Ak8Rows &r, long long k, long long R, long long total,
                                             Ak8Cursor &c) {
    long long x = k * total / R;
    if (x >= total) return total;
    c.at(r, x);
    if (c.blocks <= kAk8Short) {
        x -= c.blk;
        c.blk = 0;
    }
    return x;
}
__device__ __forceinline__ long long ak8_runs(long long total, int warps) {
    return min((long long)warps, (total + kAk8MinRun - 1) / kAk8MinRun);
}

// One stage of a warp's ring, in bytes: K, V, the queries of `cols` columns, positions
// of the block, positions of the row's last 32 slots, the two scales.
template <int D>
struct Ak8Stage {
    static constexpr int kCount = 256 / D, kQ = 2 * kKv8Block * D;
    __host__ __device__ static constexpr int pos(int cols) { return kQ + cols * D * 2; }
    __host__ __device__ static constexpr int bytes(int cols) { return (pos(cols) + 256 + 16 + 127) / 128 * 128; }
    // the ring of a CTA and an mbarrier per stage
    __host__ __device__ static constexpr int smem(int cols) { return kAk8Warps * kCount * (bytes(cols) + 8); }
};

__device__ __forceinline__ void ak8_async4(const void *dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(tc_smem(dst)), "l"(src) : "memory");
}

// Columns of a chunk: query c = t * group + i of a key head, t the token, i the query head.
template <int D, bool E4M3, int NT>
__global__ void __launch_bounds__(kAk8Threads, NT == 1 ? 3 : 2) attn_kv8_kernel(const AttnKv8Args a) {
    constexpr int HS = D / 64, VW = D / 32, W = 8 * NT;   // K segments of 16 bytes a lane; V words a key
    using Stage = Ak8Stage<D>;
    constexpr int ST = Stage::kCount;
    extern __shared__ __align__(128) unsigned char ak8_raw[];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, g = lane >> 2, t4 = lane & 3;
    const int cols = a.part_cols, sbytes = Stage::bytes(cols);
    unsigned char *ring = ak8_raw + w * ST * sbytes;
    uint64_t *bar = reinterpret_cast<uint64_t *>(ak8_raw + kAk8Warps * ST * sbytes) + w * ST;
    if (lane == 0) {
        for (int i = 0; i < ST; ++i) tc_mbar_init(&bar[i], 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncwarp();
    griddep_launch();
    griddep_wait();

    const int group = a.n / a.kv, C = group * a.T, chunks = (C + W - 1) / W;
    const Ak8Rows rows{a.lens, a.B, a.max_seq, a.kv * chunks};
    if (a.err && blockIdx.x == 0)
        for (int b = threadIdx.x; b < a.B; b += kAk8Threads)
            if (a.lens[b] > a.max_seq) atomicOr(a.err, kErrSlot);
    const long long total = ak8_total(rows), R = ak8_runs(total, (int)gridDim.x * kAk8Warps);
    const int run = w * (int)gridDim.x + (int)blockIdx.x;   // runs spread over the CTAs first
    if (run >= R) return;
    Ak8Cursor cur, ahead;
    const long long x1 = ak8_cut(rows, run + 1, R, total, ahead);
    const long long x0 = ak8_cut(rows, run, R, total, cur);
    if (x0 >= x1) return;
    ahead = cur;

    // block xa of the run into stage `st`; one cp.async group, empty beyond the end
    long long xa = x0;
    auto issue = [&](int st) {
        if (xa < x1) {
            unsigned char *stage = ring + st * sbytes;
            const int base = ahead.blk * kKv8Block, n = min(kKv8Block, ahead.len - base);   // n <= 0: no keys
            const int h = ahead.head / chunks;
            const long long bh = (long long)ahead.b * a.kv + h;
            if (lane == 0) {
                const uint32_t br = tc_smem(&bar[st]);
                if (n > 0) {
                    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(br), "r"(2 * n * D) : "memory");
#pragma unroll
                    for (int v = 0; v < 2; ++v)
                        asm volatile(
                            "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                                tc_smem(stage + v * kKv8Block * D)),
                            "l"((v ? a.vc : a.kc) + (bh * a.max_seq + base) * D), "r"(n * D), "r"(br)
                            : "memory");
                } else {
                    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(br) : "memory");
                }
            }
            int *pos = reinterpret_cast<int *>(stage + Stage::pos(cols));
            const int *rowpos = a.pos + (long long)ahead.b * a.max_seq;
            if (lane < n) ak8_async4(pos + lane, rowpos + base + lane);
            else pos[lane] = -1;
            if (lane < 2 && n > 0)
                ak8_async4(pos + 64 + lane, (lane ? a.vs : a.ks) + bh * a.blocks + base / kKv8Block);
            if (xa == x0 || ahead.blk == 0) {   // the first block of a (row, head) in this run
                if (ahead.len - 1 - lane >= 0) ak8_async4(pos + 32 + lane, rowpos + ahead.len - 1 - lane);
                else pos[32 + lane] = -1;
                const int c0 = ahead.head % chunks * W, nc = min(W, C - c0);
                for (int i = lane; i < nc * (D / 8); i += 32) {
                    const int c = c0 + i / (D / 8), e = i % (D / 8) * 8;
                    cp_async16(stage + Stage::kQ + (i / (D / 8) * D + e) * 2,
                               a.q + (((long long)ahead.b * a.T + c / group) * a.n + h * group + c % group) * D + e);
                }
            }
            ++xa;
            ahead.next(rows);
        }
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < ST; ++i) issue(i);

    constexpr float kLog2e = 1.4426950408889634f;
    uint32_t qf[NT][D / 16][2];
    float qinv[NT][2], slope[NT][2], m[NT][2], M[NT][2], l[NT][2], acc[D / 16][NT][4];
    int lim[NT][2];                // slots that a column sees
    int ref = 0, st = 0;
    uint32_t parity = 0;
    long long seg0 = x0;           // first block of the current (row, head) in this run
    bool fresh = true;
    for (long long x = x0; x < x1; ++x) {
        const int chunk = cur.head % chunks, h = cur.head / chunks;
        const int ncol = min(W, C - chunk * W);
        unsigned char *stage = ring + st * sbytes;
        const int *pos = reinterpret_cast<const int *>(stage + Stage::pos(cols));
        // ---- the block's copies
        cp_async_wait<ST - 1>();
        const bool ok = __all_sync(0xffffffffu, tc_mbar_wait(&bar[st], parity, 0));
        if (!ok) {   // report; a second bounded wait, so that no copy lands later; the block is skipped
            if (a.err) atomicOr(a.err, kErrTimeout);
            tc_mbar_wait(&bar[st], parity, kTcWaitNs);
        }
        __syncwarp();
        if (fresh) {
            fresh = false;
            seg0 = x;
            ref = __reduce_max_sync(0xffffffffu, pos[32 + lane]);
            for (int k0 = cur.len - 32; k0 > 0 && ref < 0; k0 -= 32)   // pads alone at the row's end
                ref = __reduce_max_sync(0xffffffffu, k0 - 1 - lane >= 0 ? a.pos[(long long)cur.b * a.max_seq + k0 - 1 - lane] : -1);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                // B fragments: column g, elements 64 s + 16 t4 + 4 u + (0, 1 | 2, 3)
                uint4 raw[HS][2];
                uint32_t amax = 0;
#pragma unroll
                for (int s = 0; s < HS; ++s) {
                    raw[s][0] = raw[s][1] = make_uint4(0u, 0u, 0u, 0u);
                    if (nt * 8 + g < ncol) {
                        const uint4 *q = reinterpret_cast<const uint4 *>(stage + Stage::kQ + ((nt * 8 + g) * D + 64 * s + 16 * t4) * 2);
                        raw[s][0] = q[0];
                        raw[s][1] = q[1];
                    }
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        amax = __vmaxu2(amax, raw[s][u].x & 0x7fff7fffu);
                        amax = __vmaxu2(amax, raw[s][u].y & 0x7fff7fffu);
                        amax = __vmaxu2(amax, raw[s][u].z & 0x7fff7fffu);
                        amax = __vmaxu2(amax, raw[s][u].w & 0x7fff7fffu);
                    }
                }
                amax = max(amax & 0xffffu, amax >> 16);
                amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                // 2^up brings the largest element to [2^14, 2^15); at most 2^126
                const int up = amax >= 0x7f80u ? 0 : min(126, 14 + 127 - (int)(amax >> 7));
                const float mul = __uint_as_float((uint32_t)(127 + up) << 23);
                float inv = __uint_as_float((uint32_t)(127 - up) << 23);
                if (amax >= 0x7f80u) inv = __uint_as_float(0x7fc00000u);   // every score NaN
#pragma unroll
                for (int s = 0; s < HS; ++s)
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const uint32_t *p = &raw[s][u >> 1].x + 2 * (u & 1);
                        qf[nt][4 * s + u][0] = ak8_pack_f16(bf_lo(p[0]) * mul, bf_hi(p[0]) * mul);
                        qf[nt][4 * s + u][1] = ak8_pack_f16(bf_lo(p[1]) * mul, bf_hi(p[1]) * mul);
                    }
#pragma unroll
                for (int e = 0; e < 2; ++e) {   // accumulator columns 2 t4 + e
                    const int cc = chunk * W + nt * 8 + 2 * t4 + e;
                    qinv[nt][e] = __shfl_sync(0xffffffffu, inv, (2 * t4 + e) * 4);
                    slope[nt][e] = a.slopes && cc < C ? a.slopes[h * group + cc % group] * kLog2e : 0.f;
                    lim[nt][e] = cc < C ? cur.len - a.T + 1 + cc / group : 0;
                    m[nt][e] = M[nt][e] = -INFINITY;
                    l[nt][e] = 0.f;
                }
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[i][nt][e] = 0.f;
            }
        }
        const int base = cur.blk * kKv8Block;
        {
            const uint8_t *ks = stage, *vs = stage + kKv8Block * D;
            // ---- scores: 16 slots x columns per mt
            float s[2][NT][4];
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
                uint4 ka[HS], kb[HS];
#pragma unroll
                for (int i = 0; i < HS; ++i) {
                    ka[i] = *reinterpret_cast<const uint4 *>(ks + (mt * 16 + g) * D + 64 * i + 16 * t4);
                    kb[i] = *reinterpret_cast<const uint4 *>(ks + (mt * 16 + 8 + g) * D + 64 * i + 16 * t4);
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[mt][nt][e] = 0.f;
#pragma unroll
                for (int i = 0; i < HS; ++i)
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        uint32_t a0, a1, a2, a3;
                        ak8_widen<E4M3>(ak8_bias<E4M3>((&ka[i].x)[u]), a0, a2);
                        ak8_widen<E4M3>(ak8_bias<E4M3>((&kb[i].x)[u]), a1, a3);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            ak8_mma(s[mt][nt], a0, a1, a2, a3, qf[nt][4 * i + u][0], qf[nt][4 * i + u][1]);
                    }
            }
            // ---- softmax
            const float kscale = reinterpret_cast<const float *>(pos)[64], vscale = reinterpret_cast<const float *>(pos)[65];
            // vscale = mant * 2^ev
            const uint32_t vb = __float_as_uint(vscale), vexp = (vb >> 23) & 255u;
            const float ev = vexp == 255u ? 0.f : vexp == 0u ? -126.f : (float)((int)vexp - 127);
            const float mant = vexp == 255u ? vscale : vexp == 0u ? vscale * 0x1p126f : __uint_as_float((vb & 0x807fffffu) | 0x3f800000u);
            int pk[4];
            float dp[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                pk[i] = ok ? pos[8 * i + g] : -1;
                dp[i] = (float)(pk[i] - ref);
            }
            uint32_t pb[2][NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float wt[2][4];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float f = kscale * qinv[nt][e] * (a.scale * kLog2e);
                    float bm = -INFINITY;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {   // slot 8 i + g
                        float &v = s[i >> 1][nt][2 * (i & 1) + e];
                        v = v * f + slope[nt][e] * dp[i];
                        if (pk[i] < 0 || base + 8 * i + g >= lim[nt][e]) v = -INFINITY;
                        bm = fmaxf(bm, v);
                    }
                    bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 4));
                    bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 8));
                    bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 16));
                    const float mn = fmaxf(m[nt][e], bm), Mn = fmaxf(M[nt][e], bm + ev);
                    const float mf = ak8_finite(mn), Mf = ak8_finite(Mn) - 14.f - ev;
                    l[nt][e] *= ak8_exp2(m[nt][e] - mf);
                    if (__any_sync(0xffffffffu, Mn > M[nt][e])) {
                        const float r = ak8_exp2(M[nt][e] - ak8_finite(Mn));
#pragma unroll
                        for (int i = 0; i < D / 16; ++i) {
                            acc[i][nt][e] *= r;
                            acc[i][nt][2 + e] *= r;
                        }
                    }
                    m[nt][e] = mn;
                    M[nt][e] = Mn;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float v = s[i >> 1][nt][2 * (i & 1) + e];
                        l[nt][e] += ak8_exp2(v - mf);
                        wt[i >> 1][2 * (i & 1) + e] = v == -INFINITY ? 0.f : ak8_exp2(v - Mf) * mant;
                    }
                }
#pragma unroll
                for (int mt = 0; mt < 2; ++mt) {   // [slot][column] -> [column][slot] fragments
                    pb[mt][nt][0] = ak8_transpose(ak8_pack_f16(wt[mt][0], wt[mt][1]));
                    pb[mt][nt][1] = ak8_transpose(ak8_pack_f16(wt[mt][2], wt[mt][3]));
                }
            }
            // ---- values: D elements x columns, 16 slots per mt
            // slots that take no part may hold e4m3 NaNs: their codes count as 0
            const bool clean = !E4M3 || !__any_sync(0xffffffffu, pk[0] < 0 || pk[1] < 0 || pk[2] < 0 || pk[3] < 0);
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
                uint32_t v[4][VW];   // slots 2 t4 + 0, 1, 8, 9
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int slot = mt * 16 + 2 * t4 + (i & 1) + 8 * (i >> 1);
                    const uint8_t *p = vs + slot * D + g * (D / 8);
                    if (D == 128) {
                        const uint4 r = *reinterpret_cast<const uint4 *>(p);
                        v[i][0] = r.x; v[i][1] = r.y; v[i][VW - 2] = r.z; v[i][VW - 1] = r.w;
                    } else {
                        const uint2 r = *reinterpret_cast<const uint2 *>(p);
                        v[i][0] = r.x; v[i][1] = r.y;
                    }
                    if (!clean && (!ok || pos[slot] < 0)) {
#pragma unroll
                        for (int u = 0; u < VW; ++u) v[i][u] = 0;
                    }
#pragma unroll
                    for (int u = 0; u < VW; ++u) v[i][u] = ak8_bias<E4M3>(v[i][u]);
                }
#pragma unroll
                for (int u = 0; u < VW; ++u) {
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {   // elements 4 u + 2 hh, + 1 of two slots, side by side
                        const uint32_t sel = hh ? 0x7362u : 0x5140u;
                        uint32_t a0, a1, a2, a3;
                        ak8_widen<E4M3>(__byte_perm(v[0][u], v[1][u], sel), a0, a1);
                        ak8_widen<E4M3>(__byte_perm(v[2][u], v[3][u], sel), a2, a3);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            ak8_mma(acc[2 * u + hh][nt], a0, a1, a2, a3, pb[mt][nt][0], pb[mt][nt][1]);
                    }
                }
            }
        }
        __syncwarp();   // the stage has been read
        issue(st);
        if (++st == ST) {
            st = 0;
            parity ^= 1u;
        }
        const Ak8Cursor here = cur;
        cur.next(rows);
        if (cur.blk != 0 && x + 1 < x1) continue;

        // ---- the end of a (row, head), or of the run
        fresh = true;
        const bool whole = here.blk + 1 == here.blocks && x - here.blk >= seg0;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float sum = l[nt][e];
                sum += __shfl_xor_sync(0xffffffffu, sum, 4);
                sum += __shfl_xor_sync(0xffffffffu, sum, 8);
                sum += __shfl_xor_sync(0xffffffffu, sum, 16);
                const int c = nt * 8 + 2 * t4 + e;
                if (c >= ncol) continue;
                if (whole) {
                    const int cc = chunk * W + c;
                    const float inv = sum == 0.f ? 0.f : ak8_exp2(ak8_finite(M[nt][e]) - ak8_finite(m[nt][e])) / sum;
                    uint4 *o = reinterpret_cast<uint4 *>(
                        a.o + (((long long)here.b * a.T + cc / group) * a.n + h * group + cc % group) * D + g * (D / 8));
#pragma unroll
                    for (int i = 0; i < HS; ++i) {
                        uint32_t r[4];
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            r[u] = pack_bf2(acc[4 * i + u][nt][e] * 0x1p-14f * inv, acc[4 * i + u][nt][2 + e] * 0x1p-14f * inv);
                        o[i] = make_uint4(r[0], r[1], r[2], r[3]);
                    }
                } else {   // slot 0 of this run: its first (row, head); 1: its last
                    float *p = a.part + ((long long)(2 * run + (seg0 == x0 ? 0 : 1)) * cols + c) * (D + kAk8Part);
                    if (g == 0) {
                        p[D] = m[nt][e];
                        p[D + 1] = M[nt][e];
                        p[D + 2] = sum;
                    }
#pragma unroll
                    for (int i = 0; i < D / 32; ++i)
                        reinterpret_cast<float4 *>(p + g * (D / 8))[i] =
                            make_float4(acc[2 * i][nt][e], acc[2 * i][nt][2 + e], acc[2 * i + 1][nt][e], acc[2 * i + 1][nt][2 + e]);
                }
            }
    }
    cp_async_wait_all();
}

// Joins the partial results of one (row, head), in the order of the runs.  Block x
// is the (row, head) x where those are fewer than the runs; else the one that run
// x began and did not end.  Warps take the partials in turn, lanes D / 32 elements.
template <int D, int NT>
__global__ void __launch_bounds__(128) attn_kv8_join_kernel(const AttnKv8Args a, int warps, int by_head) {
    constexpr int W = 8 * NT, E = D / 32;
    __shared__ float sm_o[4][D], sm_l[4], sm_m[4][2];
    griddep_launch();
    griddep_wait();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int group = a.n / a.kv, C = group * a.T, chunks = (C + W - 1) / W;
    const Ak8Rows rows{a.lens, a.B, a.max_seq, a.kv * chunks};
    const long long total = ak8_total(rows), R = ak8_runs(total, warps);
    int b, head;
    long long first, end;   // its blocks
    if (by_head) {
        b = blockIdx.x / rows.heads;
        head = blockIdx.x % rows.heads;
        int before = 0;
        for (int i = lane; i < b; i += 32) before += rows.blocks(i);
        const int blocks = rows.blocks(b);
        if (blocks <= kAk8Short) return;
        first = (long long)__reduce_add_sync(0xffffffffu, before) * rows.heads + (long long)head * blocks;
        end = first + blocks;
    } else {
        if (blockIdx.x + 1 >= R) return;
        Ak8Cursor c;
        const long long x1 = (blockIdx.x + 1) * total / R;
        c.at(rows, x1);
        if (c.blocks <= kAk8Short || c.blk == 0) return;   // the cut lies between two
        b = c.b;
        head = c.head;
        first = x1 - c.blk;
        end = first + c.blocks;
        if (blockIdx.x * total / R > first) return;        // an earlier run began it
    }
    const int r0 = (int)(((first + 1) * R - 1) / total), r1 = (int)((end * R - 1) / total);   // the runs it lies in
    if (r0 == r1) return;
    // run r0 may have begun with an earlier (row, head)
    Ak8Cursor c;
    const int slot0 = ak8_cut(rows, r0, R, total, c) != first;
    const int chunk = head % chunks, h = head / chunks, ncol = min(W, C - chunk * W);
    for (int col = blockIdx.y; col < ncol; col += gridDim.y) {
        auto part = [&](int r) {
            return a.part + ((long long)(2 * r + (r == r0 ? slot0 : 0)) * a.part_cols + col) * (D + kAk8Part);
        };
        float mm = -INFINITY, MM = -INFINITY;
        for (int r = r0 + (int)threadIdx.x; r <= r1; r += 128) {
            const float2 v = *reinterpret_cast<const float2 *>(part(r) + D);
            mm = fmaxf(mm, v.x);
            MM = fmaxf(MM, v.y);
        }
        mm = warp_max(mm);
        MM = warp_max(MM);
        __syncthreads();   // the previous column's values have been read
        if (lane == 0) {
            sm_m[w][0] = mm;
            sm_m[w][1] = MM;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            mm = fmaxf(mm, sm_m[i][0]);
            MM = fmaxf(MM, sm_m[i][1]);
        }
        float o[E] = {}, ll = 0.f;
#pragma unroll 4
        for (int r = r0 + w; r <= r1; r += 4) {
            const float *p = part(r);
            const float4 st = *reinterpret_cast<const float4 *>(p + D);
            const float f = ak8_exp2(st.y - ak8_finite(MM));
            ll += st.z * ak8_exp2(st.x - ak8_finite(mm));
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] += p[32 * e + lane] * f;
        }
#pragma unroll
        for (int e = 0; e < E; ++e) sm_o[w][32 * e + lane] = o[e];
        if (lane == 0) sm_l[w] = ll;
        __syncthreads();
        ll = sm_l[0] + sm_l[1] + sm_l[2] + sm_l[3];
        const int d = threadIdx.x, cc = chunk * W + col;
        if (d < D) {
            const float inv = ll == 0.f ? 0.f : ak8_exp2(ak8_finite(MM) - ak8_finite(mm)) / ll;
            const float v = (sm_o[0][d] + sm_o[1][d] + sm_o[2][d] + sm_o[3][d]) * 0x1p-14f * inv;
            a.o[(((long long)b * a.T + cc / group) * a.n + h * group + cc % group) * D + d] = f2bf(v);
        }
    }
}

// CTAs per SM of a variant with its shared memory, found once per device.
template <int D, bool E4M3, int NT>
static cudaError_t ak8_launch(AttnKv8Args a, int sms, cudaStream_t s) {
    constexpr int kDevices = 64, W = 8 * NT;
    static std::atomic<int> known[kDevices][W + 1];
    const auto kern = attn_kv8_kernel<D, E4M3, NT>;
    const int group = a.n / a.kv, C = group * a.T, chunks = (C + W - 1) / W;
    a.part_cols = C < W ? C : W;
    const int smem = Ak8Stage<D>::smem(a.part_cols);
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    int per_sm = dev < kDevices ? known[dev][a.part_cols].load(std::memory_order_relaxed) : 0;
    if (per_sm == 0) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Ak8Stage<D>::smem(W));
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, kAk8Threads, smem);
        if (e != cudaSuccess) return e;
        per_sm = per_sm < 1 ? 1 : per_sm > kAk8MaxPerSm ? kAk8MaxPerSm : per_sm;
        if (dev < kDevices) known[dev][a.part_cols].store(per_sm, std::memory_order_relaxed);
    }
    const long long heads = (long long)a.B * a.kv * chunks;
    const long long most = heads * ((a.max_seq + kKv8Block - 1) / kKv8Block);
    const long long runs = (most + kAk8MinRun - 1) / kAk8MinRun;
    const int G = (int)(runs < (long long)sms * per_sm ? runs : (long long)sms * per_sm), warps = G * kAk8Warps;
    e = launch_pdl_smem(kern, dim3(G), dim3(kAk8Threads), smem, s, a);
    if (e != cudaSuccess || a.max_seq <= kAk8Short * kKv8Block) return e;   // nothing can have been cut
    const int by_head = heads < warps, blocks = by_head ? (int)heads : warps;
    int y = 2 * warps / blocks;   // columns apart while that keeps the grid small
    y = y < 1 ? 1 : y > a.part_cols ? a.part_cols : y;
    return launch_pdl(attn_kv8_join_kernel<D, NT>, dim3(blocks, y), dim3(128), s, a, warps, by_head);
}

size_t attn_kv8_workspace(int n, int kv, int T, int max_seq, int d, int sms) {
    const int C = n / kv * T, W = C <= 8 ? 8 : 16;
    if (max_seq <= kAk8Short * kKv8Block) return 0;
    return (size_t)sms * kAk8MaxPerSm * kAk8Warps * 2 * (C < W ? C : W) * (d + kAk8Part) * 4;
}

cudaError_t launch_attn_kv8(const AttnKv8Args &a, int d, int e4m3, int sms, cudaStream_t s) {
    // more than 8 columns: two column tiles a pass, or the codes would be read and widened twice
    const bool wide = a.n / a.kv * a.T > 8;
    if (d == 64) {
        if (wide) return e4m3 ? ak8_launch<64, true, 2>(a, sms, s) : ak8_launch<64, false, 2>(a, sms, s);
        return e4m3 ? ak8_launch<64, true, 1>(a, sms, s) : ak8_launch<64, false, 1>(a, sms, s);
    }
    if (wide) return e4m3 ? ak8_launch<128, true, 2>(a, sms, s) : ak8_launch<128, false, 2>(a, sms, s);
    return e4m3 ? ak8_launch<128, true, 1>(a, sms, s) : ak8_launch<128, false, 1>(a, sms, s);
}

}  // namespace bloom
