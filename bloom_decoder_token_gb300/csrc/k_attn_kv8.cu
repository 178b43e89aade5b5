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
//  * Work is cut evenly whatever the lengths: the tiles (128 slots) of all rows and
//    key heads are numbered in one sequence, and each of as many CTAs as are
//    resident takes an equal run of it.  A (row, key head) that falls into
//    several runs leaves partial results, which a second kernel joins in order.
//  * Each warp takes 32 slots (one scale block) of a tile and keeps its own ring of
//    stages ahead of it: two bulk copies (K, V) a stage, completing on an
//    mbarrier, and positions and scales by cp.async.  No barrier of the block
//    until a (row, key head) ends.
#include <atomic>
#include <math.h>

#include "common.cuh"
#include "kernels.h"
#include "kv8_ops.cuh"
#include "tc_ops.cuh"

namespace bloom {

constexpr int kAk8Warps = 4, kAk8Threads = 32 * kAk8Warps;
constexpr int kAk8Tile = kAk8Warps * kKv8Block;   // slots per tile
constexpr int kAk8Part = 4;                       // floats beside a partial's accumulator: m, M, l

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

// ---- where a tile number lies
struct Ak8Rows {
    const int *lens;
    int B, max_seq, heads;   // heads: (key head, column chunk) pairs of a row
    __device__ __forceinline__ int len(int b) const { return max(0, min(lens[b], max_seq)); }
    // tiles of one head of row b; at least one, so that every output is written
    __device__ __forceinline__ int tiles(int b) const { return max(1, (len(b) + kAk8Tile - 1) / kAk8Tile); }
};
// Tiles per head of all rows together, and the row that holds tile number x (with
// the number of its first tile), by the whole warp.
__device__ __forceinline__ long long ak8_total(const Ak8Rows &r) {
    const int lane = threadIdx.x & 31;
    int t = 0;
    for (int b = lane; b < r.B; b += 32) t += r.tiles(b);
    return (long long)__reduce_add_sync(0xffffffffu, t) * r.heads;
}
__device__ __forceinline__ int ak8_find(const Ak8Rows &r, long long x, long long &first) {
    const int lane = threadIdx.x & 31;
    long long before = 0;
    for (int b0 = 0; b0 < r.B; b0 += 32) {
        const int mine = b0 + lane < r.B ? r.tiles(b0 + lane) : 0;
        int sum = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += y;
        }
        const unsigned past = __ballot_sync(0xffffffffu, before + (long long)sum * r.heads > x);
        if (past) {
            const int src = __ffs(past) - 1;
            first = before + (long long)__shfl_sync(0xffffffffu, sum - mine, src) * r.heads;
            return b0 + src;
        }
        before += (long long)__shfl_sync(0xffffffffu, sum, 31) * r.heads;
    }
    first = before;
    return r.B;
}
struct Ak8Cursor {   // a tile: row, head, tile of that head
    int b, head, tile, len, tiles;
    __device__ __forceinline__ void at(const Ak8Rows &r, long long x) {
        long long first;
        b = ak8_find(r, x, first);
        row(r);
        head = (int)((x - first) / tiles);
        tile = (int)((x - first) % tiles);
    }
    __device__ __forceinline__ void row(const Ak8Rows &r) {
        len = b < r.B ? r.len(b) : 0;
        tiles = b < r.B ? r.tiles(b) : 1;
    }
    __device__ __forceinline__ void next(const Ak8Rows &r) {
        if (++tile < tiles) return;
        tile = 0;
        if (++head < r.heads) return;
        head = 0;
        ++b;
        row(r);
    }
};

template <int D, int NT>
struct Ak8Smem {
    static constexpr int kStages = 256 / D;
    uint8_t kv[kAk8Warps][kStages][2][kKv8Block * D];
    int pos[kAk8Warps][kStages][kKv8Block];
    float scale[kAk8Warps][kStages][2];
    uint64_t bar[kAk8Warps][kStages];
    float stat[kAk8Warps][8 * NT][3];   // m, M, l of a warp
    // then accumulators [kAk8Warps][columns][D]
};

// Columns of a chunk: query c = t * group + i of a key head, t the token, i the query head.
template <int D, bool E4M3, int NT>
__global__ void __launch_bounds__(kAk8Threads, NT == 1 ? 3 : 2) attn_kv8_kernel(const AttnKv8Args a) {
    constexpr int HS = D / 64, VW = D / 32, W = 8 * NT;   // K segments of 16 bytes a lane; V words a key
    using Smem = Ak8Smem<D, NT>;
    constexpr int ST = Smem::kStages;
    extern __shared__ __align__(128) unsigned char ak8_raw[];
    Smem &sm = *reinterpret_cast<Smem *>(ak8_raw);
    float *sm_acc = reinterpret_cast<float *>(ak8_raw + sizeof(Smem));
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, g = lane >> 2, t4 = lane & 3;
    if (lane == 0) {
        for (int i = 0; i < ST; ++i) tc_mbar_init(&sm.bar[w][i], 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncwarp();
    griddep_launch();
    griddep_wait();

    const int group = a.n / a.kv, C = group * a.T, chunks = (C + W - 1) / W;
    const Ak8Rows rows{a.lens, a.B, a.max_seq, a.kv * chunks};
    const long long total = ak8_total(rows), G = min((long long)gridDim.x, total);   // no run is empty
    if (blockIdx.x >= G) return;
    const long long x0 = blockIdx.x * total / G, x1 = (blockIdx.x + 1) * total / G;
    if (a.err && blockIdx.x == 0)
        for (int b = tid; b < a.B; b += kAk8Threads)
            if (a.lens[b] > a.max_seq) atomicOr(a.err, kErrSlot);
    Ak8Cursor cur, ahead;
    cur.at(rows, x0);
    ahead = cur;

    // the next tile with keys for this warp into stage `st`; one cp.async group, empty at the end
    long long xa = x0;
    auto issue = [&](int st) {
        for (; xa < x1; ++xa, ahead.next(rows)) {
            const int base = ahead.tile * kAk8Tile + w * kKv8Block, n = min(kKv8Block, ahead.len - base);
            if (n <= 0) continue;
            const long long bh = (long long)ahead.b * a.kv + ahead.head / chunks;
            if (lane == 0) {
                const uint32_t bar = tc_smem(&sm.bar[w][st]);
                asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(2 * n * D) : "memory");
#pragma unroll
                for (int v = 0; v < 2; ++v)
                    asm volatile(
                        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                            tc_smem(&sm.kv[w][st][v][0])),
                        "l"((v ? a.vc : a.kc) + (bh * a.max_seq + base) * D), "r"(n * D), "r"(bar)
                        : "memory");
            }
            if (lane < n)
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(tc_smem(&sm.pos[w][st][lane])),
                             "l"(a.pos + (long long)ahead.b * a.max_seq + base + lane)
                             : "memory");
            else
                sm.pos[w][st][lane] = -1;
            if (lane < 2)
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(tc_smem(&sm.scale[w][st][lane])),
                             "l"((lane ? a.vs : a.ks) + bh * a.blocks + base / kKv8Block)
                             : "memory");
            ++xa;
            ahead.next(rows);
            break;
        }
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < ST; ++i) issue(i);

    constexpr float kLog2e = 1.4426950408889634f;
    uint32_t qf[NT][D / 16][2];
    float qinv[NT][2], slope[NT][2], m[NT][2], M[NT][2], l[NT][2], acc[D / 16][NT][4];
    int lim[NT][2];                // slots that a column sees
    int ref = 0, ref_row = -1, st = 0;
    uint32_t parity = 0;
    long long seg0 = x0;           // first tile of the current (row, head) in this run
    bool fresh = true;
    for (long long x = x0; x < x1; ++x) {
        const int chunk = cur.head % chunks, h = cur.head / chunks;
        const int ncol = min(W, C - chunk * W);
        if (fresh) {
            fresh = false;
            seg0 = x;
            if (ref_row != cur.b) {
                ref_row = cur.b;
                ref = -1;
                const int *pos = a.pos + (long long)cur.b * a.max_seq;
                for (int k0 = cur.len; k0 > 0 && ref < 0; k0 -= 32)
                    ref = __reduce_max_sync(0xffffffffu, k0 - 1 - lane >= 0 ? pos[k0 - 1 - lane] : -1);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                // B fragments: column g, elements 64 s + 16 t4 + 4 u + (0, 1 | 2, 3)
                const int c = chunk * W + nt * 8 + g;
                uint4 raw[HS][2];
                uint32_t amax = 0;
#pragma unroll
                for (int s = 0; s < HS; ++s) {
                    raw[s][0] = raw[s][1] = make_uint4(0u, 0u, 0u, 0u);
                    if (c < C) {
                        const uint4 *q = reinterpret_cast<const uint4 *>(
                            a.q + (((long long)cur.b * a.T + c / group) * a.n + h * group + c % group) * D + 64 * s + 16 * t4);
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
        const int base = cur.tile * kAk8Tile + w * kKv8Block;
        if (cur.len > base) {   // this warp has keys in the tile: the stage's turn
            cp_async_wait<ST - 1>();
            bool ok = tc_mbar_wait(&sm.bar[w][st], parity, 0);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) {   // report; a second bounded wait, so that no copy lands later; the block is skipped
                if (a.err) atomicOr(a.err, kErrTimeout);
                tc_mbar_wait(&sm.bar[w][st], parity, kTcWaitNs);
            }
            __syncwarp();
            const uint8_t *ks = &sm.kv[w][st][0][0], *vs = &sm.kv[w][st][1][0];
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
            const float kscale = sm.scale[w][st][0], vscale = sm.scale[w][st][1];
            // vscale = mant * 2^ev
            const uint32_t vb = __float_as_uint(vscale), vexp = (vb >> 23) & 255u;
            const float ev = vexp == 255u ? 0.f : vexp == 0u ? -126.f : (float)((int)vexp - 127);
            const float mant = vexp == 255u ? vscale : vexp == 0u ? vscale * 0x1p126f : __uint_as_float((vb & 0x807fffffu) | 0x3f800000u);
            int pk[4];
            float dp[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                pk[i] = ok ? sm.pos[w][st][8 * i + g] : -1;
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
                    if (!clean && (!ok || sm.pos[w][st][slot] < 0)) {
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
            __syncwarp();   // the stage has been read
            issue(st);
            if (++st == ST) {
                st = 0;
                parity ^= 1u;
            }
        }
        const Ak8Cursor here = cur;
        cur.next(rows);
        if (cur.tile != 0 && x + 1 < x1) continue;

        // ---- the end of a (row, head), or of the run: join the four warps
        fresh = true;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float sum = l[nt][e];
                sum += __shfl_xor_sync(0xffffffffu, sum, 4);
                sum += __shfl_xor_sync(0xffffffffu, sum, 8);
                sum += __shfl_xor_sync(0xffffffffu, sum, 16);
                const int c = nt * 8 + 2 * t4 + e;
                if (c < ncol) {
                    if (g == 0) {
                        sm.stat[w][c][0] = m[nt][e];
                        sm.stat[w][c][1] = M[nt][e];
                        sm.stat[w][c][2] = sum;
                    }
                    float2 *dst = reinterpret_cast<float2 *>(sm_acc + (w * ncol + c) * D + g * (D / 8));
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) dst[i] = make_float2(acc[i][nt][e], acc[i][nt][2 + e]);
                }
            }
        __syncthreads();
        const bool whole = here.tile + 1 == here.tiles && x - here.tile >= seg0;
        for (int i = tid; i < ncol * D; i += kAk8Threads) {
            const int c = i / D, d = i % D;
            float mm = -INFINITY, MM = -INFINITY, ll = 0.f, oo = 0.f;
#pragma unroll
            for (int k = 0; k < kAk8Warps; ++k) {
                mm = fmaxf(mm, sm.stat[k][c][0]);
                MM = fmaxf(MM, sm.stat[k][c][1]);
            }
#pragma unroll
            for (int k = 0; k < kAk8Warps; ++k) {
                ll += sm.stat[k][c][2] * ak8_exp2(sm.stat[k][c][0] - ak8_finite(mm));
                oo += sm_acc[(k * ncol + c) * D + d] * ak8_exp2(sm.stat[k][c][1] - ak8_finite(MM));
            }
            if (whole) {
                const int cc = chunk * W + c;
                const float o = ll == 0.f ? 0.f : oo * 0x1p-14f * ak8_exp2(ak8_finite(MM) - ak8_finite(mm)) / ll;
                a.o[(((long long)here.b * a.T + cc / group) * a.n + h * group + cc % group) * D + d] = f2bf(o);
            } else {   // slot 0 of this CTA: the run's first (row, head); 1: its last
                float *p = a.part + ((long long)(2 * blockIdx.x + (seg0 == x0 ? 0 : 1)) * a.part_cols + c) * (D + kAk8Part);
                p[d] = oo;
                if (d == 0) {
                    p[D] = mm;
                    p[D + 1] = MM;
                    p[D + 2] = ll;
                }
            }
        }
        __syncthreads();
    }
    cp_async_wait_all();
}

// Joins the partial results of the (row, head) that CTA blockIdx.x of the kernel
// above began and did not end, in the order of the runs.
template <int D, int NT>
__global__ void __launch_bounds__(D) attn_kv8_join_kernel(const AttnKv8Args a, int ctas) {
    constexpr int W = 8 * NT;
    griddep_launch();
    griddep_wait();
    const int group = a.n / a.kv, C = group * a.T, chunks = (C + W - 1) / W;
    const Ak8Rows rows{a.lens, a.B, a.max_seq, a.kv * chunks};
    const long long total = ak8_total(rows), G = min((long long)ctas, total);
    if (blockIdx.x >= G) return;
    const long long x0 = blockIdx.x * total / G, x1 = (blockIdx.x + 1) * total / G;
    Ak8Cursor last;
    last.at(rows, x1 - 1);
    const long long first = x1 - 1 - last.tile, end = first + last.tiles;   // tiles of that (row, head)
    if (first < x0 || end <= x1) return;   // begun by an earlier CTA, or ended here
    const int c1 = (int)((end * G - 1) / total);                            // the CTA that ends it
    const int chunk = last.head % chunks, h = last.head / chunks, ncol = min(W, C - chunk * W), d = threadIdx.x;
    for (int c = blockIdx.y; c < ncol; c += gridDim.y) {
        auto part = [&](int cta) {
            return a.part + ((long long)(2 * cta + (cta == (int)blockIdx.x && first != x0)) * a.part_cols + c) * (D + kAk8Part);
        };
        float mm = -INFINITY, MM = -INFINITY, ll = 0.f, oo = 0.f;
        for (int k = blockIdx.x; k <= c1; ++k) {
            const float *p = part(k);
            mm = fmaxf(mm, p[D]);
            MM = fmaxf(MM, p[D + 1]);
        }
        for (int k = blockIdx.x; k <= c1; ++k) {
            const float *p = part(k);
            ll += p[D + 2] * ak8_exp2(p[D] - ak8_finite(mm));
            oo += p[d] * ak8_exp2(p[D + 1] - ak8_finite(MM));
        }
        const int cc = chunk * W + c;
        const float o = ll == 0.f ? 0.f : oo * 0x1p-14f * ak8_exp2(ak8_finite(MM) - ak8_finite(mm)) / ll;
        a.o[(((long long)last.b * a.T + cc / group) * a.n + h * group + cc % group) * D + d] = f2bf(o);
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
    const size_t smem = sizeof(Ak8Smem<D, NT>) + (size_t)kAk8Warps * a.part_cols * D * 4;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    int per_sm = dev < kDevices ? known[dev][a.part_cols].load(std::memory_order_relaxed) : 0;
    if (per_sm == 0) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)(sizeof(Ak8Smem<D, NT>) + (size_t)kAk8Warps * W * D * 4));
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, kAk8Threads, smem);
        if (e != cudaSuccess) return e;
        per_sm = per_sm < 1 ? 1 : per_sm > kAk8MaxPerSm ? kAk8MaxPerSm : per_sm;
        if (dev < kDevices) known[dev][a.part_cols].store(per_sm, std::memory_order_relaxed);
    }
    const long long most = (long long)a.B * a.kv * chunks * ((a.max_seq + kAk8Tile - 1) / kAk8Tile);
    const int G = (int)(most < (long long)sms * per_sm ? most : (long long)sms * per_sm);
    e = launch_pdl_smem(kern, dim3(G), dim3(kAk8Threads), smem, s, a);
    // rows of one tile are never cut
    if (e == cudaSuccess && a.max_seq > kAk8Tile)
        e = launch_pdl(attn_kv8_join_kernel<D, NT>, dim3(G, a.part_cols < 4 ? a.part_cols : 4), dim3(D), s, a, G);
    return e;
}

size_t attn_kv8_workspace(int n, int kv, int T, int max_seq, int d, int sms) {
    const int C = n / kv * T, W = C <= 8 ? 8 : 16;
    if (max_seq <= kAk8Tile) return 0;
    return (size_t)sms * kAk8MaxPerSm * 2 * (C < W ? C : W) * (d + kAk8Part) * 4;
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
