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
//    (int8: one; exact for both code types; V's codes in the forms with several
//    columns: two instructions to bf16) and, in V, half a byte permutation that pairs
//    two keys.  tcgen05 would want the codes in f16 in shared memory first.
//  * q is multiplied by a power of two that brings its largest element to
//    [2^14, 2^15), where bf16 -> f16 is exact from 2^-28 of that element on
//    (smaller ones are off by 2^-39 of it at most); the scores are float32 sums
//    of exact products.
//  * The softmax is one pass: running maxima and sums in float32, in powers of
//    two.  The weight of V_k carries the block's V scale: exp2(s_k + log2 scale -
//    M) with a reference M of its own, the largest such sum.  Both references
//    move, and what was summed is rescaled, only when a score passes one by
//    more than 2^8.
//  * The weights, multiplied with exact codes into float32 accumulators, keep 16
//    bits at least and a float's range: a key of zeros, or a block that is large in
//    other channels only, may lie any number of binades above the keys that make an
//    output.  Several columns: two bf16 parts (8 + 8 bits, from 2^-126 of the
//    reference on), a product each.  One column: the other seven columns of the same
//    product are free, so the weight goes in as f16 parts (11 + 11 bits) in one of
//    four column pairs by its size, 28 binades each (from 2^-104 of the reference
//    on, fewer bits to 2^-114, then 0).  Weights of one f16 part, 2^-31 of the
//    reference at least, lost such outputs; they took 29 against 34 us for 16 rows x 4
//    tokens over 1025..4090 slots, 32 heads on 8, and the same time in the one-column form.
//  * Work is cut evenly whatever the lengths: the blocks (32 slots at d = 128, 64 at
//    64) of all rows and key heads are numbered in one sequence, and each resident
//    warp takes an equal run of it.  A (row, key head) of at most kAk8Whole slots
//    is left whole; a longer one that falls into several runs leaves partial
//    results, which a second kernel joins in order.
//  * A warp keeps its own ring of stages ahead of it, one block each: K and V by TMA
//    (swizzled by the row's width, and the slots dealt to the fragments' rows, so
//    that the fragment loads meet no bank twice), and by cp.async positions,
//    scales and, at the first block of a (row, key head), its queries.  Warps
//    never wait for one another.
// Measured (codes' bytes over time, join included): 4 rows of 30-33k slots, 32 x 128,
// e4m3, 168 us = 6.2 TB/s; 32 rows of 130..2011, int8, 54 us = 5.3 TB/s; 16 rows x 4
// tokens over 1025..4090 slots, 32 heads on 8, 34 us, bound by the latency of eight
// warps' instructions an SM; one row of 2000, 9.6 us; one of 41
// slots, 16 x 64, 4.8 us.  What short jobs lose is about 5 us from launch to the first
// block's data and 3 us for the join.
#include <atomic>
#include <math.h>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "kv8_ops.cuh"
#include "tc_ops.cuh"

namespace bloom {

constexpr int kAk8Warps = 4, kAk8Threads = 32 * kAk8Warps;
// Slots of a block of work: 4 KB of K and of V, one scale block at d = 128, two at 64.
__host__ __device__ constexpr int ak8_slots(int D) { return 4096 / D; }
// A (row, key head) of up to so many slots is never cut, and caches of at most so many need no
// join: a launch, a workspace and about 5 us of the host less a call.  On the GPU (32 x 128,
// int8, 160 slots, 128 against 192), a cache of 160: 1 row 8.0, 8.8 us; 8 rows 8.8, 10.7; 32 rows
// 14.9, 13.2; a cache of 2048, where the join runs all the same: 7.7, 9.7; 8.7, 11.2; 14.9,
// 13.9.  256 would cost more: 1 row of 250 11.3 against 7.3 us, 8 rows 13.9 against 8.4.
constexpr int kAk8Whole = 192;
constexpr int kAk8MinRun = 64;    // slots a warp takes at least (one sequence of 2000, 32 heads x 128: 32, 64, 128,
                                  // 256 slots at least: 10.9, 9.6, 11.1, 14.5 us)
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
// The same to bf16 pairs, exact too (a NaN code stays NaN); int8 codes come without the bias.
__device__ __forceinline__ uint32_t ak8_s8x2_bf16(uint32_t w, uint32_t sel) {
    // 0x4300 | byte is 128 + its low seven bits where the sign bit is taken out; less 128 or, negative, 256
    const uint32_t t = __byte_perm(w, 0x43434343u, sel);
    uint32_t r;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(t & 0xff7fff7fu), "r"(t & 0xff80ff80u));
    return r;
}
template <bool E4M3>
__device__ __forceinline__ void ak8_widen_bf16(uint32_t w, uint32_t &lo, uint32_t &hi) {
    if (E4M3) {
        float f[4];
        kv8_widen_e4m3(w, f);
        lo = __byte_perm(__float_as_uint(f[0]), __float_as_uint(f[1]), 0x7632);
        hi = __byte_perm(__float_as_uint(f[2]), __float_as_uint(f[3]), 0x7632);
    } else {
        lo = ak8_s8x2_bf16(w, 0x4140);
        hi = ak8_s8x2_bf16(w, 0x4342);
    }
}

__device__ __forceinline__ void ak8_mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ak8_mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
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
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));   // relative error 2^-22
    return r;
}
__device__ __forceinline__ float ak8_finite(float m) { return m == -INFINITY ? 0.f : m; }

constexpr float kAk8Lift = 6.f;   // weights carry 2^6: up to 2^15
// The one-column form's f16 weights: column pair j takes those from 2^(-20 - 28 j) to 2^(8 - 28 j)
// of the reference (the last pair all smaller ones), times 2^(28 j), as two parts: eleven bits,
// and what is left of the weight times 2^11.
constexpr float kAk8Band = 28.f, kAk8Low = -20.f;

// The output of an accumulated value, from the references and the sum: v 2^(M - m - lift) / l,
// in two steps, for M - m may pass the range of a float's exponent; 0 where nothing was seen.
struct Ak8Last {
    float a, b;
    __device__ __forceinline__ Ak8Last(float m, float M, float l) {
        a = ak8_exp2(0.5f * (ak8_finite(M) - ak8_finite(m) - kAk8Lift));
        b = l == 0.f ? 0.f : a / l;
    }
    __device__ __forceinline__ float of(float v) const { return v * a * b; }
};

// ---- where a block number lies
template <int D>
struct Ak8Rows {
    static constexpr int kSlots = ak8_slots(D);
    const int *lens;
    int B, max_seq, heads;   // heads: (key head, column chunk) pairs of a row
    __device__ __forceinline__ int len(int b) const { return max(0, min(lens[b], max_seq)); }
    // blocks of one head of row b; at least one, so that every output is written
    __device__ __forceinline__ int blocks(int b) const { return max(1, (len(b) + kSlots - 1) / kSlots); }
};
template <int D>
__device__ __forceinline__ int ak8_total(const Ak8Rows<D> &r) {   // by the whole warp
    int t = 0;
    for (int b = threadIdx.x & 31; b < r.B; b += 32) t += r.blocks(b);
    return __reduce_add_sync(0xffffffffu, t) * r.heads;
}
struct Ak8Cursor {   // a block: its row, head, place in that head; the row's length and blocks a head
    int b, head, blk, len, blocks;
    // block number x < total, by the whole warp
    template <int D>
    __device__ __forceinline__ void at(const Ak8Rows<D> &r, int x) {
        const int lane = threadIdx.x & 31;
        int before = 0;
        for (int b0 = 0;; b0 += 32) {
            const int mine = b0 + lane < r.B ? r.blocks(b0 + lane) * r.heads : 0;
            int sum = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += y;
            }
            const unsigned past = __ballot_sync(0xffffffffu, before + sum > x);
            if (past || b0 + 32 >= r.B) {
                const int src = past ? __ffs(past) - 1 : 31;
                b = b0 + src;
                x -= before + __shfl_sync(0xffffffffu, sum - mine, src);
                break;
            }
            before += __shfl_sync(0xffffffffu, sum, 31);
        }
        row(r);
        head = x / blocks;
        blk = x - head * blocks;
    }
    template <int D>
    __device__ __forceinline__ void row(const Ak8Rows<D> &r) {
        len = b < r.B ? r.len(b) : 0;
        blocks = b < r.B ? r.blocks(b) : 1;
    }
    template <int D>
    __device__ __forceinline__ void next(const Ak8Rows<D> &r) {
        if (++blk < blocks) return;
        blk = 0;
        if (++head < r.heads) return;
        head = 0;
        ++b;
        row(r);
    }
};
// The runs: R equal shares of `total` blocks, the first `rem` one longer.
template <int D>
struct Ak8Runs {
    static constexpr int kWhole = kAk8Whole / ak8_slots(D), kMin = kAk8MinRun / ak8_slots(D);   // in blocks
    int total, R, q, rem;
    __device__ __forceinline__ Ak8Runs(int t, int warps) : total(t) {
        R = min(warps, (t + kMin - 1) / kMin);
        q = t / R;
        rem = t - q * R;
    }
    __device__ __forceinline__ int start(int k) const { return k * q + min(k, rem); }
    __device__ __forceinline__ int of(int x) const {   // the run that block x falls into
        const int y = x - rem * (q + 1);
        return y < 0 ? x / (q + 1) : rem + y / q;
    }
    // where run k begins in earnest: a short (row, head) belongs to the run of its last block
    __device__ __forceinline__ int cut(const Ak8Rows<D> &r, int k, Ak8Cursor &c) const {
        int x = start(k);
        if (x >= total) return total;
        c.at(r, x);
        if (c.blocks <= kWhole) {
            x -= c.blk;
            c.blk = 0;
        }
        return x;
    }
};

struct Ak8Maps {   // K and V codes as rows of D bytes
    CUtensorMap k, v;
};

// CTAs an SM, by registers.  One column: two with three stages a warp rather than three
// with two (HBM serves 1216 streams better than 1824; e4m3, 4 x 30-33k slots, 32 x 128:
// 162 against 187 us; 32 x 130..2011 slots, 16 x 64: 20.5 against 22.5 us).
constexpr int ak8_per_sm(int NT, bool ONE) { return NT == 2 || ONE ? 2 : 3; }

// Shared memory of a CTA: stages of K and V [warps][stages], 1024-byte aligned; beside
// each stage its queries [cols][D], positions of the block, of the row's last 32
// slots, slopes [16], scales [2 or 4]; an mbarrier per stage.
template <int D, bool ONE>
struct Ak8Smem {
    static constexpr int kStages = ONE ? 3 : 2, kSlots = ak8_slots(D), kStage = 2 * kSlots * D;
    static constexpr int kAll = kAk8Warps * kStages, kPos = 4 * (kSlots + 32);   // bytes of positions
    __host__ __device__ static constexpr int side(int cols) { return cols * D * 2 + kPos + 64 + 16; }
    __host__ __device__ static constexpr int bytes(int cols) { return 1024 + kAll * (kStage + side(cols) + 8); }
};

__device__ __forceinline__ void ak8_async4(const void *dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(tc_smem(dst)), "l"(src) : "memory");
}

// Wait for the phase `parity` of `bar`: tc_mbar_wait, or, where the caller set a bound,
// without its try_wait, which may itself sleep for longer than a bound of microseconds.
__device__ __forceinline__ bool ak8_wait(uint64_t *bar, uint32_t parity, unsigned long long limit_ns) {
    if (limit_ns == 0) return tc_mbar_wait(bar, parity);
    const unsigned long long t0 = tc_now_ns();
    for (;;) {
        uint32_t done;
        asm volatile("{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
                     : "=r"(done)
                     : "r"(tc_smem(bar)), "r"(parity)
                     : "memory");
        if (done) return true;
        if (tc_now_ns() - t0 > limit_ns) return false;
    }
}

// The slot (of 8) that row r of a fragment takes.  With 16-byte pieces c of a row at
// c ^ slot % 8 (D = 128) or c ^ slot / 2 % 4 (D = 64), the eight lanes of a K access
// (rows 2 i and 2 i + 1, four pieces each) and those of a V access (rows 0, 2, 4, 6
// or 1, 3, 5, 7, two pieces each; 8 bytes and sixteen lanes at D = 64) cover all banks.
template <int D>
__device__ __forceinline__ int ak8_slot(int r) {
    return (int)((D == 128 ? 0x37621540u : 0x65742130u) >> (4 * r)) & 7;
}

// Columns of a chunk: query c = t * group + i of a key head, t the token, i the query
// head.  ONE: a single column in all (T = 1, as many key heads as query heads).
template <int D, bool E4M3, int NT, bool ONE>
__global__ void __launch_bounds__(kAk8Threads, ak8_per_sm(NT, ONE))
    attn_kv8_kernel(const __grid_constant__ AttnKv8Args a, const __grid_constant__ Ak8Maps maps) {
    constexpr int HS = D / 64, VW = D / 32, W = 8 * NT, NE = ONE ? 1 : 2;
    constexpr int SL = ak8_slots(D), MT = SL / 16, NB = SL / kKv8Block;   // slots, fragments of 16, scale blocks of a block
    using Smem = Ak8Smem<D, ONE>;
    constexpr int ST = Smem::kStages;
    constexpr float kLog2e = 1.4426950408889634f, kSlack = 8.f;
    extern __shared__ __align__(1024) unsigned char ak8_raw[];
    unsigned char *smem = ak8_raw + ((0u - tc_smem(ak8_raw)) & 1023u);
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, g = lane >> 2, t4 = lane & 3;
    const int cols = a.part_cols, side_bytes = Smem::side(cols);
    unsigned char *ring = smem + w * ST * Smem::kStage;
    unsigned char *sides = smem + Smem::kAll * Smem::kStage + w * ST * side_bytes;
    uint64_t *bar = reinterpret_cast<uint64_t *>(smem + Smem::kAll * (Smem::kStage + side_bytes)) + w * ST;
    if (lane == 0) {
        for (int i = 0; i < ST; ++i) tc_mbar_init(&bar[i], 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncwarp();
    griddep_wait();
    griddep_launch();   // after the wait: what the join kernel finds when it starts is final but for the partials

    const int group = ONE ? 1 : a.n / a.kv, C = ONE ? 1 : group * a.T, chunks = ONE ? 1 : (C + W - 1) / W;
    const Ak8Rows<D> rows{a.lens, a.B, a.max_seq, a.kv * chunks};
    if (a.err && blockIdx.x == 0)
        for (int b = threadIdx.x; b < a.B; b += kAk8Threads)
            if (a.lens[b] > a.max_seq) atomicOr(a.err, kErrSlot);
    const Ak8Runs<D> runs(ak8_total(rows), (int)gridDim.x * kAk8Warps);
    const int run = w * (int)gridDim.x + (int)blockIdx.x;   // runs spread over the CTAs first
    if (run >= runs.R) return;
    Ak8Cursor cur = {}, ahead = {};
    const int x1 = runs.cut(rows, run + 1, ahead), x0 = runs.cut(rows, run, cur);
    if (x0 >= x1) return;
    ahead = cur;

    // block xa of the run into stage `st`; one cp.async group, empty beyond the end
    int xa = x0, bh = 0;   // bh: row * key heads + key head of block xa
    auto issue = [&](int st) {
        if (xa < x1) {
            unsigned char *stage = ring + st * Smem::kStage, *side = sides + st * side_bytes;
            int *pos = reinterpret_cast<int *>(side + cols * D * 2);   // [SL], [32], slopes, scales
            const int base = ahead.blk * SL;
            const int *rowpos = a.pos + (long long)ahead.b * a.max_seq;
            if (xa == x0 || ahead.blk == 0) {   // the first block of a (row, head) in this run
                const int h = ONE ? ahead.head : ahead.head / chunks, c0 = (ahead.head - h * chunks) * W;
                bh = ahead.b * a.kv + h;
                if (ahead.len - 1 - lane >= 0) ak8_async4(pos + SL + lane, rowpos + ahead.len - 1 - lane);
                else pos[SL + lane] = -1;
                const int nc = ONE ? 1 : min(W, C - c0);
                if (a.slopes && lane < nc) ak8_async4(pos + SL + 32 + lane, a.slopes + h * group + (c0 + lane) % group);
                for (int i = lane; i < nc * (D / 8); i += 32) {
                    const int c = c0 + i / (D / 8), e = i % (D / 8) * 8;
                    cp_async16(side + (i / (D / 8) * D + e) * 2,
                               a.q + (((long long)ahead.b * a.T + c / group) * a.n + h * group + c % group) * D + e);
                }
            }
            if (lane == 0 && ahead.len == 0) {   // an idle row
                asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(tc_smem(&bar[st])) : "memory");
            } else if (lane == 0) {
                // slots beyond the row's length come along; they are masked
                asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(tc_smem(&bar[st])), "r"(Smem::kStage)
                             : "memory");
                tc_tma_2d(stage, &maps.k, 0, bh * a.max_seq + base, &bar[st]);
                tc_tma_2d(stage + SL * D, &maps.v, 0, bh * a.max_seq + base, &bar[st]);
            }
#pragma unroll
            for (int i = 0; i < SL; i += 32) {
                if (base + i + lane < ahead.len) ak8_async4(pos + i + lane, rowpos + base + i + lane);
                else pos[i + lane] = -1;
            }
            if (lane < 2 * NB)   // K, V; the row's last block may have no second scale
                ak8_async4(pos + SL + 48 + lane, (lane & 1 ? a.vs : a.ks) + (long long)bh * a.blocks + min(ahead.blk * NB + (lane >> 1), a.blocks - 1));
            ++xa;
            ahead.next(rows);
        }
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < ST; ++i) issue(i);

    // this lane's places in a stage: K rows g (8 slots further: + 8 D), V slots of rows
    // 2 t4 and 2 t4 + 1
    const int slot_g = ak8_slot<D>(g), va = ak8_slot<D>(2 * t4), vb = ak8_slot<D>(2 * t4 + 1);
    int koff[HS], voff[2];
    if (D == 128) {
#pragma unroll
        for (int i = 0; i < HS; ++i) koff[i] = slot_g * D + ((4 * i + t4) ^ slot_g) * 16;
        voff[0] = va * D + (g ^ va) * 16;
        voff[1] = vb * D + (g ^ vb) * 16;
    } else {   // 8 slots are two periods of the swizzle: the offset is the same
        koff[0] = slot_g * D + (t4 ^ (slot_g >> 1)) * 16;
        voff[0] = va * D + ((g >> 1) ^ (va >> 1)) * 16 + (g & 1) * 8;
        voff[1] = vb * D + ((g >> 1) ^ (vb >> 1)) * 16 + (g & 1) * 8;
    }

    // ONE: the weights of this lane's column pair, in binades below the reference, and their factor
    const float band_lo = t4 == 3 ? -INFINITY : kAk8Low - kAk8Band * t4, band_hi = t4 == 0 ? INFINITY : kAk8Low - kAk8Band * (t4 - 1);
    const float band_up = ak8_exp2(kAk8Lift + kAk8Band * t4), band_down = ak8_exp2(-kAk8Band * t4);

    uint32_t qf[NT][D / 16][2];
    float qs[NT][NE], slope[NT][NE], m[NT][NE], M[NT][NE], l[NT][NE], acc[D / 16][NT][4];
    int lim[NT][NE];               // slots that a column sees
    int chunk = 0, h = 0, ncol = 1, all = 0;   // all: slots that every column sees
    int ref = 0, st = 0, seg0 = x0;            // seg0: first block of the current (row, head) in this run
    uint32_t parity = 0;
    bool fresh = true;

    // A wait for block x expired: report it, wait (with a bound again) for the copies in
    // flight, so that none lands later, and give up the rest of the run: NaN for every
    // (row, head) that it has blocks of.
    auto give_up = [&](int x) {
        if (a.err && lane == 0) atomicOr(a.err, kErrTimeout);
        for (int y = x; y < xa; ++y) {
            tc_mbar_wait(&bar[st], parity, kTcWaitNs);
            if (++st == ST) {
                st = 0;
                parity ^= 1u;
            }
        }
        for (;;) {
            if (fresh) seg0 = x;
            const int hd = ONE ? cur.head : cur.head / chunks, c0 = (cur.head - hd * chunks) * W, nc = ONE ? 1 : min(W, C - c0);
            const int last = min(cur.blocks - 1, cur.blk + (x1 - 1 - x));   // of its blocks in this run
            x += last + 1 - cur.blk;
            cur.blk = last;
            if (last + 1 == cur.blocks && x - 1 - last >= seg0) {
                for (int i = lane; i < nc * (D / 8); i += 32) {
                    const int cc = c0 + i / (D / 8);
                    reinterpret_cast<uint4 *>(a.o + (((long long)cur.b * a.T + cc / group) * a.n + hd * group + cc % group) * D)[i % (D / 8)] =
                        make_uint4(0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u);
                }
            } else if (lane < nc) {   // a partial result whose sum is NaN
                float *p = a.part + ((long long)(2 * run + (seg0 == x0 ? 0 : 1)) * cols + lane) * (D + kAk8Part);
                *reinterpret_cast<float4 *>(p + D) = make_float4(-INFINITY, -INFINITY, __uint_as_float(0x7fc00000u), 0.f);
            }
            if (x >= x1) break;
            cur.next(rows);
            fresh = true;
        }
    };
    for (int x = x0; x < x1; ++x) {
        unsigned char *stage = ring + st * Smem::kStage;
        const int *pos = reinterpret_cast<const int *>(sides + st * side_bytes + cols * D * 2);
        // ---- the block's copies
        cp_async_wait<ST - 1>();
        if (!__all_sync(0xffffffffu, ak8_wait(&bar[st], parity, a.wait_ns))) {
            give_up(x);
            break;
        }
        __syncwarp();
        if (fresh) {
            fresh = false;
            seg0 = x;
            h = ONE ? cur.head : cur.head / chunks;
            chunk = cur.head - h * chunks;
            ncol = ONE ? 1 : min(W, C - chunk * W);
            all = cur.len - a.T + 1 + (ONE ? 0 : chunk * W / group);
            ref = __reduce_max_sync(0xffffffffu, pos[SL + lane]);
            for (int k0 = cur.len - 33 - lane; ref < 0 && k0 + lane >= 0; k0 -= 512) {   // pads alone at the row's end
                int best = -1;
#pragma unroll
                for (int u = 0; u < 16; ++u)   // as many loads in flight
                    if (k0 - 32 * u >= 0) best = max(best, a.pos[(long long)cur.b * a.max_seq + k0 - 32 * u]);
                ref = __reduce_max_sync(0xffffffffu, best);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                // B fragments: column g, elements 64 s + 16 t4 + 4 u + (0, 1 | 2, 3)
                uint4 raw[HS][2];
                uint32_t amax = 0;
#pragma unroll
                for (int s = 0; s < HS; ++s) {
                    raw[s][0] = raw[s][1] = make_uint4(0u, 0u, 0u, 0u);
                    const int col = ONE ? 0 : nt * 8 + g;   // ONE: the query in every column
                    if (col < ncol) {
                        const uint4 *q = reinterpret_cast<const uint4 *>(
                            sides + st * side_bytes + (col * D + 64 * s + 16 * t4) * 2);
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
                // 2^up brings the largest element to [2^14, 2^15); at most 2^120, so that
                // scale / 2^up is a normal number
                const int up = amax >= 0x7f80u ? 0 : min(120, 14 + 127 - (int)(amax >> 7));
                const float mul = __uint_as_float((uint32_t)(127 + up) << 23);
                float inv = __uint_as_float((uint32_t)(127 - up) << 23) * (a.scale * kLog2e);
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
                for (int e = 0; e < NE; ++e) {   // accumulator columns 2 t4 + e
                    const int c = ONE ? 0 : nt * 8 + 2 * t4 + e, cc = chunk * W + c;
                    qs[nt][e] = __shfl_sync(0xffffffffu, inv, (2 * t4 + e) * 4);
                    slope[nt][e] = a.slopes && c < ncol ? __int_as_float(pos[SL + 32 + c]) * kLog2e : 0.f;
                    lim[nt][e] = c < ncol ? cur.len - a.T + 1 + (ONE ? 0 : cc / group) : 0;
                    m[nt][e] = M[nt][e] = -INFINITY;
                    l[nt][e] = 0.f;
                }
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[i][nt][e] = 0.f;
            }
        }
        const int base = cur.blk * SL;
        // ---- scores: 16 slots x columns per mt
        float s[MT][NT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[mt][nt][e] = 0.f;
#pragma unroll
            for (int i = 0; i < HS; ++i) {
                const uint4 ka = *reinterpret_cast<const uint4 *>(stage + mt * 16 * D + koff[i]);
                const uint4 kb = *reinterpret_cast<const uint4 *>(stage + (mt * 16 + 8) * D + koff[i]);
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    uint32_t a0, a1, a2, a3;
                    ak8_widen<E4M3>(ak8_bias<E4M3>((&ka.x)[u]), a0, a2);
                    ak8_widen<E4M3>(ak8_bias<E4M3>((&kb.x)[u]), a1, a3);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        ak8_mma(s[mt][nt], a0, a1, a2, a3, qf[nt][4 * i + u][0], qf[nt][4 * i + u][1]);
                }
            }
        }
        // V scale = mant * 2^ev
        float kscale[NB], ev[NB], mant[NB];
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            kscale[i] = __int_as_float(pos[SL + 48 + 2 * i]);
            const uint32_t vbits = (uint32_t)pos[SL + 49 + 2 * i], vexp = (vbits >> 23) & 255u;
            const float vscale = __uint_as_float(vbits);
            ev[i] = vexp == 255u ? 0.f : vexp == 0u ? -126.f : (float)((int)vexp - 127);
            mant[i] = vexp == 255u ? vscale : vexp == 0u ? vscale * 0x1p126f : __uint_as_float((vbits & 0x807fffffu) | 0x3f800000u);
            if (ONE) mant[i] *= band_up;
        }
        int pk[2 * MT], least = 0;
        float dp[2 * MT];
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i) {
            pk[i] = pos[8 * i + slot_g];
            least = min(least, pk[i]);
            dp[i] = (float)(pk[i] - ref);
        }
        // does every column see every slot of the block?
        const bool clean = __all_sync(0xffffffffu, base + SL <= all && least >= 0);
        // ---- softmax, then values: D elements x columns, 16 slots per mt
        auto rest = [&](auto is_clean) {
            constexpr bool CLEAN = decltype(is_clean)::value;
            uint32_t pb[MT][NT][2], pl[MT][ONE ? 1 : NT][2];   // the weights' first and second parts (ONE: both in pb)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float wt[MT][4], bm[NE], bM[NE];   // the block's maxima: of scores, and with the V scale
                bool move = false;
#pragma unroll
                for (int e = 0; e < NE; ++e) {
                    bm[e] = bM[e] = -INFINITY;
#pragma unroll
                    for (int j = 0; j < NB; ++j) {
                        const float f = kscale[j] * qs[nt][e];
                        float top = -INFINITY;
#pragma unroll
                        for (int i = 4 * j; i < 4 * j + 4; ++i) {   // slot 8 i + slot_g
                            float &v = s[i >> 1][nt][2 * (i & 1) + e];
                            v = v * f + slope[nt][e] * dp[i];
                            if (!CLEAN && (pk[i] < 0 || base + 8 * i + slot_g >= lim[nt][e])) v = -INFINITY;
                            top = fmaxf(top, v);
                        }
                        bm[e] = fmaxf(bm[e], top);
                        bM[e] = fmaxf(bM[e], top + ev[j]);
                    }
                    move |= bm[e] > m[nt][e] + kSlack || bM[e] > M[nt][e] + kSlack;
                }
                if (__any_sync(0xffffffffu, move)) {
#pragma unroll
                    for (int e = 0; e < NE; ++e) {
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) {
                            bm[e] = fmaxf(bm[e], __shfl_xor_sync(0xffffffffu, bm[e], o));
                            bM[e] = fmaxf(bM[e], __shfl_xor_sync(0xffffffffu, bM[e], o));
                        }
                        const float mn = fmaxf(m[nt][e], bm[e]), Mn = fmaxf(M[nt][e], bM[e]);
                        l[nt][e] *= ak8_exp2(m[nt][e] - ak8_finite(mn));
                        const float r = ak8_exp2(M[nt][e] - ak8_finite(Mn));
#pragma unroll
                        for (int i = 0; i < D / 16; ++i) {
                            acc[i][nt][e] *= r;
                            acc[i][nt][2 + e] *= r;
                            if (ONE) {
                                acc[i][nt][1] *= r;
                                acc[i][nt][3] *= r;
                            }
                        }
                        m[nt][e] = mn;
                        M[nt][e] = Mn;
                    }
                }
#pragma unroll
                for (int e = 0; e < NE; ++e) {
                    const float mf = ak8_finite(m[nt][e]), Mf = ak8_finite(M[nt][e]) - (ONE ? 0.f : kAk8Lift);
#pragma unroll
                    for (int i = 0; i < 2 * MT; ++i) {
                        const float v = s[i >> 1][nt][2 * (i & 1) + e];
                        l[nt][e] += ak8_exp2(v - mf);
                        const float x = v - (Mf - ev[i / 4]), p = ak8_exp2(x) * mant[i / 4];
                        const bool none = ONE ? x < band_lo || x >= band_hi : false;
                        wt[i >> 1][2 * (i & 1) + e] = none || (!CLEAN && v == -INFINITY) ? 0.f : p;
                    }
                }
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)   // [slot][column] -> [column][slot] fragments
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float w0 = wt[mt][2 * i], w1 = ONE ? 0.f : wt[mt][2 * i + 1];
                        if (ONE) {   // columns 2 t4 and 2 t4 + 1: the first eleven bits, the rest
                            const float h = __uint_as_float(__float_as_uint(w0) & 0xffffe000u);
                            pb[mt][nt][i] = ak8_transpose(ak8_pack_f16(h, (w0 - h) * 2048.f));
                        } else {     // the first eight bits, the rest
                            const uint32_t u0 = __float_as_uint(w0), u1 = __float_as_uint(w1);
                            pb[mt][nt][i] = ak8_transpose(__byte_perm(u0, u1, 0x7632));
                            pl[mt][nt][i] = ak8_transpose(kv8_bf16x2(w0 - __uint_as_float(u0 & 0xffff0000u), w1 - __uint_as_float(u1 & 0xffff0000u)));
                        }
                    }
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                uint32_t v[4][VW];   // slots of rows 2 t4, 2 t4 + 1, and 8 further
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const unsigned char *p = stage + (SL + mt * 16 + 8 * (i >> 1)) * D + voff[i & 1];
                    if (D == 128) {
                        const uint4 r = *reinterpret_cast<const uint4 *>(p);
                        v[i][0] = r.x; v[i][1] = r.y; v[i][VW - 2] = r.z; v[i][VW - 1] = r.w;
                    } else {
                        const uint2 r = *reinterpret_cast<const uint2 *>(p);
                        v[i][0] = r.x; v[i][1] = r.y;
                    }
                    // slots that take no part may hold e4m3 NaNs: their codes count as 0
                    if (E4M3 && !CLEAN && pos[mt * 16 + 8 * (i >> 1) + (i & 1 ? vb : va)] < 0) {
#pragma unroll
                        for (int u = 0; u < VW; ++u) v[i][u] = 0;
                    }
                    if (ONE) {
#pragma unroll
                        for (int u = 0; u < VW; ++u) v[i][u] = ak8_bias<E4M3>(v[i][u]);
                    }
                }
#pragma unroll
                for (int u = 0; u < VW; ++u) {
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {   // elements 4 u + 2 hh, + 1 of two slots, side by side
                        const uint32_t sel = hh ? 0x7362u : 0x5140u;
                        uint32_t a0, a1, a2, a3;
                        const uint32_t va2 = __byte_perm(v[0][u], v[1][u], sel), vb2 = __byte_perm(v[2][u], v[3][u], sel);
                        if (ONE) {
                            ak8_widen<E4M3>(va2, a0, a1);
                            ak8_widen<E4M3>(vb2, a2, a3);
                            ak8_mma(acc[2 * u + hh][0], a0, a1, a2, a3, pb[mt][0][0], pb[mt][0][1]);
                        } else {
                            ak8_widen_bf16<E4M3>(va2, a0, a1);
                            ak8_widen_bf16<E4M3>(vb2, a2, a3);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                ak8_mma_bf16(acc[2 * u + hh][nt], a0, a1, a2, a3, pb[mt][nt][0], pb[mt][nt][1]);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                ak8_mma_bf16(acc[2 * u + hh][nt], a0, a1, a2, a3, pl[mt][nt][0], pl[mt][nt][1]);
                        }
                    }
                }
            }
        };
        if (clean) rest(std::true_type{});
        else rest(std::false_type{});
        __syncwarp();   // the stage has been read
        issue(st);
        if (++st == ST) {
            st = 0;
            parity ^= 1u;
        }
        const bool ends = cur.blk + 1 == cur.blocks;
        if (!ends && x + 1 < x1) {
            ++cur.blk;
            continue;
        }

        // ---- the end of a (row, head), or of the run
        fresh = true;
        const bool whole = ends && x - cur.blk >= seg0;
        if (ONE) {   // the parts of all column pairs together
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                    float v = (acc[i][0][e] + acc[i][0][e + 1] * 0x1p-11f) * band_down;
                    v += __shfl_xor_sync(0xffffffffu, v, 1);
                    v += __shfl_xor_sync(0xffffffffu, v, 2);
                    acc[i][0][e] = v;
                }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < NE; ++e) {
                float sum = l[nt][e];
                sum += __shfl_xor_sync(0xffffffffu, sum, 4);
                sum += __shfl_xor_sync(0xffffffffu, sum, 8);
                sum += __shfl_xor_sync(0xffffffffu, sum, 16);
                const int c = nt * 8 + 2 * t4 + e;
                if (c >= ncol) continue;
                if (whole) {
                    const int cc = chunk * W + c;
                    const Ak8Last last(m[nt][e], M[nt][e], sum);
                    uint4 *o = reinterpret_cast<uint4 *>(
                        a.o + (((long long)cur.b * a.T + cc / group) * a.n + h * group + cc % group) * D + g * (D / 8));
#pragma unroll
                    for (int i = 0; i < HS; ++i) {
                        uint32_t r[4];
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            r[u] = pack_bf2(last.of(acc[4 * i + u][nt][e]), last.of(acc[4 * i + u][nt][2 + e]));
                        o[i] = make_uint4(r[0], r[1], r[2], r[3]);
                    }
                } else {   // slot 0 of this run: its first (row, head); 1: its last
                    float *p = a.part + ((long long)(2 * run + (seg0 == x0 ? 0 : 1)) * cols + c) * (D + kAk8Part);
                    if (g == 0) *reinterpret_cast<float4 *>(p + D) = make_float4(m[nt][e], M[nt][e], sum, 0.f);
#pragma unroll
                    for (int i = 0; i < D / 32; ++i)
                        reinterpret_cast<float4 *>(p + g * (D / 8))[i] =
                            make_float4(acc[2 * i][nt][e], acc[2 * i][nt][2 + e], acc[2 * i + 1][nt][e], acc[2 * i + 1][nt][2 + e]);
                }
            }
        cur.next(rows);
    }
    cp_async_wait_all();
}

// Running joint of partial results (references m and M, sum l, accumulator o).
template <int E>
struct Ak8Joint {
    float m = -INFINITY, M = -INFINITY, l = 0.f, o[E] = {};
    // U partials at once: st (m, M, l, -) and v
    template <int U>
    __device__ __forceinline__ void add(const float4 (&st)[U], const float (&v)[U][E]) {
        float mn = m, Mn = M;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            mn = fmaxf(mn, st[u].x);
            Mn = fmaxf(Mn, st[u].y);
        }
        const float mf = ak8_finite(mn), Mf = ak8_finite(Mn), f = ak8_exp2(M - Mf);
        l *= ak8_exp2(m - mf);
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] *= f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            l += st[u].z * ak8_exp2(st[u].x - mf);
            const float k = ak8_exp2(st[u].y - Mf);
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] += v[u][e] * k;
        }
        m = mn;
        M = Mn;
    }
};

// Joins the partial results of one column of one (row, head), in the order of the
// runs.  Item i is the (row, head) i where those are fewer than the runs; else the
// one that run i began and did not end.  NW > 1: one CTA an item and column, its NW
// warps take the partials in turn; NW = 1: one warp does it all, four to a CTA.  Lanes
// hold D / 32 elements, neighbours side by side.
template <int D, int NT, int NW>
__global__ void __launch_bounds__(NW == 1 ? 128 : 32 * NW) attn_kv8_join_kernel(const AttnKv8Args a, int warps, int by_head, int items) {
    constexpr int W = 8 * NT, E = D / 32, U = NW == 1 ? 8 : 4;
    griddep_launch();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int id = NW > 1 ? (int)blockIdx.x : (int)blockIdx.x * 4 + w;
    const int item = id / a.part_cols, col = id - item * a.part_cols;
    const int group = a.n / a.kv, C = group * a.T, chunks = (C + W - 1) / W;
    const Ak8Rows<D> rows{a.lens, a.B, a.max_seq, a.kv * chunks};
    int b = by_head ? min(item, items - 1) / rows.heads : 0, head = 0, before = 0, total = 0;
    for (int i = lane; i < a.B; i += 32) {
        const int n = rows.blocks(i);
        total += n;
        if (i < b) before += n;
    }
    const Ak8Runs<D> runs(__reduce_add_sync(0xffffffffu, total) * rows.heads, warps);
    int first = 0, end = 0, blocks = 0;   // its blocks
    if (by_head) {
        head = item - b * rows.heads;
        blocks = item < items ? rows.blocks(b) : 0;
        first = __reduce_add_sync(0xffffffffu, before) * rows.heads + head * blocks;
        end = first + blocks;
    } else if (item + 1 < runs.R) {
        Ak8Cursor c = {};
        const int x1 = runs.start(item + 1);
        c.at(rows, x1);
        b = c.b;
        head = c.head;
        first = x1 - c.blk;
        end = first + c.blocks;
        // begun by this run, and not just before the cut
        blocks = c.blk != 0 && runs.start(item) <= first ? c.blocks : 0;
    }
    const int r0 = blocks ? runs.of(first) : 0, r1 = blocks ? runs.of(end - 1) : 0;   // the runs it lies in
    const int slot0 = runs.start(r0) != first;             // run r0 began with an earlier (row, head)
    const int h = head / chunks, chunk = head - h * chunks, ncol = min(W, C - chunk * W);
    griddep_wait();                                        // the partials (lengths were final before)
    if (blocks <= Ak8Runs<D>::kWhole || r0 == r1 || col >= ncol) return;   // whole

    Ak8Joint<E> sum;
    for (int rr = r0 + (NW > 1 ? w : 0); rr <= r1; rr += NW * U) {   // U partials in flight
        float4 st[U];
        float v[U][E];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = rr + NW * u;
            st[u] = make_float4(-INFINITY, -INFINITY, 0.f, 0.f);
#pragma unroll
            for (int e = 0; e < E; ++e) v[u][e] = 0.f;
            if (r <= r1) {
                const float *p = a.part + ((long long)(2 * r + (r == r0 ? slot0 : 0)) * a.part_cols + col) * (D + kAk8Part);
                st[u] = *reinterpret_cast<const float4 *>(p + D);
#pragma unroll
                for (int e = 0; e < E; ++e) v[u][e] = p[32 * e + lane];
            }
        }
        sum.add(st, v);
    }
    if (NW > 1) {
        __shared__ float sm_o[NW][D];
        __shared__ float4 sm_st[NW];
#pragma unroll
        for (int e = 0; e < E; ++e) sm_o[w][32 * e + lane] = sum.o[e];
        if (lane == 0) sm_st[w] = make_float4(sum.m, sum.M, sum.l, 0.f);
        __syncthreads();
        if (w != 0) return;
        sum = Ak8Joint<E>();
        for (int i = 0; i < NW; i += 4) {
            float4 st[4];
            float v[4][E];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                st[u] = sm_st[i + u];
#pragma unroll
                for (int e = 0; e < E; ++e) v[u][e] = sm_o[i + u][32 * e + lane];
            }
            sum.add(st, v);
        }
    }
    const int cc = chunk * W + col;
    const Ak8Last last(sum.m, sum.M, sum.l);
    uint16_t *o = a.o + (((long long)b * a.T + cc / group) * a.n + h * group + cc % group) * D;
#pragma unroll
    for (int e = 0; e < E; ++e) o[32 * e + lane] = f2bf(last.of(sum.o[e]));
}

// CTAs per SM of a variant with its shared memory, found once per device.
template <int D, bool E4M3, int NT, bool ONE>
static cudaError_t ak8_launch(AttnKv8Args a, int sms, cudaStream_t s) {
    constexpr int kDevices = 64, W = 8 * NT;
    static std::atomic<int> known[kDevices][W + 1];
    const auto kern = attn_kv8_kernel<D, E4M3, NT, ONE>;
    const int group = a.n / a.kv, C = group * a.T, chunks = (C + W - 1) / W;
    a.part_cols = C < W ? C : W;
    const int smem = Ak8Smem<D, ONE>::bytes(a.part_cols);
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    int per_sm = dev < kDevices ? known[dev][a.part_cols].load(std::memory_order_relaxed) : 0;
    if (per_sm == 0) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Ak8Smem<D, ONE>::bytes(W));
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, kAk8Threads, smem);
        if (e != cudaSuccess) return e;
        per_sm = per_sm < 1 ? 1 : per_sm > kAk8MaxPerSm ? kAk8MaxPerSm : per_sm;
        if (dev < kDevices) known[dev][a.part_cols].store(per_sm, std::memory_order_relaxed);
    }
    Ak8Maps maps;
    const long long slots = (long long)a.B * a.kv * a.max_seq;
    if (!make_map_rows_u8(&maps.k, a.kc, slots, D, ak8_slots(D)) || !make_map_rows_u8(&maps.v, a.vc, slots, D, ak8_slots(D)))
        return cudaErrorInvalidValue;
    const int heads = a.B * a.kv * chunks;
    const long long most = (long long)heads * ((a.max_seq + ak8_slots(D) - 1) / ak8_slots(D));
    const long long runs = (most + Ak8Runs<D>::kMin - 1) / Ak8Runs<D>::kMin;
    const int G = (int)(runs < (long long)sms * per_sm ? runs : (long long)sms * per_sm), warps = G * kAk8Warps;
    e = launch_pdl_smem(kern, dim3(G), dim3(kAk8Threads), smem, s, a, maps);
    if (e != cudaSuccess || a.max_seq <= kAk8Whole) return e;   // nothing can have been cut
    const int by_head = heads < warps, items = by_head ? heads : warps;
    const int todo = items * a.part_cols;
    // many partials an item: four warps share them (from 16 on: two rounds of one warp's
    // loads), or sixteen (one key head of 131000 slots, 1216 partials: 57 us with four, 35 with
    // sixteen; four keep room beside the main kernel's CTAs)
    if (warps > 64 * items)
        return launch_pdl(attn_kv8_join_kernel<D, NT, 16>, dim3(todo), dim3(512), s, a, warps, by_head, items);
    if (warps > 16 * items)
        return launch_pdl(attn_kv8_join_kernel<D, NT, 4>, dim3(todo), dim3(128), s, a, warps, by_head, items);
    return launch_pdl(attn_kv8_join_kernel<D, NT, 1>, dim3((todo + 3) / 4), dim3(128), s, a, warps, by_head, items);
}

bool attn_kv8_fits(int B, int n, int kv, int T, int max_seq) {
    const long long C = (long long)n / kv * T, chunks = C <= 8 ? 1 : (C + 15) / 16;
    return (long long)B * kv * max_seq < (1ll << 31) &&
           (long long)B * kv * chunks * ((max_seq + kKv8Block - 1) / kKv8Block) < (1ll << 31);
}

size_t attn_kv8_workspace(int n, int kv, int T, int max_seq, int d, int sms) {
    const int C = n / kv * T, W = C <= 8 ? 8 : 16;
    if (max_seq <= kAk8Whole) return 0;
    return (size_t)sms * kAk8MaxPerSm * kAk8Warps * 2 * (C < W ? C : W) * (d + kAk8Part) * 4;
}

template <int D, bool E4M3>
static cudaError_t ak8_launch_cols(const AttnKv8Args &a, int sms, cudaStream_t s) {
    // more than 8 columns: two column tiles a pass, or the codes would be read and widened twice
    const int C = a.n / a.kv * a.T;
    if (C == 1) return ak8_launch<D, E4M3, 1, true>(a, sms, s);
    return C <= 8 ? ak8_launch<D, E4M3, 1, false>(a, sms, s) : ak8_launch<D, E4M3, 2, false>(a, sms, s);
}

cudaError_t launch_attn_kv8(const AttnKv8Args &a, int d, int e4m3, int sms, cudaStream_t s) {
    if (d == 64) return e4m3 ? ak8_launch_cols<64, true>(a, sms, s) : ak8_launch_cols<64, false>(a, sms, s);
    return e4m3 ? ak8_launch_cols<128, true>(a, sms, s) : ak8_launch_cols<128, false>(a, sms, s);
}

}  // namespace bloom
