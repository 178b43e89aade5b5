// Sampling with temperature, top-k, top-p and min-p, each row with settings of its
// own, from given uniform numbers.  For a row of logits z at temperature t:
//   p_i proportional to exp((z_i - max z) / t);
//   the tokens ordered by probability, highest first (equal logits: lower index first);
//   the kept ones are a prefix of that order: the first top_k, of those the shortest
//   prefix with top_p of their mass, of those the ones with p >= min_p * max p;
//   a draw u takes the token where the kept mass, summed in vocabulary order, first
//   exceeds u times the whole of it.
//
// All three filters keep a prefix, so what is looked for is one cut: a logit (as
// an order-preserving key) and how many of the tokens that have it are kept, the first by index.
// Masses are 2^-40 fixed point of a float32 exponential and summed in 64-bit integers:
// sums do not depend on their order, and the same logits give the same tokens.  The
// exponent (max z - z) log2(e) / t is carried in two floats, or the rounding of 1 / t would
// shift all far tokens the same way.
//
// Normal logits of deviation 2.5 at temperature 0.8.  A few rows are read once from HBM and then from L2,
// bound by the latency of their phases (1 x 250880: greedy 7.6 us, top-k 50 10.4, min-p 0.05 or no filter
// 11.9, top-p 0.95 30).  Of many rows more are under way than L2 holds, and every pass reads HBM (509 x
// 250880, 76 us to read once): greedy 183 and top-k 50 185 us, two readings at 70 % of the DRAM's peak;
// min-p 226, no filter 249, two; top-p 452, three, and bound by instructions too, some 70 a logit at 60 %
// of the issue slots.  One cluster of up to 16 CTAs a row, each a slice of the vocabulary:
//  1. the maximum and minimum, and every thread's own maximum;
//  2. where few tokens can be kept, these come to the first CTA, which ranks them and does the
//     rest: of the top 192, those that reach a bound from the maxima of groups of threads; the
//     maximum's ties;
//  3. else (top-p, or a larger k) a histogram of counts over the exponent, in 2048 bins, and
//     the whole mass.  A bin's tokens have masses within its edges', so the counts alone
//     bound where the cut's mass is reached to a band of bins.  (A histogram of masses needs
//     64-bit atomics for every token.)  If all down to the band are few: 2.
//  4. the exact mass above the band, by segments of the slices, and the band's tokens to
//     the first CTA, which finds the cut among them by radix over their keys.  A band of more
//     tokens than fit there is divided by another histogram, of masses over its range of
//     keys, until it fits or is a single logit.
//  5. the kept mass by segments; the segment of a draw is walked to the token.
#include <atomic>
#include <math.h>
#include <stdint.h>

#include "common.cuh"
#include "kernels.h"

namespace bloom {

typedef unsigned long long sf_u64;

constexpr int kSfMaxCluster = 16;
constexpr int kSfBins = 2048;
constexpr int kSfList = 4096;                  // tokens that a CTA lists
constexpr int kSfRank = 512;                   // that the first CTA ranks
constexpr int kSfBound = 192;                  // a top-k up to which maxima of groups of threads give a bound
constexpr int kSfMarks = 8;                    // of a rank's maxima: every ceil(k / 8)-th
constexpr int kSfDigits = 1024;
constexpr int kSfBatch = 8;                    // logits of a lane at a time
constexpr int kSfSegments = 64;                // of a slice; before them its ragged head, after them its tail
constexpr float kSfUnit = 1099511627776.f;     // 2^40
constexpr float kSfFar = 40.f;                 // binades below the maximum from which on a mass is 0
// Bounds of a bin's masses allow for the rounding of exponents (40 * 2^-23) and exponentials.  (The
// bins by keys have exact masses: with bounds a band of two logits next to a border never shrank.)
constexpr float kSfSlack = 1.f / 65536.f;

// Slots of the values that the ranks tell one another.  A slot is written again only after a
// barrier that follows its reading.
enum { kSfRange, kSfCount, kSfBandMass, kSfAbove, kSfFound, kSfLeft, kSfWhole, kSfBand, kSfHeld, kSfMass, kSfTies, kSfSlots };

template <int THREADS>
struct alignas(16) SfSmem {
    static constexpr int kWarps = THREADS / 32;
    sf_u64 list[kSfList];                      // key << 32 | ~index; first CTA: of all ranks
    union {
        uint32_t hist[kSfBins];                // this CTA's counts
        sf_u64 digit[kSfDigits];               // first CTA, looking through the list
    };
    uint32_t counts[kSfBins];                  // the cluster's
    sf_u64 seg_mass[kSfSegments + 2];
    uint32_t seg_ties[kSfSegments + 2];
    alignas(16) uint32_t own_max[THREADS / 2];
    alignas(16) uint32_t marks[kSfMaxCluster * kSfMarks];
    sf_u64 scan[2][kWarps];
    uint32_t scan_n[kWarps];
    sf_u64 part[kWarps][3];
    sf_u64 xch[kSfSlots][kSfMaxCluster];       // a value of every rank
    sf_u64 found[4];
    double real;
    float unit[2], least;
    int bin[4];
    uint32_t nlist;
};

// ---- cluster
__device__ __forceinline__ void sf_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void sf_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void sf_sync() {
    sf_arrive();
    sf_wait();
}
__device__ __forceinline__ uint32_t sf_at(const void *p, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    return r;
}
__device__ __forceinline__ void sf_put(void *p, uint32_t rank, sf_u64 v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(sf_at(p, rank)), "l"(v) : "memory");
}
__device__ __forceinline__ sf_u64 sf_get(const void *p, uint32_t rank) {
    sf_u64 v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(sf_at(p, rank)) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t sf_get32(const void *p, uint32_t rank) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(sf_at(p, rank)) : "memory");
    return v;
}

// ---- a row's exponents and masses
__device__ __forceinline__ uint32_t sf_key(float z) { return ordered_key(z + 0.f); }   // -0 as +0
__device__ __forceinline__ float sf_unkey(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

struct SfRow {
    float top;         // the maximum
    float c, c_low;    // log2(e) / t, in two floats
    // The maximum is finite (rows with infinite ones have a way of their own).  Of -inf and NaN logits, and of
    // those whose difference to it is no float, the exponent is infinite or NaN, and the mass 0.
    __device__ __forceinline__ float exponent(float z) const { return (top - z) * c; }
    // The mass as n * f, f 512 or 1: from 2^-9 on in steps of 2^-31, which a float has there, below in
    // steps of 2^-40.  Adding n * f is one instruction.
    __device__ __forceinline__ uint32_t mass(float z, float &x, uint32_t &f) const {
        const float d = top - z;
        x = d * c;
        const float low = fmaf(d, c_low, fmaf(d, c, -x));   // what the product and c lost
        float y;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(-x));
        y = fmaf(y * -0.6931471805599453f, low, y);
        const bool near = y >= 0x1p-9f;
        f = near ? 512u : 1u;
        return __float2uint_rz(y * (near ? 0x1p31f : kSfUnit));   // 0 from kSfFar on
    }
    __device__ __forceinline__ sf_u64 mass(float z) const {
        float x;
        uint32_t f;
        const uint32_t n = mass(z, x, f);
        return (sf_u64)n * f;
    }
    __device__ __forceinline__ void add(sf_u64 &sum, float z) const {
        float x;
        uint32_t f;
        const uint32_t n = mass(z, x, f);
        sum += (sf_u64)n * f;
    }
};

// How the tokens are dealt to bins: by exponent (rounded to the nearest of per_binade a
// binade), or by key from `high` down.
struct SfBins {
    bool keys;
    float per_binade;
    uint32_t high, low;
    int shift;
    __device__ __forceinline__ int near(float x) const {   // x < kSfFar
        return __float_as_int(fmaf(x, per_binade, 8388608.f)) & (kSfBins - 1);
    }
    // the bin of a logit that takes part; -1: above all bins, kSfBins: below them
    __device__ __forceinline__ int of(const SfRow &row, float z) const {
        if (keys) {
            const uint32_t k = sf_key(z);
            return k > high ? -1 : k < low ? kSfBins : (int)((high - k) >> shift);
        }
        const float x = row.exponent(z);
        return x < kSfFar ? near(x) : kSfBins;
    }
    // bounds of the masses in bin i, by exponent
    __device__ __forceinline__ sf_u64 most(int i) const {
        const sf_u64 m = (sf_u64)((per_binade > 0.f ? exp2f(-fmaxf((float)i - 0.5f, 0.f) / per_binade) : 1.f) * kSfUnit);
        return m + (sf_u64)((float)m * kSfSlack) + 2ull;
    }
    __device__ __forceinline__ float middle(int i) const {
        return (per_binade > 0.f ? exp2f(-(float)i / per_binade) : 1.f) * kSfUnit;
    }
    __device__ __forceinline__ sf_u64 least(int i) const {
        const sf_u64 m = (sf_u64)((per_binade > 0.f ? exp2f(-((float)i + 0.5f) / per_binade) : 1.f) * kSfUnit);
        const sf_u64 less = (sf_u64)((float)m * kSfSlack) + 2ull;
        return m > less ? m - less : 0ull;
    }
};

// part * whole, 0 <= part < 1, rounded down or (up) up.  In integers: an SM has next to no 64-bit floating-point units.
__device__ __forceinline__ sf_u64 sf_part(float part, sf_u64 whole, bool up) {
    const uint32_t bits = __float_as_uint(part) & 0x7fffffffu, e = bits >> 23, m = (bits & 0x7fffffu) | (e ? 0x800000u : 0u);
    const int shift = 150 - (int)(e ? e : 1u);   // part = m * 2^-shift, shift >= 24
    const sf_u64 low = whole * m, high = __umul64hi(whole, m);
    const sf_u64 n = shift < 64 ? low >> shift | high << (64 - shift) : shift < 128 ? high >> (shift - 64) : 0ull;
    const bool more = shift < 64 ? (low & ((1ull << shift) - 1ull)) != 0ull : true;   // of 64 and more digits some are not 0
    return n + (up && more ? 1ull : 0ull);
}

__device__ __forceinline__ sf_u64 sf_warp_sum(sf_u64 v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ sf_u64 sf_warp_scan(sf_u64 v) {   // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const sf_u64 y = __shfl_up_sync(0xffffffffu, v, o);
        if ((int)(threadIdx.x & 31) >= o) v += y;
    }
    return v;
}
// Exclusive scan over the block in thread order; `total` of all.
template <int THREADS>
__device__ __forceinline__ sf_u64 sf_block_scan(SfSmem<THREADS> &sm, sf_u64 v, sf_u64 &total) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const sf_u64 in = sf_warp_scan(v);
    __syncthreads();
    if (lane == 31) sm.scan[0][w] = in;
    __syncthreads();
    sf_u64 before = 0ull;
    total = 0ull;
#pragma unroll
    for (int i = 0; i < SfSmem<THREADS>::kWarps; ++i) {
        if (i < w) before += sm.scan[0][i];
        total += sm.scan[0][i];
    }
    return before + in - v;
}

// A cut: kept are keys above `key`, and the first `ties` tokens by index that have it.
struct SfCut {
    uint32_t key, ties;
    __device__ __forceinline__ void tighten(uint32_t k, uint32_t n) {
        if (k > key) {
            key = k;
            ties = n;
        } else if (k == key && n < ties) {
            ties = n;
        }
    }
};

// In the first CTA's list (n tokens, keys from `least` to `most`): the key at which the weights of the
// highest keys, one a token or its mass, reach `target`, and what of the target is left for its ties.
template <int THREADS>
__device__ __forceinline__ uint32_t sf_select(SfSmem<THREADS> &sm, const SfRow &row, int n, uint32_t most, uint32_t least,
                                              bool by_mass, sf_u64 &target) {
    constexpr int kBits = 10, PT = kSfDigits / THREADS;
    const int tid = threadIdx.x;
    uint32_t found = 0;   // of most - key, the bits above `shift`
    for (int shift = max(0, 32 - __clz((int)(most - least)) - kBits);; shift = max(0, shift - kBits)) {
        __syncthreads();
        for (int i = tid; i < kSfDigits; i += THREADS) sm.digit[i] = 0ull;
        __syncthreads();
        for (int i = tid; i < n; i += THREADS) {
            const uint32_t k = (uint32_t)(sm.list[i] >> 32), far = (most - k) >> shift;
            if (far >= found && far - found < kSfDigits) atomicAdd(&sm.digit[far - found], by_mass ? row.mass(sf_unkey(k)) : 1ull);
        }
        __syncthreads();
        sf_u64 own[PT], sum = 0ull, total;
#pragma unroll
        for (int e = 0; e < PT; ++e) sum += own[e] = sm.digit[tid * PT + e];
        sf_u64 run = sf_block_scan(sm, sum, total);
#pragma unroll
        for (int e = 0; e < PT; ++e) {
            if (run < target && run + own[e] >= target) {
                sm.found[0] = (sf_u64)(tid * PT + e);
                sm.found[1] = target - run;
            }
            run += own[e];
        }
        __syncthreads();
        found += (uint32_t)sm.found[0];
        target = sm.found[1];
        if (shift == 0) return most - found;
        found <<= min(shift, kBits);
    }
}

// The first CTA's end of a row whose kept tokens are all listed (n of them, at most kSfRank): ranks
// them, cuts, and draws.  k: top-k or 0; part: of the listed tokens' mass after top-k that is kept, or
// target: the mass itself; floor: least key kept.
template <int THREADS>
__device__ __forceinline__ void sf_finish(SfSmem<THREADS> &sm, const SfRow &row, const SampleFilteredArgs &a, int b, int n, int k,
                                          float part, sf_u64 target, uint32_t floor, float first_u) {
    constexpr int PT = kSfRank / THREADS;
    const int tid = threadIdx.x;
    sf_u64 *sorted = sm.list + kSfRank, *mass = sorted + kSfRank;   // highest first
    if (tid == 0 && (n & 1)) sm.list[n] = 0ull;
    __syncthreads();
    const int parts = 4 * n <= THREADS ? 4 : 1;   // threads a token
    for (int i0 = 0; i0 < n; i0 += THREADS) {
        const int i = i0 + tid / parts;
        const sf_u64 mine = i < n ? sm.list[i] : 0ull;
        int above = 0;
        if (i < n)
#pragma unroll 4
            for (int j = 2 * (tid % parts); j < n; j += 2 * parts) {
                const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(&sm.list[j]);
                above += (v.x > mine) + (v.y > mine);
            }
        for (int o = 1; o < parts; o *= 2) above += __shfl_xor_sync(0xffffffffu, above, o);
        if (i < n && tid % parts == 0) {
            sorted[above] = mine;
            mass[above] = row.mass(sf_unkey((uint32_t)(mine >> 32)));
        }
    }
    __syncthreads();
    const int upto = k > 0 ? min(n, k) : n;
    sf_u64 own[PT], sum = 0ull, total;
#pragma unroll
    for (int e = 0; e < PT; ++e) {
        const int i = tid * PT + e;
        sum += own[e] = i < upto ? mass[i] : 0ull;
    }
    sf_u64 run = sf_block_scan(sm, sum, total);
    if (part < 1.f) {
        target = max(sf_part(part, total, true), 1ull);
    }
    // of the tokens up to top-k: those before which the target is not reached, down to the floor
    uint32_t kept = 0;
#pragma unroll
    for (int e = 0; e < PT; ++e) {
        const int i = tid * PT + e;
        if (i < upto && run < target && (uint32_t)(sorted[i] >> 32) >= floor) ++kept;
        run += own[e];
    }
    sf_u64 m;
    sf_block_scan(sm, kept, m);
    m = m ? m : 1ull;
    sum = 0ull;
#pragma unroll
    for (int e = 0; e < PT; ++e) sum += tid * PT + e < (int)m ? own[e] : 0ull;
    sf_block_scan(sm, sum, total);
    // the kept tokens' places in vocabulary order: the mass before each
    sf_u64 from[PT], at[PT];
#pragma unroll
    for (int e = 0; e < PT; ++e) {
        const int i = tid + e * THREADS;
        from[e] = 0ull;
        at[e] = 0ull;
        if (i < (int)m) {
            const uint32_t mine = (uint32_t)sorted[i];   // ~index
            for (int j = 0; j < (int)m; ++j) from[e] += (uint32_t)sorted[j] > mine ? mass[j] : 0ull;
            at[e] = from[e] + mass[i];
        }
    }
    sf_u64 *pos = sm.digit;
    for (int j0 = 0; j0 < a.J; j0 += kSfDigits) {
        __syncthreads();
        const int nj = min(a.J - j0, kSfDigits);
        for (int j = tid; j < nj; j += THREADS) {
            const float u = j0 + j == tid ? first_u : a.u[(long long)b * a.J + j0 + j];
            pos[j] = u < 1.f ? sf_part(fmaxf(u, 0.f), total, false) : u >= 1.f ? total - 1ull : 0ull;
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < PT; ++e) {
            if (at[e] == from[e]) continue;
            for (int j = 0; j < nj; ++j)
                if (from[e] <= pos[j] && pos[j] < at[e]) a.out[(long long)b * a.J + j0 + j] = (int)~(uint32_t)sorted[tid + e * THREADS];
        }
    }
}

template <int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) sample_filtered_kernel(const SampleFilteredArgs a) {
    constexpr int WARPS = THREADS / 32;
    extern __shared__ __align__(16) unsigned char sf_raw[];
    SfSmem<THREADS> &sm = *reinterpret_cast<SfSmem<THREADS> *>(sf_raw);
    griddep_launch();
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int b = blockIdx.y, CS = (int)gridDim.x;
    uint32_t rank;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    if (tid == 0) sm.nlist = 0u;
    if (tid < kSfMaxCluster * kSfMarks) sm.marks[tid] = 0u;
    sf_arrive();   // every CTA runs, and its marks are empty: waited for before the first store to another
    griddep_wait();
    const float *z = a.logits + (long long)b * a.ld;
    // the row's settings and its first draws, on their way while the row is read
    float t = a.temperature ? a.temperature[b] : 1.f;
    int k = a.top_k ? a.top_k[b] : 0;
    const float p = a.top_p ? a.top_p[b] : 1.f, mp = a.min_p ? a.min_p[b] : 0.f;
    const float first_u = rank == 0 && tid < a.J ? a.u[(long long)b * a.J + tid] : 0.f;

    // this CTA's slice: whole float4s [at0, at0 + 4 nq) of the row's aligned body in segments of sq, and
    // beside them the row's ragged head (first CTA) and tail (last): indexes [s0, s1)
    const int head = min(a.V, (int)((0u - (uint32_t)(uintptr_t)z >> 2) & 3u));
    const int quads = (a.V - head) >> 2, per = (quads + CS - 1) / CS;
    const int q0 = min(quads, (int)rank * per), nq = min(quads, q0 + per) - q0, at0 = head + 4 * q0;
    const int s0 = rank == 0 ? 0 : at0, s1 = (int)rank == CS - 1 ? a.V : at0 + 4 * nq;
    const int sq = max(32, (nq + 32 * kSfSegments - 1) / (32 * kSfSegments) * 32);
    const float4 *body = reinterpret_cast<const float4 *>(z + at0);
    // Every logit of the slice: warps take segments in turn (0: the head, then kSfSegments of the body,
    // then the tail), lanes kSfBatch logits at a time (value e at index at + (e & 3) + 128 (e >> 2); -inf beyond
    // the end); done(segment) after each.  Both are called by whole warps.
    auto each = [&](auto see, auto done) {
        constexpr int Q = kSfBatch / 4;
        float4 f[Q];   // the next batch, on its way
        auto load = [&](int s, int i) {
            const int i1 = min(nq, (s + 1) * sq);
#pragma unroll
            for (int k = 0; k < Q; ++k) {
                const int at = i + lane + 32 * k;
                f[k] = at < i1 ? body[at] : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
            }
        };
        load(w, w * sq);
        for (int s = w; s < kSfSegments; s += WARPS) {
            const int i1 = min(nq, (s + 1) * sq);
            for (int i = s * sq; i < i1; i += 32 * Q) {
                float v[kSfBatch];
#pragma unroll
                for (int k = 0; k < Q; ++k) {
                    v[4 * k] = f[k].x;
                    v[4 * k + 1] = f[k].y;
                    v[4 * k + 2] = f[k].z;
                    v[4 * k + 3] = f[k].w;
                }
                if (i + 32 * Q < i1) load(s, i + 32 * Q);
                else if (s + WARPS < kSfSegments) load(s + WARPS, (s + WARPS) * sq);
                see(v, at0 + 4 * (i + lane));
            }
            done(s + 1);
        }
        if (w < 2) {
            const int i0 = (w ? at0 + 4 * nq : s0) + lane, i1 = w ? s1 : at0;
            float v[kSfBatch];
#pragma unroll
            for (int e = 0; e < kSfBatch; ++e) v[e] = -INFINITY;
            if (i0 < i1) v[0] = z[i0];
            see(v, i0);
            done(w ? kSfSegments + 1 : 0);
        }
    };
    auto index_of = [](int at, int e) { return at + (e & 3) + 128 * (e >> 2); };
    // the masses of those that reach `from`, into `sum`; nothing where none of the warp's does
    auto add_from = [&](const SfRow &row, const float (&v)[kSfBatch], float from, bool above_only, sf_u64 &sum) {
        const bool few = from > -INFINITY;   // else all
#pragma unroll
        for (int e = 0; e < kSfBatch; ++e) {
            const bool on = above_only ? v[e] > from : v[e] >= from;
            if (few && !__any_sync(0xffffffffu, on)) continue;
            float x;
            uint32_t f;
            const uint32_t n = row.mass(v[e], x, f);
            sum += (sf_u64)(on ? n : 0u) * f;
        }
    };
    auto any_from = [&](const float (&v)[kSfBatch], float from) {
        float m = v[0];
#pragma unroll
        for (int e = 1; e < kSfBatch; ++e) m = fmaxf(m, v[e]);
        return __any_sync(0xffffffffu, m >= from);
    };
    auto no_segment = [](int) {};
    // a value of every rank, in all of them after the next sf_sync()
    auto publish = [&](int slot, sf_u64 v) {
        if (tid < CS) sf_put(&sm.xch[slot][rank], (uint32_t)tid, v);
    };
    auto block_sum = [&](sf_u64 v) {   // every thread gets it
        v = sf_warp_sum(v);
        __syncthreads();
        if (lane == 0) sm.part[w][0] = v;
        __syncthreads();
        v = 0ull;
#pragma unroll
        for (int i = 0; i < WARPS; ++i) v += sm.part[i][0];
        return v;
    };
    auto block_range = [&](uint32_t &most, uint32_t &least) {
        most = __reduce_max_sync(0xffffffffu, most);
        least = __reduce_min_sync(0xffffffffu, least);
        __syncthreads();
        if (lane == 0) sm.part[w][1] = (sf_u64)most << 32 | least;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < WARPS; ++i) {
            most = max(most, (uint32_t)(sm.part[i][1] >> 32));
            least = min(least, (uint32_t)sm.part[i][1]);
        }
    };

    // ---- 1. maximum and minimum, as keys (0: nothing takes part)
    uint32_t kmax = 0u, kmin = ~0u;
    {
        float mx = -INFINITY, mn = INFINITY;
        auto see = [&](float v) {
            mx = fmaxf(mx, v);
            mn = fminf(mn, v > -INFINITY ? v : INFINITY);
        };
        for (int i = tid; i < nq; i += 6 * THREADS) {
            float4 v[6];
#pragma unroll
            for (int k = 0; k < 6; ++k)
                v[k] = i + k * THREADS < nq ? body[i + k * THREADS] : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
#pragma unroll
            for (int k = 0; k < 6; ++k) {
                see(v[k].x);
                see(v[k].y);
                see(v[k].z);
                see(v[k].w);
            }
        }
        if (tid < at0 - s0) see(z[s0 + tid]);
        else if (tid < at0 - s0 + s1 - at0 - 4 * nq) see(z[at0 + 4 * nq + tid - (at0 - s0)]);
        if (mx > -INFINITY) {
            kmax = sf_key(mx);
            kmin = sf_key(mn);
        }
    }
    const uint32_t thread_max = kmax;
    block_range(kmax, kmin);

    // ---- the row's settings
    k = max(k, 0);
    const bool nucleus = p < 1.f && p > 0.f;   // NaN: off
    if (!(t > 0.f)) {
        t = 1.f;
        k = 1;
    }
    // log2(e) / t stays finite.  (Differences times a power of two would allow for smaller t, and for logits that are
    // 2^128 apart: 437 -> 448 us for 4000 rows of 8000, top-p.)
    t = fmaxf(t, 0x1p-126f);
    if (p <= 0.f) k = 1;
    // 2. Of the maxima of groups of threads every step-th largest goes to all ranks, `step` of them
    // reaching the first mark, 2 step the second, ...: the eighth largest of all ranks' marks is
    // reached by 8 step >= k tokens.
    const bool bounded = k > 1 && k <= kSfBound;
    const int step = (k + kSfMarks - 1) / kSfMarks;
    if (bounded) {
        const int wide = k <= 64 ? 4 : 2, groups = THREADS / wide;
        uint32_t g = max(thread_max, __shfl_xor_sync(0xffffffffu, thread_max, 1));
        if (wide == 4) g = max(g, __shfl_xor_sync(0xffffffffu, g, 2));
        const int part = tid % wide;             // of the group's threads
        if (part == 0) sm.own_max[tid / wide] = g;
        __syncthreads();
        int above = 0, upto = 0;
#pragma unroll 4
        for (int i = 4 * part; i < groups; i += 4 * wide) {
            const uint4 o = *reinterpret_cast<const uint4 *>(&sm.own_max[i]);
            above += (o.x > g) + (o.y > g) + (o.z > g) + (o.w > g);
            upto += (o.x >= g) + (o.y >= g) + (o.z >= g) + (o.w >= g);
        }
        for (int o = 1; o < wide; o *= 2) {
            above += __shfl_xor_sync(0xffffffffu, above, o);
            upto += __shfl_xor_sync(0xffffffffu, upto, o);
        }
        sf_wait();
        // marks that fall on this value; equal ones write the same
        for (int i = above / step; g && i < kSfMarks && (i + 1) * step <= upto; ++i)
            for (int r = part; r < CS; r += wide)
                asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(sf_at(&sm.marks[rank * kSfMarks + i], (uint32_t)r)), "r"(g) : "memory");
    } else {
        sf_wait();
    }
    publish(kSfRange, (sf_u64)kmax << 32 | kmin);
    sf_arrive();
    const bool floored = mp > 0.f && mp < 1.f;
    if (tid == 0) {
        // log2(e) / t: the quotient, and what it leaves of the numerator
        constexpr float kLog2e = 1.4426950408889634f, kLog2eLow = (float)(1.4426950408889634 - (double)1.4426950408889634f);
        const float c = __fdiv_rn(kLog2e, t), low = __fdiv_rn(fmaf(-c, t, kLog2e) + kLog2eLow, t);
        sm.unit[0] = c;
        sm.unit[1] = fabsf(low) < c * 1e-6f ? low : 0.f;   // 0 where t is infinite
        // in 64 bits, by one thread: few of an SM's units have them
        if (floored) sm.real = (double)t * log((double)mp);
    }
    __syncwarp();
    sf_wait();
    __syncthreads();   // the settings, written after that thread's arrival
    {
        const sf_u64 one = sm.xch[kSfRange][min(lane, CS - 1)];
        kmax = __reduce_max_sync(0xffffffffu, (uint32_t)(one >> 32));
        kmin = __reduce_min_sync(0xffffffffu, (uint32_t)one);
    }
    if (kmax == 0u) {
        if (rank == 0)
            for (int j = tid; j < a.J; j += THREADS) a.out[(long long)b * a.J + j] = -1;
        return;
    }
    uint32_t bound = 0u;                         // 0: none
    if (bounded) {
        if (tid == 0) sm.found[0] = 0ull;
        __syncthreads();
        constexpr int PARTS = THREADS / (kSfMaxCluster * kSfMarks);   // threads a mark
        const uint32_t mine = sm.marks[tid / PARTS];
        int above = 0, upto = 0;
#pragma unroll 4
        for (int i = 4 * (tid % PARTS); i < CS * kSfMarks; i += 4 * PARTS) {
            const uint4 o = *reinterpret_cast<const uint4 *>(&sm.marks[i]);
            above += (o.x > mine) + (o.y > mine) + (o.z > mine) + (o.w > mine);
            upto += (o.x >= mine) + (o.y >= mine) + (o.z >= mine) + (o.w >= mine);
        }
#pragma unroll
        for (int o = 1; o < PARTS; o *= 2) {
            above += __shfl_xor_sync(0xffffffffu, above, o);
            upto += __shfl_xor_sync(0xffffffffu, upto, o);
        }
        if (mine && above < kSfMarks && kSfMarks <= upto) sm.found[0] = mine;
        __syncthreads();
        bound = (uint32_t)sm.found[0];
    }
    SfRow row;
    row.top = sf_unkey(kmax);
    row.c = sm.unit[0];
    row.c_low = sm.unit[1];
    SfCut cut = {0u, ~0u};
    if (mp > 0.f) {   // the least logit with exp((z - top) / t) >= min_p
        float least = row.top;
        if (floored && row.top < INFINITY) {
            if (tid == 0) sm.least = fminf(__double2float_ru((double)row.top + sm.real), row.top);
            __syncthreads();
            least = sm.least;
        }
        cut.tighten(sf_key(least), ~0u);
    }
    const uint32_t floor_key = cut.key;
    if (k == 1) cut.tighten(kmax, 1u);

    // Lists the tokens from key `least` on in every CTA; their number in all.
    auto collect = [&](uint32_t least) {
        const float from = sf_unkey(least);
        each([&](const float (&v)[kSfBatch], int at) {
            uint32_t in = 0;
#pragma unroll
            for (int e = 0; e < kSfBatch; ++e) in |= v[e] >= from ? 1u << e : 0u;
            if (in == 0u) return;
            uint32_t n = atomicAdd(&sm.nlist, (uint32_t)__popc(in));
#pragma unroll
            for (int e = 0; e < kSfBatch; ++e)
                if (in >> e & 1u) {
                    if (n < kSfList) sm.list[n] = (sf_u64)sf_key(v[e]) << 32 | (uint32_t)~index_of(at, e);
                    ++n;
                }
        }, no_segment);
        __syncthreads();
        publish(kSfCount, sm.nlist);
        sf_sync();
        return __reduce_add_sync(0xffffffffu, lane < CS ? (uint32_t)sm.xch[kSfCount][lane] : 0u);   // below 2^23
    };
    // The first CTA: the other ranks' lists behind its own.
    auto gather = [&]() {
        uint32_t end[kSfMaxCluster], at = min(sm.nlist, (uint32_t)kSfList);
        const uint32_t own = at;
#pragma unroll
        for (int r = 0; r < kSfMaxCluster; ++r) {
            if (r > 0 && r < CS) at += min((uint32_t)sm.xch[kSfCount][r], kSfList - at);
            end[r] = at;
        }
        for (uint32_t i = own + tid; i < at; i += THREADS) {
            int r = 0;
            uint32_t begin = 0;
#pragma unroll
            for (int q = 0; q + 1 < kSfMaxCluster; ++q)
                if (i >= end[q]) {
                    r = q + 1;
                    begin = end[q];
                }
            sm.list[i] = sf_get(&sm.list[i - begin], (uint32_t)r);
        }
        __syncthreads();
        return (int)at;
    };
    // All that can be kept is listed, `n` in all: the first CTA ends the row.
    auto finish = [&](float part, sf_u64 target) {
        if (rank == 0) {
            const int n = min(gather(), kSfRank);
            sf_finish(sm, row, a, b, n, k, part, target, max(floor_key, 1u), first_u);
        }
        sf_sync();   // the lists have been read
    };

    // An infinite maximum: its tokens share the mass, all else has none.
    const bool infinite = row.top == INFINITY;
    if (infinite) {
        sf_u64 n = 0ull;
        each([&](const float (&v)[kSfBatch], int) {
#pragma unroll
            for (int e = 0; e < kSfBatch; ++e) n += v[e] == INFINITY ? 1u : 0u;
        }, no_segment);
        publish(kSfWhole, block_sum(n));
        sf_sync();
        n = 0ull;
        for (int r = 0; r < CS; ++r) n += sm.xch[kSfWhole][r];
        if (k > 0) n = min(n, (sf_u64)k);
        if (nucleus && k != 1) n = max(1ull, min(n, sf_part(p, n, true)));
        cut.tighten(kmax, (uint32_t)n);
    }

    // ---- 2. few tokens
    if (!infinite) {
        uint32_t least = k == 1 ? kmax : bound;
        if (least == 0u && k != 1 && (k > 1 || nucleus) && a.V <= kSfRank) least = kmin;
        if (least && !nucleus) least = max(least, floor_key);   // with top-p the mass of what lies below counts
        if (least) {
            const uint32_t n = collect(least);
            if (n <= kSfRank) {
                finish(nucleus ? p : 1.f, ~0ull);
                return;
            }
            __syncthreads();
            if (tid == 0) sm.nlist = 0u;
            sf_sync();   // the counts have been read
        }
    }

    // ---- 3., 4. the cuts of top-k and top-p
    bool ready = false;   // the segments' masses are those of the cut
    if (!infinite && k != 1 && (k > 1 || nucleus)) {
        const float far = fminf(row.exponent(sf_unkey(kmin)), kSfFar);
        SfBins bins = {false, far > 0.f ? (kSfBins - 2) / far : 0.f, 0u, 0u, 0};
        if (!(bins.per_binade < 1e30f)) bins.per_binade = 0.f;   // logits that differ by next to nothing
        // the cluster's counts of `bins`; by exponent with the whole mass, by keys with the bins'
        // masses, in the place of the list
        sf_u64 *mass_own = sm.list, *mass_all = sm.list + kSfBins;
        // by exponent there: what the masses of 2^-9 and more differ from their bins' middles, in 2^-20 of
        // them.  Few tokens hold most of the mass; the many others' differences cancel.
        int *rest_own = reinterpret_cast<int *>(mass_own), *rest_all = reinterpret_cast<int *>(mass_all);
        auto count = [&](sf_u64 *whole) {
            for (int i = tid; i < kSfBins; i += THREADS) {
                sm.hist[i] = 0u;
                if (bins.keys) mass_own[i] = 0ull;
                else rest_own[i] = 0;
            }
            __syncthreads();
            sf_u64 own = 0ull;
            if (whole) {
                const float binades = bins.per_binade > 0.f ? 1.f / bins.per_binade : 0.f;
                each([&](const float (&v)[kSfBatch], int) {
#pragma unroll
                    for (int e = 0; e < kSfBatch; ++e) {
                        float x;
                        uint32_t f;
                        const uint32_t n = row.mass(v[e], x, f);
                        own += (sf_u64)n * f;
                        const int i = x < kSfFar ? bins.near(x) : kSfBins - 1;   // NaN too: to the bin that no other logit has
                        atomicAdd(&sm.hist[i], 1u);
                        if (f > 1u) atomicAdd(&rest_own[i], (int)(((float)i * binades - x) * (0.6931471805599453f * 1048576.f)));
                    }
                }, no_segment);
                publish(kSfWhole, block_sum(own));
            } else {
                each([&](const float (&v)[kSfBatch], int) {
#pragma unroll
                    for (int e = 0; e < kSfBatch; ++e) {
                        if (!(v[e] > -INFINITY)) continue;   // nor NaN
                        const int i = bins.of(row, v[e]);
                        if (i < 0 || i >= kSfBins) continue;
                        atomicAdd(&sm.hist[i], 1u);
                        if (bins.keys) atomicAdd(&mass_own[i], row.mass(v[e]));
                    }
                }, no_segment);
            }
            if (whole && tid == 0) sm.hist[kSfBins - 1] = 0u;
            sf_sync();
            const int share = kSfBins / CS;    // this rank adds up its share of the bins for all
            for (int i = (int)rank * share + tid; i < ((int)rank + 1) * share; i += THREADS) {
                uint32_t n = 0, c[kSfMaxCluster];
                int rest = 0, d[kSfMaxCluster];
                sf_u64 m = 0ull, x[kSfMaxCluster];
#pragma unroll
                for (int r = 0; r < kSfMaxCluster; ++r) {
                    c[r] = r < CS ? sf_get32(&sm.hist[i], (uint32_t)r) : 0u;
                    d[r] = r < CS && !bins.keys ? (int)sf_get32(&rest_own[i], (uint32_t)r) : 0;
                    x[r] = r < CS && bins.keys ? sf_get(&mass_own[i], (uint32_t)r) : 0ull;
                }
#pragma unroll
                for (int r = 0; r < kSfMaxCluster; ++r) {
                    n += c[r];
                    rest += d[r];
                    m += x[r];
                }
                for (int r = 0; r < CS; ++r) {
                    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(sf_at(&sm.counts[i], (uint32_t)r)), "r"(n) : "memory");
                    if (bins.keys) sf_put(&mass_all[i], (uint32_t)r, m);
                    else asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(sf_at(&rest_all[i], (uint32_t)r)), "r"(rest) : "memory");
                }
            }
            sf_sync();
            if (whole) {
                *whole = 0ull;
                for (int r = 0; r < CS; ++r) *whole += sm.xch[kSfWhole][r];
            }
        };
        auto sum_all = [&]() {
            sf_u64 own = 0ull;
            each([&](const float (&v)[kSfBatch], int) { add_from(row, v, -INFINITY, true, own); }, no_segment);
            publish(kSfWhole, block_sum(own));
            sf_sync();
            own = 0ull;
            for (int r = 0; r < CS; ++r) own += sm.xch[kSfWhole][r];
            return own;
        };
        // The bins [lo, hi] in which the weights from the top, `base` above all bins, reach
        // `target`; tokens before lo and up to hi.  False: they do not.
        // Estimated: by the masses of the bins' middles, and a bin on either side.
        auto bracket = [&](bool by_mass, bool estimated, sf_u64 base, sf_u64 target, int &lo, int &hi, uint32_t &before, uint32_t &upto) {
            constexpr int PT = kSfBins / THREADS;
            uint32_t c[PT], n = 0;
            sf_u64 u[PT], l[PT], su = 0ull, sl = 0ull;
#pragma unroll
            for (int e = 0; e < PT; ++e) {
                const int i = tid * PT + e;
                c[e] = sm.counts[i];
                u[e] = l[e] = c[e];
                if (by_mass && bins.keys) {
                    u[e] = l[e] = mass_all[i];
                } else if (by_mass && estimated) {
                    if (c[e]) u[e] = (sf_u64)(((float)c[e] + (float)rest_all[i] * 0x1p-20f) * bins.middle(i));
                    l[e] = u[e];
                } else if (by_mass && c[e]) {
                    u[e] *= bins.most(i);
                    l[e] *= bins.least(i);
                }
                n += c[e];
                su += u[e];
                sl += l[e];
            }
            sf_u64 iu = sf_warp_scan(su), il = sf_warp_scan(sl);
            const uint32_t in = (uint32_t)sf_warp_scan(n);
            __syncthreads();
            if (lane == 31) {
                sm.scan[0][w] = iu;
                sm.scan[1][w] = il;
                sm.scan_n[w] = in;
            }
            if (tid < 4) sm.bin[tid] = tid < 2 ? kSfBins : 0;
            __syncthreads();
            sf_u64 ru = base + iu - su, rl = base + il - sl;
            uint32_t rn = in - n;
            for (int i = 0; i < w; ++i) {
                ru += sm.scan[0][i];
                rl += sm.scan[1][i];
                rn += sm.scan_n[i];
            }
#pragma unroll
            for (int e = 0; e < PT; ++e) {
                if (ru < target && ru + u[e] >= target) {
                    sm.bin[0] = tid * PT + e;
                    sm.bin[2] = (int)rn;
                }
                rn += c[e];
                if (rl < target && rl + l[e] >= target) {
                    sm.bin[1] = tid * PT + e;
                    sm.bin[3] = (int)rn;
                }
                ru += u[e];
                rl += l[e];
            }
            if (tid == THREADS - 1 && rl < target) sm.bin[3] = (int)rn;   // to the last bin
            __syncthreads();
            lo = sm.bin[0];
            hi = min(sm.bin[1], kSfBins - 1);
            before = (uint32_t)sm.bin[2];
            upto = (uint32_t)sm.bin[3];
            if (estimated && by_mass && lo < kSfBins) {
                if (lo > 0) before -= sm.counts[--lo];
                if (hi < kSfBins - 1) upto += sm.counts[++hi];
            }
            return lo < kSfBins;
        };
        // The least key whose bin is at most i, by the warp, five bits a step (0: all are below it).
        auto least_key = [&](int i) {
            uint32_t key = kmin;   // its bin is more than i, if any of the row's is
            if (bins.of(row, sf_unkey(kmin)) <= i) return kmin;
            uint32_t span = kmax - kmin;   // kmax's bin is 0 or, by keys, above: at most i
            while (span > 1) {             // bin(key) > i >= bin(key + span)
                const uint32_t step = span / 32 + (span % 32 ? 1 : 0);
                const uint32_t mine = (uint32_t)min((sf_u64)span, (sf_u64)step * (uint32_t)(lane + 1));
                const unsigned in = __ballot_sync(0xffffffffu, bins.of(row, sf_unkey(key + mine)) <= i);
                const uint32_t first = step * (uint32_t)(__ffs(in) - 1);   // the last lane's is in
                span = min(span - first, step);
                key += first;
            }
            return key + 1;
        };
        bool divided = false;
        bool low_set = false;
        // The cut where the weights reach `target`; by_mass: a mass, else a count.  `held`: the
        // mass that the cut keeps, where want_held.  2: the row has been ended.
        auto find = [&](bool by_mass, sf_u64 target, bool want_held, SfCut &result, sf_u64 &held) {
            const SfBins coarse = bins;
            int lo = 0, hi = kSfBins - 1;
            uint32_t before = 0, upto = (uint32_t)a.V;
            if (divided) {   // an earlier search's finer counts are in place of the row's
                count(nullptr);
                divided = false;
            }
            // the estimate's band has far fewer tokens; whether the cut lies there is seen from the exact masses
            bool guess = by_mass && k <= 1 && bracket(true, true, 0ull, target, lo, hi, before, upto) && upto > kSfRank;
            if (!guess && !bracket(by_mass, false, 0ull, target, lo, hi, before, upto)) return 0;
            if (!guess && upto <= kSfRank) {   // few after all
                if (w == 0) {
                    const uint32_t key = least_key(hi);
                    if (lane == 0) sm.found[2] = key;
                }
                __syncthreads();
                collect((uint32_t)sm.found[2]);
                finish(by_mass ? 1.f : nucleus ? p : 1.f, by_mass ? target : ~0ull);
                return 2;
            }
            // by keys a band is one bin, 2^-10 of the last band's keys at most: three divisions reach a single one
            for (int round = 0; round < 8; ++round) {
                const bool fits = upto - before <= kSfList;
                if (w < 2) {   // logits above the band, and from its end on
                    uint32_t key = ~0u;        // none
                    if (w) key = least_key(hi);
                    else if (lo > 0) key = least_key(lo - 1);
                    else if (bins.keys && bins.high < kmax) key = bins.high + 1u;
                    if (lane == 0) sm.found[2 + w] = key;
                }
                __syncthreads();
                const float over = (uint32_t)sm.found[2] == ~0u ? __uint_as_float(0x7fc00000u) : sf_unkey((uint32_t)sm.found[2]);
                const float from = sf_unkey((uint32_t)sm.found[3]);
                sf_u64 own = 0ull, seg = 0ull, in_band = 0ull;
                uint32_t most = 0u, least = ~0u;
                const bool weigh = by_mass || want_held;
                each([&](const float (&v)[kSfBatch], int at) {
                    if (!any_from(v, from)) return;
                    if (weigh) add_from(row, v, over, false, seg);
                    uint32_t band = 0;
#pragma unroll
                    for (int e = 0; e < kSfBatch; ++e) band |= v[e] >= from && !(v[e] >= over) ? 1u << e : 0u;
                    if (!__any_sync(0xffffffffu, band != 0u)) return;
#pragma unroll
                    for (int e = 0; e < kSfBatch; ++e) {
                        if (!(band >> e & 1u)) continue;
                        const uint32_t key = sf_key(v[e]);
                        most = max(most, key);
                        least = min(least, key);
                        if (guess) row.add(in_band, v[e]);
                        if (fits) {
                            const uint32_t n = atomicAdd(&sm.nlist, 1u);
                            if (n < kSfList) sm.list[n] = (sf_u64)key << 32 | (uint32_t)~index_of(at, e);
                        }
                    }
                }, [&](int s) {
                    seg = sf_warp_sum(seg);
                    if (lane == 0) sm.seg_mass[s] = seg;
                    own += lane == 0 ? seg : 0ull;
                    seg = 0ull;
                });
                block_range(most, least);
                publish(kSfBand, (sf_u64)most << 32 | least);
                publish(kSfAbove, block_sum(own));
                if (guess) publish(kSfBandMass, block_sum(in_band));
                publish(kSfCount, sm.nlist);
                sf_sync();
                sf_u64 above = 0ull;
                in_band = 0ull;
                for (int r = 0; r < CS; ++r) {
                    above += sm.xch[kSfAbove][r];
                    if (guess) in_band += sm.xch[kSfBandMass][r];
                    most = max(most, (uint32_t)(sm.xch[kSfBand][r] >> 32));
                    least = min(least, (uint32_t)sm.xch[kSfBand][r]);
                }
                if (guess && !(above < target && target <= above + in_band)) {
                    guess = false;
                    __syncthreads();
                    if (tid == 0) sm.nlist = 0u;
                    sf_sync();                 // what was published has been read
                    if (!bracket(true, false, 0ull, target, lo, hi, before, upto)) return 0;
                    continue;
                }
                guess = false;
                if (most < least) return 0;    // the band is empty
                sf_u64 left = target - (by_mass ? above : (sf_u64)before);
                if (!fits && most != least) {  // divide the band by keys
                    int shift = 0;
                    while ((most - least) >> shift >= kSfBins) ++shift;
                    bins = SfBins{true, 0.f, most, least, shift};
                    divided = true;
                    const uint32_t top = before;
                    sf_sync();                 // what was published has been read
                    count(nullptr);
                    if (!bracket(by_mass, false, by_mass ? above : (sf_u64)before, target, lo, hi, before, upto)) return 0;
                    before += top;
                    upto += top;
                    continue;
                }
                uint32_t own_listed = sm.nlist;
                if (fits) {
                    if (rank == 0) {
                        const int n = gather();
                        const uint32_t key = sf_select(sm, row, n, most, least, by_mass, left);
                        publish(kSfFound, key);
                        publish(kSfLeft, left);
                        sf_u64 m = 0ull;
                        if (want_held)
                            for (int i = tid; i < n; i += THREADS) {
                                const uint32_t one = (uint32_t)(sm.list[i] >> 32);
                                if (one > key) m += row.mass(sf_unkey(one));
                            }
                        publish(kSfHeld, block_sum(m));
                    }
                    sf_sync();
                    result.key = (uint32_t)sm.xch[kSfFound][0];
                    left = sm.xch[kSfLeft][0];
                } else {
                    result.key = most;
                }
                const sf_u64 each_mass = row.mass(sf_unkey(result.key));
                if (by_mass) left = each_mass ? (left + each_mass - 1ull) / each_mass : 1ull;
                result.ties = (uint32_t)min(left, 0xffffffffull);
                if (want_held) held = above + (fits ? sm.xch[kSfHeld][0] : 0ull) + left * each_mass;
                // the segments' masses: what of the band is kept, from this rank's own list (the first
                // CTA's has the others' behind it)
                low_set = fits && weigh;
                if (low_set) {
                    if (tid < kSfSegments + 2) sm.seg_ties[tid] = 0u;
                    __syncthreads();
                    own_listed = min(own_listed, (uint32_t)kSfList);
                    for (uint32_t i = tid; i < own_listed; i += THREADS) {
                        const uint32_t key = (uint32_t)(sm.list[i] >> 32);
                        const int at = (int)~(uint32_t)sm.list[i];
                        const int s = at < at0 ? 0 : at >= at0 + 4 * nq ? kSfSegments + 1 : 1 + (at - at0) / 4 / sq;
                        if (key > result.key) atomicAdd(&sm.seg_mass[s], row.mass(sf_unkey(key)));
                        else if (key == result.key) atomicAdd(&sm.seg_ties[s], 1u);
                    }
                }
                __syncthreads();
                if (tid == 0) sm.nlist = 0u;
                bins = coarse;
                sf_sync();   // what was published has been read, and the lists
                return 1;
            }
            return 0;
        };

        sf_u64 whole = 0ull;
        count(nucleus && k <= 1 ? &whole : nullptr);
        if (k > 1) {
            SfCut by_k = {0u, ~0u};
            const int r = find(false, (sf_u64)k, nucleus, by_k, whole);
            if (r == 2) return;
            if (r == 1) {
                cut.tighten(by_k.key, by_k.ties);
                ready = low_set && cut.key == by_k.key && cut.ties == by_k.ties;
            } else if (nucleus) {   // all take part
                whole = sum_all();
            }
        }
        if (nucleus) {
            const sf_u64 target = max(sf_part(p, whole, true), 1ull);
            SfCut by_p = {0u, ~0u};
            sf_u64 held;
            const int r = find(true, target, false, by_p, held);
            if (r == 2) return;
            if (r == 1) {
                cut.tighten(by_p.key, by_p.ties);
                ready = low_set && cut.key == by_p.key && cut.ties == by_p.ties;
            }
        }
    }

    // ---- 5. kept mass by segments of the slice
    const float cut_at = cut.key ? sf_unkey(cut.key) : -INFINITY;
    if (!ready) {
        sf_u64 seg = 0ull;
        uint32_t ties = 0;
        each([&](const float (&v)[kSfBatch], int) {
            if (!any_from(v, cut_at)) return;
            add_from(row, v, cut_at, true, seg);
#pragma unroll
            for (int e = 0; e < kSfBatch; ++e) ties += v[e] == cut_at ? 1u : 0u;
        }, [&](int s) {
            seg = sf_warp_sum(seg);
            ties = __reduce_add_sync(0xffffffffu, ties);
            if (lane == 0) {
                sm.seg_mass[s] = seg;
                sm.seg_ties[s] = ties;
            }
            seg = 0ull;
            ties = 0;
        });
    }
    __syncthreads();
    const sf_u64 tie_mass = infinite ? 1ull << 40 : cut.key ? row.mass(cut_at) : 0ull;
    // every warp: the head's, the segments' and the tail's, three a lane
    static_assert(kSfSegments + 2 <= 3 * 32, "three places a lane");
    sf_u64 sm3[3], st3[3], mass_sum = 0ull, tie_sum = 0ull;
#pragma unroll
    for (int e = 0; e < 3; ++e) {
        const int s = 3 * lane + e;
        sm3[e] = s < kSfSegments + 2 ? sm.seg_mass[s] : 0ull;
        st3[e] = s < kSfSegments + 2 && cut.key ? sm.seg_ties[s] : 0ull;
        mass_sum += sm3[e];
        tie_sum += st3[e];
    }
    publish(kSfMass, sf_warp_sum(mass_sum));
    publish(kSfTies, sf_warp_sum(tie_sum));
    sf_sync();
    sf_u64 start = 0ull, kept = 0ull, ties_before = 0ull, seen = 0ull;
    for (int r = 0; r < CS; ++r) {
        if (r == (int)rank) {
            start = kept;
            ties_before = seen;
        }
        const sf_u64 n = sm.xch[kSfTies][r], left = seen < cut.ties ? cut.ties - seen : 0ull;
        kept += sm.xch[kSfMass][r] + min(n, left) * tie_mass;
        seen += n;
    }
    // a warp a draw
    for (int j = w; j < a.J; j += WARPS) {
        const long long out = (long long)b * a.J + j;
        const float u = a.u[out];
        const sf_u64 pos = u < 1.f ? sf_part(fmaxf(u, 0.f), kept, false) : u >= 1.f ? kept - 1ull : 0ull;
        // the place whose mass the draw falls into, with the ties and the mass before it
        sf_u64 tb = ties_before + sf_warp_scan(tie_sum) - tie_sum, own = 0ull, m3[3], t3[3];
#pragma unroll
        for (int e = 0; e < 3; ++e) {
            t3[e] = tb;
            m3[e] = sm3[e] + (tb < cut.ties ? min(st3[e], (sf_u64)cut.ties - tb) : 0ull) * tie_mass;
            own += m3[e];
            tb += st3[e];
        }
        sf_u64 run = start + sf_warp_scan(own) - own;
        int mine = -1;
        sf_u64 at_mass = 0ull, at_ties = 0ull;
#pragma unroll
        for (int e = 0; e < 3; ++e) {
            if (run <= pos && pos < run + m3[e]) {
                mine = 3 * lane + e;
                at_mass = run;
                at_ties = t3[e];
            }
            run += m3[e];
        }
        const unsigned hit = __ballot_sync(0xffffffffu, mine >= 0);
        if (!hit) continue;   // another rank's
        const int src = __ffs(hit) - 1, s = __shfl_sync(0xffffffffu, mine, src);
        run = __shfl_sync(0xffffffffu, at_mass, src);
        sf_u64 tied = __shfl_sync(0xffffffffu, at_ties, src);
        const int i0 = s == 0 ? s0 : at0 + 4 * min(nq, (s - 1) * sq);
        const int i1 = s == 0 ? at0 : s == kSfSegments + 1 ? s1 : at0 + 4 * min(nq, s * sq);
        for (int i = s == kSfSegments + 1 ? at0 + 4 * nq : i0; i < i1; i += 32) {
            const float v = i + lane < i1 ? z[i + lane] : -INFINITY;
            const bool tie = cut.key && v == cut_at;
            const unsigned ties = __ballot_sync(0xffffffffu, tie);
            sf_u64 m = 0ull;
            if (v > cut_at) m = row.mass(v);
            else if (tie && tied + __popc(ties & ((1u << lane) - 1u)) < cut.ties) m = tie_mass;
            const sf_u64 sum = run + sf_warp_scan(m);
            const unsigned past = __ballot_sync(0xffffffffu, m != 0ull && sum > pos);
            if (past) {
                if (lane == __ffs(past) - 1) a.out[out] = i + lane;
                break;
            }
            run = __shfl_sync(0xffffffffu, sum, 31);
            tied += __popc(ties);
        }
    }
}

template <int THREADS>
static cudaError_t sf_launch(const SampleFilteredArgs &a, int cluster, cudaStream_t s) {
    constexpr int kDevices = 64;
    static std::atomic<bool> ready[kDevices];
    const auto kern = sample_filtered_kernel<THREADS>;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= kDevices) return cudaErrorInvalidDevice;
    if (!ready[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(SfSmem<THREADS>));
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        ready[dev].store(true, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)cluster, (unsigned)a.B);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = sizeof(SfSmem<THREADS>);
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
    return cudaLaunchKernelEx(&cfg, kern, a);
}

cudaError_t launch_sample_filtered(const SampleFilteredArgs &a, cudaStream_t s) {
    const int sms = bloom_device_sms();
    // CTAs of 512 threads, two an SM, in one resident wave, each of 4096 logits at least; clusters of 16
    // for a few rows (top-p 0.95, clusters of 2, 4, 8, 16: 4 rows of 250880 87, 54, 37, 31 us; 16 rows
    // 95, 57, 48, 64; 64 rows 117, 78, 97, 174; 300 rows of 32000, from 1 on: 62, 84, 146, 251).
    // More rows than that: CTAs of 256 threads, four an SM, hide one another's phases; long rows on
    // two CTAs (509 rows of 250880, clusters of 1, 2, 4, 8: 511, 443, 451, 504 us; of 512 threads
    // 491, 463, 499, 664; 2000 rows of 8000: 228 against 266).
    if (a.B > 2 * sms) return sf_launch<256>(a, a.V >= 65536 ? 2 : 1, s);
    int cluster = 1;
    while (a.V / (2 * cluster) >= 4096 && (cluster < 8 ? a.B * cluster <= sms : cluster < kSfMaxCluster && 32 * a.B <= sms)) cluster *= 2;
    return sf_launch<512>(a, cluster, s);
}

}  // namespace bloom
