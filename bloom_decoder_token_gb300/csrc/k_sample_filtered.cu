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
// Bound by the logits' first read; then by the passes over them in shared memory or
// L2.  One cluster of up to 8 CTAs a row, each a slice of the vocabulary:
//  1. the maximum and minimum;
//  2. (top-k or top-p) a histogram of counts over the exponent, in 2048 bins, and the whole
//     mass.  A bin's tokens have masses within its edges', so the counts alone bound
//     where the cut's mass is reached to a band of bins.  (A histogram of masses needs 64-bit
//     atomics for every token.)
//  3. the exact mass above the band, and the band's tokens to the first CTA, which finds
//     the cut among them by radix over their keys.  A band of more tokens than fit
//     there is divided by another histogram, of masses over its range of keys, until it fits
//     or is a single logit.
//     Top-k and then top-p: one list serves both where it holds all of the top k.
//  4. the kept mass of 64 segments of each slice; the segment of a draw is walked to
//     the token.
#include <atomic>
#include <math.h>
#include <stdint.h>

#include "common.cuh"
#include "kernels.h"

namespace bloom {

typedef unsigned long long sf_u64;

constexpr int kSfMaxCluster = 8;
constexpr int kSfThreads = 512;
constexpr int kSfWarps = kSfThreads / 32;
constexpr int kSfBins = 2048;
constexpr int kSfList = 4096;                  // tokens of a band that the first CTA looks through
constexpr int kSfSegments = 64;                // of a slice
constexpr float kSfUnit = 1099511627776.f;     // 2^40
constexpr float kSfFar = 40.f;                 // binades below the maximum from which on a mass is 0
// Bounds of a bin's masses allow for the rounding of exponents (40 * 2^-23) and exponentials.  (The
// bins by keys have exact masses: with bounds a band of two logits next to a border never shrank.)
constexpr float kSfSlack = 1.f / 65536.f;

// Slots of the values that the ranks tell one another.  A slot is written again only after a
// barrier that follows its reading.
enum { kSfRange, kSfAbove, kSfFound, kSfLeft, kSfWhole, kSfBand, kSfHeld, kSfMass, kSfTies, kSfSlots };

struct alignas(16) SfSmem {   // the cached slice follows, in float4s
    sf_u64 list[kSfList];                      // first CTA: key << 32 | ~index
    uint32_t hist[kSfBins];                    // this CTA's counts
    uint32_t counts[kSfBins];                  // the cluster's
    sf_u64 digit[256];
    sf_u64 seg_mass[kSfSegments];
    uint32_t seg_ties[kSfSegments];
    sf_u64 scan[2][kSfWarps];
    uint32_t scan_n[kSfWarps];
    sf_u64 part[kSfWarps][3];
    sf_u64 xch[kSfSlots][kSfMaxCluster];       // a value of every rank
    sf_u64 found[4];
    double real[2];
    int bin[4];
    uint32_t nlist;
};

// ---- cluster
__device__ __forceinline__ void sf_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t sf_at(const void *p, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    return r;
}
__device__ __forceinline__ void sf_put(void *p, uint32_t rank, sf_u64 v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(sf_at(p, rank)), "l"(v) : "memory");
}

// ---- a row's exponents and masses
__device__ __forceinline__ uint32_t sf_key(float z) { return ordered_key(z + 0.f); }   // -0 as +0
__device__ __forceinline__ float sf_unkey(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}
__device__ __forceinline__ bool sf_takes_part(float z) { return z > -INFINITY; }   // nor NaN

struct SfRow {
    float top;         // the maximum
    float c, c_low;    // log2(e) / t, in two floats
    // (top - z) c in two floats; at least kSfFar where no mass is left
    __device__ __forceinline__ float exponent(float z, float &low) const {
        low = 0.f;
        if (z == top) return 0.f;
        const float d = top - z, w = d - top;
        const float e = (top - (d - w)) - (z + w);     // what d lost
        if (d == INFINITY) return kSfFar;              // an infinite maximum, or too far
        const float x = d * c;
        low = fmaf(d, c, -x) + fmaf(d, c_low, e * c);
        return x;
    }
    __device__ __forceinline__ sf_u64 mass(float z) const {
        float low;
        const float x = exponent(z, low);
        if (!(x < kSfFar)) return 0ull;
        float y;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(-x));
        y = fmaf(y * -0.6931471805599453f, low, y);
        return (sf_u64)(y * kSfUnit);
    }
};

// How the tokens are dealt to bins: by exponent, or by key from `high` down.
struct SfBins {
    bool keys;
    float per_binade;
    uint32_t high, low;
    int shift;
    // the bin; -1: above all bins, kSfBins: below them
    __device__ __forceinline__ int of(const SfRow &row, float z) const {
        if (keys) {
            const uint32_t k = sf_key(z);
            return k > high ? -1 : k < low ? kSfBins : (int)((high - k) >> shift);
        }
        float low_part;
        const float x = row.exponent(z, low_part);
        return x < kSfFar ? min(kSfBins - 1, (int)(x * per_binade)) : kSfBins;
    }
    // bounds of the masses in bin i, by exponent
    __device__ __forceinline__ sf_u64 most(int i) const {
        return up((sf_u64)((per_binade > 0.f ? exp2f(-(float)i / per_binade) : 1.f) * kSfUnit));   // 0: one exponent
    }
    __device__ __forceinline__ sf_u64 least(int i) const {
        if (i == kSfBins - 1) return 0ull;
        return down((sf_u64)((per_binade > 0.f ? exp2f(-(float)(i + 1) / per_binade) : 1.f) * kSfUnit));
    }
    static __device__ __forceinline__ sf_u64 up(sf_u64 m) { return m + (sf_u64)((float)m * kSfSlack) + 2ull; }
    static __device__ __forceinline__ sf_u64 down(sf_u64 m) {
        const sf_u64 less = (sf_u64)((float)m * kSfSlack) + 2ull;
        return m > less ? m - less : 0ull;
    }
};

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

// In the first CTA's list (n tokens): the key at which the weights of the highest keys,
// one a token or its mass, reach `target`, and what of the target is left for its ties.
__device__ __forceinline__ uint32_t sf_select(SfSmem &sm, const SfRow &row, int n, bool by_mass, sf_u64 &target) {
    const int tid = threadIdx.x, lane = tid & 31;
    uint32_t found = 0;
    for (int shift = 24; shift >= 0; shift -= 8) {
        if (tid < 256) sm.digit[tid] = 0ull;
        __syncthreads();
        for (int i = tid; i < n; i += kSfThreads) {
            const uint32_t k = (uint32_t)(sm.list[i] >> 32);
            if (shift < 24 && (k >> (shift + 8)) != found >> (shift + 8)) continue;
            atomicAdd(&sm.digit[k >> shift & 255u], by_mass ? row.mass(sf_unkey(k)) : 1ull);
        }
        __syncthreads();
        if (tid < 32) {   // digits from 255 down, eight a lane
            sf_u64 own = 0ull;
#pragma unroll
            for (int e = 0; e < 8; ++e) own += sm.digit[255 - 8 * lane - e];
            const sf_u64 upto = sf_warp_scan(own);
            const unsigned reach = __ballot_sync(0xffffffffu, upto >= target);
            const int src = reach ? __ffs(reach) - 1 : 31;
            if (lane == src) {
                sf_u64 run = upto - own;
                int e = 0;
                for (; e < 7 && run + sm.digit[255 - 8 * lane - e] < target; ++e) run += sm.digit[255 - 8 * lane - e];
                sm.found[0] = (sf_u64)(255 - 8 * lane - e);
                sm.found[1] = target - run;
            }
        }
        __syncthreads();
        found |= (uint32_t)sm.found[0] << shift;
        target = sm.found[1];
        __syncthreads();
    }
    return found;
}

__global__ void __launch_bounds__(kSfThreads) sample_filtered_kernel(const SampleFilteredArgs a) {
    extern __shared__ __align__(16) unsigned char sf_raw[];
    SfSmem &sm = *reinterpret_cast<SfSmem *>(sf_raw);
    griddep_launch();
    griddep_wait();
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int b = blockIdx.y, CS = (int)gridDim.x;
    uint32_t rank;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    const float *z = a.logits + (long long)b * a.ld;

    // this CTA's slice: whole float4s [at0, at0 + 4 nq) of the row's aligned body, and beside
    // them the row's ragged head (first CTA) and tail (last): indexes [s0, s1)
    const int head = min(a.V, (int)((0u - (uint32_t)(uintptr_t)z >> 2) & 3u));
    const int quads = (a.V - head) >> 2, per = (quads + CS - 1) / CS;
    const int q0 = min(quads, (int)rank * per), nq = min(quads, q0 + per) - q0, at0 = head + 4 * q0;
    const int s0 = rank == 0 ? 0 : at0, s1 = (int)rank == CS - 1 ? a.V : at0 + 4 * nq;
    float4 *cache = reinterpret_cast<float4 *>(sf_raw + sizeof(SfSmem));
    const float4 *body = a.cached ? cache : reinterpret_cast<const float4 *>(z + at0);
    const int ends = (at0 - s0) + (s1 - at0 - 4 * nq);   // at most six
    auto end_at = [&](int i) { return i < at0 - s0 ? s0 + i : at0 + 4 * nq + i - (at0 - s0); };
    auto each = [&](auto see) {   // every logit of the slice, in no order
        for (int i = tid; i < nq; i += 4 * kSfThreads) {
            float4 v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                v[k] = i + k * kSfThreads < nq ? body[i + k * kSfThreads] : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int at = at0 + 4 * (i + k * kSfThreads);
                see(v[k].x, at);
                see(v[k].y, at + 1);
                see(v[k].z, at + 2);
                see(v[k].w, at + 3);
            }
        }
        if (tid < ends) see(z[end_at(tid)], end_at(tid));
    };
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
        for (int i = 0; i < kSfWarps; ++i) v += sm.part[i][0];
        return v;
    };
    auto block_range = [&](uint32_t &most, uint32_t &least) {
        most = __reduce_max_sync(0xffffffffu, most);
        least = __reduce_min_sync(0xffffffffu, least);
        __syncthreads();
        if (lane == 0) sm.part[w][1] = (sf_u64)most << 32 | least;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kSfWarps; ++i) {
            most = max(most, (uint32_t)(sm.part[i][1] >> 32));
            least = min(least, (uint32_t)sm.part[i][1]);
        }
    };

    // ---- 1. maximum and minimum, as keys (0: nothing takes part)
    if (tid == 0) sm.nlist = 0u;
    sf_sync();   // every CTA runs, its counter is 0
    uint32_t kmax = 0u, kmin = ~0u;
    if (a.cached)
        for (int i = tid; i < nq; i += kSfThreads) cache[i] = reinterpret_cast<const float4 *>(z + at0)[i];   // a thread reads back its own below
    {
        float mx = -INFINITY, mn = INFINITY;
        each([&](float v, int) {
            mx = fmaxf(mx, v);
            mn = fminf(mn, v > -INFINITY ? v : INFINITY);
        });
        if (mx > -INFINITY) {
            kmax = sf_key(mx);
            kmin = sf_key(mn);
        }
    }
    block_range(kmax, kmin);
    publish(kSfRange, (sf_u64)kmax << 32 | kmin);
    sf_sync();
    for (int r = 0; r < CS; ++r) {
        kmax = max(kmax, (uint32_t)(sm.xch[kSfRange][r] >> 32));
        kmin = min(kmin, (uint32_t)sm.xch[kSfRange][r]);
    }
    if (kmax == 0u) {
        if (rank == 0)
            for (int j = tid; j < a.J; j += kSfThreads) a.out[(long long)b * a.J + j] = -1;
        sf_sync();   // no rank leaves while another's stores to it are under way
        return;
    }

    // ---- the row's settings
    float t = a.temperature ? a.temperature[b] : 1.f;
    int k = a.top_k ? a.top_k[b] : 0;
    const float p = a.top_p ? a.top_p[b] : 1.f, mp = a.min_p ? a.min_p[b] : 0.f;
    const bool nucleus = p < 1.f && p > 0.f;   // NaN: off
    if (!(t > 0.f)) {
        t = 1.f;
        k = 1;
    }
    if (p <= 0.f) k = 1;
    SfRow row;
    row.top = sf_unkey(kmax);
    const bool floored = mp > 0.f && mp < 1.f && row.top < INFINITY;
    if (tid == 0) {   // in 64 bits, by one thread: few of an SM's units have them
        sm.real[0] = fmin(1.4426950408889634 / (double)t, 3e38);
        if (floored) sm.real[1] = (double)row.top + (double)t * log((double)mp);
    }
    __syncthreads();
    row.c = (float)sm.real[0];
    row.c_low = (float)(sm.real[0] - (double)row.c);
    SfCut cut = {0u, ~0u};
    if (mp > 0.f) {   // the least logit with exp((z - top) / t) >= min_p
        float least = row.top;
        if (floored) least = fminf(__double2float_ru(sm.real[1]), row.top);
        cut.tighten(sf_key(least), ~0u);
    }
    if (k == 1) cut.tighten(kmax, 1u);

    // ---- 2., 3. the cuts of top-k and top-p
    if (k != 1 && (k > 1 || nucleus)) {
        float far_low;
        const float far = fminf(row.exponent(sf_unkey(kmin), far_low), kSfFar);
        SfBins bins = {false, far > 0.f ? 0.9999f * kSfBins / far : 0.f, 0u, 0u, 0};
        const bool all = a.V <= kSfList;       // the list holds the row: no histogram
        if (all) bins.per_binade = 0.f;
        // the cluster's counts of `bins`; by exponent with the whole mass, by keys with the bins'
        // masses, in the place of the list
        sf_u64 *mass_own = sm.list, *mass_all = sm.list + kSfBins;
        auto count = [&](sf_u64 *whole) {
            for (int i = tid; i < kSfBins; i += kSfThreads) {
                sm.hist[i] = 0u;
                if (bins.keys) mass_own[i] = 0ull;
            }
            __syncthreads();
            sf_u64 own = 0ull;
            each([&](float v, int) {
                if (!sf_takes_part(v)) return;
                const int i = bins.of(row, v);
                if (whole) own += row.mass(v);
                if (i < 0 || i >= kSfBins) return;
                atomicAdd(&sm.hist[i], 1u);
                if (bins.keys) atomicAdd(&mass_own[i], row.mass(v));
            });
            if (whole) publish(kSfWhole, block_sum(own));
            sf_sync();
            const int share = kSfBins / CS;    // this rank adds up its share of the bins for all
            for (int i = (int)rank * share + tid; i < ((int)rank + 1) * share; i += kSfThreads) {
                uint32_t n = 0;
                for (int r = 0; r < CS; ++r) {
                    uint32_t x;
                    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(x) : "r"(sf_at(&sm.hist[i], (uint32_t)r)) : "memory");
                    n += x;
                }
                for (int r = 0; r < CS; ++r)
                    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(sf_at(&sm.counts[i], (uint32_t)r)), "r"(n) : "memory");
                if (!bins.keys) continue;
                sf_u64 m = 0ull;
                for (int r = 0; r < CS; ++r) {
                    sf_u64 x;
                    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(x) : "r"(sf_at(&mass_own[i], (uint32_t)r)) : "memory");
                    m += x;
                }
                for (int r = 0; r < CS; ++r) sf_put(&mass_all[i], (uint32_t)r, m);
            }
            sf_sync();
            if (whole) {
                *whole = 0ull;
                for (int r = 0; r < CS; ++r) *whole += sm.xch[kSfWhole][r];
            }
        };
        // The bins [lo, hi] in which the weights from the top, `base` above all bins, reach
        // `target`; tokens before lo and up to hi.  False: they do not.
        auto bracket = [&](bool by_mass, sf_u64 base, sf_u64 target, int &lo, int &hi, uint32_t &before, uint32_t &upto) {
            constexpr int PT = kSfBins / kSfThreads;
            uint32_t c[PT], n = 0;
            sf_u64 u[PT], l[PT], su = 0ull, sl = 0ull;
#pragma unroll
            for (int e = 0; e < PT; ++e) {
                const int i = tid * PT + e;
                c[e] = sm.counts[i];
                u[e] = l[e] = c[e];
                if (by_mass && bins.keys) {
                    u[e] = l[e] = mass_all[i];
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
            if (tid == kSfThreads - 1 && rl < target) sm.bin[3] = (int)rn;   // to the last bin
            __syncthreads();
            lo = sm.bin[0];
            hi = min(sm.bin[1], kSfBins - 1);
            before = (uint32_t)sm.bin[2];
            upto = (uint32_t)sm.bin[3];
            return lo < kSfBins;
        };
        bool divided = false;
        int listed = 0;          // tokens in the first CTA's list: all from the top on
        uint32_t list_from = 0;  // number of tokens above the list
        sf_u64 above = 0ull;     // their mass
        // The cut where the weights reach `target`; by_mass: a mass, else a count.  `held`: the
        // mass that the cut keeps, where want_held.
        auto find = [&](bool by_mass, sf_u64 target, bool want_held, SfCut &result, sf_u64 &held) {
            const SfBins coarse = bins;
            int lo = 0, hi = kSfBins - 1;
            uint32_t before = 0, upto = (uint32_t)a.V;
            if (divided) {   // an earlier search's finer counts are in place of the row's
                count(nullptr);
                divided = false;
            }
            if (!all && !bracket(by_mass, 0ull, target, lo, hi, before, upto)) return false;
            if (!by_mass && upto <= kSfList) {   // all of the top k
                lo = 0;
                before = 0;
            }
            // by keys a band is one bin, 2^-10 of the last band's keys at most: three divisions reach a single one
            for (int division = 0; division < 8; ++division) {
                const bool fits = upto - before <= kSfList;
                sf_u64 own = 0ull;
                uint32_t most = 0u, least = ~0u;
                each([&](float v, int at) {
                    if (!sf_takes_part(v)) return;
                    const int i = bins.of(row, v);
                    if (i < lo) {
                        if (by_mass || want_held) own += row.mass(v);
                    } else if (i <= hi) {
                        const uint32_t key = sf_key(v);
                        most = max(most, key);
                        least = min(least, key);
                        if (fits) {
                            uint32_t n;
                            asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(n) : "r"(sf_at(&sm.nlist, 0u)), "r"(1u) : "memory");
                            if (n < kSfList) sf_put(&sm.list[n], 0u, (sf_u64)key << 32 | (uint32_t)~at);
                        }
                    }
                });
                block_range(most, least);
                publish(kSfBand, (sf_u64)most << 32 | least);
                publish(kSfAbove, block_sum(own));
                sf_sync();
                above = 0ull;
                for (int r = 0; r < CS; ++r) {
                    above += sm.xch[kSfAbove][r];
                    most = max(most, (uint32_t)(sm.xch[kSfBand][r] >> 32));
                    least = min(least, (uint32_t)sm.xch[kSfBand][r]);
                }
                sf_u64 left = target - (by_mass ? above : (sf_u64)before);
                if (fits || most == least) {
                    if (fits) {
                        if (rank == 0) {
                            listed = (int)min(sm.nlist, (uint32_t)kSfList);
                            __syncthreads();
                            if (tid == 0) sm.nlist = 0u;
                            const bool short_of = !by_mass && (sf_u64)listed < left;   // fewer take part: no cut
                            if (short_of) left = (sf_u64)listed;
                            const uint32_t key = sf_select(sm, row, listed, by_mass, left);
                            publish(kSfFound, (sf_u64)key << 32 | (short_of ? 1u : 0u));
                            publish(kSfLeft, left);
                        }
                        sf_sync();
                        result.key = (uint32_t)(sm.xch[kSfFound][0] >> 32);
                        left = sm.xch[kSfLeft][0];
                        if ((uint32_t)sm.xch[kSfFound][0]) return false;
                        list_from = before;
                    } else {
                        result.key = most;
                        sf_sync();
                        list_from = ~0u;
                    }
                    const sf_u64 each_mass = row.mass(sf_unkey(result.key));
                    if (by_mass) left = each_mass ? (left + each_mass - 1ull) / each_mass : 1ull;
                    result.ties = (uint32_t)min(left, (sf_u64)0xffffffffull);
                    if (want_held) {
                        held = above + left * each_mass;
                        if (fits) {
                            if (rank == 0) {
                                sf_u64 m = 0ull;
                                for (int i = tid; i < listed; i += kSfThreads) {
                                    const uint32_t key = (uint32_t)(sm.list[i] >> 32);
                                    if (key > result.key) m += row.mass(sf_unkey(key));
                                }
                                publish(kSfHeld, block_sum(m));
                            }
                            sf_sync();
                            held += sm.xch[kSfHeld][0];
                        }
                    }
                    bins = coarse;
                    return true;
                }
                // divide the band by keys
                int shift = 0;
                while ((most - least) >> shift >= kSfBins) ++shift;
                bins = SfBins{true, 0.f, most, least, shift};
                divided = true;
                const uint32_t top = before;
                sf_sync();   // what was published has been read
                count(nullptr);
                if (!bracket(by_mass, by_mass ? above : (sf_u64)before, target, lo, hi, before, upto)) return false;
                before += top;
                upto += top;
            }
            return false;
        };

        auto sum_all = [&]() {
            sf_u64 own = 0ull;
            each([&](float v, int) {
                if (sf_takes_part(v)) own += row.mass(v);
            });
            publish(kSfWhole, block_sum(own));
            sf_sync();
            own = 0ull;
            for (int r = 0; r < CS; ++r) own += sm.xch[kSfWhole][r];
            return own;
        };
        sf_u64 whole = 0ull;
        if (!all) count(nucleus && k <= 1 ? &whole : nullptr);
        else if (nucleus && k <= 1) whole = sum_all();
        bool have_list = false;
        if (k > 1) {
            SfCut by_k;
            if (find(false, (sf_u64)k, nucleus, by_k, whole)) {
                cut.tighten(by_k.key, by_k.ties);
                have_list = list_from == 0u;
            } else if (nucleus) {   // all take part
                whole = sum_all();
            }
        }
        if (nucleus) {
            __syncthreads();
            if (tid == 0) {
                const double want = ceil((double)p * (double)whole);
                sm.found[2] = want < 1.0 ? 1ull : min((sf_u64)want, whole);
            }
            __syncthreads();
            const sf_u64 target = sm.found[2];
            SfCut by_p = {0u, ~0u};
            if (have_list) {   // the top k are listed
                if (rank == 0) {
                    sf_u64 left = target;
                    const uint32_t key = sf_select(sm, row, listed, true, left);
                    const sf_u64 m = row.mass(sf_unkey(key));
                    publish(kSfFound, (sf_u64)key << 32 | (uint32_t)(m ? (left + m - 1ull) / m : 1ull));
                }
                sf_sync();
                by_p.key = (uint32_t)(sm.xch[kSfFound][0] >> 32);
                by_p.ties = (uint32_t)sm.xch[kSfFound][0];
                cut.tighten(by_p.key, by_p.ties);
            } else {
                sf_u64 held;
                sf_sync();   // after a search for the top k: what it published has been read
                if (find(true, target, false, by_p, held)) cut.tighten(by_p.key, by_p.ties);
            }
        }
    }

    // ---- 4. kept mass by segments of the slice
    const int len = s1 - s0, sl = ((len + kSfSegments - 1) / kSfSegments + 31) / 32 * 32;
    const float *flat = reinterpret_cast<const float *>(body);
    auto logit = [&](int i) { return i >= at0 && i < at0 + 4 * nq ? flat[i - at0] : z[i]; };
    for (int s = w; s < kSfSegments; s += kSfWarps) {
        const int i1 = min(s1, s0 + (s + 1) * sl);
        sf_u64 m = 0ull;
        uint32_t ties = 0;
        for (int i = s0 + s * sl + lane; i < i1; i += 4 * 32) {
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = i + 32 * e < i1 ? logit(i + 32 * e) : -INFINITY;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (!sf_takes_part(v[e])) continue;
                const uint32_t key = sf_key(v[e]);
                if (key > cut.key) m += row.mass(v[e]);
                else if (key == cut.key) ++ties;
            }
        }
        m = sf_warp_sum(m);
        ties = __reduce_add_sync(0xffffffffu, ties);
        if (lane == 0) {
            sm.seg_mass[s] = m;
            sm.seg_ties[s] = ties;
        }
    }
    __syncthreads();
    static_assert(kSfSegments == 64, "two segments a lane");
    const sf_u64 tie_mass = row.mass(sf_unkey(cut.key));
    sf_u64 own_mass = 0ull, own_ties = 0ull;
    if (w == 0) {
        own_mass = sf_warp_sum(sm.seg_mass[lane] + sm.seg_mass[lane + 32]);
        own_ties = sf_warp_sum((sf_u64)sm.seg_ties[lane] + sm.seg_ties[lane + 32]);
        if (lane == 0) {
            sm.found[2] = own_mass;
            sm.found[3] = own_ties;
        }
    }
    __syncthreads();
    publish(kSfMass, sm.found[2]);
    publish(kSfTies, sm.found[3]);
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
    for (int j = w; j < a.J; j += kSfWarps) {
        const long long at = (long long)b * a.J + j;
        const float u = a.u[at];
        sf_u64 pos = u > 0.f ? (sf_u64)((double)u * (double)kept) : 0ull;
        if (pos >= kept) pos = kept - 1ull;
        // segments 2 lane and 2 lane + 1: ties, then masses before them
        const sf_u64 t0 = sm.seg_ties[2 * lane], t1 = sm.seg_ties[2 * lane + 1];
        const sf_u64 tb = ties_before + sf_warp_scan(t0 + t1) - t0 - t1;
        auto of = [&](sf_u64 n, sf_u64 before) { return before < cut.ties ? min(n, (sf_u64)cut.ties - before) : 0ull; };
        const sf_u64 m0 = sm.seg_mass[2 * lane] + of(t0, tb) * tie_mass, m1 = sm.seg_mass[2 * lane + 1] + of(t1, tb + t0) * tie_mass;
        const sf_u64 upto = start + sf_warp_scan(m0 + m1), from = upto - m0 - m1;
        const unsigned mine = __ballot_sync(0xffffffffu, from <= pos && pos < upto);
        if (!mine) continue;   // another rank's
        const int src = __ffs(mine) - 1;
        const int second = __shfl_sync(0xffffffffu, (int)(pos >= from + m0), src);
        sf_u64 run = __shfl_sync(0xffffffffu, second ? from + m0 : from, src);
        sf_u64 tied = __shfl_sync(0xffffffffu, second ? tb + t0 : tb, src);
        const int s = 2 * src + second, i1 = min(s1, s0 + (s + 1) * sl);
        for (int i0 = s0 + s * sl; i0 < i1; i0 += 32) {
            const float v = i0 + lane < i1 ? logit(i0 + lane) : -INFINITY;
            const uint32_t key = sf_takes_part(v) ? sf_key(v) : 0u;
            const unsigned ties = __ballot_sync(0xffffffffu, key != 0u && key == cut.key);
            sf_u64 m = 0ull;
            if (key > cut.key) m = row.mass(v);
            else if (key != 0u && key == cut.key && tied + __popc(ties & ((1u << lane) - 1u)) < cut.ties) m = tie_mass;
            const sf_u64 sum = run + sf_warp_scan(m);
            const unsigned past = __ballot_sync(0xffffffffu, m != 0ull && sum > pos);
            if (past) {
                if (lane == __ffs(past) - 1) a.out[at] = i0 + lane;
                break;
            }
            run = __shfl_sync(0xffffffffu, sum, 31);
            tied += __popc(ties);
        }
    }
    sf_sync();   // no rank leaves while another's stores to it are under way
}

cudaError_t launch_sample_filtered(SampleFilteredArgs a, cudaStream_t s) {
    constexpr int kDevices = 64, kMost = 220 * 1024;
    static std::atomic<bool> ready[kDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= kDevices) return cudaErrorInvalidDevice;
    if (!ready[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(sample_filtered_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
        if (e != cudaSuccess) return e;
        ready[dev].store(true, std::memory_order_release);
    }
    const int sms = bloom_device_sms();
    int cluster = 1;
    while (cluster < kSfMaxCluster && a.V / (2 * cluster) >= 4096 && (long long)a.B * cluster < 4ll * sms) cluster *= 2;
    const size_t slice = ((size_t)(a.V / 4 + cluster - 1) / cluster + 1) * 16;
    a.cached = sizeof(SfSmem) + slice <= 100 * 1024 || ((long long)a.B * cluster <= sms && sizeof(SfSmem) + slice <= kMost);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)cluster, (unsigned)a.B);
    cfg.blockDim = dim3(kSfThreads);
    cfg.dynamicSmemBytes = sizeof(SfSmem) + (a.cached ? slice : 0);
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
    return cudaLaunchKernelEx(&cfg, sample_filtered_kernel, a);
}

}  // namespace bloom
