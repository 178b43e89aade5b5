// Quantising bf16 weights to 4 bits with group scales, and reading them back
// (w4_ops.cuh has the format).
//
// scale = bf16(amax / 7), code = w / scale rounded half to even.  Both come out as
// in exact arithmetic: amax and w have 8 significant bits, so amax / 7 lies 2^-13 of
// itself or more from a border between two bf16 numbers (below 2^-126: 2^-137 or more),
// while a product with the float 1 / 7 is off by 2^-23 of itself and 2^-150; and
// w / scale is a half or lies 2^-10 or more from one, so a product with 1 / scale, off
// by 2^-19 at most (rcp.approx: 2^-23 of itself), rounded to multiples of 2^-13, is a
// half where the quotient is.
//
// Bound by HBM: 2 bytes a weight in and half a byte out, or the other way round.  One
// warp a tile; a row's 8 columns are one 16-byte access, 64 bytes of a row for the
// four lanes that hold it.  57344 x 14336 in groups of 64: quantised in 311 us, 6690
// GB/s (as a copy), read back in 331, 6290; 14336 x 57344 in groups of 32: 342 and 328;
// 16384 x 4096 in groups of 64: 31 and 30.  (With scales by IEEE division, and codes by conversions
// to integers and comparisons, it was bound by instructions: 88 us for these two.)
#include "common.cuh"
#include "kernels.h"
#include "w4_ops.cuh"

namespace bloom {

constexpr int kW4Threads = 128;

// A word from its pairs, each as w4_pair() gives it.
__device__ __forceinline__ uint32_t w4_word(const uint32_t (&p)[4]) {
    return p[0] | p[1] >> 4 | p[2] >> 8 | __funnelshift_l(p[3], p[3], 4);
}

struct W4Scale {
    float inv, up;    // |code| = |x| * inv, rounded; where `rare`, min(|x| * up * inv, 7), rounded
    uint16_t bits;
    bool rare;        // a scale whose reciprocal may be no float or whose bits are few, or NaN
    __device__ __forceinline__ explicit W4Scale(uint32_t amax) {   // |bf16| bits
        asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(bits) : "f"(bf2f((uint16_t)amax) * (1.f / 7.f)));
        if (amax >= 0x7f80u) bits = 0x7fc0u;
        const float s = bf2f(bits);
        rare = amax != 0u && !(s >= 0x1p-64f);
        up = rare ? 0x1p64f : 1.f;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s * up));
        inv = s > 0.f ? inv : 0.f;    // 0 and NaN: codes 0
    }
};

// Two codes of the bf16 numbers x, as w4_pair() gives them.  |x| * inv + 1536 is a multiple of 2^-13, and
// adding what is missing to 1.5 * 2^23 rounds it to an integer, the code in the last byte.
template <bool RARE>
__device__ __forceinline__ uint32_t w4_codes(uint32_t x, const W4Scale &s) {
    float t[2] = {fabsf(bf_lo(x)), fabsf(bf_hi(x))};
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        if (RARE) t[e] = s.inv > 0.f ? fminf(t[e] * s.up * s.inv, 7.f) : 0.f;
        else t[e] = __fmul_rn(t[e], s.inv);
        t[e] = __fadd_rn(__fadd_rn(t[e], 1536.f), 12582912.f - 1536.f);
    }
    const uint32_t m = __byte_perm(__float_as_uint(t[0]), __float_as_uint(t[1]), 0x4501);   // |code| << 8
    return m | (x & (m * 16u + 0x70007000u) & 0x80008000u);                                 // 0 has no sign
}

template <int G>
__global__ void __launch_bounds__(kW4Threads) w4_quantize_kernel(const W4Args a) {
    constexpr int U = 128, J = U / 32, GJ = G / 32;   // columns of a pass (64 and 256: the same); 32-column steps of it, of a group
    griddep_wait();
    const long long tile = (long long)blockIdx.x * (kW4Threads / 32) + (threadIdx.x >> 5);
    const int ktiles = (a.K + kW4Cols - 1) / kW4Cols, row_tiles = (a.N + kW4Rows - 1) / kW4Rows;
    if (tile >= (long long)ktiles * row_tiles) return;
    const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int kt = (int)(tile / row_tiles), rt = (int)(tile - (long long)kt * row_tiles), k0 = kt * kW4Cols;
    const int row[2] = {rt * kW4Rows + g, rt * kW4Rows + g + 8};
    unsigned char *out = a.tiles + tile * w4_tile_bytes(G);
#pragma unroll
    for (int u = 0; u < kW4Cols / U; ++u) {
        uint4 x[J][2];
        const int ku = k0 + u * U + 8 * q;
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                x[j][r] = make_uint4(0u, 0u, 0u, 0u);
                if (row[r] < a.N && ku + 32 * j < a.K)
                    x[j][r] = *reinterpret_cast<const uint4 *>(a.w + row[r] * a.ld + ku + 32 * j);
            }
        uint32_t words[J][2];
#pragma unroll
        for (int gr = 0; gr < J / GJ; ++gr) {
            uint32_t scales = 0;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                uint32_t m2 = 0;
#pragma unroll
                for (int j = gr * GJ; j < (gr + 1) * GJ; ++j) {
                    m2 = __vmaxu2(m2, x[j][r].x & 0x7fff7fffu);
                    m2 = __vmaxu2(m2, x[j][r].y & 0x7fff7fffu);
                    m2 = __vmaxu2(m2, x[j][r].z & 0x7fff7fffu);
                    m2 = __vmaxu2(m2, x[j][r].w & 0x7fff7fffu);
                }
                uint32_t amax = max(m2 & 0xffffu, m2 >> 16);
                amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                const W4Scale s(amax);
                scales |= (uint32_t)s.bits << (16 * r);
                const bool rare = __any_sync(0xffffffffu, s.rare);
#pragma unroll
                for (int j = gr * GJ; j < (gr + 1) * GJ; ++j) {
                    const uint32_t v[4] = {x[j][r].x, x[j][r].y, x[j][r].z, x[j][r].w};
                    uint32_t p[4];
                    if (rare) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) p[e] = w4_codes<true>(v[e], s);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e) p[e] = w4_codes<false>(v[e], s);
                    }
                    words[j][r] = w4_word(p);
                }
            }
            if (q == 0) *reinterpret_cast<uint32_t *>(out + 2048 + ((u * U) / G + gr) * 32 + g * 4) = scales;
        }
#pragma unroll
        for (int j = 0; j < J; j += 2)
            *reinterpret_cast<uint4 *>(out + (u * U / 64 + j / 2) * 512 + lane * 16) =
                make_uint4(words[j][0], words[j][1], words[j + 1][0], words[j + 1][1]);
    }
}

// Codes 2 i and 2 i + 1 of a word times the scale, as bf16: 128 + |code| is a bf16 number, and the
// product is rounded once.
__device__ __forceinline__ uint32_t w4_values(uint32_t w, int i, uint32_t scales) {
    const uint32_t p = w4_pair(w, i), m = (p >> 8 & 0x00070007u) | 0x43004300u, s = scales ^ (p & 0x80008000u);
    uint32_t c, v;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(c) : "r"(m), "r"(0x43004300u));
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(v) : "r"(c), "r"(s));
    return v;
}

template <int G>
__global__ void __launch_bounds__(kW4Threads) w4_read_kernel(const W4Args a) {
    // No early start of the kernel after this one: the matrix may be a model's weights, which its layers load before
    // they wait.
    griddep_wait();
    const long long tile = (long long)blockIdx.x * (kW4Threads / 32) + (threadIdx.x >> 5);
    const int ktiles = (a.K + kW4Cols - 1) / kW4Cols, row_tiles = (a.N + kW4Rows - 1) / kW4Rows;
    if (tile >= (long long)ktiles * row_tiles) return;
    const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int kt = (int)(tile / row_tiles), rt = (int)(tile - (long long)kt * row_tiles), k0 = kt * kW4Cols;
    const unsigned char *in = a.tiles + tile * w4_tile_bytes(G);
    uint4 v[4];
    uint32_t s[kW4Cols / G];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const uint4 *>(in + i * 512 + lane * 16);
#pragma unroll
    for (int i = 0; i < kW4Cols / G; ++i) s[i] = *reinterpret_cast<const uint32_t *>(in + 2048 + i * 32 + g * 4);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int k = k0 + 32 * j + 8 * q;
        if (k >= a.K) continue;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = rt * kW4Rows + g + 8 * r;
            if (row >= a.N) continue;
            const uint32_t w = (&v[j / 2].x)[2 * (j & 1) + r];
            const uint32_t scales = __byte_perm(s[32 * j / G], 0u, r ? 0x3232 : 0x1010);
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = w4_values(w, i, scales);
            *reinterpret_cast<uint4 *>(a.w + row * a.ld + k) = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
    __threadfence();
}

template <typename K>
static cudaError_t w4_launch(K k32, K k64, K k128, const W4Args &a, cudaStream_t s) {
    const long long tiles = (long long)((a.K + kW4Cols - 1) / kW4Cols) * ((a.N + kW4Rows - 1) / kW4Rows);
    const long long ctas = (tiles + kW4Threads / 32 - 1) / (kW4Threads / 32);
    if (ctas > 0x7fffffffll) return cudaErrorInvalidValue;
    return launch_pdl(a.group == 32 ? k32 : a.group == 64 ? k64 : k128, dim3((unsigned)ctas), dim3(kW4Threads), s, a);
}

cudaError_t launch_w4_quantize(const W4Args &a, cudaStream_t s) {
    return w4_launch(w4_quantize_kernel<32>, w4_quantize_kernel<64>, w4_quantize_kernel<128>, a, s);
}

cudaError_t launch_w4_read(const W4Args &a, cudaStream_t s) {
    return w4_launch(w4_read_kernel<32>, w4_read_kernel<64>, w4_read_kernel<128>, a, s);
}

}  // namespace bloom
