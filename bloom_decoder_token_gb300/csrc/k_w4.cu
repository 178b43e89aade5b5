// Quantising bf16 weights to 4 bits with group scales, and reading them back
// (w4_ops.cuh has the format).
//
// scale = bf16(amax / 7), code = w / scale rounded half to even.  Both come out as
// in exact arithmetic: amax and w have 8 significant bits, so amax / 7 lies 2^-13 of
// itself or more from a border between two bf16 numbers (float32 division is off by
// 2^-24), and w / scale is a half or lies 2^-10 or more from one, so a product with
// 1 / scale, off by 2^-20 at most, rounded to multiples of 2^-13, is a half where
// the quotient is.  A division an element would cost more than the loads.
//
// Bound by HBM: 2 bytes a weight in and half a byte out, or the other way round.  One
// warp a tile; a row's 8 columns are one 16-byte access, 64 bytes of a row for the
// four lanes that hold it.
#include "common.cuh"
#include "kernels.h"
#include "w4_ops.cuh"

namespace bloom {

constexpr int kW4Threads = 128;

// A word from its eight codes, for w4_pair().
__device__ __forceinline__ uint32_t w4_word(const int (&c)[8]) {
    uint32_t w = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t half = (uint32_t)abs(c[e]) << 8 | (c[e] < 0 ? 0x8000u : 0u);
        const uint32_t both = half << (16 * (e & 1));
        w |= e < 6 ? __funnelshift_r(both, both, 4 * (e >> 1)) : __funnelshift_l(both, both, 4);
    }
    return w;
}

struct W4Scale {
    float up, inv;    // code = (x * up) * inv rounded
    uint16_t bits;
    __device__ __forceinline__ explicit W4Scale(uint32_t amax) {   // |bf16| bits
        bits = amax >= 0x7f80u ? (uint16_t)0x7fc0u : f2bf(__fdiv_rn(bf2f((uint16_t)amax), 7.f));
        const float s = bf2f(bits);
        up = s < 0x1p-64f ? 0x1p64f : 1.f;    // 1 / scale stays a float
        inv = s > 0.f ? __frcp_rn(s * up) : 0.f;   // 0 and NaN: codes 0
    }
    __device__ __forceinline__ int code(float x) const {
        const float t = inv > 0.f ? x * up * inv : 0.f;
        return max(-7, min(7, __float2int_rn((t + 1536.f) - 1536.f)));
    }
};

template <int G>
__global__ void __launch_bounds__(kW4Threads) w4_quantize_kernel(const W4Args a) {
    constexpr int U = G < 64 ? 64 : G, J = U / 32, GJ = G / 32;   // columns of a pass; 32-column steps of it, of a group
    griddep_launch();
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
#pragma unroll
                for (int j = gr * GJ; j < (gr + 1) * GJ; ++j) {
                    float f[8];
                    unpack8(x[j][r], f);
                    int c[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) c[e] = s.code(f[e]);
                    words[j][r] = w4_word(c);
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

// Code e of the eight of a word.
__device__ __forceinline__ float w4_code(uint32_t w, int e) {
    const uint32_t half = w4_pair(w, e >> 1) >> (16 * (e & 1));
    const float m = (float)(half >> 8 & 7u);
    return half & 0x8000u ? -m : m;
}

template <int G>
__global__ void __launch_bounds__(kW4Threads) w4_read_kernel(const W4Args a) {
    griddep_launch();
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
            const float scale = r ? bf_hi(s[32 * j / G]) : bf_lo(s[32 * j / G]);
            uint32_t o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = pack_bf2(w4_code(w, 2 * e) * scale, w4_code(w, 2 * e + 1) * scale);
            *reinterpret_cast<uint4 *>(a.w + row * a.ld + k) = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
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
