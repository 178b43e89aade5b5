// 4-bit weights with group scales: what a tile holds, shared by the kernels that
// quantise, read back and multiply.
//
// value = code * scale, codes -7 .. 7, one bf16 scale for every `group` (32, 64 or
// 128) neighbouring weights of a row.  The matrix [N][K] lies in tiles of 16 rows x
// 256 columns, [ceil(N / 16)][ceil(K / 256)], zeros beyond N and K, so that a warp
// streams whole tiles with one bulk copy each and finds its fragments of mma.sync
// m16n8k32 in place:
//  * codes, 2048 bytes: lane (g, q) = 4 g + q holds rows g and g + 8, of every 32
//    columns j the eight 8 q .. 8 q + 7: 16-byte piece i (at i * 512 + lane * 16) =
//    words (row g, j = 2 i), (row g + 8, 2 i), (row g, 2 i + 1), (row g + 8, 2 i + 1);
//  * scales, 32 bytes a group: rows g and g + 8 side by side, for g = 0 .. 7.
// Byte b of a word holds columns 8 q + b and 8 q + 4 + b as sign and magnitude, laid so
// that the word itself and the word turned right by 4 bits, masked with 0x87 in
// every byte, are four e4m3 numbers each: the magnitude (0 .. 7) in the last three bits
// of an e4m3 is a subnormal, magnitude * 2^-9.  Eight codes cost three instructions.
#pragma once

#include <stdint.h>

#include "common.cuh"

namespace bloom {

constexpr int kW4Rows = 16, kW4Cols = 256;
constexpr uint32_t kW4Mask = 0x87878787u;
__host__ __device__ constexpr int w4_tile_bytes(int group) { return 2048 + 8192 / group; }

__device__ __forceinline__ uint32_t w4_low(uint32_t w) { return w & kW4Mask; }
__device__ __forceinline__ uint32_t w4_high(uint32_t w) { return __funnelshift_r(w, w, 4) & kW4Mask; }

}  // namespace bloom
