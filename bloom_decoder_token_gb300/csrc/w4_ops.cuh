// 4-bit weights with group scales: what a tile holds, shared by the kernels that
// quantise, read back and multiply.
//
// value = code * scale, codes -7 .. 7, one bf16 scale for every `group` (32, 64 or
// 128) neighbouring weights of a row.  The matrix [N][K] lies in tiles of 16 rows x
// 256 columns, [ceil(K / 256)][ceil(N / 16)], zeros beyond N and K, so that a warp
// streams whole tiles with one bulk copy each and finds its fragments of mma.sync
// m16n8k16 in place:
//  * codes, 2048 bytes: lane (g, q) = 4 g + q holds rows g and g + 8, of every 32
//    columns j the eight 8 q .. 8 q + 7: 16-byte piece i (at i * 512 + lane * 16) =
//    words (row g, j = 2 i), (row g + 8, 2 i), (row g, 2 i + 1), (row g + 8, 2 i + 1);
//  * scales, 32 bytes a group: rows g and g + 8 side by side, for g = 0 .. 7.
// A word's pair i is columns 8 q + 2 i and 8 q + 2 i + 1, each as sign and magnitude, laid
// so that the word, shifted (w4_pair) and masked with 0x87008700, is the two codes as f16
// numbers: with the magnitude (0 .. 7) in bits 8 to 10, the last two bits of its place in
// the fraction and the last of the exponent, an f16 is magnitude * 2^-16.  Eight codes cost
// seven instructions, and nothing has to be subtracted.  (In the last three bits, as
// subnormals of 2^-24, they cost the tensor cores' sums seven bits: products are
// aligned by exponent.)
#pragma once

#include <stdint.h>

#include "common.cuh"

namespace bloom {

constexpr int kW4Rows = 16, kW4Cols = 256;
__host__ __device__ constexpr int w4_tile_bytes(int group) { return 2048 + 8192 / group; }

// Codes 2 i and 2 i + 1 of a word, times 2^-16, as f16x2.  Shifts to the left can run on
// another pipe than the masks; the last pair takes a turn, for one sign bit is left at the other end.
__device__ __forceinline__ uint32_t w4_pair(uint32_t w, int i) {
    return (i < 3 ? w << (4 * i) : __funnelshift_r(w, w, 4)) & 0x87008700u;
}

}  // namespace bloom
