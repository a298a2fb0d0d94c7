// Packed 4-bit weights: where the codes, scales and zero points of a matrix lie (the layout that strata_moe_ops.h
// describes), for the packers and for the kernels that read them.
//
// 16 rows (a slab) x 128 columns (a chunk) are one contiguous run: 1,024 bytes of codes in the order in which the lanes
// of a warp take them as operands of mma.m16n8k16, then scales, then zero points.  Lane (g, c) = 4g + c holds rows g and g + 8; of each
// 32 columns (a block) it holds columns 8c .. 8c + 7, one 32-bit word a row: four blocks are 16 bytes a row, one wide load.
#pragma once
#include "ops_common.cuh"
#include "q4_sizes.h"

namespace strata {
namespace q4 {

__host__ __device__ constexpr int groups_of(int group) { return CHUNK / group; }             // in a chunk
__host__ __device__ constexpr int scale_bytes(int group) { return 4 * groups_of(group); }    // rows g, g + 8 of a chunk
__host__ __device__ constexpr int zero_bytes(int group) {                                    // the same, to 4 bytes at least
  return 2 * groups_of(group) < 4 ? 4 : 2 * groups_of(group);
}
__host__ __device__ constexpr int meta_bytes(int group, bool zeros) {
  return 8 * (scale_bytes(group) + (zeros ? zero_bytes(group) : 0));
}
__host__ __device__ constexpr int chunk_bytes(int group, bool zeros) { return ROWS * CHUNK / 2 + meta_bytes(group, zeros); }
__host__ __device__ constexpr int64_t slab_bytes(int d_in, int group, bool zeros) {  // the last chunk may hold 1 to 3 blocks
  return (int64_t)(d_in / CHUNK) * chunk_bytes(group, zeros) +
         (d_in % CHUNK ? ROWS * (d_in % CHUNK) / 2 + meta_bytes(group, zeros) : 0);
}
inline int64_t matrix_bytes(const strata_q4_t& q) {
  return (int64_t)((q.n_out + ROWS - 1) / ROWS) * slab_bytes(q.d_in, q.group, q.zeros != 0);
}
// The row of the matrix in row r (0 .. 15) of slab s, or -1 behind its end.
__host__ __device__ inline int source_row(int n_out, int paired, int64_t s, int r) {
  if (paired) return (int)(8 * s + (r & 7) + (r >> 3) * (n_out / 2));
  const int64_t row = ROWS * s + r;
  return row < n_out ? (int)row : -1;
}
// Codes 0 .. 7 of a word of the matrix to the order of a packed word: code 2j at bits 4j, code 2j + 1 at bits 16 + 4j,
// so that (word >> 4j) & 0x000f000f is the pair (2j, 2j + 1).
__host__ __device__ inline uint32_t pair_codes(uint32_t w) {
  uint32_t p = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) p |= (w >> (8 * j) & 15u) << (4 * j) | (w >> (8 * j + 4) & 15u) << (16 + 4 * j);
  return p;
}

bool valid(const strata_q4_t& q);  // q4_pack.cu

}  // namespace q4

void pack_q4_host(const strata_q4_t& q, const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros, uint8_t* packed,
                  int64_t n_matrix);
cudaError_t launch_pack_q4(const strata_q4_t& q, const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros,
                           uint8_t* packed, int64_t n_matrix, cudaStream_t s);

}  // namespace strata
