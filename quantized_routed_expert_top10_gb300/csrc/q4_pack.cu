// Packing of 4-bit weights (strata_pack_q4, strata_pack_q4_device): a permutation of the codes, scales and zero points.
// A packed matrix is seen as units of 4 bytes (a word of codes; the two scales of a group; four zero points), each of
// which is gathered by itself, so the host and the device run the same function.  Once for a model's weights, so it is kept plain: a word a thread,
// stored in 4 bytes, 1.4 GB in 2.2 ms, five times a copy.
#include "q4_format.cuh"

namespace strata {
namespace q4 {

bool valid(const strata_q4_t& q) {
  if (q.group != 32 && q.group != 64 && q.group != 128) return false;
  if (q.n_out < 1 || q.n_out > STRATA_Q4_ROWS_MAX || q.d_in < q.group || q.d_in > STRATA_Q4_COLUMNS_MAX || q.d_in % q.group)
    return false;
  if (q.scale_type != STRATA_BF16 && q.scale_type != STRATA_F16) return false;
  if ((q.zeros != 0 && q.zeros != 1) || (q.paired != 0 && q.paired != 1)) return false;
  return !q.paired || q.n_out % ROWS == 0;
}

// Word `at` (0 .. slab_bytes / 4 - 1) of slab s; codes, scales and zeros are this matrix's.  wide: codes lie on 4-byte boundaries.
__host__ __device__ inline uint32_t packed_word(const strata_q4_t& q, const uint8_t* codes, const uint16_t* scales,
                                                const uint8_t* zeros, int64_t s, int at, bool wide) {
  const int chunk = chunk_bytes(q.group, q.zeros != 0) / 4;  // words
  const int ch = at / chunk;
  int w = at % chunk;
  const int left = q.d_in - ch * CHUNK;
  const int blocks = left >= CHUNK ? 4 : left / BLOCK;
  if (w < 64 * blocks) {  // codes: [row half][lane][block]
    const int half = w / (32 * blocks), lane = w / blocks % 32, b = w % blocks;
    const int row = source_row(q.n_out, q.paired, s, (lane >> 2) + 8 * half);
    if (row < 0) return 0;
    const uint8_t* p = codes + (int64_t)row * (q.d_in / 2) + ch * (CHUNK / 2) + b * (BLOCK / 2) + (lane & 3) * 4;
    if (wide) return pair_codes(*reinterpret_cast<const uint32_t*>(p));
    return pair_codes((uint32_t)p[0] | (uint32_t)p[1] << 8 | (uint32_t)p[2] << 16 | (uint32_t)p[3] << 24);
  }
  w -= 64 * blocks;
  const int n_group = q.d_in / q.group, first = ch * groups_of(q.group), per = groups_of(q.group);
  if (w < 8 * per) {  // scales: [g][group]{row g, row g + 8}
    const int g = w / per, gr = first + w % per;
    uint32_t v = 0;
    for (int half = 0; half < 2; ++half) {
      const int row = source_row(q.n_out, q.paired, s, g + 8 * half);
      if (row >= 0 && gr < n_group) v |= (uint32_t)scales[(int64_t)row * n_group + gr] << (16 * half);
    }
    return v;
  }
  w -= 8 * per;
  const int words = zero_bytes(q.group) / 4, g = w / words;  // zero points: [g][group]{row g, row g + 8}
  uint32_t v = 0;
  for (int i = 0; i < 4; ++i) {
    const int in = (w % words) * 2 + i / 2, gr = first + in;
    const int row = source_row(q.n_out, q.paired, s, g + 8 * (i & 1));
    if (in < per && row >= 0 && gr < n_group) v |= (uint32_t)(zeros[(int64_t)row * n_group + gr] & 15u) << (8 * i);
  }
  return v;
}

namespace {

// Source and destination of matrix m.
struct Place {
  int64_t codes, scales, packed;
};
__host__ __device__ inline Place place(const strata_q4_t& q, int64_t m, int64_t bytes) {
  const int64_t n_group = q.d_in / q.group;
  return Place{m * q.n_out * (q.d_in / 2), m * q.n_out * n_group, m * bytes};
}

// A slab of a matrix a block at a time: its words by 32-bit arithmetic (1.4 GB in 2.2 ms; 2.6 where every word found its matrix by 64 bits).
__global__ void pack_q4_kernel(strata_q4_t q, const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros, uint8_t* packed,
                               int64_t bytes, int64_t slabs, bool wide) {
  const int words = (int)(slab_bytes(q.d_in, q.group, q.zeros != 0) / 4);
  const int64_t of_matrix = bytes / (4 * words);
  for (int64_t i = blockIdx.x; i < slabs; i += gridDim.x) {
    const int64_t m = i / of_matrix, slab = i % of_matrix;
    const Place p = place(q, m, bytes);
    uint32_t* to = reinterpret_cast<uint32_t*>(packed + p.packed) + slab * words;
    for (int at = threadIdx.x; at < words; at += blockDim.x)
      to[at] = packed_word(q, codes + p.codes, scales + p.scales, zeros + (zeros ? p.scales : 0), slab, at, wide);
  }
}

}  // namespace
}  // namespace q4

void pack_q4_host(const strata_q4_t& q, const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros, uint8_t* packed,
                  int64_t n_matrix) {
  const int64_t bytes = q4::matrix_bytes(q), slab = q4::slab_bytes(q.d_in, q.group, q.zeros != 0) / 4;
  for (int64_t m = 0; m < n_matrix; ++m) {
    const q4::Place p = q4::place(q, m, bytes);
    for (int64_t at = 0; at < bytes / 4; ++at) {
      const uint32_t w =
          q4::packed_word(q, codes + p.codes, scales + p.scales, zeros + (zeros ? p.scales : 0), at / slab, (int)(at % slab), false);
      for (int b = 0; b < 4; ++b) packed[p.packed + 4 * at + b] = (uint8_t)(w >> (8 * b));
    }
  }
}

cudaError_t launch_pack_q4(const strata_q4_t& q, const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros,
                           uint8_t* packed, int64_t n_matrix, cudaStream_t s) {
  const int64_t bytes = q4::matrix_bytes(q), slabs = n_matrix * (bytes / q4::slab_bytes(q.d_in, q.group, q.zeros != 0));
  const bool wide = ((uintptr_t)codes & 3) == 0;  // d_in / 2 is a multiple of 16
  STRATA_LAUNCH(KID_PACK_Q4, s,
                q4::pack_q4_kernel<<<(unsigned)(slabs < 152 * 64 ? slabs : 152 * 64), 256, 0, s>>>(q, codes, scales, zeros, packed, bytes, slabs,
                                                                                                 wide));
  return cudaGetLastError();
}

}  // namespace strata
