// What the kernels of strata_moe_linear and strata_moe_q4_experts share: weights streamed through a ring that each lane
// keeps for itself, 4-bit codes widened to bf16, products by mma.m16n8k16 and the activations' bf16 terms.
//
// Mathematics.  y[row] = sum over groups of s[row][group] * (sum over its columns of (code - zero) * x).  code - zero is a whole
// number of magnitude below 16 and exact in bf16; x enters as 1 to 3 bf16 terms that add up to it exactly (bf16: 1, fp16: 2, fp32: 3),
// each a column of the products, so all products are exact and their sums fp32; the scale multiplies a group's fp32 sum.
// What bounds it: the weights' bytes, each read once and by no other warp.  16 rows x 32 columns of codes (256 bytes) are two MMAs
// for up to 8 columns of terms; at the measured copy rate a scheduler has 44 cycles for them, an MMA takes 8 (measured, 4 warps and
// more a scheduler or 4 accumulators and more a warp), so up to two tiles of 8 columns cost nothing.  Warp-level MMAs take the
// operands where dequantisation leaves them, in registers; tcgen05 would have four times the codes' bytes pass shared memory.
#pragma once
#include "device_common.cuh"
#include "elements.cuh"
#include "q4_format.cuh"

namespace strata {
namespace q4 {

constexpr int WARPS = 16;           // of a CTA; one CTA an SM
constexpr int THREADS = 32 * WARPS;
constexpr int SMEM_MAX = 227 * 1024;
constexpr int TILES_MAX = 3;        // tiles of 8 term columns that a warp accumulates at once
constexpr int PART_STRIDE = 20;     // floats between two columns of a warp's sums: 16 rows and 4 against bank conflicts

// ---- activations ------------------------------------------------------------------------------------
// Terms of a type: bf16 holds 8 significant bits, fp16 11, fp32 24.
__host__ __device__ constexpr int terms_of(int type) { return type == STRATA_BF16 ? 1 : type == STRATA_F16 ? 2 : 3; }
// Bytes between rows of `columns` (a multiple of 32) bf16 in shared memory: 64 past a multiple of 128, so that the 16-byte
// operand loads of 8 lanes, 64 bytes of each of two rows, meet all banks once.
__host__ __device__ constexpr int row_bytes(int columns) { return (2 * columns) | 64; }

// Columns i .. i + 7 of a row into `terms` rows of shared memory; behind the last column zeros.
__device__ __forceinline__ void stage8(const void* x, int64_t row0, int i, int columns, int type, int terms, char* dst, int stride) {
  float f[8] = {};
  if (i < columns) widen8(load8(x, row0 + i, type), type, f);
  for (int t = 0; t < terms; ++t) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      w[j] = narrow2(f[2 * j], f[2 * j + 1], STRATA_BF16);
      f[2 * j] -= __uint_as_float(w[j] << 16);  // exact: the rest has fewer bits
      f[2 * j + 1] -= __uint_as_float(w[j] & 0xffff0000u);
    }
    *reinterpret_cast<uint4*>(dst + t * stride) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// ---- copies ------------------------------------------------------------------------------------------
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory"); }
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds4(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}

// ---- products ----------------------------------------------------------------------------------------
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Pair j of a packed word as bf16 code - zero; zero128 holds 128 + zero twice.  0x4300 | code is 128 + code.
__device__ __forceinline__ uint32_t widen_pair(uint32_t w, int j, uint32_t zero128) {
  const uint32_t v = ((w >> (4 * j)) & 0x000f000fu) | 0x43004300u;
  const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v), *reinterpret_cast<const __nv_bfloat162*>(&zero128));
  return *reinterpret_cast<const uint32_t*>(&d);
}
__device__ __forceinline__ float2 scales_of(uint32_t w, bool f16) {
  return f16 ? __half22float2(*reinterpret_cast<const __half2*>(&w))
             : make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// 4-bit weights of groups of GROUP columns: a chunk's bytes in the ring and its products.
template <int GROUP, bool ZEROS>
struct Q4 {
  static constexpr int COLUMNS = CHUNK;
  static constexpr int SB = scale_bytes(GROUP), ZB = ZEROS ? zero_bytes(GROUP) : 0;
  static constexpr int SLOT = 1024 + 32 * (SB + ZB);  // of a warp; scales and zero points once for each lane
  static constexpr int BYTES = chunk_bytes(GROUP, ZEROS);

  const uint8_t* base;  // of the matrix
  int64_t slab;         // bytes of a slab
  int columns;
  bool f16;             // scales are fp16

  __device__ __forceinline__ int blocks(int ch) const { return min(4, columns / BLOCK - 4 * ch); }
  __device__ __forceinline__ void load(uint32_t slot, int64_t s, int ch, int lane) const {
    const uint8_t* p = base + s * slab + (int64_t)ch * BYTES;
    const int nb = blocks(ch), g = lane >> 2;
    if (nb == 4) {
      copy_async<16>(slot + lane * 16, p + lane * 16);
      copy_async<16>(slot + 512 + lane * 16, p + 512 + lane * 16);
    } else {
      for (int b = 0; b < nb; ++b) {
        copy_async<4>(slot + lane * 16 + 4 * b, p + (lane * nb + b) * 4);
        copy_async<4>(slot + 512 + lane * 16 + 4 * b, p + 128 * nb + (lane * nb + b) * 4);
      }
    }
    p += 256 * nb;
    copy_async<SB>(slot + 1024 + lane * SB, p + g * SB);
    if constexpr (ZEROS) copy_async<ZB>(slot + 1024 + 32 * SB + lane * ZB, p + 8 * SB + g * ZB);
  }

  // acc[tile] += slab x columns; b[tile]: the shared address of this lane's operand row at the chunk's first column.
  template <int NT, bool WHOLE>
  __device__ __forceinline__ void products(uint32_t slot, int nb, const uint32_t (&b)[NT], int lane, float (&acc)[NT][4]) const {
    const uint4 lo4 = lds16(slot + lane * 16), hi4 = lds16(slot + 512 + lane * 16);
    const uint32_t lo[4] = {lo4.x, lo4.y, lo4.z, lo4.w}, hi[4] = {hi4.x, hi4.y, hi4.z, hi4.w};
    constexpr int PER = GROUP / BLOCK;
#pragma unroll
    for (int gr = 0; gr < groups_of(GROUP); ++gr) {
      if (!WHOLE && gr * PER >= nb) break;
      const float2 s = scales_of(lds4(slot + 1024 + lane * SB + 4 * gr), f16);
      uint32_t zlo = 0x43084308u, zhi = 0x43084308u;  // zero point 8
      if constexpr (ZEROS) {
        const uint32_t z = lds4(slot + 1024 + 32 * SB + lane * ZB + (gr >> 1) * 4) >> (16 * (gr & 1));
        zlo = (z & 15u) * 0x00010001u | 0x43004300u;
        zhi = (z >> 8 & 15u) * 0x00010001u | 0x43004300u;
      }
      float part[NT][4] = {};
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int k = gr * PER + i;
        if (!WHOLE && k >= nb) break;
        uint32_t alo[4], ahi[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          alo[j] = widen_pair(lo[k], j, zlo);
          ahi[j] = widen_pair(hi[k], j, zhi);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const uint4 x = lds16(b[t] + k * 64);
          mma(part[t], alo[0], ahi[0], alo[1], ahi[1], x.x, x.y);
          mma(part[t], alo[2], ahi[2], alo[3], ahi[3], x.z, x.w);
        }
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        acc[t][0] = fmaf(s.x, part[t][0], acc[t][0]);
        acc[t][1] = fmaf(s.x, part[t][1], acc[t][1]);
        acc[t][2] = fmaf(s.y, part[t][2], acc[t][2]);
        acc[t][3] = fmaf(s.y, part[t][3], acc[t][3]);
      }
    }
  }
};

// bf16 weights, rows as they are: 64 columns of 16 rows a chunk, 16 bytes a lane, row and block of 32 columns.
struct Bf16 {
  static constexpr int COLUMNS = 64;
  static constexpr int SLOT = 2048;

  const uint8_t* base;
  int64_t stride;  // elements
  int columns, rows;

  __device__ __forceinline__ int blocks(int ch) const { return min(2, (columns + BLOCK - 1) / BLOCK - 2 * ch); }
  __device__ __forceinline__ void load(uint32_t slot, int64_t s, int ch, int lane) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // block i / 2, row half i % 2
      const int64_t row = s * ROWS + (lane >> 2) + 8 * (i & 1);
      const int col = ch * COLUMNS + (i >> 1) * BLOCK + (lane & 3) * 8;
      const bool have = row < rows && col < columns;
      const uint8_t* p = have ? base + 2 * (row * stride + col) : base;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(slot + i * 512 + lane * 16), "l"(p), "r"(have ? 16 : 0)
                   : "memory");
    }
  }
  template <int NT, bool WHOLE>
  __device__ __forceinline__ void products(uint32_t slot, int nb, const uint32_t (&b)[NT], int lane, float (&acc)[NT][4]) const {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (!WHOLE && k >= nb) break;
      const uint4 lo = lds16(slot + k * 1024 + lane * 16), hi = lds16(slot + k * 1024 + 512 + lane * 16);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const uint4 x = lds16(b[t] + k * 64);
        mma(acc[t], lo.x, hi.x, lo.y, hi.y, x.x, x.y);
        mma(acc[t], lo.z, hi.z, lo.w, hi.w, x.z, x.w);
      }
    }
  }
};

template <int NT, class W>
__device__ __forceinline__ void chunk_products(const W& w, uint32_t slot, int ch, const uint32_t (&rows)[NT], uint32_t column0,
                                               int lane, float (&acc)[NT][4]) {
  uint32_t b[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) b[t] = rows[t] + column0 * 2;
  const int nb = w.blocks(ch);
  if (nb == W::COLUMNS / BLOCK) w.template products<NT, true>(slot, nb, b, lane, acc);
  else w.template products<NT, false>(slot, nb, b, lane, acc);
}

// A warp's sums to its place in shared memory, [column][16 rows].
template <int NT>
__device__ __forceinline__ void store_part(float* part, int lane, const float (&acc)[NT][4]) {
  const int g = lane >> 2, c = lane & 3;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    float* p = part + (8 * t + 2 * c) * PART_STRIDE + g;
    p[0] = acc[t][0];
    p[PART_STRIDE] = acc[t][1];
    p[8] = acc[t][2];
    p[PART_STRIDE + 8] = acc[t][3];
  }
}
// Row `row` of token j of a block over its terms and the S warps of its group (the first warp's part, parts `step` floats apart).
__device__ __forceinline__ float sum_part(const float* part, int step, int S, int terms, int j, int row) {
  float v = 0.f;
  for (int s = 0; s < S; ++s)
    for (int t = terms - 1; t >= 0; --t) v += part[s * step + (j * terms + t) * PART_STRIDE + row];
  return v;
}

// The S (1, 2, 4, 8 or 16) warps that share a unit meet.
__device__ __forceinline__ void group_sync(int group, int S) {
  if (S == 1) __syncwarp();
  else if (S == WARPS) __syncthreads();
  else named_barrier(1 + group, 32 * S);
}

// Warps to a unit (16 rows x all chunks): the split with the fewest chunks one after the other; equal: fewer warps a unit,
// which leaves fewer sums to join.
__host__ __device__ inline int choose_split(int units_of_cta, int chunks, int most = WARPS) {
  int best = 1, cost = 1 << 30;
  for (int S = 1; S <= WARPS && S <= most; S *= 2) {
    const int groups = WARPS / S;
    const int c = (units_of_cta + groups - 1) / groups * ((chunks + S - 1) / S);
    if (c < cost) best = S, cost = c;
  }
  return best;
}

}  // namespace q4
}  // namespace strata
