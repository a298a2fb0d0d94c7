// What the kernels of strata_moe_linear and strata_moe_q4_experts share: weights streamed through a ring that each warp keeps for itself, codes
// widened in registers, products by warp-level MMAs with terms of the activations.
//
// Mathematics.  y[row] = sum over groups of s[row][group] * (sum over its columns of (code - zero) * x).  code - zero is a whole number of magnitude
// below 16, exact in fp16; x enters as fp16 terms (stage8), each a column of the products, so the products are exact and their sums fp32; the
// scale multiplies a group's fp32 sum, the activations' power of two a chunk's.
// What bounds it: no pipe alone.  16 rows x 128 columns leave a scheduler 190 cycles at the measured copy rate (1 KB of codes; 214 with the scales of
// groups of 32).  Widening takes 5 integer instructions a word of 8 codes (2 cycles each) and 4 subtractions, 8 words a lane: 80 cycles of the
// integer pipe; with scales, sums and copies a chunk comes to 176 instructions, 152 in units of 32 rows (2,560 -> 131,072 rows, one token: 189 MB in 38.2
// and 36.6 us, 5.2 TB/s).  There a chunk takes a scheduler 280 cycles: its four warps issue in 67% of the cycles in which the SM is active, and wait for
// the integer and tensor pipes, for dispatch and for fixed latencies in the others; a fifth of the call is its start and its end.  bf16 operands, with 7 mantissa bits, take 7 integer instructions a word: 57 us.  An MMA takes 8 cycles (measured, with 4 warps a scheduler), 8 of them
// a chunk and tile of 8 columns, so two tiles are hidden.  Warp-level MMAs take the operands where widening leaves them, in registers; tcgen05 would
// have four times the codes' bytes pass shared memory.
// Tried and not kept: codes as e4m3 bytes (a code in the low bits of a byte is code * 2^-9 without further work): mma.sync of e4m3 turns into
// conversions and fp16 MMAs here, 215 instructions a chunk; codes as fp16 subnormals, with the zero point in the MMA's starting value: 157
// instructions, the same time, and more work on x.
#pragma once
#include "device_common.cuh"
#include "elements.cuh"
#include "q4_format.cuh"

namespace strata {
namespace q4 {

// ---- activations ------------------------------------------------------------------------------------
// How x enters the products.  Beside 4-bit codes: fp16 terms of x divided by a power of two for each token and chunk of 128 columns, so
// that the largest lies in [2^14, 2^15); one term holds all bits of a bf16 or fp16 (down to 2^-40 of the chunk's largest), two hold 22 of an
// fp32's 24.  Beside bf16 weights: bf16 terms as they are, 8 bits each.
__host__ __device__ constexpr int terms_of(int type, bool f16) {
  return type == STRATA_BF16 ? 1 : type == STRATA_F16 ? (f16 ? 1 : 2) : (f16 ? 2 : 3);
}

// The place in shared memory of CTA `peer` of the cluster where this CTA has p.
__device__ __forceinline__ uint32_t peer_address(const void* p, int peer) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(peer));
  return at;
}
// All threads of the cluster meet, and see what was stored to one another's shared memory.
__device__ __forceinline__ void cluster_meet() {
  __syncwarp();  // .aligned: all lanes together
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Eight columns, first i of a row, into `terms` rows at dst; F16: after their chunk's power of two, which goes to *scale.  By the 16 lanes of
// a chunk; in: they are columns of x, else zeros; store: they are laid out.  PAIR: to the same places of CTA `peer` too.
// The terms unrolled: 64 tokens to a router's 512, three terms each, 11.0 us with a loop and 9.9 without.
template <bool F16, bool PAIR>
__device__ __forceinline__ void stage8(const Raw8& raw, int type, bool in, bool store, int terms, char* dst, int stride, float* scale, int peer) {
  float f[8] = {};
  if (in) widen8(raw, type, f);
  if (F16) {
    float most = 0.f;  // a NaN counts for nothing here and stays one
#pragma unroll
    for (int j = 0; j < 8; ++j) most = fmaxf(most, fabsf(f[j]));
    const uint32_t top = __reduce_max_sync(0xffffu << (threadIdx.x & 16), __float_as_uint(most));
    const uint32_t e = max(top >> 23, 15u);  // 2^(e - 127) <= largest; below 2^-112 all count as 2^-112
    const float up = __uint_as_float((268u - e) << 23);
    if ((threadIdx.x & 15) == 0) {
      *scale = __uint_as_float((e - 14u) << 23);
      if (PAIR) asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(peer_address(scale, peer)), "r"((e - 14u) << 23) : "memory");
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] *= up;
  }
  if (!store) return;
#pragma unroll
  for (int t = 0; t < (F16 ? 2 : 3); ++t) {
    if (t == terms) break;
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = narrow2(f[2 * j], f[2 * j + 1], F16 ? STRATA_F16 : STRATA_BF16);
    *reinterpret_cast<uint4*>(dst + t * stride) = make_uint4(w[0], w[1], w[2], w[3]);
    if (PAIR)
      asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(peer_address(dst + t * stride, peer)), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                   "r"(w[3])
                   : "memory");
    if (t + 1 == terms) break;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 v = widen2(w[j], F16 ? STRATA_F16 : STRATA_BF16);
      f[2 * j] -= v.x;  // exact: the rest has fewer bits
      f[2 * j + 1] -= v.y;
    }
  }
}
// Columns c0 .. c1 - 1 (c0 a multiple of 128, c1 of 32) of n rows of x as `terms` rows each at dst; behind the last column zeros.  Nothing is stored
// behind c1, where the next row begins.
// Row j is x's row j, or row index[j] / d (inverse: of d, see divide) where there is an index.  By `halves` half warps, this one `half`, a chunk of
// a row each, four of them asked for at once.  PAIR: see stage8.
struct StageArgs {
  const void* x;
  int64_t x_stride;
  int type, columns, terms;
  char* rows;
  int row_stride;
  float* scale;
  int scale_stride;
  const uint16_t* index;
  uint32_t inverse;
  int peer;  // PAIR: the CTA of the cluster that gets the same rows
};
// n / d by inverse = ceil(2^32 / d), or 0 for d = 1; exact while n * d < 2^32.
__device__ __forceinline__ int divide(int n, uint32_t inverse) { return inverse ? __umulhi(n, inverse) : n; }
inline uint32_t inverse_of(int d) { return d == 1 ? 0 : (uint32_t)(((1ull << 32) + d - 1) / d); }

template <bool F16, bool PAIR = false>
__device__ __noinline__ void stage_rows(const StageArgs s, int n, int c0, int c1, int half, int halves) {
  constexpr int AHEAD = 4;
  const int lane = threadIdx.x & 15, last = min(s.columns, c1), chunks = (c1 - c0 + CHUNK - 1) / CHUNK;
  const uint32_t chunks_inverse = chunks == 1 ? 0u : 0xffffffffu / (uint32_t)chunks + 1u;  // inverse_of(chunks); n * chunks^2 stays far below 2^32
  for (int first = half; first < n * chunks; first += AHEAD * halves) {
    Raw8 raw[AHEAD];
    int row[AHEAD], at[AHEAD];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      const int task = first + u * halves;
      row[u] = divide(task, chunks_inverse);
      at[u] = (task - row[u] * chunks) * CHUNK + lane * 8;
      raw[u] = Raw8{};
      if (row[u] < n && c0 + at[u] < last) {
        const int from = s.index ? divide(s.index[row[u]], s.inverse) : row[u];
        raw[u] = load8(s.x, from * s.x_stride + c0 + at[u], s.type);
      }
    }
#pragma unroll
    for (int u = 0; u < AHEAD; ++u)
      if (row[u] < n)
        stage8<F16, PAIR>(raw[u], s.type, c0 + at[u] < last, c0 + at[u] < c1, s.terms, s.rows + row[u] * s.terms * s.row_stride + at[u] * 2,
                    s.row_stride, s.scale + row[u] * s.scale_stride + at[u] / CHUNK, s.peer);
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
template <bool F16>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same on a sum of 0, fp16 operands.
__device__ __forceinline__ void mma_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t sub2(uint32_t a, uint32_t b) {
  const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&d);
}
// (w & mask) | set, in one instruction: written out, since the compiler makes two of two constants.
__device__ __forceinline__ uint32_t mask_set(uint32_t w, uint32_t mask, uint32_t set) {
  uint32_t v;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(v) : "r"(w), "r"(mask), "r"(set));
  return v;
}
// A packed word as four pairs of fp16 code - zero.  In the mantissa of fp16, 0x6400 | code is 1024 + code and 0x5400 | code << 4 is
// 64 + code, so two pairs of nibbles need no shift; z0 holds 1024 + zero twice, z1 64 + zero.
__device__ __forceinline__ void widen_word(uint32_t w, uint32_t z0, uint32_t z1, uint32_t (&a)[4]) {
  const uint32_t v = w >> 8;
  a[0] = sub2(mask_set(w, 0x000f000fu, 0x64006400u), z0);
  a[1] = sub2(mask_set(w, 0x00f000f0u, 0x54005400u), z1);
  a[2] = sub2(mask_set(v, 0x000f000fu, 0x64006400u), z0);
  a[3] = sub2(mask_set(v, 0x00f000f0u, 0x54005400u), z1);
}

// z0 and z1 of rows g (byte 0 of z) and g + 8 (byte 1).
__device__ __forceinline__ void zero_pairs(uint32_t z, uint32_t& z0lo, uint32_t& z1lo, uint32_t& z0hi, uint32_t& z1hi) {
  const uint32_t l = (z & 15u) * 0x00010001u, h = (z >> 8 & 15u) * 0x00010001u;
  z0lo = l | 0x64006400u, z1lo = l << 4 | 0x54005400u;
  z0hi = h | 0x64006400u, z1hi = h << 4 | 0x54005400u;
}

// 4-bit weights of groups of GROUP columns, units of SLABS (1 or 2) slabs: their chunk's bytes in the ring and its products.
template <int GROUP, bool ZEROS, bool SCALE_F16, int SLABS_ = 1>
struct Q4 {
  static constexpr bool F16 = true;  // the products' operands
  static constexpr int SLABS = SLABS_;
  static constexpr int COLUMNS = CHUNK;
  static constexpr int SB = scale_bytes(GROUP), ZB = ZEROS ? zero_bytes(GROUP) : 0;
  static constexpr int META = meta_bytes(GROUP, ZEROS);
  static constexpr int ONE = 1024 + META;  // of a slab
  static constexpr int SLOT = SLABS * ONE;
  static constexpr int BYTES = chunk_bytes(GROUP, ZEROS);

  struct Cursor {  // this lane's part of a chunk
    const uint8_t* at;
    int64_t second;  // bytes to the second slab's (0 behind the last slab: the first again, and its results are not used)
  };
  const uint8_t* base;  // of the matrix
  int64_t slab;         // bytes of a slab
  int slabs;

  __device__ __forceinline__ Cursor cursor(int64_t unit, int ch, int lane) const {
    return {base + unit * SLABS * slab + ch * BYTES + lane * 16, SLABS == 2 && unit * 2 + 1 < slabs ? slab : 0};
  }
  static __device__ __forceinline__ void load(uint32_t slot, const Cursor& c, int lane) {
#pragma unroll
    for (int h = 0; h < SLABS; ++h) {
      const uint8_t* p = h ? c.at + c.second : c.at;
      copy_async<16>(slot + h * ONE + lane * 16, p);
      copy_async<16>(slot + h * ONE + 512 + lane * 16, p + 512);
      if (lane < META / 16) copy_async<16>(slot + h * ONE + 1024 + lane * 16, p + 1024);
    }
  }
  // A last chunk of `left` (32, 64 or 96) columns.
  static __device__ __forceinline__ void load_tail(uint32_t slot, const Cursor& c, int left, int lane) {
    const int nb = left / BLOCK;
#pragma unroll 1
    for (int h = 0; h < SLABS; ++h) {
      const uint8_t* p = c.at - lane * 16 + (h ? c.second : 0);
      const uint32_t to = slot + h * ONE;
#pragma unroll 1
      for (int b = 0; b < nb; ++b) {
        copy_async<4>(to + lane * 16 + 4 * b, p + (lane * nb + b) * 4);
        copy_async<4>(to + 512 + lane * 16 + 4 * b, p + 128 * nb + (lane * nb + b) * 4);
      }
      if (lane < META / 16) copy_async<16>(to + 1024 + lane * 16, p + 256 * nb + lane * 16);
    }
  }
  static __device__ __forceinline__ float2 scales_of(uint32_t w) { return widen2(w, SCALE_F16 ? STRATA_F16 : STRATA_BF16); }

  // acc[slab * NT + tile] += chunk x columns.  b[tile]: shared address of this lane's operand row at the chunk's first column; cs[tile]: the powers
  // of two of this lane's two result columns in this chunk.  An operand of x is loaded once for all slabs.
  template <int NT>
  static __device__ __forceinline__ void products(uint32_t slot, const uint32_t (&b)[NT], const float2 (&cs)[NT], int lane,
                                                  float (&acc)[SLABS * NT][4]) {
    const int g = lane >> 2;
    uint32_t codes[SLABS][8], scales[SLABS][4], zeros[SLABS][2];
#pragma unroll
    for (int h = 0; h < SLABS; ++h) {
      const uint32_t at = slot + h * ONE;
      const uint4 lo = lds16(at + lane * 16), hi = lds16(at + 512 + lane * 16);
      codes[h][0] = lo.x, codes[h][1] = lo.y, codes[h][2] = lo.z, codes[h][3] = lo.w;
      codes[h][4] = hi.x, codes[h][5] = hi.y, codes[h][6] = hi.z, codes[h][7] = hi.w;
      if constexpr (SB == 16) {
        const uint4 v = lds16(at + 1024 + g * 16);
        scales[h][0] = v.x, scales[h][1] = v.y, scales[h][2] = v.z, scales[h][3] = v.w;
      } else {
#pragma unroll
        for (int i = 0; i < SB / 4; ++i) scales[h][i] = lds4(at + 1024 + g * SB + 4 * i);
      }
      if constexpr (ZEROS) {
#pragma unroll
        for (int i = 0; i < ZB / 4; ++i) zeros[h][i] = lds4(at + 1024 + 8 * SB + g * ZB + 4 * i);
      }
    }
    constexpr int PER = GROUP / BLOCK;
    float sum[SLABS * NT][4] = {};
#pragma unroll
    for (int gr = 0; gr < groups_of(GROUP); ++gr) {
      float part[SLABS * NT][4];
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int k = gr * PER + i;
        uint4 x[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) x[t] = lds16(b[t] + k * 64);
#pragma unroll
        for (int h = 0; h < SLABS; ++h) {
          uint32_t z0lo = 0x64086408u, z1lo = 0x54805480u, z0hi = z0lo, z1hi = z1lo;  // zero point 8
          if constexpr (ZEROS) zero_pairs(zeros[h][gr >> 1] >> (16 * (gr & 1)), z0lo, z1lo, z0hi, z1hi);
          uint32_t alo[4], ahi[4];
          widen_word(codes[h][k], z0lo, z1lo, alo);
          widen_word(codes[h][4 + k], z0hi, z1hi, ahi);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            float(&d)[4] = part[h * NT + t];
            if (i == 0) mma_first(d, alo[0], ahi[0], alo[1], ahi[1], x[t].x, x[t].y);
            else mma<true>(d, alo[0], ahi[0], alo[1], ahi[1], x[t].x, x[t].y);
            mma<true>(d, alo[2], ahi[2], alo[3], ahi[3], x[t].z, x[t].w);
          }
        }
      }
#pragma unroll
      for (int h = 0; h < SLABS; ++h) {
        const float2 s = scales_of(scales[h][gr]);
#pragma unroll
        for (int t = h * NT; t < (h + 1) * NT; ++t) {
          sum[t][0] = fmaf(s.x, part[t][0], sum[t][0]);
          sum[t][1] = fmaf(s.x, part[t][1], sum[t][1]);
          sum[t][2] = fmaf(s.y, part[t][2], sum[t][2]);
          sum[t][3] = fmaf(s.y, part[t][3], sum[t][3]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < SLABS * NT; ++i) {
      const float2 c = cs[i % NT];
      acc[i][0] = fmaf(c.x, sum[i][0], acc[i][0]);
      acc[i][1] = fmaf(c.y, sum[i][1], acc[i][1]);
      acc[i][2] = fmaf(c.x, sum[i][2], acc[i][2]);
      acc[i][3] = fmaf(c.y, sum[i][3], acc[i][3]);
    }
  }

  // The same for a last chunk of nb (1 to 3) blocks, block by block.
  template <int NT>
  static __device__ __forceinline__ void tail(uint32_t slot, int nb, const uint32_t (&b)[NT], const float2 (&cs)[NT], int lane,
                                              float (&acc)[SLABS * NT][4]) {
    const int g = lane >> 2;
#pragma unroll 1
    for (int k = 0; k < nb; ++k) {
      const int gr = k * BLOCK / GROUP;
#pragma unroll
      for (int h = 0; h < SLABS; ++h) {
        const uint32_t at = slot + h * ONE;
        const float2 s = scales_of(lds4(at + 1024 + g * SB + 4 * gr));
        uint32_t z0lo = 0x64086408u, z1lo = 0x54805480u, z0hi = z0lo, z1hi = z1lo;
        if constexpr (ZEROS) zero_pairs(lds4(at + 1024 + 8 * SB + g * ZB + 4 * (gr >> 1)) >> (16 * (gr & 1)), z0lo, z1lo, z0hi, z1hi);
        uint32_t alo[4], ahi[4];
        widen_word(lds4(at + lane * 16 + 4 * k), z0lo, z1lo, alo);
        widen_word(lds4(at + 512 + lane * 16 + 4 * k), z0hi, z1hi, ahi);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const uint4 x = lds16(b[t] + k * 64);
          float part[4];
          mma_first(part, alo[0], ahi[0], alo[1], ahi[1], x.x, x.y);
          mma<true>(part, alo[2], ahi[2], alo[3], ahi[3], x.z, x.w);
          float(&d)[4] = acc[h * NT + t];
          d[0] = fmaf(cs[t].x * s.x, part[0], d[0]);
          d[1] = fmaf(cs[t].y * s.x, part[1], d[1]);
          d[2] = fmaf(cs[t].x * s.y, part[2], d[2]);
          d[3] = fmaf(cs[t].y * s.y, part[3], d[3]);
        }
      }
    }
  }
};

// bf16 weights, rows as they are: 64 columns of 16 rows a chunk, 16 bytes a lane, row and block of 32 columns.
struct Bf16 {
  static constexpr bool F16 = false;
  static constexpr int SLABS = 1;
  static constexpr int COLUMNS = 64;
  static constexpr int SLOT = 2048;
  static constexpr int BYTES = 2 * COLUMNS;

  struct Cursor {
    const uint8_t* at;
    int64_t eight;  // to the row 8 further
  };
  const uint8_t* base;
  int64_t stride;  // elements
  int rows;

  __device__ __forceinline__ Cursor cursor(int64_t s, int ch, int lane) const {
    // rows behind the last read another, and their results are not used
    const int64_t row = s * ROWS + (lane >> 2);
    return {base + 2 * ((row < rows ? row : 0) * stride) + ch * BYTES + (lane & 3) * 16, row + 8 < rows ? 16 * stride : 0};
  }
  static __device__ __forceinline__ void load(uint32_t slot, const Cursor& c, int lane) {
    copy_async<16>(slot + lane * 16, c.at);
    copy_async<16>(slot + 512 + lane * 16, c.at + c.eight);
    copy_async<16>(slot + 1024 + lane * 16, c.at + 64);
    copy_async<16>(slot + 1536 + lane * 16, c.at + c.eight + 64);
  }
  // A last chunk of `left` (8 .. 56) columns; behind them zeros.
  static __device__ __forceinline__ void load_tail(uint32_t slot, const Cursor& c, int left, int lane) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // block i / 2, row half i % 2
      const bool have = (i >> 1) * BLOCK + (lane & 3) * 8 < left;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(slot + i * 512 + lane * 16),
                   "l"(have ? c.at + (i & 1 ? c.eight : 0) + (i >> 1) * 64 : c.at - (lane & 3) * 16), "r"(have ? 16 : 0)
                   : "memory");
    }
  }
  template <int NT>
  static __device__ __forceinline__ void products(uint32_t slot, const uint32_t (&b)[NT], const float2 (&)[NT], int lane,
                                                  float (&acc)[NT][4]) {
    block<NT>(slot, 0, b, lane, acc);
    block<NT>(slot, 1, b, lane, acc);
  }
  template <int NT>
  static __device__ __forceinline__ void tail(uint32_t slot, int nb, const uint32_t (&b)[NT], const float2 (&)[NT], int lane,
                                              float (&acc)[NT][4]) {
    for (int k = 0; k < nb; ++k) block<NT>(slot, k, b, lane, acc);
  }
  template <int NT>
  static __device__ __forceinline__ void block(uint32_t slot, int k, const uint32_t (&b)[NT], int lane, float (&acc)[NT][4]) {
    const uint4 lo = lds16(slot + k * 1024 + lane * 16), hi = lds16(slot + k * 1024 + 512 + lane * 16);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const uint4 x = lds16(b[t] + k * 64);
      mma<false>(acc[t], lo.x, hi.x, lo.y, hi.y, x.x, x.y);
      mma<false>(acc[t], lo.z, hi.z, lo.w, hi.w, x.z, x.w);
    }
  }
};

// A value that all lanes of the warp hold, as one that the compiler knows they do (a reduction's result).
__device__ __forceinline__ int uniform(int v) { return __reduce_min_sync(0xffffffffu, v); }
__device__ __forceinline__ int warp_index() { return uniform(threadIdx.x >> 5); }

// A warp's share of a unit: chunks member, member + S, ...; the last of the unit may be a shorter one.
struct Share {
  int whole;  // its whole chunks
  int tail;   // columns of its shorter one, or 0
  __device__ __forceinline__ Share(int columns, int chunk, int member, int log_split) {
    const int S = 1 << log_split, wholes = columns / chunk;
    whole = wholes > member ? (wholes - member + S - 1) >> log_split : 0;
    tail = (wholes & (S - 1)) == member ? columns - wholes * chunk : 0;
  }
};

// A warp's ring of DEPTH chunks of SLOT bytes, filled DEPTH - 1 ahead: one group of copies a chunk used, empty when none is left.
// U walks the warp's units: next() sets out for the next one and tells whether there is one; its cursor, whole and tail are then taken from it.
template <class W, int DEPTH, class U>
struct Feed {
  U units;
  uint32_t ring, used;  // shared addresses: of the ring, of the slot that was used last and is filled next
  typename W::Cursor cursor;
  int left, tail, stride;  // of the unit: whole chunks and columns of a shorter one to copy; bytes from one chunk of this warp to its next
  int lane;
  bool more;  // units, as far as is known

  __device__ __forceinline__ Feed(const U& u, uint32_t at, int l) : units(u), ring(at), used(at), left(0), tail(0), lane(l), more(true) {
#pragma unroll 1
    for (int i = 0; i < DEPTH - 1; ++i) {
      fill();
      used += W::SLOT;
    }
  }
  __device__ __forceinline__ void fill() {
    if (left == 0) {  // a shorter chunk, or on to the next unit
      if (tail == 0 && more) {
        more = units.next();
        if (more) cursor = units.cursor, left = units.whole, tail = units.tail, stride = units.stride;
      }
      if (left == 0 && tail) {
        W::load_tail(used, cursor, tail, lane);
        tail = 0;
      }
    }
    if (left) {
      W::load(used, cursor, lane);
      cursor.at += stride;
      --left;
    }
    copy_commit();
  }
  // The next chunk's slot, once it is there.
  __device__ __forceinline__ uint32_t take() {
    copy_wait<DEPTH - 2>();
    __syncwarp();  // its scales were copied by other lanes; and all have read the slot that is filled now
    fill();
    used = used == ring + (DEPTH - 1) * W::SLOT ? ring : used + W::SLOT;
    return used;
  }
};

// Products of a warp's next `whole` chunks, then of one of `tail` columns.  b[tile] and cs[tile] are this lane's shared addresses for the
// activations of the first of them; one chunk of this warp to the next is S of the unit's.
template <int NT, class W, class F>
__device__ __forceinline__ void run_chunks(F& feed, int whole, int tail, int S, uint32_t (&b)[NT], uint2 (&cs)[NT],
                                           float (&acc)[W::SLABS * NT][4]) {
  auto scales = [&](float2 (&v)[NT]) {
#pragma unroll
    for (int t = 0; t < NT; ++t)
      if (W::F16) v[t] = make_float2(__uint_as_float(lds4(cs[t].x)), __uint_as_float(lds4(cs[t].y)));
  };
  float2 v[NT];
#pragma unroll 1
  for (int i = 0; i < whole; ++i) {
    const uint32_t slot = feed.take();
    scales(v);
    W::template products<NT>(slot, b, v, feed.lane, acc);
#pragma unroll
    for (int t = 0; t < NT; ++t) b[t] += S * 2 * W::COLUMNS, cs[t].x += 4 * S, cs[t].y += 4 * S;
  }
  if (tail) {
    const uint32_t slot = feed.take();
    scales(v);
    W::template tail<NT>(slot, (tail + BLOCK - 1) / BLOCK, b, v, feed.lane, acc);
  }
}
// A warp's sums to its place in shared memory, [column][rows of the unit].
template <int NT, int SLABS>
__device__ __forceinline__ void store_part(float* part, int lane, const float (&acc)[SLABS * NT][4]) {
  const int g = lane >> 2, c = lane & 3;
  constexpr int STRIDE = part_stride(SLABS);
#pragma unroll
  for (int i = 0; i < SLABS * NT; ++i) {
    float* p = part + (8 * (i % NT) + 2 * c) * STRIDE + i / NT * ROWS + g;
    p[0] = acc[i][0];
    p[STRIDE] = acc[i][1];
    p[8] = acc[i][2];
    p[STRIDE + 8] = acc[i][3];
  }
}
// Row `row` of token j of a block over its terms and the S warps of its group (the first warp's part, parts `step` floats apart).
template <int SLABS>
__device__ __forceinline__ float sum_part(const float* part, int step, int S, int terms, int j, int row) {
  float v = 0.f;
  for (int s = 0; s < S; ++s)
    for (int t = terms - 1; t >= 0; --t) v += part[s * step + (j * terms + t) * part_stride(SLABS) + row];
  return v;
}

// The S (a power of two up to WARPS) warps that share a unit meet.
template <int WARPS>
__device__ __forceinline__ void group_sync(int group, int S) {
  if (S == 1) __syncwarp();
  else if (S == WARPS) __syncthreads();
  else named_barrier(1 + group, 32 * S);
}

}  // namespace q4
}  // namespace strata
