// Low-rank adapters of many requests beside a shared projection (strata_moe_adapters), sm_103a:
//   y[t] = base[t] + scale[a] * B_a (A_a x[t]),  a the adapter of t's segment.
// Two kernels: shrink, v = A_a x (partial sums over slices of d_in, kept apart in the workspace and added in a
// fixed order), and expand, base + B_a (scale v).  Both walk tiles of up to 16 MT tokens of one segment; the products
// are warp-level bf16 MMAs with fp32 accumulators.  A wider activation is the exact sum of bf16 terms (an fp16 two, an
// fp32 three), each multiplied on its own.
#include <atomic>

#include "device_common.cuh"
#include "elements.cuh"
#include "tc_common.cuh"

namespace strata {
namespace {

constexpr int AD_WARPS = 8;
constexpr int AD_THREADS = 32 * AD_WARPS;
constexpr int SPLIT_MAX = 8;           // slices of d_in
constexpr int V_FLOATS = 1024;         // scratch per token: SPLIT_MAX * rank <= 1024

struct AdapterArgs {
  const uint16_t* a;
  const uint16_t* b;
  const float* scale;
  int64_t a_stride, b_stride, x_stride, base_stride, y_stride;
  const int32_t* seg_off;
  const int32_t* seg_adapter;
  const void* x;
  const void* base;
  void* y;
  float* v;  // [split][T][rank]
  int* status;
  int n_seg, n_adapter, rank, d_in, d_out, T, x_type, y_type, split, k_slice;
};

struct Tile {
  int row, rows, adapter;
};

// Tile number `want` of the segments cut into tiles of `height` tokens, found by the whole CTA; false if there is
// none or the segments are not valid (recorded in the status word).  Every CTA checks all segments, so either all
// work or none does.
__device__ bool find_tile(const AdapterArgs& a, int want, int height, Tile* out) {
  __shared__ int s_warp[AD_WARPS];
  __shared__ int s_tile[3];
  __shared__ int s_bad;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    s_bad = 0;
    s_tile[1] = 0;
  }
  __syncthreads();
  const int per = (a.n_seg + AD_THREADS - 1) / AD_THREADS;
  const int s0 = min(tid * per, a.n_seg), s1 = min(s0 + per, a.n_seg);
  int count = 0;
  bool bad = false;
  for (int s = s0; s < s1; ++s) {
    const int lo = __ldg(a.seg_off + s), hi = __ldg(a.seg_off + s + 1), ad = __ldg(a.seg_adapter + s);
    if (lo < 0 || hi < lo || hi > a.T || ad < -1 || ad >= a.n_adapter) {
      bad = true;
      break;
    }
    count += (hi - lo + height - 1) / height;
  }
  if (bad) s_bad = 1;
  int v = count;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int n = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += n;
  }
  if (lane == 31) s_warp[warp] = v;
  __syncthreads();
  if (s_bad) {
    if (tid == 0) set_status(a.status, ST_CORRUPT);
    return false;
  }
  int at = v - count;  // tiles before this thread's segments
  for (int w = 0; w < warp; ++w) at += s_warp[w];
  if (want >= at && want < at + count) {
    for (int s = s0; s < s1; ++s) {
      const int lo = __ldg(a.seg_off + s), hi = __ldg(a.seg_off + s + 1);
      const int n = (hi - lo + height - 1) / height;
      if (want < at + n) {
        s_tile[0] = lo + (want - at) * height;
        s_tile[1] = min(height, hi - s_tile[0]);
        s_tile[2] = __ldg(a.seg_adapter + s);
        break;
      }
      at += n;
    }
  }
  __syncthreads();
  *out = Tile{s_tile[0], s_tile[1], s_tile[2]};
  return out->rows > 0;
}

// D (16 x 8, fp32) += A (16 x 16, bf16) * B (16 x 8, bf16).
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// f as TERMS bf16 terms whose sum it is (to 8 TERMS bits), eight values at a time: term i in t[i], two values a word.
template <int TERMS>
__device__ __forceinline__ void split8(float (&f)[8], uint32_t (&t)[TERMS][4]) {
#pragma unroll
  for (int i = 0; i < TERMS; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      t[i][q] = narrow2(f[2 * q], f[2 * q + 1], STRATA_BF16);
      if (i + 1 < TERMS) {
        f[2 * q] -= __uint_as_float(t[i][q] << 16);
        f[2 * q + 1] -= __uint_as_float(t[i][q] & 0xffff0000u);
      }
    }
}

// Both kernels read operands straight into MMA fragments, 16 bytes a thread.  An MMA's k index may be permuted as long as
// A and B agree: of 32 consecutive k, the thread of quarter q (lane & 3) takes the 8 at 8 q, as k 2q, 2q+1, 2q+8, 2q+9 of
// two MMAs; so four lanes read 64 contiguous bytes of a row.

// v[slice][token][r] = sum over the slice's k of A_a[r][k] x[token][k].  CTA: one tile, one slice; its warps take 32
// k each in turn and their sums are added in warp order.
template <int NT, int MT, int TERMS>
__global__ void __launch_bounds__(AD_THREADS) shrink_kernel(AdapterArgs a) {
  __shared__ float s_v[16 * MT * NT * 8];
  Tile tile;
  griddep_launch_dependents();
  griddep_wait();
  if (!find_tile(a, blockIdx.x, 16 * MT, &tile) || tile.adapter < 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int r0 = blockIdx.z * NT * 8;
  const uint16_t* A = a.a + (int64_t)tile.adapter * a.a_stride;
  const int k0 = blockIdx.y * a.k_slice, k1 = min(a.d_in, k0 + a.k_slice);
  float acc[MT][NT][4];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.f;
  const Raw8 zero{make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
  for (int k = k0 + 32 * warp + 8 * q; k - 8 * q < k1; k += 32 * AD_WARPS) {
    const bool in = k < k1;
    uint4 w[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = r0 + 8 * n + g;
      w[n] = in && r < a.rank ? __ldg(reinterpret_cast<const uint4*>(A + (int64_t)r * a.d_in + k)) : zero.lo;
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      uint32_t t0[TERMS][4], t1[TERMS][4];
      const int row0 = 16 * m + g, row1 = row0 + 8;
      const Raw8 x0 = in && row0 < tile.rows ? load8(a.x, (int64_t)(tile.row + row0) * a.x_stride + k, a.x_type) : zero;
      const Raw8 x1 = in && row1 < tile.rows ? load8(a.x, (int64_t)(tile.row + row1) * a.x_stride + k, a.x_type) : zero;
      if constexpr (TERMS == 1) {
        t0[0][0] = x0.lo.x; t0[0][1] = x0.lo.y; t0[0][2] = x0.lo.z; t0[0][3] = x0.lo.w;
        t1[0][0] = x1.lo.x; t1[0][1] = x1.lo.y; t1[0][2] = x1.lo.z; t1[0][3] = x1.lo.w;
      } else {
        float f[8];
        widen8(x0, a.x_type, f);
        split8<TERMS>(f, t0);
        widen8(x1, a.x_type, f);
        split8<TERMS>(f, t1);
      }
#pragma unroll
      for (int i = TERMS - 1; i >= 0; --i) {
        const uint32_t a0[4] = {t0[i][0], t1[i][0], t0[i][1], t1[i][1]};
        const uint32_t a1[4] = {t0[i][2], t1[i][2], t0[i][3], t1[i][3]};
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          mma_bf16(acc[m][n], a0, w[n].x, w[n].y);
          mma_bf16(acc[m][n], a1, w[n].z, w[n].w);
        }
      }
    }
  }
  for (int i = threadIdx.x; i < 16 * MT * NT * 8; i += AD_THREADS) s_v[i] = 0.f;
  for (int w = 0; w < AD_WARPS; ++w) {
    __syncthreads();
    if (w != warp) continue;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) s_v[(16 * m + g + 8 * (i >> 1)) * (NT * 8) + 8 * n + 2 * q + (i & 1)] += acc[m][n][i];
  }
  __syncthreads();
  const int cols = min(NT * 8, a.rank - r0);
  float* v = a.v + ((int64_t)blockIdx.y * a.T + tile.row) * a.rank + r0;
  for (int i = threadIdx.x; i < tile.rows * NT * 8; i += AD_THREADS) {
    const int row = i / (NT * 8), c = i % (NT * 8);
    if (c < cols) v[(int64_t)row * a.rank + c] = s_v[i];
  }
}

// y = base + B_a (scale v).  CTA: one tile, a share of the columns; a warp takes 32 columns at a time, all tokens of the
// tile.  Columns may be permuted over the MMAs' n as k above: the thread of quarter q ends with 8 consecutive columns of
// a row (column 8 q + 2 j + i from MMA j), which it reads and writes 16 bytes at a time.
template <int MT, int TERMS>
__global__ void __launch_bounds__(AD_THREADS) expand_kernel(AdapterArgs a) {
  Tile tile;
  griddep_launch_dependents();
  griddep_wait();
  if (!find_tile(a, blockIdx.x, 16 * MT, &tile)) return;
  if (tile.adapter < 0 && a.base == a.y) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const uint16_t* B = a.b + (int64_t)max(tile.adapter, 0) * a.b_stride;
  const float sc = a.scale && tile.adapter >= 0 ? __ldg(a.scale + tile.adapter) : 1.f;
  const int rank = tile.adapter >= 0 ? a.rank : 0;
  for (int c0 = 32 * (blockIdx.y * AD_WARPS + warp); c0 < a.d_out; c0 += 32 * AD_WARPS * gridDim.y) {
    float acc[MT][4][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][j][i] = 0.f;
    for (int k = 8 * q; k - 8 * q < rank; k += 32) {
      uint4 w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = c0 + 8 * (g >> 1) + 2 * j + (g & 1);
        w[j] = k < rank && c < a.d_out ? __ldg(reinterpret_cast<const uint4*>(B + (int64_t)c * rank + k))
                                       : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        uint32_t t[2][TERMS][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int row = 16 * m + g + 8 * h;
          float f[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] = 0.f;
          if (k < rank && row < tile.rows)
            for (int s = 0; s < a.split; ++s) {
              const float4* p = reinterpret_cast<const float4*>(a.v + ((int64_t)s * a.T + tile.row + row) * rank + k);
              const float4 u0 = __ldcg(p), u1 = __ldcg(p + 1);
              f[0] += u0.x; f[1] += u0.y; f[2] += u0.z; f[3] += u0.w;
              f[4] += u1.x; f[5] += u1.y; f[6] += u1.z; f[7] += u1.w;
            }
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] *= sc;
          split8<TERMS>(f, t[h]);
        }
#pragma unroll
        for (int i = TERMS - 1; i >= 0; --i) {
          const uint32_t a0[4] = {t[0][i][0], t[1][i][0], t[0][i][1], t[1][i][1]};
          const uint32_t a1[4] = {t[0][i][2], t[1][i][2], t[0][i][3], t[1][i][3]};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            mma_bf16(acc[m][j], a0, w[j].x, w[j].y);
            mma_bf16(acc[m][j], a1, w[j].z, w[j].w);
          }
        }
      }
    }
    const int c = c0 + 8 * q;
    if (c >= a.d_out) continue;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = 16 * m + g + 8 * h;
        if (row >= tile.rows) continue;
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = 0.f;
        if (a.base) widen8(load8(a.base, (int64_t)(tile.row + row) * a.base_stride + c, a.y_type), a.y_type, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] += acc[m][i >> 1][2 * h + (i & 1)];
        store8(a.y, (int64_t)(tile.row + row) * a.y_stride + c, a.y_type, f);
      }
  }
}

// ---- Tiles of up to 128 tokens on the 5th-generation tensor cores -----------------------------------------
// Operands go through registers into the tensor cores' K-major shared-memory layout, 16 bytes a thread, so that one kernel
// serves all three types (a wider activation leaves as its bf16 terms) and any row stride.  TMEM is allocated after
// griddep_wait and before the next kernel may start, so no CTA holds it while it waits for another.
constexpr int TC_ROWS = 128;
constexpr uint32_t TC_TILE = TC_ROWS * 128;  // 128 rows of 64 bf16

__host__ __device__ __forceinline__ uint32_t idesc_bf16(int M, int N) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// A wait that ran out is recorded; the CTA's later waits are then skipped (the call's result is void).
struct Waiter {
  int* status;
  volatile int* dead;
  __device__ __forceinline__ void wait(uint64_t* bar, uint32_t parity) const {
    if (!*dead && !mbar_wait(bar, parity, status)) *dead = 1;
  }
};

// The eight values of a 16-byte (fp32: 32-byte) piece as TERMS bf16 pieces.
template <int TERMS>
__device__ __forceinline__ void put_terms(const Raw8& r, int type, uint8_t* tile, uint32_t tile_step, uint32_t off) {
  if constexpr (TERMS == 1) {
    *reinterpret_cast<uint4*>(tile + off) = r.lo;
  } else {
    float f[8];
    uint32_t t[TERMS][4];
    widen8(r, type, f);
    split8<TERMS>(f, t);
#pragma unroll
    for (int i = 0; i < TERMS; ++i)
      *reinterpret_cast<uint4*>(tile + i * tile_step + off) = make_uint4(t[i][0], t[i][1], t[i][2], t[i][3]);
  }
}

// v[slice][token][r] for a tile of up to 128 tokens: D[128 x rank] in TMEM, 64 k a stage.
template <int TERMS>
__global__ void __launch_bounds__(AD_THREADS, 2) shrink_tc_kernel(AdapterArgs a, int np, int stages) {
  constexpr int AHEAD = TERMS == 3 ? 1 : 2;  // stages on their way in registers
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  __shared__ uint64_t s_empty[4], s_done;
  __shared__ uint32_t s_tmem;
  __shared__ int s_dead;
  Tile tile;
  griddep_wait();
  if (!find_tile(a, blockIdx.x, TC_ROWS, &tile) || tile.adapter < 0) return;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t cols = np <= 32 ? 32 : np <= 64 ? 64 : 128;
  if (warp == 0) {
    tc::tmem_alloc(&s_tmem, cols);
    tc::tmem_relinquish();
  }
  if (tid == 32) {
    for (int i = 0; i < stages; ++i) mbar_init(&s_empty[i], 1);
    mbar_init(&s_done, 1);
    s_dead = 0;
    fence_mbar_init();
  }
  const uint16_t* A = a.a + (int64_t)tile.adapter * a.a_stride;
  const int k0 = blockIdx.y * a.k_slice, k1 = min(a.d_in, k0 + a.k_slice);
  const int blocks = k0 < k1 ? (k1 - k0 + 63) / 64 : 0;
  const int chunk = tid & 7, row0 = tid >> 3;
  const uint32_t stage_bytes = TERMS * TC_TILE + (uint32_t)np * 128;
  const Raw8 zero{make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
  struct Piece {
    Raw8 x[4];
    uint4 w[4];
  };
  Piece piece[AHEAD];
  const auto fetch = [&](int kb, Piece& p) {
    const int k = k0 + 64 * kb + 8 * chunk;
    const bool in = k < k1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = row0 + 32 * i;
      p.x[i] = in && r < tile.rows ? load8(a.x, (int64_t)(tile.row + r) * a.x_stride + k, a.x_type) : zero;
      if (32 * i < np) p.w[i] = in && r < a.rank ? __ldg(reinterpret_cast<const uint4*>(A + (int64_t)r * a.d_in + k)) : zero.lo;
    }
  };
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) fetch(i, piece[i]);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  griddep_launch_dependents();
  const uint32_t tmem = s_tmem;
  const uint32_t idesc = idesc_bf16(TC_ROWS, np);
  const Waiter waiter{a.status, &s_dead};
  int stage = 0;
  uint32_t turn = 0;
  for (int kb0 = 0; kb0 < blocks; kb0 += AHEAD) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const int kb = kb0 + i;
      if (kb >= blocks) break;
      uint8_t* at = smem + stage * stage_bytes;
      if (turn) waiter.wait(&s_empty[stage], (turn - 1) & 1);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t off = tc::swz_off(row0 + 32 * j, chunk);
        put_terms<TERMS>(piece[i].x[j], a.x_type, at, TC_TILE, off);
        if (row0 + 32 * j < np) *reinterpret_cast<uint4*>(at + TERMS * TC_TILE + off) = piece[i].w[j];
      }
      fetch(kb + AHEAD, piece[i]);
      tc::fence_proxy_async_smem();
      __syncthreads();
      if (tid == 0) {
        tc::fence_after_sync();
        const uint64_t bd = tc::smem_desc_sw128(smem_u32(at + TERMS * TC_TILE));
#pragma unroll
        for (int t = TERMS - 1; t >= 0; --t) {
          const uint64_t ad = tc::smem_desc_sw128(smem_u32(at + t * TC_TILE));
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc::mma_f16(tmem, ad + 2 * kk, bd + 2 * kk, idesc, (kb > 0 || t < TERMS - 1 || kk > 0) ? 1u : 0u);
        }
        tc::mma_commit(&s_empty[stage]);
      }
      if (++stage == stages) {
        stage = 0;
        ++turn;
      }
    }
  }
  if (tid == 0) tc::mma_commit(&s_done);
  waiter.wait(&s_done, 0);
  tc::fence_after_sync();
  // rows: the warp's TMEM quadrant; columns: warps 0-3 the even 16, warps 4-7 the odd
  const int row = 32 * (warp & 3) + lane;
  float* v = a.v + ((int64_t)blockIdx.y * a.T + tile.row + row) * a.rank;
  for (int c = 16 * (warp >> 2); c < np; c += 32) {
    float f[16];
    tc::tmem_ld16(tmem + ((uint32_t)(32 * (warp & 3)) << 16) + (uint32_t)c, f);
    if (row < tile.rows)
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        if (c + i < a.rank)
          *reinterpret_cast<float4*>(v + c + i) =
              blocks ? make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 0) tc::tmem_dealloc(tmem, cols);
}

// y = base + B_a (scale v) for a tile of up to 128 tokens and `blocks` blocks of 128 columns.  The tile's scaled v (its
// bf16 terms) stays in shared memory; a block's product is in one of two TMEM accumulators while the block before it is
// read back, turned to rows of 8 consecutive columns a thread through shared memory, added to base and stored.
template <int TERMS>
__global__ void __launch_bounds__(AD_THREADS, 2) expand_tc_kernel(AdapterArgs a, int blocks_per_cta) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  __shared__ uint64_t s_full[2];
  __shared__ uint32_t s_tmem;
  __shared__ int s_dead;
  Tile tile;
  griddep_wait();
  if (!find_tile(a, blockIdx.x, TC_ROWS, &tile)) return;
  if (tile.adapter < 0 && a.base == a.y) return;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool product = tile.adapter >= 0;
  if (warp == 0 && product) {
    tc::tmem_alloc(&s_tmem, 256);
    tc::tmem_relinquish();
  }
  if (tid == 32) {
    mbar_init(&s_full[0], 1);
    mbar_init(&s_full[1], 1);
    s_dead = 0;
    fence_mbar_init();
  }
  const int kblocks = (a.rank + 63) / 64, ksteps = (a.rank + 15) / 16, chunks = 2 * ksteps;
  uint8_t* const sv = smem;                                  // [TERMS][kblocks] tiles
  uint8_t* const sb = sv + TERMS * kblocks * TC_TILE;        // [2][kblocks] tiles
  uint8_t* const stage = sb + 2 * kblocks * TC_TILE + warp * 4096;  // 32 rows x 32 fp32
  const uint16_t* B = a.b + (int64_t)max(tile.adapter, 0) * a.b_stride;
  const int first = blockIdx.y * blocks_per_cta;
  const int blocks = min(blocks_per_cta, (a.d_out + 127) / 128 - first);
  // the block's B rows (columns of y), 16 bytes a thread and turn
  uint4 w[8];
  const auto fetch_b = [&](int blk) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (256 * i >= 128 * chunks) break;
      const int at = tid + 256 * i, r = at / chunks, c = at - r * chunks;
      const int col = 128 * (first + blk) + r, k = 8 * c;
      w[i] = product && blk < blocks && col < a.d_out && k < a.rank
                 ? __ldg(reinterpret_cast<const uint4*>(B + (int64_t)col * a.rank + k))
                 : make_uint4(0u, 0u, 0u, 0u);
    }
  };
  // base of the warp's next 32 x 32 piece (8 columns of 4 rows a lane)
  const int q = warp & 3, half = warp >> 2;
  const int prow = 32 * q + (lane >> 2), pcol = 64 * half + 8 * (lane & 3);
  const Raw8 zero{make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
  Raw8 base[4];
  const auto fetch_base = [&](int blk, int sub) {
    const int col = 128 * (first + blk) + 32 * sub + pcol;
    const bool in = a.base && blk < blocks && col < a.d_out;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = prow + 8 * i;
      base[i] = in && r < tile.rows ? load8(a.base, (int64_t)(tile.row + r) * a.base_stride + col, a.y_type) : zero;
    }
  };
  fetch_b(0);
  fetch_base(0, 0);
  if (product) {
    const float sc = a.scale ? __ldg(a.scale + tile.adapter) : 1.f;
    for (int at = tid; at < TC_ROWS * chunks; at += AD_THREADS) {
      const int r = at / chunks, c = at - r * chunks, k = 8 * c;
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = 0.f;
      if (r < tile.rows && k < a.rank)
        for (int s = 0; s < a.split; ++s) {
          const float4* p = reinterpret_cast<const float4*>(a.v + ((int64_t)s * a.T + tile.row + r) * a.rank + k);
          const float4 u0 = __ldcg(p), u1 = __ldcg(p + 1);
          f[0] += u0.x; f[1] += u0.y; f[2] += u0.z; f[3] += u0.w;
          f[4] += u1.x; f[5] += u1.y; f[6] += u1.z; f[7] += u1.w;
        }
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] *= sc;
      uint32_t t[TERMS][4];
      split8<TERMS>(f, t);
      const uint32_t off = (uint32_t)(c >> 3) * TC_TILE + tc::swz_off(r, c & 7);
#pragma unroll
      for (int i = 0; i < TERMS; ++i)
        *reinterpret_cast<uint4*>(sv + i * kblocks * TC_TILE + off) = make_uint4(t[i][0], t[i][1], t[i][2], t[i][3]);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  griddep_launch_dependents();
  const uint32_t tmem = product ? s_tmem : 0u;
  const uint32_t idesc = idesc_bf16(TC_ROWS, 128);
  const Waiter waiter{a.status, &s_dead};
  for (int blk = 0; blk <= blocks; ++blk) {
    if (product && blk < blocks) {
      uint8_t* const tb = sb + (blk & 1) * kblocks * TC_TILE;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (256 * i >= 128 * chunks) break;
        const int at = tid + 256 * i, r = at / chunks, c = at - r * chunks;
        if (r < 128) *reinterpret_cast<uint4*>(tb + (uint32_t)(c >> 3) * TC_TILE + tc::swz_off(r, c & 7)) = w[i];
      }
      fetch_b(blk + 1);
      tc::fence_proxy_async_smem();
      tc::fence_before_sync();  // this thread's reads of the accumulator two blocks back
      __syncthreads();
      if (tid == 0) {
        tc::fence_after_sync();
        for (int t = TERMS - 1; t >= 0; --t)
          for (int kk = 0; kk < ksteps; ++kk) {
            const uint64_t ad = tc::smem_desc_sw128(smem_u32(sv + (t * kblocks + (kk >> 2)) * TC_TILE));
            const uint64_t bd = tc::smem_desc_sw128(smem_u32(tb + (kk >> 2) * TC_TILE));
            tc::mma_f16(tmem + 128u * (blk & 1), ad + 2 * (kk & 3), bd + 2 * (kk & 3), idesc,
                        (t < TERMS - 1 || kk > 0) ? 1u : 0u);
          }
        tc::mma_commit(&s_full[blk & 1]);
      }
    }
    if (blk == 0) continue;
    const int b = blk - 1;
    if (product) {
      waiter.wait(&s_full[b & 1], (b >> 1) & 1);
      tc::fence_after_sync();
      __syncwarp();
    }
#pragma unroll
    for (int sub = 0; sub < 2; ++sub) {
      if (product) {
        uint32_t u[2][16];
        const uint32_t at = tmem + ((uint32_t)(32 * q) << 16) + 128u * (b & 1) + 64u * half + 32u * sub;
        tc::tmem_ld16_async(at, u[0]);
        tc::tmem_ld16_async(at + 16, u[1]);
        tc::tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 8; ++c)
          *reinterpret_cast<uint4*>(stage + lane * 128 + ((c ^ (lane & 7)) << 4)) =
              make_uint4(u[c >> 2][4 * (c & 3)], u[c >> 2][4 * (c & 3) + 1], u[c >> 2][4 * (c & 3) + 2], u[c >> 2][4 * (c & 3) + 3]);
        __syncwarp();
      }
      const int col = 128 * (first + b) + 32 * sub + pcol;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int rr = (lane >> 2) + 8 * i, r = 32 * q + rr;
        float f[8];
        widen8(base[i], a.y_type, f);
        if (product) {
          const float4 d0 = *reinterpret_cast<const float4*>(stage + rr * 128 + (((2 * (lane & 3)) ^ (rr & 7)) << 4));
          const float4 d1 = *reinterpret_cast<const float4*>(stage + rr * 128 + (((2 * (lane & 3) + 1) ^ (rr & 7)) << 4));
          f[0] += d0.x; f[1] += d0.y; f[2] += d0.z; f[3] += d0.w;
          f[4] += d1.x; f[5] += d1.y; f[6] += d1.z; f[7] += d1.w;
        }
        if (r < tile.rows && col < a.d_out) store8(a.y, (int64_t)(tile.row + r) * a.y_stride + col, a.y_type, f);
      }
      fetch_base(sub == 0 ? b : b + 1, sub ^ 1);
      __syncwarp();
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 0 && product) tc::tmem_dealloc(tmem, 256);
}

template <int MT, int TERMS>
void launch_shrink(const AdapterArgs& a, int tiles, cudaStream_t s) {
  // rank in pieces of up to 64
  const int NT = a.rank <= 16 ? 2 : a.rank <= 32 ? 4 : 8;
  const dim3 grid(tiles, a.split, (a.rank + 8 * NT - 1) / (8 * NT));
  if (NT == 2) launch_pdl(shrink_kernel<2, MT, TERMS>, grid, AD_THREADS, 0, s, a);
  else if (NT == 4) launch_pdl(shrink_kernel<4, MT, TERMS>, grid, AD_THREADS, 0, s, a);
  else launch_pdl(shrink_kernel<8, MT, TERMS>, grid, AD_THREADS, 0, s, a);
}

template <int MT>
cudaError_t launch_both(const AdapterArgs& a, int tiles, int col_split, cudaStream_t s) {
  kernel_begin(KID_ADAPTER_SHRINK, s);
  if (a.x_type == STRATA_BF16) launch_shrink<MT, 1>(a, tiles, s);
  else if (a.x_type == STRATA_F16) launch_shrink<MT, 2>(a, tiles, s);
  else launch_shrink<MT, 3>(a, tiles, s);
  kernel_end(KID_ADAPTER_SHRINK, s);
  const dim3 grid(tiles, col_split);
  kernel_begin(KID_ADAPTER_EXPAND, s);
  if (a.y_type == STRATA_F32) launch_pdl(expand_kernel<MT, 3>, grid, AD_THREADS, 0, s, a);
  else launch_pdl(expand_kernel<MT, 2>, grid, AD_THREADS, 0, s, a);
  kernel_end(KID_ADAPTER_EXPAND, s);
  return cudaGetLastError();
}

// The dynamic shared memory a kernel may use, raised once per kernel and device.
template <auto* KERNEL>
cudaError_t allow_smem(size_t bytes) {
  static std::atomic<uint64_t> done{0};  // bit d: raised on device d
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (bit && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
  err = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (err == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return err;
}
constexpr size_t TC_SMEM_MAX = 226 * 1024;

template <int TERMS>
cudaError_t launch_shrink_tc(const AdapterArgs& a, int tiles, cudaStream_t s) {
  cudaError_t err = allow_smem<shrink_tc_kernel<TERMS>>(TC_SMEM_MAX);
  if (err != cudaSuccess) return err;
  const int np = (a.rank + 15) / 16 * 16;
  const size_t stage = (size_t)TERMS * TC_TILE + (size_t)np * 128;
  // two CTAs an SM
  int stages = (int)((110 * 1024) / stage);
  stages = stages > 4 ? 4 : stages < 2 ? 2 : stages;
  STRATA_LAUNCH(KID_ADAPTER_SHRINK, s,
                err = launch_pdl(shrink_tc_kernel<TERMS>, dim3(tiles, a.split), AD_THREADS, stages * stage + 1024, s, a, np, stages));
  return err;
}

template <int TERMS>
cudaError_t launch_expand_tc(const AdapterArgs& a, int tiles, cudaStream_t s) {
  cudaError_t err = allow_smem<expand_tc_kernel<TERMS>>(TC_SMEM_MAX);
  if (err != cudaSuccess) return err;
  const int kblocks = (a.rank + 63) / 64, col_blocks = (a.d_out + 127) / 128;
  const size_t smem = (size_t)(TERMS + 2) * kblocks * TC_TILE + AD_WARPS * 4096 + 1024;
  int per = 1;
  while (per < col_blocks && tiles * ((col_blocks + per - 1) / per) > 2 * 304) ++per;
  const dim3 grid(tiles, (col_blocks + per - 1) / per);
  STRATA_LAUNCH(KID_ADAPTER_EXPAND, s, err = launch_pdl(expand_tc_kernel<TERMS>, grid, AD_THREADS, smem, s, a, per));
  return err;
}

cudaError_t launch_tc(AdapterArgs a, cudaStream_t s) {
  const int tiles = a.T / TC_ROWS + (a.n_seg < a.T ? a.n_seg : a.T);
  int split = 1;
  while (split < SPLIT_MAX && tiles * split < 228 && a.d_in / (2 * split) >= 256 && 2 * split * a.rank <= V_FLOATS) split *= 2;
  a.split = split;
  a.k_slice = ((a.d_in + split - 1) / split + 63) / 64 * 64;
  const cudaError_t err = a.x_type == STRATA_BF16  ? launch_shrink_tc<1>(a, tiles, s)
                          : a.x_type == STRATA_F16 ? launch_shrink_tc<2>(a, tiles, s)
                                                   : launch_shrink_tc<3>(a, tiles, s);
  if (err != cudaSuccess) return err;
  return a.y_type == STRATA_F32 ? launch_expand_tc<3>(a, tiles, s) : launch_expand_tc<2>(a, tiles, s);
}

}  // namespace

cudaError_t launch_adapters(const strata_adapters_t& ad, const int32_t* seg_off, const int32_t* seg_adapter, int n_seg,
                            const void* x, int T, const void* base, void* y, float* v_parts, int* status,
                            cudaStream_t s) {
  AdapterArgs a{};
  a.a = ad.a; a.b = ad.b; a.scale = ad.scale; a.a_stride = ad.a_stride; a.b_stride = ad.b_stride;
  a.x_stride = ad.x_stride; a.base_stride = ad.base_stride; a.y_stride = ad.y_stride;
  a.seg_off = seg_off; a.seg_adapter = seg_adapter; a.n_seg = n_seg; a.n_adapter = ad.n_adapter;
  a.x = x; a.base = base; a.y = y; a.v = v_parts; a.status = status;
  a.rank = ad.rank; a.d_in = ad.d_in; a.d_out = ad.d_out; a.T = T; a.x_type = ad.x_type; a.y_type = ad.y_type;
  if (T >= 32 * n_seg) return launch_tc(a, s);
  // segments of L tokens make ceil(L / height) tiles: at most T / height + (segments that are not empty)
  const int height = T > 2 * 16 * n_seg ? 32 : 16;
  const int tiles = T / height + (n_seg < T ? n_seg : T);
  int split = 1;
  while (split < SPLIT_MAX && tiles * split < 304 && ad.d_in / (2 * split) >= 256 && 2 * split * ad.rank <= V_FLOATS)
    split *= 2;
  a.split = split;
  a.k_slice = ((ad.d_in + split - 1) / split + 31) / 32 * 32;
  int col_split = 1;
  while (tiles * col_split < 304 && 32 * AD_WARPS * col_split < ad.d_out) ++col_split;
  return height == 32 ? launch_both<2>(a, tiles, col_split, s) : launch_both<1>(a, tiles, col_split, s);
}

}  // namespace strata
