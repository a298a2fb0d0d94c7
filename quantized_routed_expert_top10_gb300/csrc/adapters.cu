// Low-rank adapters of many requests beside a shared projection (strata_moe_adapters), sm_103a:
//   y[t] = base[t] + scale[a] * B_a (A_a x[t]),  a the adapter of t's segment.
// A wider activation is the exact sum of bf16 terms (an fp16 two, an fp32 three), each multiplied on its own with fp32
// accumulators; so is A_a x, to 24 bits for an fp32 y and to 16 otherwise (a rounding of 2^-17, below y's own of 2^-9 or
// 2^-12).
//
// Segments of few tokens, or few tokens times ranks in all, go by one kernel: tiles of 8, 16 or 32 tokens of one segment, a cluster
// a tile, warp-level MMAs.  It is bound by the latency of its chain (segments, A and x, the cluster's sum, B and base), which is
// why everything that a CTA reads is asked for as early as its registers allow: one token 4.3 us, 64 tokens of 64 adapters
// (10.5 MB of them) 5.8 us; 2,048 ragged fp32 tokens, rank 32, 19.6 us (3.4 TB/s; 16 us where all of its 66 MB are in L2).  The rest go by two kernels in tiles of 128 tokens on
// the 5th-generation tensor cores, shrink (v = A_a x) and expand (base + B_a (scale v)): 8,192 tokens of 32 adapters of
// rank 64, 2,560 -> 2,560, bf16, 46.7 us (3.1 TB/s), about 18 and 28, one after the other and each below half of the memory's pace.
#include "device_common.cuh"
#include "elements.cuh"
#include "tc_common.cuh"

namespace strata {
namespace {

constexpr int AD_WARPS = 8;
constexpr int AD_THREADS = 32 * AD_WARPS;
constexpr int SPLIT_MAX = 8;           // slices of d_in
constexpr int LONG = 32;               // tokens a segment from which 128-row tiles may be taken

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
  uint16_t* v;  // [term][T][rank]
  int* status;
  int n_seg, n_adapter, rank, d_in, d_out, T, x_type, y_type, split, k_slice;
};

struct Tile {
  int row, rows, adapter;
};

// The segments cut into tiles of `height` tokens, a thread's share of them: the whole CTA calls both.
struct Segments {
  int s0, s1;     // this thread's segments
  int at, count;  // their first tile, and how many
  int total;      // tiles of all segments; -1: the segments are not valid (recorded in the status word)
};

// Every CTA checks all segments, so either all work or none does.
template <int THREADS>
__device__ Segments cut_segments(const AdapterArgs& a, int height) {
  constexpr int WARPS = THREADS / 32;
  __shared__ int s_warp[WARPS];
  __shared__ int s_bad;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) s_bad = 0;
  __syncthreads();
  const int per = (a.n_seg + THREADS - 1) / THREADS;
  Segments g;
  g.s0 = min(tid * per, a.n_seg);
  g.s1 = min(g.s0 + per, a.n_seg);
  g.count = 0;
  bool bad = false;
  for (int s = g.s0; s < g.s1; ++s) {
    const int lo = __ldg(a.seg_off + s), hi = __ldg(a.seg_off + s + 1), ad = __ldg(a.seg_adapter + s);
    if (lo < 0 || hi < lo || hi > a.T || ad < -1 || ad >= a.n_adapter) {
      bad = true;
      break;
    }
    g.count += (hi - lo + height - 1) / height;
  }
  if (bad) s_bad = 1;
  int v = g.count;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int n = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += n;
  }
  if (lane == 31) s_warp[warp] = v;
  __syncthreads();
  g.at = v - g.count;
  g.total = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) g.at += s_warp[w];
    g.total += s_warp[w];
  }
  if (s_bad) {
    if (tid == 0) set_status(a.status, ST_CORRUPT);
    g.total = -1;
  }
  return g;
}

// Tile `want` of [0, total).
__device__ Tile tile_at(const AdapterArgs& a, const Segments& g, int want, int height) {
  __shared__ int s_tile[3];
  __syncthreads();  // the tile before this one has been read
  if (want >= g.at && want < g.at + g.count) {
    int at = g.at;
    for (int s = g.s0; s < g.s1; ++s) {
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
  return Tile{s_tile[0], s_tile[1], s_tile[2]};
}

// The CTA's one tile; false if there is none.
template <int THREADS>
__device__ bool find_tile(const AdapterArgs& a, int want, int height, Tile* out) {
  const Segments g = cut_segments<THREADS>(a, height);
  if (want >= g.total) return false;
  *out = tile_at(a, g, want, height);
  return true;
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

// Operands are read straight into MMA fragments, 16 bytes a thread.  An MMA's k index may be permuted as long as
// A and B agree: of 32 consecutive k, the thread of quarter q (lane & 3) takes the 8 at 8 q, as k 2q, 2q+1, 2q+8, 2q+9 of
// two MMAs; so four lanes read 64 contiguous bytes of a row.

// (The lanes come together first: loops of different lengths come before.)
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Four floats of shared memory of CTA `rank` of the cluster, at the address that this CTA's `p` has there.
__device__ __forceinline__ float4 cluster_ld4(const void* p, int rank) {
  uint32_t at;
  float4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(at)
               : "memory");
  return v;
}

// Short segments: one cluster a tile of up to 8 H tokens.  Each CTA takes a slice of d_in, its warps 32 k each in turn, and
// adds their sums in warp order; the slices' sums are read from the cluster's shared memory and added in order by every
// CTA, which then has all of scale A_a x (fp32) and takes its share of the columns, 32 a warp at a time.  Columns may be permuted
// over the MMAs' n as k above: the thread of quarter q ends with 8 consecutive columns of a row (column 8 q + 2 j + i
// from MMA j), which it reads and writes 16 bytes at a time.  B and base of a warp's first columns are on their way from
// the start where registers allow.  NT: 8 NT ranks at a time.
template <int NT, int H, int TERMS, bool WIDE>
__global__ void __launch_bounds__(AD_THREADS, 2) short_kernel(AdapterArgs a) {
  constexpr int ROWS = 8 * H, COLS = 8 * NT, MT = (H + 1) / 2;
  constexpr int V_TERMS = WIDE ? 3 : 2;  // of an fp32 y: 24 bits of A_a x, else 16
  constexpr bool EARLY = H == 1 && NT <= 4;
  constexpr int XT = TERMS == 1 ? STRATA_BF16 : TERMS == 2 ? STRATA_F16 : STRATA_F32;
  constexpr int TURNS = H > 1 || NT > 4 ? 1 : NT == 2 && TERMS < 3 ? 3 : 2;  // whose reads are in flight together
  extern __shared__ __align__(16) float s_f[];
  const int pitch = a.rank + 4;
  float* const s_warp = s_f;                              // [warp][ROWS][COLS]
  float* const s_part = s_warp + AD_WARPS * ROWS * COLS;  // [ROWS][pitch]: this CTA's slice
  float* const s_v = s_part + ROWS * pitch;               // [ROWS][pitch]: scale A_a x
  Tile tile;
  griddep_launch_dependents();
  griddep_wait();
  // (the same for all CTAs of a cluster)
  if (!find_tile<AD_THREADS>(a, blockIdx.y, ROWS, &tile)) return;
  const bool product = tile.adapter >= 0;
  if (!product && a.base == a.y) return;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
  const uint16_t* const A = a.a + (int64_t)max(tile.adapter, 0) * a.a_stride;
  const uint16_t* const B = a.b + (int64_t)max(tile.adapter, 0) * a.b_stride;
  const int rank = product ? a.rank : 0;
  const Raw8 zero{make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
  // (d_out and the ranks come in eights: the pieces of a column of four MMAs are all inside or all outside.)
  const uint16_t* const b_at = B + (int64_t)(8 * (g >> 1) + (g & 1)) * a.rank + 8 * q;
  const auto load_b = [&](int c0, int kk, uint4 (&w)[4]) {
    const bool in = kk + 8 * q < rank && c0 + 8 * (g >> 1) < a.d_out;
    const uint16_t* const at = b_at + (int64_t)c0 * a.rank + kk;
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = in ? __ldg(reinterpret_cast<const uint4*>(at + 2 * j * a.rank)) : zero.lo;
  };
  constexpr int Y_SIZE = WIDE ? 4 : 2;
  const char* const base_at = a.base ? static_cast<const char*>(a.base) + ((int64_t)(tile.row + g) * a.base_stride + 8 * q) * Y_SIZE : nullptr;
  char* const y_at = static_cast<char*>(a.y) + ((int64_t)(tile.row + g) * a.y_stride + 8 * q) * Y_SIZE;
  const auto load_base = [&](int c0, Raw8 (&b)[H]) {
    const bool in = base_at && c0 + 8 * q < a.d_out;
#pragma unroll
    for (int h = 0; h < H; ++h)
      b[h] = in && g + 8 * h < tile.rows
                 ? load8(base_at + (8 * h * a.base_stride + c0) * Y_SIZE, 0, WIDE ? STRATA_F32 : STRATA_BF16)  // (as raw bytes)
                 : zero;
  };
  const int c_first = 32 * (warp * a.split + blockIdx.x), c_step = 32 * AD_WARPS * a.split;
  uint4 w_ahead[4], w_next[4];  // of the warp's next columns and the ones after them
  Raw8 base_ahead[H], base_next[H];
  if constexpr (EARLY) {
    load_b(c_first, 0, w_ahead);
    load_base(c_first, base_ahead);
  }
  if (product) {
    const int k0 = blockIdx.x * a.k_slice, k1 = min(a.d_in, k0 + a.k_slice);
    constexpr int X_SIZE = TERMS == 3 ? 4 : 2;
    const uint16_t* const a_at = A + (int64_t)g * a.d_in + 8 * q;
    const char* const x_at = static_cast<const char*>(a.x) + ((int64_t)(tile.row + g) * a.x_stride + 8 * q) * X_SIZE;
    for (int r0 = 0; r0 < rank; r0 += COLS) {
      float acc[MT][NT][4];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.f;
      for (int kt = k0 + 32 * warp; kt < k1; kt += TURNS * 32 * AD_WARPS) {
        uint4 w[TURNS][NT];
        Raw8 x[TURNS][H];
#pragma unroll
        for (int u = 0; u < TURNS; ++u) {
          const int k = kt + u * 32 * AD_WARPS;
          const bool in = k + 8 * q < k1;
#pragma unroll
          for (int n = 0; n < NT; ++n)
            w[u][n] = in && r0 + 8 * n + g < rank
                          ? __ldg(reinterpret_cast<const uint4*>(a_at + (int64_t)(r0 + 8 * n) * a.d_in + k)) : zero.lo;
#pragma unroll
          for (int h = 0; h < H; ++h)
            x[u][h] = in && g + 8 * h < tile.rows ? load8(x_at + (8 * h * a.x_stride + k) * X_SIZE, 0, XT) : zero;
        }
#pragma unroll
        for (int u = 0; u < TURNS; ++u) {
          if (u && kt + u * 32 * AD_WARPS >= k1) break;
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            uint32_t t[2][TERMS][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (2 * m + h >= H) {
#pragma unroll
                for (int i = 0; i < TERMS; ++i) t[h][i][0] = t[h][i][1] = t[h][i][2] = t[h][i][3] = 0u;
                continue;
              }
              const Raw8& f8 = x[u][(2 * m + h) % H];
              if constexpr (TERMS == 1) {
                t[h][0][0] = f8.lo.x; t[h][0][1] = f8.lo.y; t[h][0][2] = f8.lo.z; t[h][0][3] = f8.lo.w;
              } else {
                float f[8];
                widen8(f8, XT, f);
                split8<TERMS>(f, t[h]);
              }
            }
#pragma unroll
            for (int i = TERMS - 1; i >= 0; --i) {
              const uint32_t a0[4] = {t[0][i][0], t[1][i][0], t[0][i][1], t[1][i][1]};
              const uint32_t a1[4] = {t[0][i][2], t[1][i][2], t[0][i][3], t[1][i][3]};
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                mma_bf16(acc[m][n], a0, w[u][n].x, w[u][n].y);
                mma_bf16(acc[m][n], a1, w[u][n].z, w[u][n].w);
              }
            }
          }
        }
      }
      if (EARLY && r0 + COLS >= rank) {  // while the sums are exchanged
        load_b(c_first + c_step, 0, w_next);
        load_base(c_first + c_step, base_next);
      }
      float* const mine = s_warp + warp * ROWS * COLS + 2 * q;
#pragma unroll
      for (int h = 0; h < H; ++h)
        if (g + 8 * h < tile.rows)
#pragma unroll
          for (int n = 0; n < NT; ++n)
            *reinterpret_cast<float2*>(mine + (g + 8 * h) * COLS + 8 * n) =
                make_float2(acc[h >> 1][n][2 * (h & 1)], acc[h >> 1][n][2 * (h & 1) + 1]);
      __syncthreads();
      for (int i = tid; i < tile.rows * COLS; i += AD_THREADS) {
        const int row = i / COLS, c = r0 + i % COLS;
        float v = 0.f;
#pragma unroll
        for (int u = 0; u < AD_WARPS; ++u) v += s_warp[u * ROWS * COLS + i];
        if (c < rank) s_part[row * pitch + c] = v;
      }
      __syncthreads();
    }
    cluster_sync();
    const float sc = a.scale ? __ldg(a.scale + tile.adapter) : 1.f;
    const int pieces = rank / 4;
    for (int i = tid; i < tile.rows * pieces; i += AD_THREADS) {
      const int at = i / pieces * pitch + i % pieces * 4;
      float4 u[SPLIT_MAX], v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int s = 0; s < SPLIT_MAX; ++s) u[s] = s < a.split ? cluster_ld4(s_part + at, s) : v;
#pragma unroll
      for (int s = 0; s < SPLIT_MAX; ++s) v = make_float4(v.x + u[s].x, v.y + u[s].y, v.z + u[s].z, v.w + u[s].w);
      *reinterpret_cast<float4*>(s_v + at) = make_float4(v.x * sc, v.y * sc, v.z * sc, v.w * sc);
    }
    __syncwarp();
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");  // waited for at the end: no CTA leaves while its sums are read
    __syncthreads();
  }
  if (EARLY && !product) load_base(c_first + c_step, base_next);
  // A_a x of rows 16 m .. and k-step kk as MMA operands
  const auto load_v = [&](int m, int kk, uint32_t (&t)[2][V_TERMS][4]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = 16 * m + g + 8 * h, k = kk + 8 * q;
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = 0.f;
      if (2 * m + h < H && k < rank && row < tile.rows) {
        const float4* p = reinterpret_cast<const float4*>(s_v + row * pitch + k);
        const float4 u0 = p[0], u1 = p[1];
        f[0] = u0.x; f[1] = u0.y; f[2] = u0.z; f[3] = u0.w;
        f[4] = u1.x; f[5] = u1.y; f[6] = u1.z; f[7] = u1.w;
      }
      split8<V_TERMS>(f, t[h]);
    }
  };
  uint32_t t[MT][2][V_TERMS][4];
  if constexpr (EARLY) load_v(0, 0, t[0]);  // (rank <= 32: one step of k)
  for (int c0 = c_first; c0 < a.d_out; c0 += c_step) {
    Raw8 base[H];
    uint4 w[4];
    if constexpr (EARLY) {
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = w_ahead[j], w_ahead[j] = w_next[j];
#pragma unroll
      for (int h = 0; h < H; ++h) base[h] = base_ahead[h], base_ahead[h] = base_next[h];
      if (c0 + 2 * c_step < a.d_out) {
        load_b(c0 + 2 * c_step, 0, w_next);
        load_base(c0 + 2 * c_step, base_next);
      }
    } else {
      load_base(c0, base);
    }
    float acc[MT][4][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][j][i] = 0.f;
    for (int kk = 0; kk < rank; kk += 32) {
      if constexpr (!EARLY) {
        load_b(c0, kk, w);
#pragma unroll
        for (int m = 0; m < MT; ++m) load_v(m, kk, t[m]);
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
#pragma unroll
        for (int i = V_TERMS - 1; i >= 0; --i) {
          const uint32_t a0[4] = {t[m][0][i][0], t[m][1][i][0], t[m][0][i][1], t[m][1][i][1]};
          const uint32_t a1[4] = {t[m][0][i][2], t[m][1][i][2], t[m][0][i][3], t[m][1][i][3]};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            mma_bf16(acc[m][j], a0, w[j].x, w[j].y);
            mma_bf16(acc[m][j], a1, w[j].z, w[j].w);
          }
        }
      }
      if (EARLY) break;
    }
    if (c0 + 8 * q >= a.d_out) continue;
#pragma unroll
    for (int h = 0; h < H; ++h) {
      if (g + 8 * h >= tile.rows) continue;
      float f[8];
      widen8(base[h], WIDE ? STRATA_F32 : a.y_type, f);
      if (product) {  // (without an adapter y is base: -0 + 0 would be +0)
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] += acc[h >> 1][i >> 1][2 * (h & 1) + (i & 1)];
      }
      store8(y_at + (8 * h * a.y_stride + c0) * Y_SIZE, 0, WIDE ? STRATA_F32 : a.y_type, f);
    }
  }
  if (product) {
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
}

// ---- Tiles of up to 128 tokens on the 5th-generation tensor cores -----------------------------------------
// Operands are copied 16 bytes a thread into the tensor cores' K-major shared-memory layout (cp.async; an fp16 or fp32 x
// by registers, which split it into its bf16 terms); tensor maps, which the strides would allow, were not tried.  The shrink kernel allocates TMEM after
// griddep_wait and lets the expand kernel start only then; so an expand CTA, which allocates before its wait, waits for
// CTAs that have what they need.
constexpr int TC_ROWS = 128;
constexpr uint32_t TC_TILE = TC_ROWS * 128;  // 128 rows of 64 bf16

__host__ __device__ __forceinline__ uint32_t idesc_bf16(int M, int N) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__host__ __device__ constexpr int bf16_terms(int type) { return type == STRATA_F32 ? 3 : type == STRATA_F16 ? 2 : 1; }
// terms of A x: 16 bits for a 16-bit y, 24 for fp32
__host__ __device__ constexpr int v_terms(int y_type) { return y_type == STRATA_F32 ? 3 : 2; }

// 16 bytes global -> shared, or zeros.
__device__ __forceinline__ void copy16(void* dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All of this thread's copy groups but the last n have arrived.
__device__ __forceinline__ void copy_wait(int n) {
  if (n >= 2) asm volatile("cp.async.wait_group 2;" ::: "memory");
  else if (n == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
  else asm volatile("cp.async.wait_group 0;" ::: "memory");
}
// 16 lanes x 256 bits x 4 into registers without waiting, in the layout of a warp-level MMA's result: of the 8 columns
// 8j .. 8j + 7, thread t gets columns 2 (t % 4), + 1 of lane t / 4 in r[4j], r[4j + 1] and of lane t / 4 + 8 in
// r[4j + 2], r[4j + 3] (lanes counted from the address's lane).
__device__ __forceinline__ void tmem_ld16x256b_x4_async(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// A barrier of the CTA's producers and its issuer.  bar.sync wants whole warps, and the lanes may come from waits and loops of
// different lengths.
__device__ __forceinline__ void stage_barrier() {
  __syncwarp();
  named_barrier(1, AD_THREADS + 32);
}

// A wait that ran out is recorded; the CTA's later waits are then skipped (the call's result is void).
struct Waiter {
  int* status;
  volatile int* dead;
  __device__ __forceinline__ void wait(uint64_t* bar, uint32_t parity) const {
    if (!*dead && !mbar_wait(bar, parity, status)) *dead = 1;
  }
};

// scale A_a x of a tile of up to 128 tokens, as bf16 terms vt[term][token][r].  One cluster a tile: each CTA takes a slice of
// d_in, 64 k a stage, into a [128 x rank] accumulator in TMEM; the slices are then added in order over the cluster's
// shared memory, each CTA finishing its share of the rows.  A warp of its own issues the MMAs.
template <int XT>
__global__ void __launch_bounds__(AD_THREADS + 32, XT == STRATA_F32 ? 2 : 3) shrink_tc_kernel(AdapterArgs a, int np, int stages) {
  constexpr int TERMS = bf16_terms(XT);
  constexpr int AHEAD = 2;  // stages of x on their way in registers (TERMS > 1)
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  __shared__ uint64_t s_empty[4], s_done;
  __shared__ uint32_t s_tmem;
  __shared__ int s_dead;
  Tile tile;
  griddep_wait();
  // (the same for all CTAs of a cluster)
  if (!find_tile<AD_THREADS + 32>(a, blockIdx.x, TC_ROWS, &tile) || tile.adapter < 0) return;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool issuer = warp == AD_WARPS;
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
  const float sc = a.scale ? __ldg(a.scale + tile.adapter) : 1.f;
  const int k0 = blockIdx.y * a.k_slice, k1 = min(a.d_in, k0 + a.k_slice);
  const int blocks = (k1 - k0 + 63) / 64;  // at least one
  const int chunk = tid & 7, row0 = tid >> 3;
  const uint32_t stage_bytes = TERMS * TC_TILE + (uint32_t)np * 128;
  const int64_t x_size = XT == STRATA_F32 ? 4 : 2;
  const char* X = static_cast<const char*>(a.x) + ((int64_t)(tile.row + row0) * a.x_stride + k0 + 8 * chunk) * x_size;
  const uint16_t* W = A + (int64_t)row0 * a.d_in + k0 + 8 * chunk;
  // what goes by cp.async of k-block kb: A, and a bf16 x
  const auto copy = [&](int kb) {
    if (kb < blocks) {
      uint8_t* at = smem + (kb % stages) * stage_bytes;
      const bool in = k0 + 64 * kb + 8 * chunk < k1;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = row0 + 32 * j;
        const uint32_t off = tc::swz_off(r, chunk);
        if (TERMS == 1) {
          const bool ok = in && r < tile.rows;
          copy16(at + off, ok ? X + (32 * j * a.x_stride + 64 * kb) * x_size : static_cast<const char*>(a.x), ok);
        }
        if (r < np) {
          const bool ok = in && r < a.rank;
          copy16(at + TERMS * TC_TILE + off, ok ? W + (int64_t)32 * j * a.d_in + 64 * kb : A, ok);
        }
      }
    }
    copy_commit();
  };
  const Raw8 zero{make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
  Raw8 piece[AHEAD][4];
  const auto fetch = [&](int kb, Raw8 (&p)[4]) {
    const bool in = k0 + 64 * kb + 8 * chunk < k1;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      p[j] = in && row0 + 32 * j < tile.rows ? load8(X + (32 * j * a.x_stride + 64 * kb) * x_size, 0, XT) : zero;
  };
  if (!issuer) {
    if (TERMS > 1) {
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) fetch(i, piece[i]);
    }
    for (int i = 0; i < stages - 1; ++i) copy(i);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  griddep_launch_dependents();
  const uint32_t tmem = s_tmem;
  const uint32_t idesc = idesc_bf16(TC_ROWS, np);
  const Waiter waiter{a.status, &s_dead};
  if (issuer) {
    uint64_t desc = tc::smem_desc_sw128(smem_u32(smem));
    for (int kb = 0, stage = 0; kb < blocks; ++kb) {
      stage_barrier();  // k-block kb is in shared memory
      if (lane == 0) {
        tc::fence_after_sync();
        const uint64_t ad = desc + (uint64_t)(stage * (stage_bytes >> 4)), bd = ad + TERMS * (TC_TILE >> 4);
#pragma unroll
        for (int t = TERMS - 1; t >= 0; --t)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc::mma_f16(tmem, ad + t * (TC_TILE >> 4) + 2 * kk, bd + 2 * kk, idesc, (kb > 0 || t < TERMS - 1 || kk > 0) ? 1u : 0u);
        tc::mma_commit(&s_empty[stage]);
      }
      if (++stage == stages) stage = 0;
    }
    if (lane == 0) tc::mma_commit(&s_done);
    __syncwarp();
  } else {
    for (int kb0 = 0; kb0 < blocks; kb0 += AHEAD) {
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        const int kb = kb0 + i;
        if (kb >= blocks) break;
        if (TERMS > 1) {
          uint8_t* at = smem + (kb % stages) * stage_bytes;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float f[8];
            uint32_t t[TERMS][4];
            widen8(piece[i][j], XT, f);
            split8<TERMS>(f, t);
#pragma unroll
            for (int e = 0; e < TERMS; ++e)
              *reinterpret_cast<uint4*>(at + e * TC_TILE + tc::swz_off(row0 + 32 * j, chunk)) =
                  make_uint4(t[e][0], t[e][1], t[e][2], t[e][3]);
          }
          fetch(kb + AHEAD, piece[i]);
        }
        copy_wait(stages - 2);
        tc::fence_proxy_async_smem();
        stage_barrier();
        // the stage of k-block kb - 1 is free once its MMAs are done
        if (kb > 0) waiter.wait(&s_empty[(kb - 1) % stages], ((kb - 1) / stages) & 1);
        copy(kb + stages - 1);
      }
    }
    copy_wait(0);
  }
  waiter.wait(&s_done, 0);
  tc::fence_after_sync();
  __syncthreads();  // all have seen the last MMA: the stages are free for the sums
  const int pitch = np + 4;
  float* const part = reinterpret_cast<float*>(smem);
  if (!issuer) {
    // rows: the warp's TMEM quadrant; columns: warps 0-3 the even 16, warps 4-7 the odd
    const int row = 32 * (warp & 3) + lane;
    for (int c = 16 * (warp >> 2); c < np; c += 32) {
      float f[16];
      tc::tmem_ld16(tmem + ((uint32_t)(32 * (warp & 3)) << 16) + (uint32_t)c, f);
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        *reinterpret_cast<float4*>(part + row * pitch + c + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
    }
  }
  tc::fence_before_sync();
  cluster_sync();
  if (warp == 0) tc::tmem_dealloc(tmem, cols);
  const int chunks = a.rank >> 3, vt = v_terms(a.y_type);
  // the cluster's CTAs share the tile's rows x 8 columns out among their threads
  for (int at = issuer ? tile.rows * chunks : blockIdx.y * AD_THREADS + tid; at < tile.rows * chunks; at += a.split * AD_THREADS) {
    const int row = at / chunks, c = 8 * (at - row * chunks);
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = 0.f;
    for (int s0 = 0; s0 < a.split; s0 += 4) {  // four slices' reads at once
      float4 u0[4], u1[4];
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        u0[s] = u1[s] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (s0 + s < a.split) {
          u0[s] = cluster_ld4(part + row * pitch + c, s0 + s);
          u1[s] = cluster_ld4(part + row * pitch + c + 4, s0 + s);
        }
      }
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        f[0] += u0[s].x; f[1] += u0[s].y; f[2] += u0[s].z; f[3] += u0[s].w;
        f[4] += u1[s].x; f[5] += u1[s].y; f[6] += u1[s].z; f[7] += u1[s].w;
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] *= sc;
    uint32_t t[3][4];
    split8<3>(f, t);
    uint16_t* out = a.v + (int64_t)(tile.row + row) * a.rank + c;
#pragma unroll
    for (int e = 0; e < 3; ++e)
      if (e < vt) *reinterpret_cast<uint4*>(out + (int64_t)e * a.T * a.rank) = make_uint4(t[e][0], t[e][1], t[e][2], t[e][3]);
  }
  cluster_sync();  // no CTA leaves while another reads its sums
}

// y = base + B_a (scale A_a x).  The work is one line of units, 128 columns of a tile of up to 128 tokens each, of which every
// CTA (two an SM) takes an equal stretch.  A tile's scaled A_a x (its bf16 terms) stays in shared memory, B of the units
// ahead is on its way by cp.async into a ring; a unit's product is in one of two TMEM accumulators while the unit before it
// is read back, added to base (on its way in registers for a unit ahead) and stored.  A warp of its own issues the MMAs.
// The accumulator is read back in the layout of a warp-level MMA's result, 2 of every 8 columns a thread; B's rows are placed
// so that these are 8 consecutive columns of y: place 8 j + 2 q + b of 32 holds column 8 q + 2 j + b.  So y passes
// no shared memory, and four lanes read and write 32 columns of a row.
template <int YT>
__global__ void __launch_bounds__(AD_THREADS + 32, 2) expand_tc_kernel(AdapterArgs a, int ring) {
  constexpr int TERMS = v_terms(YT);
  constexpr int CW = 128;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  __shared__ uint64_t s_full[2];
  __shared__ uint32_t s_tmem;
  __shared__ int s_dead;
  // Until griddep_wait only what the shrink kernel does not write is read; its CTAs let this kernel start after
  // their own wait for what came before them.
  const Segments g = cut_segments<AD_THREADS + 32>(a, TC_ROWS);
  const int col_blocks = (a.d_out + CW - 1) / CW;
  const int units = g.total * col_blocks;  // far inside 32 bits: a few hundred tiles of 128
  const int u1 = (int)((int64_t)units * (blockIdx.x + 1) / gridDim.x);
  int u = (int)((int64_t)units * blockIdx.x / gridDim.x);
  if (u >= u1) {
    griddep_wait();
    return;
  }
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool issuer = warp == AD_WARPS;
  if (warp == 0) {
    tc::tmem_alloc(&s_tmem, 2 * CW);
    tc::tmem_relinquish();
  }
  if (tid == 32) {
    mbar_init(&s_full[0], 1);
    mbar_init(&s_full[1], 1);
    s_dead = 0;
    fence_mbar_init();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  griddep_launch_dependents();
  const uint32_t tmem = s_tmem;
  const int kblocks = (a.rank + 63) / 64, ksteps = (a.rank + 15) / 16;
  const uint32_t b_slot = kblocks * TC_TILE;
  uint8_t* const sv = smem;                             // [TERMS][kblocks] tiles
  uint8_t* const sb = sv + TERMS * kblocks * TC_TILE;   // [ring][kblocks] tiles
  const uint32_t idesc = idesc_bf16(TC_ROWS, CW);
  const uint64_t v_desc = tc::smem_desc_sw128(smem_u32(sv)), b_desc = tc::smem_desc_sw128(smem_u32(sb));
  const Waiter waiter{a.status, &s_dead};
  const uint16_t* vt = a.v;
  // the warp's part of a unit: TMEM quadrant q4 (32 tokens) and 64 columns in two pieces; a lane has 8 columns of 4 rows of
  // a piece
  const int q4 = warp & 3, half = warp >> 2;
  const int mrow = 32 * q4 + (lane >> 2), mcol = 64 * half + 8 * (lane & 3);
  // two threads a row of B
  const int brow = tid >> 1;
  const int bcol = (brow & ~31) + 8 * ((brow >> 1) & 3) + 2 * ((brow >> 3) & 3) + (brow & 1);
  const Raw8 zero{make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
  int n = 0;  // units with a product so far: the next one's accumulator and barrier phase
  bool waited = false;
  while (u < u1) {
    const int first = u % col_blocks, blocks = min(col_blocks - first, u1 - u);
    const Tile tile = tile_at(a, g, u / col_blocks, TC_ROWS);
    u += blocks;
    const bool product = tile.adapter >= 0;
    if (!product && a.base == a.y) continue;
    if (issuer) {
      if (!waited) griddep_wait();
      waited = true;
      if (product)
        for (int blk = 0; blk < blocks; ++blk) {
          stage_barrier();  // A_a x and B of unit blk are in shared memory
          if (lane == 0) {
            tc::fence_after_sync();
            const int acc = (n + blk) & 1;
            const uint64_t bd = b_desc + (uint64_t)((blk % ring) * (b_slot >> 4));
#pragma unroll
            for (int t = TERMS - 1; t >= 0; --t)
#pragma unroll
              for (int kk = 0; kk < 8; ++kk)
                if (kk < ksteps)
                  tc::mma_f16(tmem + (uint32_t)(CW * acc), v_desc + (t * kblocks + (kk >> 2)) * (TC_TILE >> 4) + 2 * (kk & 3),
                              bd + (kk >> 2) * (TC_TILE >> 4) + 2 * (kk & 3), idesc, (t < TERMS - 1 || kk > 0) ? 1u : 0u);
            tc::mma_commit(&s_full[acc]);
          }
        }
      if (product) n += blocks;
      continue;
    }
    const uint16_t* B = a.b + (int64_t)max(tile.adapter, 0) * a.b_stride;
    const int64_t base_at = (int64_t)(tile.row + mrow) * a.base_stride + CW * first + mcol;
    const int64_t y_at = (int64_t)(tile.row + mrow) * a.y_stride + CW * first + mcol;
    uint32_t rows = 0;  // bit i: row mrow + 8 i is the tile's
#pragma unroll
    for (int i = 0; i < 4; ++i) rows |= (mrow + 8 * i < tile.rows ? 1u : 0u) << i;
    const uint16_t* const b_at = B + (int64_t)(CW * first + bcol) * a.rank;
    const auto copy_b = [&](int blk) {
      if (product && blk < blocks) {
        uint8_t* const to = sb + (blk % ring) * b_slot;
        const bool col = CW * (first + blk) + bcol < a.d_out;
        for (int c = tid & 1; c < 2 * ksteps; c += 2) {
          const bool ok = col && 8 * c < a.rank;
          copy16(to + (c >> 3) * TC_TILE + tc::swz_off(brow, c & 7), ok ? b_at + (int64_t)(CW * blk) * a.rank + 8 * c : B, ok);
        }
      }
      copy_commit();
    };
    Raw8 base[2][4];
    const auto fetch_base = [&](int blk, int sub, Raw8 (&to)[4]) {
      const bool in = a.base && blk < blocks && CW * (first + blk) + 32 * sub + mcol < a.d_out;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        to[i] = in && (rows >> i & 1u) ? load8(a.base, base_at + 8 * i * a.base_stride + CW * blk + 32 * sub, YT) : zero;
    };
    // base of the unit after the next goes to L2 (8,192 tokens: 46.6 us, one further 47.5, none 51), a row of 128 columns two threads
    const auto warm = [&](int blk) {
      const int c0 = CW * (first + blk), size = YT == STRATA_F32 ? 4 : 2;
      if (!a.base || blk >= blocks || brow >= tile.rows) return;
#pragma unroll
      for (int c = (tid & 1) * 64; c < CW; c += YT == STRATA_F32 ? (c & 32 ? 128 : 32) : 128)
        if (c0 + c < a.d_out)
          prefetch_l2(static_cast<const char*>(a.base) + ((tile.row + brow) * a.base_stride + c0 + c) * size);
    };
    for (int i = 0; i < ring - 1; ++i) copy_b(i);
    warm(1);
    fetch_base(0, 0, base[0]);
    fetch_base(0, 1, base[1]);
    if (!waited) griddep_wait();
    waited = true;
    if (product) {
      const int r = tid >> 1;
      for (int e = 0; e < TERMS; ++e)
        for (int c = tid & 1; c < 2 * ksteps; c += 2) {
          const bool ok = r < tile.rows && 8 * c < a.rank;
          copy16(sv + (e * kblocks + (c >> 3)) * TC_TILE + tc::swz_off(r, c & 7),
                 ok ? vt + ((int64_t)e * a.T + tile.row + r) * a.rank + 8 * c : vt, ok);
        }
      copy_commit();
    }
    for (int blk = 0; blk <= blocks; ++blk) {
      if (product && blk < blocks) {
        copy_wait(blk ? ring - 2 : 0);
        tc::fence_proxy_async_smem();
        tc::fence_before_sync();  // this thread's reads of the accumulator two units back
        stage_barrier();
      }
      if (blk > 0) {
        const int b = blk - 1, acc = (n + b) & 1;
        if (product) {
          waiter.wait(&s_full[acc], ((n + b) >> 1) & 1);
          tc::fence_after_sync();
        }
#pragma unroll
        for (int sub = 0; sub < 2; ++sub) {
          const bool col = CW * (first + b) + 32 * sub + mcol < a.d_out;
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // rows mrow + 16 h, + 8
            uint32_t d[16];
            if (product) {
              __syncwarp();  // (lanes whose row or column is outside store nothing)
              tmem_ld16x256b_x4_async(tmem + ((uint32_t)(32 * q4 + 16 * h) << 16) + (uint32_t)(CW * acc + 64 * half + 32 * sub), d);
              tc::tmem_wait_ld();
            }
#pragma unroll
            for (int p = 0; p < 2; ++p) {
              const int i = 2 * h + p;
              float f[8];
              widen8(base[sub][i], YT, f);
              if (product) {
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] += __uint_as_float(d[4 * (e >> 1) + 2 * p + (e & 1)]);
              }
              if (col && (rows >> i & 1u)) store8(a.y, y_at + 8 * i * a.y_stride + CW * b + 32 * sub, YT, f);
            }
          }
          fetch_base(b + 1, sub, base[sub]);
        }
      }
      // into the slot of the unit just stored, whose product's MMAs this thread has waited for
      if (blk < blocks) copy_b(blk + ring - 1);
      warm(blk + 2);
    }
    copy_wait(0);
    if (product) n += blocks;
  }
  if (!waited) griddep_wait();
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 0) tc::tmem_dealloc(tmem, 2 * CW);
}

// No more tiles than this: a segment of L > 0 tokens has ceil(L / height), at most (L + height - 1) / height.
int tiles_of(const AdapterArgs& a, int height) {
  return (a.T + (a.n_seg < a.T ? a.n_seg : a.T) * (height - 1)) / height;
}

// Clusters of `split` CTAs that the device holds at a time (a cluster lies within a part of it, so not all of two CTAs an SM).
// The split decides the order of the sums, so this goes by all that cfg depends on: the kernel, the split and the rank.
template <int NT, int H, int TERMS, bool WIDE>
int resident_clusters(cudaLaunchConfig_t cfg, int split, int rank) {
  static std::atomic<int> known[SPLIT_MAX + 1][STRATA_ADAPTER_RANK_MAX / 8 + 1];
  std::atomic<int>& k = known[split][rank / 8];
  int n = k.load(std::memory_order_relaxed);
  if (n) return n;
  cfg.gridDim = dim3(split, 1);
  cfg.attrs[1].val.clusterDim.x = split;
  if (cudaOccupancyMaxActiveClusters(&n, short_kernel<NT, H, TERMS, WIDE>, &cfg) != cudaSuccess || n < 1) {
    cudaGetLastError();
    n = 1;
  }
  k.store(n, std::memory_order_relaxed);
  return n;
}

template <int NT, int H, int TERMS, bool WIDE>
cudaError_t launch_short_v(AdapterArgs a, cudaStream_t s) {
  cudaError_t err = allow_smem<short_kernel<NT, H, TERMS, WIDE>>(110 * 1024);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(AD_THREADS);
  cfg.dynamicSmemBytes = sizeof(float) * 8 * H * (AD_WARPS * 8 * NT + 2 * (a.rank + 4));
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  // CTAs a tile: as many as leave all tiles resident at once, where a segment's last tile is taken to be half full (a second
  // round costs more than shorter slices gain: 64 single tokens 7.2 us with 4 CTAs each, 11.5 with 5; a tile alone 15.6, 4.1
  // with 8).  No more than warps have turns.
  const int m = a.n_seg < a.T ? a.n_seg : a.T, half = a.T / (8 * H) + m / 2, tiles = half > m ? half : m;
  const int most = ((a.d_in > a.d_out ? a.d_in : a.d_out) + 32 * AD_WARPS - 1) / (32 * AD_WARPS);
  a.split = 1;
  while (a.split < SPLIT_MAX && a.split < most && tiles + tiles / 32 <= resident_clusters<NT, H, TERMS, WIDE>(cfg, a.split + 1, a.rank))
    ++a.split;
  a.k_slice = ((a.d_in + 31) / 32 + a.split - 1) / a.split * 32;
  cfg.gridDim = dim3(a.split, tiles_of(a, 8 * H));
  attr[1].val.clusterDim.x = a.split;
  STRATA_LAUNCH(KID_ADAPTERS, s, err = cudaLaunchKernelEx(&cfg, short_kernel<NT, H, TERMS, WIDE>, a));
  return err;
}

template <int H, int TERMS, bool WIDE>
cudaError_t launch_short_r(const AdapterArgs& a, cudaStream_t s) {
  return a.rank <= 16   ? launch_short_v<2, H, TERMS, WIDE>(a, s)
         : a.rank <= 32 ? launch_short_v<4, H, TERMS, WIDE>(a, s)
                        : launch_short_v<8, H, TERMS, WIDE>(a, s);
}

template <int H, int TERMS>
cudaError_t launch_short_y(const AdapterArgs& a, cudaStream_t s) {
  return a.y_type == STRATA_F32 ? launch_short_r<H, TERMS, true>(a, s) : launch_short_r<H, TERMS, false>(a, s);
}

template <int H>
cudaError_t launch_short(const AdapterArgs& a, cudaStream_t s) {
  return a.x_type == STRATA_BF16  ? launch_short_y<H, 1>(a, s)
         : a.x_type == STRATA_F16 ? launch_short_y<H, 2>(a, s)
                                  : launch_short_y<H, 3>(a, s);
}

constexpr size_t TC_SMEM_MAX = 226 * 1024;

template <int XT>
cudaError_t launch_shrink_tc(const AdapterArgs& a, int tiles, cudaStream_t s) {
  cudaError_t err = allow_smem<shrink_tc_kernel<XT>>(TC_SMEM_MAX);
  if (err != cudaSuccess) return err;
  const int np = (a.rank + 15) / 16 * 16;
  const size_t stage = (size_t)bf16_terms(XT) * TC_TILE + (size_t)np * 128;
  const int ctas = XT == STRATA_F32 ? 2 : 3;  // an SM
  int stages = (int)((226 * 1024 / ctas - 2048) / stage);
  stages = stages > 4 ? 4 : stages < 2 ? 2 : stages;
  const size_t sums = (size_t)TC_ROWS * (np + 4) * sizeof(float);  // take the stages' place
  const size_t smem = (stages * stage > sums ? stages * stage : sums) + 1024;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(tiles, a.split);
  cfg.blockDim = dim3(AD_THREADS + 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1;
  attr[1].val.clusterDim.y = a.split;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  STRATA_LAUNCH(KID_ADAPTER_SHRINK, s, err = cudaLaunchKernelEx(&cfg, shrink_tc_kernel<XT>, a, np, stages));
  return err;
}

template <int YT>
cudaError_t launch_expand_tc(const AdapterArgs& a, int tiles, cudaStream_t s) {
  cudaError_t err = allow_smem<expand_tc_kernel<YT>>(TC_SMEM_MAX);
  if (err != cudaSuccess) return err;
  const int kblocks = (a.rank + 63) / 64, units = tiles * ((a.d_out + 127) / 128);
  const size_t fixed = (size_t)v_terms(YT) * kblocks * TC_TILE + 1024, slot = (size_t)kblocks * TC_TILE;
  const size_t half_sm = 113 * 1024;  // two CTAs an SM
  const int ring = fixed + 2 * slot > half_sm || fixed + 3 * slot <= half_sm ? 3 : 2;
  const size_t smem = fixed + ring * slot;
  const int fit = smem <= half_sm ? 304 : 152;
  STRATA_LAUNCH(KID_ADAPTER_EXPAND, s,
                err = launch_pdl(expand_tc_kernel<YT>, dim3(units < fit ? units : fit), AD_THREADS + 32, smem, s, a, ring));
  return err;
}

cudaError_t launch_tc(AdapterArgs a, cudaStream_t s) {
  const int tiles = tiles_of(a, TC_ROWS);
  int split = 1;
  while (split < SPLIT_MAX && 2 * tiles * split <= 152 * (a.x_type == STRATA_F32 ? 2 : 3) && a.d_in / (2 * split) >= 256) split *= 2;
  // whole blocks of 64 k a slice; every slice has one (no MMAs are committed that were not issued, no sums of nothing added)
  a.k_slice = ((a.d_in + split - 1) / split + 63) / 64 * 64;
  a.split = (a.d_in + a.k_slice - 1) / a.k_slice;
  const cudaError_t err = a.x_type == STRATA_BF16  ? launch_shrink_tc<STRATA_BF16>(a, tiles, s)
                          : a.x_type == STRATA_F16 ? launch_shrink_tc<STRATA_F16>(a, tiles, s)
                                                   : launch_shrink_tc<STRATA_F32>(a, tiles, s);
  if (err != cudaSuccess) return err;
  return a.y_type == STRATA_F32    ? launch_expand_tc<STRATA_F32>(a, tiles, s)
         : a.y_type == STRATA_BF16 ? launch_expand_tc<STRATA_BF16>(a, tiles, s)
                                   : launch_expand_tc<STRATA_F16>(a, tiles, s);
}

}  // namespace

cudaError_t launch_adapters(const strata_adapters_t& ad, const int32_t* seg_off, const int32_t* seg_adapter, int n_seg,
                            const void* x, int T, const void* base, void* y, uint16_t* v_terms, int* status,
                            cudaStream_t s) {
  AdapterArgs a{};
  a.a = ad.a; a.b = ad.b; a.scale = ad.scale; a.a_stride = ad.a_stride; a.b_stride = ad.b_stride;
  a.x_stride = ad.x_stride; a.base_stride = ad.base_stride; a.y_stride = ad.y_stride;
  a.seg_off = seg_off; a.seg_adapter = seg_adapter; a.n_seg = n_seg; a.n_adapter = ad.n_adapter;
  a.x = x; a.base = base; a.y = y; a.v = v_terms; a.status = status;
  a.rank = ad.rank; a.d_in = ad.d_in; a.d_out = ad.d_out; a.T = T; a.x_type = ad.x_type; a.y_type = ad.y_type;
  // The 128-row kernels cost a call more and a token's rank less than warp-level MMAs.  (Measured at 2,560 -> 2,560 only: other
  // widths take the same rule.)  bf16, in us, short and 128-row: rank 32, 8,192 tokens 40 and 46; rank 64, 4,096 tokens 31 and
  // 32, 8,192 tokens 59 and 50; rank 128, 2,048 tokens in 32 segments 29 and 38, in 64 57 and 45.  x or y fp32: rank 64, 8,192
  // tokens 70 to 85 and 85 to 105; rank 128, 2,048 tokens in 32 43 and 56.
  const int filled = n_seg < T ? n_seg : T;
  const bool half = T / 16 + filled / 2 <= 152;  // tiles of 16 tokens, two CTAs each, all at once (a last tile half full)
  const bool wide = a.x_type == STRATA_F32 || a.y_type == STRATA_F32;
  const bool many = (int64_t)T * a.rank > (half ? 256 : 192) * 1024 && a.rank > (wide ? 64 : 32);
  if (many && T >= LONG * n_seg) return launch_tc(a, s);
  // Tiles of 8 tokens where segments are as short or four CTAs a tile fit the device; else of 16 while two each fit; else of 32.
  // Larger tiles read A and B less often, smaller ones fill the device: 256 tokens in 8 segments, bf16, rank 16 by 8 and 16, 5.7 us
  // and 6.7; 2,048 in 24, fp32, rank 32 by 16 and 32, 16 us and 21; 4,096 in 32, bf16, rank 16, 19 and 17.
  if (T <= 8 * n_seg || T / 8 + filled / 2 <= 76) return launch_short<1>(a, s);
  return half ? launch_short<2>(a, s) : launch_short<4>(a, s);
}

}  // namespace strata
