// The norms before and after the block (strata_moe_norm, strata_moe_combine_norm), sm_103a.
//
// zwxr.cn news/242664, section "一次路由的完整旅程": moe_combine adds the experts' outputs weighted by the router's
// weights to the layer's input; the layers read a normalised activation.  Here the weighted sum, the norm of the
// block's output, its gates, the scaled residual and the next block's norm are one pass: a row is held in registers
// between its one read and its one write, both mean squares are sums over its CTA.
//
// The kernels may start while the one before them ends (griddep_wait) and let the next one start when their rows are done;
// started earlier, its CTAs took room from this one's (ten parts 44 -> 47 us).  All forms are bound by memory, or by the
// launch where rows are few (four rows 2.0 us, one token's ten parts 4.3 us), so each keeps rows on their way while another is
// summed: CTAs stay and walk the rows, and what comes next is already being read, into registers (one part or none) or a
// ring in shared memory (several).  A CTA a row without that: 39 us for the norm below, 65 us for ten parts.  On one GB300, 2,560
// columns: the norm of 8,192 rows, fp32 to bf16, 22.4 us (5.6 TB/s), a copy of 42 MB and back 15 to 20 us; 2,048 rows of ten
// fp32 parts 43.5 us (6.3 TB/s, 92% of the measured copy rate); 8,192 rows of one fp32 part with the stream in bf16 38.6 us
// (5.4 TB/s).
#include "device_common.cuh"
#include "elements.cuh"

namespace strata {
namespace {

struct NormArgs {
  const void* parts;   // null: no block output, r = x
  const float* pw;
  const void* x;
  const float* post_gain;
  const float* channel;
  const float* token;
  const float* pre_gain;
  void* out;
  void* next;
  int64_t part_stride, token_stride, x_stride, out_stride, next_stride;
  int T, n, P, part_type, x_type, next_type;
  int post, sigmoid;
  float eps, residual, block, inv_n;
  bool gains16;  // the gains given lie on 16-byte boundaries
};

// (A row is a CTA's, or where a warp has threads for all of it a warp's: blockDim.x == 32, blockDim.y rows a CTA.)
//
// Sum of v over the threads of a row: its warp, or the whole CTA (blockDim.x > 32).  red: 32 floats of shared
// memory used by this sum alone.
__device__ __forceinline__ float row_sum(float v, float* red) {
  v = warp_sum(v);
  if (blockDim.x == 32) return v;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) red[warp] = v;
  __syncthreads();
  const int warps = blockDim.x >> 5;
  return warp_sum(lane < warps ? red[lane] : 0.f);
}

// 4 consecutive elements of type T on a boundary of their size, as read (16 bytes of fp32, so that a warp's accesses are
// contiguous whatever the types of the operands).
template <int T>
struct Unit {
  uint32_t r[T == STRATA_F32 ? 4 : 2];
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    if constexpr (T == STRATA_F32) {
      const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const float*>(p) + i);
      r[0] = v.x; r[1] = v.y; r[2] = v.z; r[3] = v.w;
    } else {
      const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
      r[0] = v.x; r[1] = v.y;
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (uint32_t& v : r) v = 0u;
  }
  __device__ __forceinline__ void widen(float (&f)[4]) const {
    if constexpr (T == STRATA_F32) {
#pragma unroll
      for (int e = 0; e < 4; ++e) f[e] = __uint_as_float(r[e]);
    } else {
      const float2 a = widen2(r[0], T), b = widen2(r[1], T);
      f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
    }
  }
};
__device__ __forceinline__ void store_unit(void* p, int64_t i, int type, const float (&f)[4]) {
  if (type == STRATA_F32) *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = make_float4(f[0], f[1], f[2], f[3]);
  else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + i) = make_uint2(narrow2(f[0], f[1], type), narrow2(f[2], f[3], type));
}
// f *= g[i .. i + 3] (fp32)
__device__ __forceinline__ void times(float (&f)[4], const float* g, int i, bool aligned) {
  if (aligned) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(g + i));
    f[0] *= a.x; f[1] *= a.y; f[2] *= a.z; f[3] *= a.w;
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) f[e] *= __ldg(g + i + e);
}

constexpr int NO_PARTS = -1;

// Few rows with several parts, on boundaries of 4 elements: a CTA a row, a thread one unit of 4 columns, ten parts read at
// once.
template <int XT, int PT>
__global__ void __launch_bounds__(1024) edge_few_kernel(const __grid_constant__ NormArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  constexpr int GROUP = 10;
  __shared__ float red[2][32];
  const int t = blockIdx.x, u = threadIdx.x, lane = u & 31;
  const bool in = u < a.n / 4;
  Unit<XT> x;
  if (a.x && in) x.load(a.x, (int64_t)t * a.x_stride + u * 4);
  else x.zero();
  const float mine = lane >= a.P ? 0.f : a.pw ? __ldg(a.pw + (int64_t)t * a.P + lane) : 1.f;  // P <= 32
  float g = a.block;
  if (a.token) {
    const float s = __ldg(a.token + t);
    g *= a.sigmoid ? 1.f / (1.f + expf(-s)) : s;
  }
  float y[4] = {0.f, 0.f, 0.f, 0.f}, r[4];
  for (int k0 = 0; k0 < a.P; k0 += GROUP) {
    Unit<PT> p[GROUP];
    float w[GROUP];
#pragma unroll
    for (int k = 0; k < GROUP; ++k) {
      w[k] = k0 + k < 32 ? __shfl_sync(0xffffffffu, mine, (k0 + k) & 31) : 0.f;
      if (w[k] != 0.f && in) p[k].load(a.parts, (int64_t)t * a.token_stride + (k0 + k) * a.part_stride + u * 4);
      else p[k].zero();
    }
#pragma unroll
    for (int k = 0; k < GROUP; ++k) {
      float f[4];
      p[k].widen(f);
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = fmaf(w[k], f[e], y[e]);
    }
  }
  float rn = 1.f;
  if (a.post) {
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) ss = fmaf(y[e], y[e], ss);
    rn = rsqrtf(fmaf(row_sum(ss, red[0]), a.inv_n, a.eps));
  }
  x.widen(r);
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] *= rn;
  if (in) {
    if (a.post_gain) times(y, a.post_gain, u * 4, a.gains16);
    if (a.channel) times(y, a.channel, u * 4, a.gains16);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) r[e] = in ? fmaf(g, y[e], a.residual * r[e]) : 0.f;
  if (a.out && in) store_unit(a.out, (int64_t)t * a.out_stride + u * 4, XT, r);
  if (a.next) {
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) ss = fmaf(r[e], r[e], ss);
    rn = rsqrtf(fmaf(row_sum(ss, red[1]), a.inv_n, a.eps));
    if (in) {
#pragma unroll
      for (int e = 0; e < 4; ++e) r[e] *= rn;
      if (a.pre_gain) times(r, a.pre_gain, u * 4, a.gains16);
      store_unit(a.next, (int64_t)t * a.next_stride + u * 4, a.next_type, r);
    }
  }
}

// ---- Rows of one part or none, on boundaries of 4 elements --------------------------------------------------
// A CTA takes every gridDim.x-th row, a thread V units of 4 columns, and reads the rows AHEAD of the one it works on into
// registers, so that memory never waits for a row's sums; the gains stay in registers where they are few.
template <int XT, int PT, int V, int AHEAD>
__global__ void __launch_bounds__(512) edge_stream_kernel(const __grid_constant__ NormArgs a) {
  griddep_wait();
  const int first_row = blockIdx.x * blockDim.y + threadIdx.y, row_step = gridDim.x * blockDim.y;
  constexpr bool PART = PT != NO_PARTS, KEEP = V <= 4;
  __shared__ float red[2][2][32];
  const int tid = threadIdx.x, threads = blockDim.x, units = a.n / 4;
  bool mine[V];
  float gains[KEEP ? 2 : 1][KEEP ? V : 1][4];  // of z: post and channel; of next
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int at = (tid + v * threads) * 4;
    mine[v] = tid + v * threads < units;
    if constexpr (KEEP) {
#pragma unroll
      for (int e = 0; e < 4; ++e) gains[0][v][e] = gains[1][v][e] = 1.f;
      if (mine[v]) {
        if (a.post_gain) times(gains[0][v], a.post_gain, at, a.gains16);
        if (a.channel) times(gains[0][v], a.channel, at, a.gains16);
        if (a.pre_gain) times(gains[1][v], a.pre_gain, at, a.gains16);
      }
    }
  }
  struct Row {
    Unit<XT> x[V];
    Unit<PART ? PT : XT> p[PART ? V : 1];
    float w, token;
  };
  const auto fetch = [&](int t, Row& row) {
    const bool in = t < a.T;
    row.w = PART && in && a.pw ? __ldg(a.pw + t) : 1.f;
    row.token = PART && in && a.token ? __ldg(a.token + t) : 1.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int u = (tid + v * threads) * 4;
      if (in && a.x && mine[v]) row.x[v].load(a.x, (int64_t)t * a.x_stride + u);
      else row.x[v].zero();
      if constexpr (PART) {
        // (a part of weight 0 is not read: its weight is waited for only where there are weights)
        if (in && mine[v] && (!a.pw || row.w != 0.f)) row.p[v].load(a.parts, (int64_t)t * a.token_stride + u);
        else row.p[v].zero();
      }
    }
  };
  Row rows[AHEAD];
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) fetch(first_row + i * row_step, rows[i]);
  int turn = 0;
  for (int t0 = first_row; t0 < a.T; t0 += AHEAD * row_step) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const int t = t0 + i * row_step;
      if (t >= a.T) break;
      float r[V][4];
#pragma unroll
      for (int v = 0; v < V; ++v) rows[i].x[v].widen(r[v]);
      if constexpr (PART) {
        float y[V][4], rn = 1.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          rows[i].p[v].widen(y[v]);
#pragma unroll
          for (int e = 0; e < 4; ++e) y[v][e] *= rows[i].w;
        }
        const float token = rows[i].token;
        fetch(t + AHEAD * row_step, rows[i]);
        const float g = a.block * (!a.token ? 1.f : a.sigmoid ? 1.f / (1.f + expf(-token)) : token);
        if (a.post) {
          float ss = 0.f;
#pragma unroll
          for (int v = 0; v < V; ++v)
#pragma unroll
            for (int e = 0; e < 4; ++e) ss = fmaf(y[v][e], y[v][e], ss);
          rn = rsqrtf(fmaf(row_sum(ss, red[turn][0]), a.inv_n, a.eps));
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
#pragma unroll
          for (int e = 0; e < 4; ++e) y[v][e] *= rn;
          if constexpr (KEEP) {
#pragma unroll
            for (int e = 0; e < 4; ++e) y[v][e] *= gains[0][v][e];
          } else if (mine[v]) {
            if (a.post_gain) times(y[v], a.post_gain, (tid + v * threads) * 4, a.gains16);
            if (a.channel) times(y[v], a.channel, (tid + v * threads) * 4, a.gains16);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) r[v][e] = mine[v] ? fmaf(g, y[v][e], a.residual * r[v][e]) : 0.f;
        }
      } else {
        fetch(t + AHEAD * row_step, rows[i]);
      }
      if (PART && a.out) {
#pragma unroll
        for (int v = 0; v < V; ++v)
          if (mine[v]) store_unit(a.out, (int64_t)t * a.out_stride + (tid + v * threads) * 4, XT, r[v]);
      }
      if (a.next) {
        float ss = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
          for (int e = 0; e < 4; ++e) ss = fmaf(r[v][e], r[v][e], ss);
        const float rn = rsqrtf(fmaf(row_sum(ss, red[turn][1]), a.inv_n, a.eps));
#pragma unroll
        for (int v = 0; v < V; ++v) {
          if (!mine[v]) continue;
#pragma unroll
          for (int e = 0; e < 4; ++e) r[v][e] *= rn;
          if constexpr (KEEP) {
#pragma unroll
            for (int e = 0; e < 4; ++e) r[v][e] *= gains[1][v][e];
          } else if (a.pre_gain) {
            times(r[v], a.pre_gain, (tid + v * threads) * 4, a.gains16);
          }
          store_unit(a.next, (int64_t)t * a.next_stride + (tid + v * threads) * 4, a.next_type, r[v]);
        }
      }
      turn ^= 1;
    }
  }
  griddep_launch_dependents();
}

// Rows a CTA: four of one warp each once the SMs have as many, since an SM holds 32 CTAs at most and starts them one by one
// (8,192 x 100: 3.2 us, a row a CTA 6.7).
int rows_a_cta(const NormArgs& a, int threads) { return threads == 32 && a.T > 4 * 152 ? 4 : 1; }

template <int XT, int PT, int V, int AHEAD>
cudaError_t launch_stream_v(const NormArgs& a, cudaStream_t s) {
  const int threads = ((a.n / 4 + V - 1) / V + 31) / 32 * 32;
  const int rows = rows_a_cta(a, threads), ctas = (a.T + rows - 1) / rows;
  const int fit = 152 * resident_ctas<edge_stream_kernel<XT, PT, V, AHEAD>>(threads * rows, 0);
  return launch_pdl(edge_stream_kernel<XT, PT, V, AHEAD>, ctas < fit ? ctas : fit, dim3(threads, rows), 0, s, a);
}

// Units a thread and rows ahead (2560 columns, 8,192 rows): without a part (fp32 to bf16) 2 and 2 22.4 us, 2 and 1 25.6, 4 and
// 1 23.4; with one (fp32, the stream in bf16) 4 and 1 38.6 us, 2 and 1 39.7, 2 and 2 50, 5 and 1 49, 10 and 1 66:
// more threads a row pay more for its two sums, more registers a thread leave fewer rows on their way.  Few rows are
// spread over more threads (four rows: 2.3 us).
template <int XT, int PT>
cudaError_t launch_stream(const NormArgs& a, cudaStream_t s) {
  const int units = a.n / 4;
  if (units > 2048) return launch_stream_v<XT, PT, 8, 1>(a, s);
  if (units > 1024 || (units > 64 && units <= 128) || (PT != NO_PARTS && a.T > 152)) return launch_stream_v<XT, PT, 4, 1>(a, s);
  return launch_stream_v<XT, PT, 2, PT == NO_PARTS ? 2 : 1>(a, s);
}

// ---- Rows with parts, on boundaries of 4 elements -----------------------------------------------------------
// A CTA takes every gridDim.x-th row, a thread V units of 4 columns.  What a row needs is a line of steps, its parts of weight
// other than 0 in order and then x; the steps of this row and the next ones are on their way by cp.async into a ring of
// shared memory, where a thread finds the pieces that it copied itself: no barrier, and memory never waits for
// a row's sums.  The gains stay in registers where they are few.
template <int XT, int PT, int V, int RING>
__global__ void __launch_bounds__(512) edge_ring_kernel(const __grid_constant__ NormArgs a) {
  griddep_wait();
  const int first_row = blockIdx.x * blockDim.y + threadIdx.y, row_step = gridDim.x * blockDim.y;
  extern __shared__ __align__(16) uint4 s_rings[];  // [blockDim.y][ring][V][threads]
  __shared__ float red[2][2][32];
  const int tid = threadIdx.x, threads = blockDim.x, lane = tid & 31, units = a.n / 4;
  const int slot_units = V * threads;
  uint4* const s_ring = s_rings + threadIdx.y * RING * slot_units;
  bool mine[V];
#pragma unroll
  for (int v = 0; v < V; ++v) mine[v] = tid + v * threads < units;
  constexpr bool KEEP = V <= 4;
  float gains[KEEP ? 2 : 1][KEEP ? V : 1][4];  // of z: post and channel; of next
  if constexpr (KEEP) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int at = (tid + v * threads) * 4;
#pragma unroll
      for (int e = 0; e < 4; ++e) gains[0][v][e] = gains[1][v][e] = 1.f;
      if (mine[v]) {
        if (a.post_gain) times(gains[0][v], a.post_gain, at, a.gains16);
        if (a.channel) times(gains[0][v], a.channel, at, a.gains16);
        if (a.pre_gain) times(gains[1][v], a.pre_gain, at, a.gains16);
      }
    }
  }
  const auto weight = [&](int t) { return t >= a.T || lane >= a.P ? 0.f : a.pw ? __ldg(a.pw + (int64_t)t * a.P + lane) : 1.f; };
  constexpr int P_SIZE = PT == STRATA_F32 ? 4 : 2, X_SIZE = XT == STRATA_F32 ? 4 : 2;
  const uint32_t s_mine = smem_u32(s_ring + tid);
  const auto copy = [&](int slot, const char* from, int size) {
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (mine[v]) {
        const uint32_t to = s_mine + (uint32_t)(slot * slot_units + v * threads) * 16u;
        const char* const at = from + (size_t)(tid + v * threads) * (4 * size);
        if (size == 4) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(at) : "memory");
        else asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(at) : "memory");
      }
  };
  // the step to be copied next: part `ffs(todo)` of row tc, or its x
  int tc = first_row, cslot = 0;
  float wc = weight(tc), wn = weight(tc + row_step);
  uint32_t todo = __ballot_sync(0xffffffffu, wc != 0.f);
  bool x_to_do = a.x != nullptr;
  const auto copy_next = [&]() {
    while (tc < a.T && !todo && !x_to_do) {
      tc += row_step;
      wc = wn;
      wn = weight(tc + row_step);
      todo = __ballot_sync(0xffffffffu, wc != 0.f);
      x_to_do = a.x != nullptr;
    }
    if (tc < a.T) {
      if (todo) {
        const int k = __ffs(todo) - 1;
        todo &= todo - 1;
        copy(cslot, static_cast<const char*>(a.parts) + ((int64_t)tc * a.token_stride + k * a.part_stride) * P_SIZE, P_SIZE);
      } else {
        x_to_do = false;
        copy(cslot, static_cast<const char*>(a.x) + (int64_t)tc * a.x_stride * X_SIZE, X_SIZE);
      }
      cslot = cslot + 1 == RING ? 0 : cslot + 1;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  for (int i = 0; i < RING - 1; ++i) copy_next();
  int slot = 0, turn = 0;
  float w = weight(first_row);
  for (int t = first_row; t < a.T; t += row_step, turn ^= 1) {
    const float w_next = weight(t + row_step);
    const float tok = a.token ? __ldg(a.token + t) : 1.f;
    float y[V][4], r[V][4];
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int e = 0; e < 4; ++e) y[v][e] = r[v][e] = 0.f;
    for (uint32_t parts = __ballot_sync(0xffffffffu, w != 0.f); parts; parts &= parts - 1) {
      const float wk = __shfl_sync(0xffffffffu, w, __ffs(parts) - 1);
      asm volatile("cp.async.wait_group %0;" ::"n"(RING - 2) : "memory");
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (mine[v]) {
          Unit<PT> p;
          float f[4];
          p.load(s_ring + slot * slot_units + v * threads + tid, 0);
          p.widen(f);
#pragma unroll
          for (int e = 0; e < 4; ++e) y[v][e] = fmaf(wk, f[e], y[v][e]);
        }
      slot = slot + 1 == RING ? 0 : slot + 1;
      copy_next();  // into the slot before the one just read
    }
    w = w_next;
    if (a.x) {
      asm volatile("cp.async.wait_group %0;" ::"n"(RING - 2) : "memory");
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (mine[v]) {
          Unit<XT> p;
          p.load(s_ring + slot * slot_units + v * threads + tid, 0);
          p.widen(r[v]);
        }
      slot = slot + 1 == RING ? 0 : slot + 1;
      copy_next();
    }
    const float g = a.block * (!a.token ? 1.f : a.sigmoid ? 1.f / (1.f + expf(-tok)) : tok);
    float rn = 1.f;
    if (a.post) {
      float ss = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int e = 0; e < 4; ++e) ss = fmaf(y[v][e], y[v][e], ss);
      rn = rsqrtf(fmaf(row_sum(ss, red[turn][0]), a.inv_n, a.eps));
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int u = tid + v * threads;
#pragma unroll
      for (int e = 0; e < 4; ++e) y[v][e] *= rn;
      if constexpr (KEEP) {
#pragma unroll
        for (int e = 0; e < 4; ++e) y[v][e] *= gains[0][v][e];
      } else if (mine[v]) {
        if (a.post_gain) times(y[v], a.post_gain, u * 4, a.gains16);
        if (a.channel) times(y[v], a.channel, u * 4, a.gains16);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) r[v][e] = mine[v] ? fmaf(g, y[v][e], a.residual * r[v][e]) : 0.f;
      if (a.out && mine[v]) store_unit(a.out, (int64_t)t * a.out_stride + (int64_t)u * 4, XT, r[v]);
    }
    if (a.next) {
      float ss = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int e = 0; e < 4; ++e) ss = fmaf(r[v][e], r[v][e], ss);
      rn = rsqrtf(fmaf(row_sum(ss, red[turn][1]), a.inv_n, a.eps));
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (!mine[v]) continue;
        const int u = tid + v * threads;
#pragma unroll
        for (int e = 0; e < 4; ++e) r[v][e] *= rn;
        if constexpr (KEEP) {
#pragma unroll
          for (int e = 0; e < 4; ++e) r[v][e] *= gains[1][v][e];
        } else if (a.pre_gain) {
          times(r[v], a.pre_gain, u * 4, a.gains16);
        }
        store_unit(a.next, (int64_t)t * a.next_stride + (int64_t)u * 4, a.next_type, r[v]);
      }
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  griddep_launch_dependents();
}

template <int XT, int PT, int V, int RING>
cudaError_t launch_ring_v(const NormArgs& a, cudaStream_t s) {
  const int threads = ((a.n / 4 + V - 1) / V + 31) / 32 * 32, rows = rows_a_cta(a, threads), smem = rows * RING * V * threads * 16;
  const cudaError_t err = allow_smem<edge_ring_kernel<XT, PT, V, RING>>(224 * 1024);
  if (err != cudaSuccess) return err;
  const int ctas = (a.T + rows - 1) / rows, fit = 152 * resident_ctas<edge_ring_kernel<XT, PT, V, RING>>(threads * rows, smem);
  return launch_pdl(edge_ring_kernel<XT, PT, V, RING>, ctas < fit ? ctas : fit, dim3(threads, rows), smem, s, a);
}

// Slots: 6 of up to 16 KB, or 3 of up to 64 KB.
template <int XT, int PT>
cudaError_t launch_ring(const NormArgs& a, cudaStream_t s) {
  const int units = a.n / 4;
  if (units <= 1024 && a.T <= 152) {
    return launch_pdl(edge_few_kernel<XT, PT>, a.T, (units + 31) / 32 * 32, 0, s, a);
  }
  if (units > 2048) return launch_ring_v<XT, PT, 8, 3>(a, s);
  if (units > 1024 || (units > 64 && units <= 128)) return launch_ring_v<XT, PT, 4, 3>(a, s);  // (a warp's rows up to 512 wide)
  return launch_ring_v<XT, PT, 2, 6>(a, s);
}

// ---- Rows that are not on boundaries of 4 elements ----------------------------------------------------------
// The same line of steps, copied as the 16-byte pieces that hold a row's bytes, wherever in them it starts, and
// taken out of shared memory a column at a time: a warp has 32 V columns in a row, a thread every 32nd (so a row's
// addresses differ by constants: these rows are bound by instructions, issued in 50 to 69% of cycles).  A thread
// reads what others copied, so that a step costs a barrier; it also frees the slot read before.  2,559 columns: the norm of
// 8,192 rows from fp32 to bf16 24.4 us (5.1 TB/s), 2,048 rows of ten fp32 parts 52 us (5.2 TB/s).
// f(v) for a lane's columns, v of V; all of a warp inside its row as a rule.
template <int V, class F>
__device__ __forceinline__ void each_column(int left, F f) {
  if (__all_sync(0xffffffffu, left > 32 * (V - 1))) {
#pragma unroll
    for (int v = 0; v < V; ++v) f(v);
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (32 * v < left) f(v);
  }
}
template <int T, int V>
__device__ __forceinline__ void store_columns(void* p, int64_t at, int left, const float (&f)[V]) {
  void* const to = static_cast<unsigned char*>(p) + at * (T == STRATA_F32 ? 4 : 2);
  each_column<V>(left, [&](int v) { store1(to, 32 * v, T, f[v]); });
}
template <int XT, int PT, int V, int RING>
__global__ void __launch_bounds__(512, V <= 8 ? 2 : 1) edge_columns_kernel(const __grid_constant__ NormArgs a, int slot_bytes) {
  griddep_wait();
  const int first_row = blockIdx.x * blockDim.y + threadIdx.y, row_step = gridDim.x * blockDim.y;
  extern __shared__ __align__(16) unsigned char s_bytes_all[];  // [blockDim.y][ring][slot_bytes]
  unsigned char* const s_bytes = s_bytes_all + threadIdx.y * RING * slot_bytes;
  __shared__ float red[2][2][32];
  constexpr bool PARTS = PT != NO_PARTS;
  constexpr int P_SIZE = PT == STRATA_F32 ? 4 : 2, X_SIZE = XT == STRATA_F32 ? 4 : 2;
  const int tid = threadIdx.x, threads = blockDim.x, lane = tid & 31;
  const int first = (tid - lane) * V + lane, left = a.n - first;  // its columns: first + 32 v, while 32 v < left
  constexpr bool KEEP = V <= 16;
  float gains[KEEP ? 2 : 1][KEEP ? V : 1];  // of z: post and channel; of next
  if constexpr (KEEP) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int u = first + 32 * v;
      gains[0][v] = gains[1][v] = 1.f;
      if (32 * v < left) {
        if (PARTS && a.post_gain) gains[0][v] = __ldg(a.post_gain + u);
        if (PARTS && a.channel) gains[0][v] *= __ldg(a.channel + u);
        if (a.pre_gain) gains[1][v] = __ldg(a.pre_gain + u);
      }
    }
  }
  const auto weight = [&](int t) { return t >= a.T || lane >= a.P ? 0.f : a.pw ? __ldg(a.pw + (int64_t)t * a.P + lane) : 1.f; };
  const auto part_at = [&](int t, int k) {
    return static_cast<const unsigned char*>(a.parts) + ((int64_t)t * a.token_stride + k * a.part_stride) * P_SIZE;
  };
  const auto x_at = [&](int t) { return static_cast<const unsigned char*>(a.x) + (int64_t)t * a.x_stride * X_SIZE; };
  const uint32_t s_mine = smem_u32(s_bytes) + tid * 16;
  // The pieces of `bytes` bytes at `from`.  The first may begin before the row: a piece that holds one byte of an
  // allocation lies inside it at that end.  The last is cut at the row's end.
  const auto copy = [&](int slot, const unsigned char* from, int bytes) {
    const int off = (int)(reinterpret_cast<uintptr_t>(from) & 15);
    const unsigned char* at = from - off + tid * 16;
    uint32_t to = s_mine + slot * slot_bytes;
    for (int left = bytes + off - tid * 16; left > 0; left -= threads * 16, at += threads * 16, to += threads * 16)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(at), "r"(left < 16 ? left : 16) : "memory");
  };
  int tc = first_row, cslot = 0;
  float wc = PARTS ? weight(tc) : 0.f, wn = PARTS ? weight(tc + row_step) : 0.f;
  uint32_t todo = PARTS ? __ballot_sync(0xffffffffu, wc != 0.f) : 0u;
  bool x_to_do = a.x != nullptr;
  const auto copy_next = [&]() {
    while (tc < a.T && !todo && !x_to_do) {
      tc += row_step;
      if constexpr (PARTS) {
        wc = wn;
        wn = weight(tc + row_step);
        todo = __ballot_sync(0xffffffffu, wc != 0.f);
      }
      x_to_do = a.x != nullptr;
    }
    if (tc < a.T) {
      if (todo) {
        const int k = __ffs(todo) - 1;
        todo &= todo - 1;
        copy(cslot, part_at(tc, k), a.n * P_SIZE);
      } else {
        x_to_do = false;
        copy(cslot, x_at(tc), a.n * X_SIZE);
      }
      cslot = cslot + 1 == RING ? 0 : cslot + 1;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  int slot = 0, turn = 0;
  // the step's bytes as this thread's first column finds them
  const auto next_slot = [&](const unsigned char* from, int size) {
    asm volatile("cp.async.wait_group %0;" ::"n"(RING - 2) : "memory");
    if (threads == 32) __syncwarp();
    else __syncthreads();
    const unsigned char* const at = s_bytes + slot * slot_bytes + (int)(reinterpret_cast<uintptr_t>(from) & 15) + first * size;
    slot = slot + 1 == RING ? 0 : slot + 1;
    copy_next();  // into the slot read before this one
    return at;
  };
  for (int i = 0; i < RING - 1; ++i) copy_next();
  float w = PARTS ? weight(first_row) : 0.f;
  for (int t = first_row; t < a.T; t += row_step, turn ^= 1) {
    const float w_next = PARTS ? weight(t + row_step) : 0.f;
    const float tok = PARTS && a.token ? __ldg(a.token + t) : 1.f;
    float y[V], r[V];
#pragma unroll
    for (int v = 0; v < V; ++v) y[v] = r[v] = 0.f;
    if constexpr (PARTS) {
      for (uint32_t parts = __ballot_sync(0xffffffffu, w != 0.f); parts; parts &= parts - 1) {
        const int k = __ffs(parts) - 1;
        const float wk = __shfl_sync(0xffffffffu, w, k);
        const unsigned char* const at = next_slot(part_at(t, k), P_SIZE);
        each_column<V>(left, [&](int v) { y[v] = fmaf(wk, load1(at, 32 * v, PT), y[v]); });
      }
    }
    w = w_next;
    if (a.x) {
      const unsigned char* const at = next_slot(x_at(t), X_SIZE);
      each_column<V>(left, [&](int v) { r[v] = load1(at, 32 * v, XT); });
    }
    if constexpr (PARTS) {
      const float g = a.block * (!a.token ? 1.f : a.sigmoid ? 1.f / (1.f + expf(-tok)) : tok);
      float rn = 1.f;
      if (a.post) {
        float ss = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) ss = fmaf(y[v], y[v], ss);
        rn = rsqrtf(fmaf(row_sum(ss, red[turn][0]), a.inv_n, a.eps));
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int u = first + 32 * v;
        const bool in = 32 * v < left;
        float z = y[v] * rn;
        if constexpr (KEEP) {
          z *= gains[0][v];
        } else {
          if (a.post_gain && in) z *= __ldg(a.post_gain + u);
          if (a.channel && in) z *= __ldg(a.channel + u);
        }
        r[v] = in ? fmaf(g, z, a.residual * r[v]) : 0.f;
      }
    }
    if (PARTS && a.out) store_columns<XT>(a.out, (int64_t)t * a.out_stride + first, left, r);
    if (a.next) {
      float ss = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) ss = fmaf(r[v], r[v], ss);
      const float rn = rsqrtf(fmaf(row_sum(ss, red[turn][1]), a.inv_n, a.eps));
#pragma unroll
      for (int v = 0; v < V; ++v) {
        r[v] *= rn;
        if constexpr (KEEP) r[v] *= gains[1][v];
        else if (a.pre_gain && 32 * v < left) r[v] *= __ldg(a.pre_gain + first + 32 * v);
      }
      const int64_t at = (int64_t)t * a.next_stride + first;
      if (a.next_type == STRATA_F32) store_columns<STRATA_F32>(a.next, at, left, r);
      else if (a.next_type == STRATA_BF16) store_columns<STRATA_BF16>(a.next, at, left, r);
      else store_columns<STRATA_F16>(a.next, at, left, r);
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  griddep_launch_dependents();
}

template <int XT, int PT, int V, int RING>
cudaError_t launch_columns_v(const NormArgs& a, cudaStream_t s) {
  const int threads = ((a.n + V - 1) / V + 31) / 32 * 32;
  // a slot: all of the threads' columns and the 15 bytes that a row may start behind a piece, 16 a warp (so that shared memory
  // goes with the number of threads alone, as resident_ctas has it)
  constexpr int SIZE = XT == STRATA_F32 || PT == STRATA_F32 ? 4 : 2;
  const int slot = threads / 32 * (32 * V * SIZE + 16);
  const cudaError_t err = allow_smem<edge_columns_kernel<XT, PT, V, RING>>(224 * 1024);
  if (err != cudaSuccess) return err;
  const int rows = rows_a_cta(a, threads), ctas = (a.T + rows - 1) / rows, smem = rows * RING * slot;
  const int fit = 152 * resident_ctas<edge_columns_kernel<XT, PT, V, RING>>(threads * rows, smem);
  return launch_pdl(edge_columns_kernel<XT, PT, V, RING>, ctas < fit ? ctas : fit, dim3(threads, rows), smem, s, a, slot);
}

// Slots: 4 of up to 16 KB, or 3 of up to 64 KB.
template <int XT, int PT>
cudaError_t launch_columns(const NormArgs& a, cudaStream_t s) {
  if (a.n > 8192) return launch_columns_v<XT, PT, 32, 3>(a, s);
  if (a.n > 4096) return launch_columns_v<XT, PT, 16, 3>(a, s);
  // 2,559 columns in us, a lane 16 or 8 of them: the norm of 8,192 rows 24.8 and 25.4 (bf16 18.9 and 23.5), one part 57 and 66,
  // 2,048 rows of ten parts 57 and 53.
  if (a.n > 1024 && a.P <= 1) return launch_columns_v<XT, PT, 16, 3>(a, s);
  return launch_columns_v<XT, PT, 8, 4>(a, s);
}

// Every row of the operand starts on a boundary of four elements.
bool rows4(const void* p, int64_t stride, int type) {
  const int64_t size = type == STRATA_F32 ? 4 : 2;
  return !p || (((uintptr_t)p & (4 * size - 1)) == 0 && stride % 4 == 0);
}

template <int XT, int PT>
cudaError_t launch_parts(const NormArgs& a, bool vec, cudaStream_t s) {
  if constexpr (PT != NO_PARTS)
    if (vec && a.P > 1) return launch_ring<XT, PT>(a, s);
  return vec ? launch_stream<XT, PT>(a, s) : launch_columns<XT, PT>(a, s);
}

template <int XT>
cudaError_t launch_types(const NormArgs& a, bool vec, cudaStream_t s) {
  if (!a.parts) return launch_parts<XT, NO_PARTS>(a, vec, s);
  return a.part_type == STRATA_F32    ? launch_parts<XT, STRATA_F32>(a, vec, s)
         : a.part_type == STRATA_BF16 ? launch_parts<XT, STRATA_BF16>(a, vec, s)
                                      : launch_parts<XT, STRATA_F16>(a, vec, s);
}

cudaError_t launch_edge(NormArgs a, int kid, cudaStream_t s) {
  const bool vec = a.n % 4 == 0 && rows4(a.parts, a.part_stride, a.part_type) &&
                   rows4(a.parts, a.token_stride, a.part_type) && rows4(a.x, a.x_stride, a.x_type) &&
                   rows4(a.out, a.out_stride, a.x_type) && rows4(a.next, a.next_stride, a.next_type);
  a.inv_n = 1.f / (float)a.n;
  a.gains16 = (((uintptr_t)a.post_gain | (uintptr_t)a.channel | (uintptr_t)a.pre_gain) & 15) == 0;
  kernel_begin(kid, s);
  const cudaError_t err = a.x_type == STRATA_F32    ? launch_types<STRATA_F32>(a, vec, s)
                          : a.x_type == STRATA_BF16 ? launch_types<STRATA_BF16>(a, vec, s)
                                                    : launch_types<STRATA_F16>(a, vec, s);
  kernel_end(kid, s);
  return err;
}

}  // namespace

cudaError_t launch_norm(const strata_norm_t& nd, const void* x, int T, const float* gain, void* out, cudaStream_t s) {
  NormArgs a{};
  a.x = x; a.x_stride = nd.x_stride; a.x_type = nd.x_type;
  a.next = out; a.next_stride = nd.out_stride; a.next_type = nd.out_type;
  a.pre_gain = gain; a.T = T; a.n = nd.n; a.eps = nd.eps;
  return launch_edge(a, KID_NORM, s);
}

cudaError_t launch_combine_norm(const strata_combine_norm_t& cn, const void* parts, const float* part_weights,
                                const void* x, int T, const float* post_gain, const float* channel_gate,
                                const float* token_gate, const float* pre_gain, void* out, void* next, cudaStream_t s) {
  NormArgs a{};
  a.parts = parts; a.pw = part_weights; a.P = cn.n_part; a.part_type = cn.part_type;
  a.part_stride = cn.part_stride; a.token_stride = cn.token_stride;
  a.x = x; a.x_stride = cn.x_stride; a.x_type = cn.x_type;
  a.post = (cn.flags & STRATA_POST_NORM) ? 1 : 0; a.post_gain = post_gain;
  a.sigmoid = (cn.flags & STRATA_TOKEN_SIGMOID) ? 1 : 0; a.channel = channel_gate; a.token = token_gate;
  a.pre_gain = pre_gain; a.eps = cn.eps; a.residual = cn.residual_scale; a.block = cn.block_scale;
  a.out = out; a.out_stride = cn.out_stride; a.next = next; a.next_stride = cn.next_stride; a.next_type = cn.next_type;
  a.T = T; a.n = cn.n;
  return launch_edge(a, KID_COMBINE_NORM, s);
}

}  // namespace strata
