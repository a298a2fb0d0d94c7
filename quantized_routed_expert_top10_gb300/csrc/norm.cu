// The norms before and after the block (strata_moe_norm, strata_moe_combine_norm), sm_103a.
//
// zwxr.cn news/242664, section "一次路由的完整旅程": moe_combine adds the experts' outputs weighted by the router's
// weights to the layer's input; the layers read a normalised activation.  Here the weighted sum, the norm of the
// block's output, its gates, the scaled residual and the next block's norm are one pass: a row is held in registers
// between its one read and its one write, both mean squares are sums over its CTA.
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

// W consecutive elements of type T as a unit, as read: 1, or 4 on a boundary of their size (16 bytes of fp32, so that a
// warp's accesses are contiguous whatever the types of the operands).
template <int T, int W>
struct Unit;
template <int T>
struct Unit<T, 4> {
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
template <int T>
struct Unit<T, 1> {
  float r;
  __device__ __forceinline__ void load(const void* p, int64_t i) { r = load1(p, i, T); }
  __device__ __forceinline__ void zero() { r = 0.f; }
  __device__ __forceinline__ void widen(float (&f)[1]) const { f[0] = r; }
};
template <int W>
__device__ __forceinline__ void store_unit(void* p, int64_t i, int type, const float (&f)[W]) {
  if constexpr (W == 4) {
    if (type == STRATA_F32) *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = make_float4(f[0], f[1], f[2], f[3]);
    else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + i) = make_uint2(narrow2(f[0], f[1], type), narrow2(f[2], f[3], type));
  } else {
    store1(p, i, type, f[0]);
  }
}
// f *= g[i .. i + W - 1] (fp32)
template <int W>
__device__ __forceinline__ void times(float (&f)[W], const float* g, int i, bool aligned) {
  if constexpr (W == 4) {
    if (aligned) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(g + i));
      f[0] *= a.x; f[1] *= a.y; f[2] *= a.z; f[3] *= a.w;
      return;
    }
  }
#pragma unroll
  for (int e = 0; e < W; ++e) f[e] *= __ldg(g + i + e);
}

constexpr int NO_PARTS = -1;

// One row per blockDim.x threads; a thread holds V units of W elements, blockDim.x units apart.  Memory bounds it: all
// of a row is read before the first sum (x, and GROUP parts at a time), and a row's threads are few (one warp in a long
// call), so that many rows are on their way at once and no barrier holds them.
template <int XT, int PT, int W, int V>
__global__ void __launch_bounds__(1024) edge_kernel(const __grid_constant__ NormArgs a) {
  constexpr int GROUP = PT == NO_PARTS || V == 16 ? 1 : W == 4 ? 10 : 5;
  __shared__ float red[2][32];
  const int t = blockIdx.x * blockDim.y + threadIdx.y;
  if (t >= a.T) return;  // whole warps; only one-warp rows share a CTA
  const int units = a.n / W, step = blockDim.x;
  Unit<XT, W> x[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int u = threadIdx.x + v * step;
    if (a.x && u < units) x[v].load(a.x, (int64_t)t * a.x_stride + (int64_t)u * W);
    else x[v].zero();
  }
  float r[V][W];
  if constexpr (PT != NO_PARTS) {
    const int lane = threadIdx.x & 31;
    const float mine = lane >= a.P ? 0.f : a.pw ? __ldg(a.pw + (int64_t)t * a.P + lane) : 1.f;  // P <= 32
    float g = a.block;
    if (a.token) {
      const float s = __ldg(a.token + t);
      g *= a.sigmoid ? 1.f / (1.f + expf(-s)) : s;
    }
    float y[V][W];
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int i = 0; i < W; ++i) y[v][i] = 0.f;
    for (int k0 = 0; k0 < a.P; k0 += GROUP) {
      Unit<PT, W> p[GROUP][V];
      float w[GROUP];
#pragma unroll
      for (int k = 0; k < GROUP; ++k) {
        w[k] = k0 + k < 32 ? __shfl_sync(0xffffffffu, mine, (k0 + k) & 31) : 0.f;
        const int64_t at = (int64_t)t * a.token_stride + (k0 + k) * a.part_stride;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const int u = threadIdx.x + v * step;
          if (w[k] != 0.f && u < units) p[k][v].load(a.parts, at + (int64_t)u * W);  // (a part of weight 0 is not read)
          else p[k][v].zero();
        }
      }
#pragma unroll
      for (int k = 0; k < GROUP; ++k)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          float f[W];
          p[k][v].widen(f);
#pragma unroll
          for (int i = 0; i < W; ++i) y[v][i] = fmaf(w[k], f[i], y[v][i]);
        }
    }
    float rn = 1.f;
    if (a.post) {
      float ss = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < W; ++i) ss = fmaf(y[v][i], y[v][i], ss);
      rn = rsqrtf(fmaf(row_sum(ss, red[0]), a.inv_n, a.eps));
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int u = threadIdx.x + v * step;
      float z[W], xf[W];
      x[v].widen(xf);
#pragma unroll
      for (int i = 0; i < W; ++i) z[i] = y[v][i] * rn;
      if (u < units) {
        if (a.post_gain) times<W>(z, a.post_gain, u * W, a.gains16);
        if (a.channel) times<W>(z, a.channel, u * W, a.gains16);
      }
#pragma unroll
      for (int i = 0; i < W; ++i) r[v][i] = u < units ? fmaf(g, z[i], a.residual * xf[i]) : 0.f;
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) x[v].widen(r[v]);
  }
  if (a.out) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int u = threadIdx.x + v * step;
      if (u < units) store_unit<W>(a.out, (int64_t)t * a.out_stride + (int64_t)u * W, a.x_type, r[v]);
    }
  }
  if (a.next) {
    float ss = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int i = 0; i < W; ++i) ss = fmaf(r[v][i], r[v][i], ss);
    const float rn = rsqrtf(fmaf(row_sum(ss, red[1]), a.inv_n, a.eps));
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int u = threadIdx.x + v * step;
      if (u >= units) continue;
      float f[W];
#pragma unroll
      for (int i = 0; i < W; ++i) f[i] = r[v][i] * rn;
      if (a.pre_gain) times<W>(f, a.pre_gain, u * W, a.gains16);
      store_unit<W>(a.next, (int64_t)t * a.next_stride + (int64_t)u * W, a.next_type, f);
    }
  }
}

// ---- Rows of one part or none, on boundaries of 4 elements --------------------------------------------------
// A CTA takes every gridDim.x-th row, a thread V units of 4 columns, and reads the rows AHEAD of the one it works on into
// registers, so that memory never waits for a row's sums; the gains stay in registers where they are few.
template <int XT, int PT, int V, int AHEAD>
__global__ void __launch_bounds__(512) edge_stream_kernel(const __grid_constant__ NormArgs a) {
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
        if (a.post_gain) times<4>(gains[0][v], a.post_gain, at, a.gains16);
        if (a.channel) times<4>(gains[0][v], a.channel, at, a.gains16);
        if (a.pre_gain) times<4>(gains[1][v], a.pre_gain, at, a.gains16);
      }
    }
  }
  struct Row {
    Unit<XT, 4> x[V];
    Unit<PART ? PT : XT, 4> p[PART ? V : 1];
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
  for (int i = 0; i < AHEAD; ++i) fetch(blockIdx.x + i * gridDim.x, rows[i]);
  int turn = 0;
  for (int t0 = blockIdx.x; t0 < a.T; t0 += AHEAD * gridDim.x) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const int t = t0 + i * gridDim.x;
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
        fetch(t + AHEAD * gridDim.x, rows[i]);
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
            if (a.post_gain) times<4>(y[v], a.post_gain, (tid + v * threads) * 4, a.gains16);
            if (a.channel) times<4>(y[v], a.channel, (tid + v * threads) * 4, a.gains16);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) r[v][e] = mine[v] ? fmaf(g, y[v][e], a.residual * r[v][e]) : 0.f;
        }
      } else {
        fetch(t + AHEAD * gridDim.x, rows[i]);
      }
      if (PART && a.out) {
#pragma unroll
        for (int v = 0; v < V; ++v)
          if (mine[v]) store_unit<4>(a.out, (int64_t)t * a.out_stride + (tid + v * threads) * 4, XT, r[v]);
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
            times<4>(r[v], a.pre_gain, (tid + v * threads) * 4, a.gains16);
          }
          store_unit<4>(a.next, (int64_t)t * a.next_stride + (tid + v * threads) * 4, a.next_type, r[v]);
        }
      }
      turn ^= 1;
    }
  }
}

template <int XT, int PT, int V, int AHEAD>
cudaError_t launch_stream_v(const NormArgs& a, cudaStream_t s) {
  const int threads = ((a.n / 4 + V - 1) / V + 31) / 32 * 32;
  const int fit = 152 * resident_ctas<edge_stream_kernel<XT, PT, V, AHEAD>>(threads, 0);
  edge_stream_kernel<XT, PT, V, AHEAD><<<a.T < fit ? a.T : fit, threads, 0, s>>>(a);
  return cudaGetLastError();
}

// Units a thread and rows ahead (2560 columns, 8,192 rows): without a part (fp32 to bf16) 2 and 2 22.4 us, 2 and 1 25.6, 4 and
// 1 23.4; with one (fp32, the stream in bf16) 4 and 1 38.6 us, 2 and 1 39.7, 2 and 2 50, 5 and 1 49, 10 and 1 66:
// more threads a row pay more for its two sums, more registers a thread leave fewer rows on their way.  Few rows are
// spread over more threads (four rows: 2.3 us).
template <int XT, int PT>
cudaError_t launch_stream(const NormArgs& a, cudaStream_t s) {
  const int units = a.n / 4;
  if (units > 2048) return launch_stream_v<XT, PT, 8, 1>(a, s);
  if (units > 1024 || (PT != NO_PARTS && a.T > 152)) return launch_stream_v<XT, PT, 4, 1>(a, s);
  return launch_stream_v<XT, PT, 2, PT == NO_PARTS ? 2 : 1>(a, s);
}

// ---- Rows with parts, on boundaries of 4 elements -----------------------------------------------------------
// A CTA takes every gridDim.x-th row, a thread V units of 4 columns.  What a row needs is a line of steps, its parts of weight
// other than 0 in order and then x; the steps of this row and the next ones are on their way by cp.async into a ring of
// shared memory, where a thread finds the pieces that it copied itself: no barrier, and memory never waits for
// a row's sums.  The gains stay in registers where a thread has two units.
template <int XT, int PT, int V, int RING>
__global__ void __launch_bounds__(512) edge_ring_kernel(const __grid_constant__ NormArgs a) {
  extern __shared__ __align__(16) uint4 s_ring[];  // [ring][V][threads]
  __shared__ float red[2][2][32];
  const int tid = threadIdx.x, threads = blockDim.x, lane = tid & 31, units = a.n / 4;
  const int slot_units = V * threads;
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
        if (a.post_gain) times<4>(gains[0][v], a.post_gain, at, a.gains16);
        if (a.channel) times<4>(gains[0][v], a.channel, at, a.gains16);
        if (a.pre_gain) times<4>(gains[1][v], a.pre_gain, at, a.gains16);
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
  int tc = blockIdx.x, cslot = 0;
  float wc = weight(tc), wn = weight(tc + gridDim.x);
  uint32_t todo = __ballot_sync(0xffffffffu, wc != 0.f);
  bool x_to_do = a.x != nullptr;
  const auto copy_next = [&]() {
    while (tc < a.T && !todo && !x_to_do) {
      tc += gridDim.x;
      wc = wn;
      wn = weight(tc + gridDim.x);
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
  float w = weight(blockIdx.x);
  for (int t = blockIdx.x; t < a.T; t += gridDim.x, turn ^= 1) {
    const float w_next = weight(t + gridDim.x);
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
          Unit<PT, 4> p;
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
          Unit<XT, 4> p;
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
        if (a.post_gain) times<4>(y[v], a.post_gain, u * 4, a.gains16);
        if (a.channel) times<4>(y[v], a.channel, u * 4, a.gains16);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) r[v][e] = mine[v] ? fmaf(g, y[v][e], a.residual * r[v][e]) : 0.f;
      if (a.out && mine[v]) store_unit<4>(a.out, (int64_t)t * a.out_stride + (int64_t)u * 4, XT, r[v]);
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
          times<4>(r[v], a.pre_gain, u * 4, a.gains16);
        }
        store_unit<4>(a.next, (int64_t)t * a.next_stride + (int64_t)u * 4, a.next_type, r[v]);
      }
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

template <int XT, int PT, int V, int RING>
cudaError_t launch_ring_v(const NormArgs& a, cudaStream_t s) {
  const int threads = ((a.n / 4 + V - 1) / V + 31) / 32 * 32, smem = RING * V * threads * 16;
  const cudaError_t err = allow_smem<edge_ring_kernel<XT, PT, V, RING>>(224 * 1024);
  if (err != cudaSuccess) return err;
  const int fit = 152 * resident_ctas<edge_ring_kernel<XT, PT, V, RING>>(threads, smem);
  edge_ring_kernel<XT, PT, V, RING><<<a.T < fit ? a.T : fit, threads, smem, s>>>(a);
  return cudaGetLastError();
}

// Slots: 6 of up to 16 KB, or 3 of up to 64 KB.
template <int XT, int PT>
cudaError_t launch_ring(const NormArgs& a, cudaStream_t s) {
  const int units = a.n / 4;
  if (units <= 1024 && a.T <= 152) {
    edge_kernel<XT, PT, 4, 1><<<a.T, (units + 31) / 32 * 32, 0, s>>>(a);
    return cudaGetLastError();
  }
  if (units > 2048) return launch_ring_v<XT, PT, 8, 3>(a, s);
  if (units > 1024) return launch_ring_v<XT, PT, 4, 3>(a, s);
  return launch_ring_v<XT, PT, 2, 6>(a, s);
}

// Every row of the operand starts on a boundary of four elements.
bool rows4(const void* p, int64_t stride, int type) {
  const int64_t size = type == STRATA_F32 ? 4 : 2;
  return !p || (((uintptr_t)p & (4 * size - 1)) == 0 && stride % 4 == 0);
}

// Rows that are not on boundaries of four elements go element by element.
template <int XT, int PT>
cudaError_t launch_parts(const NormArgs& a, bool vec, cudaStream_t s) {
  if (vec) {
    if constexpr (PT != NO_PARTS)
      if (a.P > 1) return launch_ring<XT, PT>(a, s);
    return launch_stream<XT, PT>(a, s);
  }
  const int V = a.n <= 4096 ? 4 : 16, threads = ((a.n + V - 1) / V + 31) / 32 * 32;
  const int rows = threads == 32 ? 4 : 1;
  const dim3 block(threads, rows), grid((a.T + rows - 1) / rows);
  if (V == 4) edge_kernel<XT, PT, 1, 4><<<grid, block, 0, s>>>(a);
  else edge_kernel<XT, PT, 1, 16><<<grid, block, 0, s>>>(a);
  return cudaGetLastError();
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
