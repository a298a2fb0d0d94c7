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
  float eps, residual, block;
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

// W consecutive elements as a unit (8 on 16-byte boundaries, or 1).
template <int W>
struct Unit;
template <>
struct Unit<8> {
  using Raw = Raw8;
  static __device__ __forceinline__ Raw load(const void* p, int64_t i, int type) { return load8(p, i, type); }
  static __device__ __forceinline__ void widen(const Raw& r, int type, float* f) {
    widen8(r, type, *reinterpret_cast<float(*)[8]>(f));
  }
  static __device__ __forceinline__ void store(void* p, int64_t i, int type, const float* f) {
    store8(p, i, type, *reinterpret_cast<const float(*)[8]>(f));
  }
};
template <>
struct Unit<1> {
  using Raw = float;
  static __device__ __forceinline__ Raw load(const void* p, int64_t i, int type) { return load1(p, i, type); }
  static __device__ __forceinline__ void widen(const Raw& r, int, float* f) { f[0] = r; }
  static __device__ __forceinline__ void store(void* p, int64_t i, int type, const float* f) { store1(p, i, type, f[0]); }
};

// One row per blockDim.x threads; a thread holds V units of W elements, blockDim.x units apart.
template <int W, int V>
__global__ void __launch_bounds__(W == 8 ? 512 : 1024) edge_kernel(NormArgs a) {
  __shared__ float red[2][32];
  const int t = blockIdx.x * blockDim.y + threadIdx.y;
  if (t >= a.T) return;  // whole warps; only one-warp rows share a CTA
  using U = Unit<W>;
  const int units = a.n / W;
  float r[V * W];
  if (a.parts) {
    float y[V * W];
#pragma unroll
    for (int i = 0; i < V * W; ++i) y[i] = 0.f;
    for (int k = 0; k < a.P; ++k) {
      const float w = a.pw ? __ldg(a.pw + (int64_t)t * a.P + k) : 1.f;
      if (w == 0.f) continue;
      const int64_t at = (int64_t)t * a.token_stride + k * a.part_stride;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int u = threadIdx.x + v * blockDim.x;
        if (u >= units) continue;
        float f[W];
        U::widen(U::load(a.parts, at + (int64_t)u * W, a.part_type), a.part_type, f);
#pragma unroll
        for (int i = 0; i < W; ++i) y[v * W + i] = fmaf(w, f[i], y[v * W + i]);
      }
    }
    float g = a.block;
    if (a.token) {
      const float s = __ldg(a.token + t);
      g *= a.sigmoid ? 1.f / (1.f + expf(-s)) : s;
    }
    float rn = 1.f;
    if (a.post) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < V * W; ++i) ss = fmaf(y[i], y[i], ss);
      rn = 1.f / sqrtf(row_sum(ss, red[0]) / (float)a.n + a.eps);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int u = threadIdx.x + v * blockDim.x;
      if (u >= units) {
#pragma unroll
        for (int i = 0; i < W; ++i) r[v * W + i] = 0.f;
        continue;
      }
      float xf[W];
#pragma unroll
      for (int i = 0; i < W; ++i) xf[i] = 0.f;
      if (a.x) U::widen(U::load(a.x, (int64_t)t * a.x_stride + (int64_t)u * W, a.x_type), a.x_type, xf);
#pragma unroll
      for (int i = 0; i < W; ++i) {
        float z = y[v * W + i] * rn;
        if (a.post_gain) z *= __ldg(a.post_gain + u * W + i);
        if (a.channel) z *= __ldg(a.channel + u * W + i);
        r[v * W + i] = fmaf(g, z, a.residual * xf[i]);
      }
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int u = threadIdx.x + v * blockDim.x;
#pragma unroll
      for (int i = 0; i < W; ++i) r[v * W + i] = 0.f;
      if (u < units) U::widen(U::load(a.x, (int64_t)t * a.x_stride + (int64_t)u * W, a.x_type), a.x_type, r + v * W);
    }
  }
  if (a.out) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int u = threadIdx.x + v * blockDim.x;
      if (u < units) U::store(a.out, (int64_t)t * a.out_stride + (int64_t)u * W, a.x_type, r + v * W);
    }
  }
  if (a.next) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < V * W; ++i) ss = fmaf(r[i], r[i], ss);
    const float rn = 1.f / sqrtf(row_sum(ss, red[1]) / (float)a.n + a.eps);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int u = threadIdx.x + v * blockDim.x;
      if (u >= units) continue;
      float f[W];
#pragma unroll
      for (int i = 0; i < W; ++i) {
        f[i] = r[v * W + i] * rn;
        if (a.pre_gain) f[i] *= __ldg(a.pre_gain + u * W + i);
      }
      U::store(a.next, (int64_t)t * a.next_stride + (int64_t)u * W, a.next_type, f);
    }
  }
}

// Every row of the operand starts on a 16-byte boundary.
bool rows16(const void* p, int64_t stride, int type) {
  const int64_t size = type == STRATA_F32 ? 4 : 2;
  return !p || (((uintptr_t)p & 15) == 0 && (stride * size) % 16 == 0);
}

cudaError_t launch_edge(const NormArgs& a, int kid, cudaStream_t s) {
  const bool vec = a.n % 8 == 0 && rows16(a.parts, a.part_stride, a.part_type) &&
                   rows16(a.parts, a.token_stride, a.part_type) && rows16(a.x, a.x_stride, a.x_type) &&
                   rows16(a.out, a.out_stride, a.x_type) && rows16(a.next, a.next_stride, a.next_type);
  const int units = vec ? a.n / 8 : a.n;
  const int V = vec ? (units <= 512 ? 1 : units <= 1024 ? 2 : 4) : (units <= 4096 ? 4 : 16);
  const int threads = ((units + V - 1) / V + 31) / 32 * 32;
  const int rows = threads == 32 ? 8 : 1;
  const dim3 block(threads, rows), grid((a.T + rows - 1) / rows);
  kernel_begin(kid, s);
  if (vec) {
    if (V == 1) edge_kernel<8, 1><<<grid, block, 0, s>>>(a);
    else if (V == 2) edge_kernel<8, 2><<<grid, block, 0, s>>>(a);
    else edge_kernel<8, 4><<<grid, block, 0, s>>>(a);
  } else {
    if (V == 4) edge_kernel<1, 4><<<grid, block, 0, s>>>(a);
    else edge_kernel<1, 16><<<grid, block, 0, s>>>(a);
  }
  kernel_end(kid, s);
  return cudaGetLastError();
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
