// Routing from logits (strata_moe_select), sm_103a: softmax or sigmoid scores, a bias for balance, groups
// of experts, stable top-k, renormalised weights.
//
// zwxr.cn news/242664, section "一次路由的完整旅程", has the step this one generalises: softmax over all
// experts, stable descending order, gather, renormalise with a lower clamp.
#include <cfloat>

#include "device_common.cuh"
#include "elements.cuh"

namespace strata {
namespace {

constexpr int SEL_WARPS = 4;          // one token each
constexpr int PER = EMAX / 32;        // experts of a lane: lane + 32 j
constexpr float SUM_MIN = 1.f / 16384.f;  // lower clamp of the weights' sum (2^-14)

struct SelectArgs {
  const void* logits;
  int64_t stride;
  const float* bias;
  int32_t* ids;
  float* weights;
  int T, E, k, softmax, G, keep, group_sum, renorm, type;
  float scale;
};

__device__ __forceinline__ double shfl_xor_d(double v, int o) { return __shfl_xor_sync(0xffffffffu, v, o); }
__device__ __forceinline__ double warp_sum_d(double v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += shfl_xor_d(v, o);
  return v;
}

// Score of logit l in 64 bits (m, z: the softmax's maximum and sum).
__device__ __forceinline__ double score_d(float l, bool softmax, float m, double z) {
  return softmax ? exp((double)l - (double)m) / z : 1.0 / (1.0 + exp(-(double)l));
}

// One token by one warp, every value in 64 bits.  l[j]: logit of expert lane + 32 j (+inf made finite); bit j of
// `usable`: the expert exists and is not masked.  val: shared [EMAX] doubles of this warp.  Lane i (< k) returns
// the id of rank i and its score.
__device__ void select_exact(const SelectArgs& a, const float (&l)[PER], uint32_t usable, double* val, int* out_id,
                             double* out_p) {
  const int lane = threadIdx.x & 31;
  float m = -FLT_MAX;
#pragma unroll
  for (int j = 0; j < PER; ++j)
    if (usable >> j & 1) m = fmaxf(m, l[j]);
  m = warp_max(m);
  double z = 1.0;
  if (a.softmax) {
    z = 0.0;
#pragma unroll 1
    for (int j = 0; j < PER; ++j)
      if (usable >> j & 1) z += exp((double)l[j] - (double)m);
    z = warp_sum_d(z);
  }
  uint32_t here = 0;  // bit j: the expert exists and its group is kept
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int e = lane + 32 * j;
    if (e < a.E) {
      here |= 1u << j;
      double v = -INFINITY;
      if (usable >> j & 1) v = score_d(l[j], a.softmax, m, z) + (a.bias ? (double)__ldg(a.bias + e) : 0.0);
      val[e] = v;
    }
  }
  __syncwarp();
  if (a.G > 1) {
    const int size = a.E / a.G;
    double b0 = -INFINITY, b1 = -INFINITY;
    if (lane < a.G)
      for (int i = 0; i < size; ++i) {
        const double v = val[lane * size + i];
        if (v > b0) {
          b1 = b0;
          b0 = v;
        } else if (v > b1) {
          b1 = v;
        }
      }
    const double gs = (a.group_sum == 2 && b1 > -INFINITY) ? b0 + b1 : b0;
    int rank = 0;
    for (int g = 0; g < a.G; ++g) {
      const double o = __shfl_sync(0xffffffffu, gs, g);
      rank += (o > gs || (o == gs && g < lane)) ? 1 : 0;
    }
    const uint32_t kept = __ballot_sync(0xffffffffu, lane < a.G && rank < a.keep);
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int e = lane + 32 * j;
      if (e < a.E && !(kept >> (e / size) & 1)) here &= ~(1u << j);
    }
  }
  // k rounds: the warp's largest (key, then lower id) among the experts that remain
  double key[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j)
    key[j] = !(here >> j & 1) ? -INFINITY : a.bias ? val[lane + 32 * j] : (usable >> j & 1) ? (double)l[j] : -INFINITY;
  int mine = 0;
  double mine_p = 0.0;
#pragma unroll 1
  for (int i = 0; i < a.k; ++i) {
    double bk = -INFINITY;
    int be = EMAX;  // no expert
#pragma unroll
    for (int j = 0; j < PER; ++j)
      if ((here >> j & 1) && (be == EMAX || key[j] > bk)) {
        bk = key[j];
        be = lane + 32 * j;
      }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const double ok = shfl_xor_d(bk, o);
      const int oe = __shfl_xor_sync(0xffffffffu, be, o);
      if (oe < EMAX && (be == EMAX || ok > bk || (ok == bk && oe < be))) {
        bk = ok;
        be = oe;
      }
    }
    double p = 0.0;
    if ((be & 31) == lane) {
      const int jw = be >> 5;
      here &= ~(1u << jw);
#pragma unroll
      for (int j = 0; j < PER; ++j)
        if (j == jw && (usable >> j & 1)) p = score_d(l[j], a.softmax, m, z);
    }
    p = __shfl_sync(0xffffffffu, p, be & 31);
    if (lane == i) {
      mine = be;
      mine_p = p;
    }
  }
  *out_id = mine;
  *out_p = mine_p;
}

__global__ void __launch_bounds__(32 * SEL_WARPS) select_kernel(SelectArgs a) {
  __shared__ double s_val[SEL_WARPS][EMAX];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x * SEL_WARPS + warp;
  if (t >= a.T) return;
  const float lowest = lowest_of(a.type);
  float l[PER];
  uint32_t usable = 0;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int e = lane + 32 * j;
    const float v = e < a.E ? load1(a.logits, (int64_t)t * a.stride + e, a.type) : lowest;
    const float b = a.bias && e < a.E ? __ldg(a.bias + e) : 0.f;
    // a comparison with NaN is false: such an expert is masked
    if (v > lowest && b > -INFINITY) usable |= 1u << j;
    l[j] = fminf(v, FLT_MAX);
  }
  int id;
  double p;
  select_exact(a, l, usable, s_val[warp], &id, &p);
  const double sum = warp_sum_d(lane < a.k ? p : 0.0);
  if (lane < a.k) {
    a.ids[(int64_t)t * a.k + lane] = id;
    a.weights[(int64_t)t * a.k + lane] =
        (float)((a.renorm ? p / fmax(sum, (double)SUM_MIN) : p) * (double)a.scale);
  }
}

}  // namespace

cudaError_t launch_select(const strata_select_t& sel, const void* logits, int T, const float* bias, int32_t* ids,
                          float* weights, cudaStream_t s) {
  const SelectArgs a{logits, sel.logits_stride, bias, ids, weights, T, sel.n_expert, sel.top_k,
                     sel.score == STRATA_SCORE_SOFTMAX, sel.n_group, sel.top_group, sel.group_sum, sel.renorm,
                     sel.logits_type, sel.scale};
  STRATA_LAUNCH(KID_SELECT, s,
                select_kernel<<<(T + SEL_WARPS - 1) / SEL_WARPS, 32 * SEL_WARPS, 0, s>>>(a));
  return cudaGetLastError();
}

}  // namespace strata
