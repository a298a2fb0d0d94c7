// Routing from logits (strata_moe_select), sm_103a: softmax or sigmoid scores, a bias for balance, groups
// of experts, stable top-k, renormalised weights.
//
// zwxr.cn news/242664, section "一次路由的完整旅程", has the step this one generalises: softmax over all
// experts, stable descending order, gather, renormalise with a lower clamp.
//
// A token is one warp's work: its logits in the warp's registers, 16 a lane for 512 experts, the choice by lane maxima and the
// few candidates not below the k-th of them.  It is bound by the chain of a token (about 1,500 instructions with groups and a
// bias, issued in 54% of cycles by the 28 warps that an SM holds; two turns at 8,192 tokens, each with its own loads) and by the
// last warp that needs a 64-bit pass; memory is at 7%.
// 512 experts, top-10: one token 2.5 us, 8,192 tokens with sigmoid scores, a bias and 4 of 16 groups 20.3 us (of which 64-bit
// passes 3.4); without groups 16.4, a softmax with a bias 31, a softmax alone 9.4.  Seven CTAs an SM: 24.4 us before the passes
// were shortened; five 24.5, eight (64 registers) 26.8.
#include <cfloat>

#include "device_common.cuh"
#include "elements.cuh"

namespace strata {
namespace {

constexpr int SEL_WARPS = 4;          // one token each
constexpr int SEL_CTAS = 7;           // an SM
constexpr float SUM_MIN = 1.f / 16384.f;  // lower clamp of the weights' sum (2^-14)

struct SelectArgs {
  const void* logits;
  int64_t stride;
  const float* bias;
  int32_t* ids;
  float* weights;
  int T, E, k, softmax, G, keep, group_sum, renorm, type;
  float scale;
  int size, magic;  // experts of a group, ceil(2^20 / size)
};

// Group of expert e: e / size, exact for e < 512 (e magic / 2^20 is above it by less than e / 2^20 < 1 / 512).
__device__ __forceinline__ int group_of(const SelectArgs& a, int e) { return (int)((unsigned)e * (unsigned)a.magic >> 20); }

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

// Softmax sum in 64 bits over the warp's usable experts.
__device__ __noinline__ double softmax_sum_d(const float* l, uint32_t usable, float m) {
  const int lane = threadIdx.x & 31;
  double z = 0.0;
#pragma unroll 4
  for (int j = 0; j < EMAX / 32; ++j)
    if (usable >> j & 1) z += exp((double)l[lane + 32 * j] - (double)m);
  return warp_sum_d(z);
}

// Token t by one warp, every value in 64 bits.  l: its logits in shared memory (+inf made finite), m the largest usable
// one; bit j of `usable`: expert lane + 32 j exists and is not masked.  val: shared [EMAX] doubles of this warp.
__device__ __noinline__ void select_exact(const SelectArgs& a, int t, const float* l, float m, uint32_t usable,
                                          double* val) {
  const int lane = threadIdx.x & 31;
  const double z = a.softmax ? softmax_sum_d(l, usable, m) : 1.0;
  uint32_t here = 0;  // bit j: the expert exists and its group is kept
#pragma unroll 1
  for (int j = 0; j < EMAX / 32; ++j) {
    const int e = lane + 32 * j;
    if (e < a.E) {
      here |= 1u << j;
      double v = -INFINITY;
      if (usable >> j & 1) v = score_d(l[e], a.softmax, m, z) + (a.bias ? (double)__ldg(a.bias + e) : 0.0);
      val[e] = v;
    }
  }
  __syncwarp();
  if (a.G > 1) {
    const int size = a.size;
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
    for (int j = 0; j < EMAX / 32; ++j) {
      const int e = lane + 32 * j;
      if (e < a.E && !(kept >> group_of(a, e) & 1)) here &= ~(1u << j);
    }
  }
  // k rounds: the warp's largest (key, then lower id) among the experts that remain
  double key[EMAX / 32];
#pragma unroll
  for (int j = 0; j < EMAX / 32; ++j)
    key[j] = !(here >> j & 1) ? -INFINITY : a.bias ? val[lane + 32 * j] : (usable >> j & 1) ? (double)l[lane + 32 * j] : -INFINITY;
  int mine = 0;
  double mine_p = 0.0;
#pragma unroll 1
  for (int i = 0; i < a.k; ++i) {
    double bk = -INFINITY;
    int be = EMAX;  // no expert
#pragma unroll
    for (int j = 0; j < EMAX / 32; ++j)
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
      here &= ~(1u << (be >> 5));
      if (usable >> (be >> 5) & 1) p = score_d(l[be], a.softmax, m, z);
    }
    p = __shfl_sync(0xffffffffu, p, be & 31);
    if (lane == i) {
      mine = be;
      mine_p = p;
    }
  }
  const double sum = warp_sum_d(lane < a.k ? mine_p : 0.0);
  if (lane < a.k) {
    a.ids[(int64_t)t * a.k + lane] = mine;
    a.weights[(int64_t)t * a.k + lane] =
        (float)((a.renorm ? mine_p / fmax(sum, (double)SUM_MIN) : mine_p) * (double)a.scale);
  }
}

// Rounding of a value of the fp32 pass, in units of u = 2^-24; exponentials are ex2(x log2 e) (the argument's two
// roundings 1.5 |x| u, the function 4 u).  A softmax score p = exp(-d) / z, d = m - l: (2.5 d + 4) u of it with d's own
// rounding, where d p <= 0.37 of the largest score; z: the same of each term, where the mean of d over the scores is at
// most ln 512 = 6.2, and 16 + 5 additions, 41 u; a quotient and a product 3 u: below 52 u of the largest score.  A
// sigmoid p = 1 / (1 + e): p (1 - p) (1.5 |l| + 4) u <= 1.4 u, the sum u, the quotient 4 u: below 8 u.  Adding the
// bias rounds once more.  (An exponential that leaves the fp32 range: 1e-37.)
constexpr float U32 = 5.9604645e-8f;
constexpr float ERR_SOFTMAX = 52.f, ERR_SIGMOID = 8.f;

// A value's place in the choice as an unsigned number: larger values larger numbers (-0 as +0).  A masked expert has the
// value -inf, and so the smallest key.
__device__ __forceinline__ uint32_t value_key(float v) {
  const int b = __float_as_int(v + 0.f);
  return (uint32_t)(b ^ ((b >> 31) | (int)0x80000000));
}
constexpr uint32_t MASKED = 0x007fffffu;  // value_key(-inf)
__device__ __forceinline__ float warp_min_key(float v) { return key_logit(__reduce_min_sync(0xffffffffu, value_key(v))); }
__device__ __forceinline__ float warp_max_key(float v) { return key_logit(__reduce_max_sync(0xffffffffu, value_key(v))); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float LOG2E = 1.44269504f;
__device__ __forceinline__ float sigmoid_fast(float l) { return rcp(1.f + ex2(l * -LOG2E)); }

constexpr int CAND = 64;
struct SelectScratch {  // one per warp
  float l[EMAX];        // for the 64-bit passes
  union {
    struct {
      float val[EMAX + EMAX / 32];  // value of expert e at e + e / 32
      uint64_t cand[CAND];          // key, then ~id: the larger number comes first
      uint64_t sel[STRATA_SELECT_K_MAX + 1];
      int kept[STRATA_SELECT_GROUP_MAX];
    };
    double exact[EMAX];  // select_exact's values
  };
};
static_assert(sizeof(SelectScratch) % 16 == 0, "one follows another");
__device__ __forceinline__ int cand_id(uint64_t c) { return (int)~(uint32_t)c; }
__device__ __forceinline__ uint32_t cand_key(uint64_t c) { return (uint32_t)(c >> 32); }

// Lanes of a group when the groups' values are read, L: all groups fit a warp.
__device__ __forceinline__ int group_lanes(int G) { return G > 16 ? 1 : G > 8 ? 2 : G > 4 ? 4 : G > 2 ? 8 : G > 1 ? 16 : 32; }

// The logits of token t once more, into shared memory for the 64-bit passes: +inf made finite; returns the usable experts
// (bit j: expert lane + 32 j) and their largest logit.
__device__ __noinline__ uint32_t read_row(const SelectArgs& a, int t, float* l, float* m) {
  const int lane = threadIdx.x & 31;
  const float lowest = lowest_of(a.type);
  uint32_t usable = 0;
  float top = -FLT_MAX, v[EMAX / 32], b[EMAX / 32];
#pragma unroll
  for (int j = 0; j < EMAX / 32; ++j) {  // every load is issued before the first is looked at
    const int e = lane + 32 * j;
    v[j] = e < a.E ? load1(a.logits, (int64_t)t * a.stride + e, a.type) : lowest;
    b[j] = a.bias && e < a.E ? __ldg(a.bias + e) : 0.f;
  }
#pragma unroll
  for (int j = 0; j < EMAX / 32; ++j) {
    if (v[j] > lowest && b[j] > -INFINITY) {
      usable |= 1u << j;
      top = fmaxf(top, fminf(v[j], FLT_MAX));
    }
    l[lane + 32 * j] = fminf(v[j], FLT_MAX);
  }
  *m = warp_max(top);
  __syncwarp();
  return usable;
}

// Logit of expert e of token t, usable, as read_row has it.
__device__ __forceinline__ float logit_at(const SelectArgs& a, int t, int e) {
  return fminf(load1(a.logits, (int64_t)t * a.stride + e, a.type), FLT_MAX);
}
// A softmax's largest usable logit and its sum where they matter: without a bias the sum divides out, and m may be any.
__device__ __forceinline__ double softmax_row(const SelectArgs& a, int t, SelectScratch& sc, float* m) {
  if (!a.softmax || !a.bias) return 1.0;
  const uint32_t usable = read_row(a, t, sc.l, m);
  return softmax_sum_d(sc.l, usable, *m);
}

// Groups kept, where the fp32 scores do not decide: the groups' scores in 64 bits, from the two largest values of each
// (val: the values with a bias, the logits without).  Lane g < G scans group g.  m: the softmax's largest logit.  *sure = false
// if a group's two largest cannot be told from its third.
__device__ __noinline__ uint32_t groups_exact(const SelectArgs& a, int t, SelectScratch& sc, float m, float err, bool* sure) {
  const int lane = threadIdx.x & 31;
  float v0 = -INFINITY, v1 = -INFINITY, v2 = -INFINITY;
  int e0 = 0, e1 = 0;
  if (lane < a.G)
#pragma unroll 8
    for (int i = 0; i < a.size; ++i) {
      const int e = lane * a.size + i;
      const float v = sc.val[e + (e >> 5)];
      const bool c0 = v > v0, c1 = v > v1;
      v2 = c1 ? v1 : fmaxf(v2, v);
      e1 = c0 ? e0 : c1 ? e : e1;
      v1 = c0 ? v0 : fmaxf(v1, v);
      e0 = c0 ? e : e0;
      v0 = fmaxf(v0, v);
    }
  const bool two = a.group_sum == 2;
  const float last = two ? v1 : v0, behind = two ? v2 : v1;
  const bool clear = !a.bias || behind == -INFINITY ||
                     last - behind > 2.f * (err + U32 * fmaxf(fabsf(last), fabsf(behind)));
  *sure = __all_sync(0xffffffffu, clear);
  const double z = softmax_row(a, t, sc, &m);
  const auto value = [&](int e, float v) {
    return v > -INFINITY ? score_d(logit_at(a, t, e), a.softmax, m, z) + (a.bias ? (double)__ldg(a.bias + e) : 0.0) : -INFINITY;
  };
  double gs;
  if (a.G <= 16) {  // lanes 16 .. take the second values
    const int e2 = __shfl_sync(0xffffffffu, e1, lane & 15);
    const float w2 = __shfl_sync(0xffffffffu, v1, lane & 15);
    const bool second = lane >= 16;
    gs = value(second ? e2 : e0, second ? (two ? w2 : -INFINITY) : v0);
    const double other = __shfl_down_sync(0xffffffffu, gs, 16);
    if (other > -INFINITY) gs += other;
  } else {
    gs = value(e0, v0);
    if (two && v1 > -INFINITY) gs += value(e1, v1);
  }
  int rank = 0;
#pragma unroll 4
  for (int g = 0; g < a.G; ++g) {
    const double o = __shfl_sync(0xffffffffu, gs, g);
    rank += (o > gs || (o == gs && g < lane)) ? 1 : 0;
  }
  return __ballot_sync(0xffffffffu, lane < a.G && rank < a.keep);
}

// Values x >= y that fp32 cannot tell apart: each is off by err and by the rounding of its sum with the bias.
__device__ __forceinline__ bool too_near(float x, float y, float err) { return !(x - y > 2.f * err + U32 * (fabsf(x) + fabsf(y))); }

// The order of C candidates (sc.cand) by their values in 64 bits into sc.sel, where neighbours among the first k (near: lane
// i and i + 1) are too near for fp32; near neighbours of the same logit and bias are true ties and stay as they are.
__device__ __noinline__ void order_exact(const SelectArgs& a, int t, SelectScratch& sc, int C, bool near, float err) {
  const int lane = threadIdx.x & 31;
  const auto same = [&](int p, int q) {
    return logit_at(a, t, p) == logit_at(a, t, q) && __ldg(a.bias + p) == __ldg(a.bias + q);
  };
  bool tie = false;  // of the last one chosen and the first one left
  if (near && same(cand_id(sc.sel[lane]), cand_id(sc.sel[lane + 1]))) {
    near = false;
    tie = lane == a.k - 1;
  }
  if (__any_sync(0xffffffffu, tie)) {
    // behind the first one left may be others too near to the last one chosen
    const uint64_t last = sc.sel[a.k - 1], left = sc.sel[a.k];
    const float x = key_logit(cand_key(last));
    for (int i = lane; i < C; i += 32) {
      const uint64_t c = sc.cand[i];
      if (c < left && too_near(x, key_logit(cand_key(c)), err) && !same(cand_id(last), cand_id(c))) near = true;
    }
  }
  if (!__any_sync(0xffffffffu, near)) return;
  float m = 0.f;
  const double z = softmax_row(a, t, sc, &m);
  double mine[CAND / 32];
#pragma unroll
  for (int h = 0; h < CAND / 32; ++h) {
    mine[h] = -INFINITY;
    if (lane + 32 * h < C) {
      const uint64_t c = sc.cand[lane + 32 * h];
      const int e = cand_id(c);
      if (cand_key(c) > MASKED) mine[h] = score_d(logit_at(a, t, e), a.softmax, m, z) + (double)__ldg(a.bias + e);
    }
  }
  int rank[CAND / 32] = {0, 0};
  for (int q = 0; q < C; ++q) {
    const double o = __shfl_sync(0xffffffffu, q < 32 ? mine[0] : mine[1], q & 31);
    const int oe = cand_id(sc.cand[q]);
#pragma unroll
    for (int h = 0; h < CAND / 32; ++h)
      if (lane + 32 * h < C) {
        const int e = cand_id(sc.cand[lane + 32 * h]);
        rank[h] += (o > mine[h] || (o == mine[h] && oe < e)) ? 1 : 0;
      }
  }
  __syncwarp();
#pragma unroll
  for (int h = 0; h < CAND / 32; ++h)
    if (lane + 32 * h < C && rank[h] < a.k) sc.sel[rank[h]] = sc.cand[lane + 32 * h];
  __syncwarp();
}

// One token per warp and turn.  VALUES: the choice goes by scores (a bias, or groups); otherwise by the logits alone.
// PER: experts of a lane (lane + 32 j), E <= 32 PER.
//
// The pass in fp32 knows how far its values may be off (err), and a choice that this could turn is made again in 64 bits:
// of the candidates' values, or of the groups' two largest; only where even that is not enough (a mass of near ties) of
// all.  64-bit arithmetic is slow on this GPU, and a token in about a thousand needs it.
template <bool VALUES, int PER>
__global__ void __launch_bounds__(32 * SEL_WARPS, SEL_CTAS) select_kernel(const __grid_constant__ SelectArgs a) {
  griddep_wait();
  __shared__ __align__(16) SelectScratch s_all[SEL_WARPS];
  __shared__ float s_bias[VALUES ? 32 * PER : 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  SelectScratch& sc = s_all[warp];
  const float lowest = lowest_of(a.type);
  const uint32_t below = (1u << lane) - 1u;
  const bool grouped = VALUES && a.G > 1;
  const int L = VALUES ? group_lanes(a.G) : 32;
  const int total = grouped ? a.keep * a.size : a.E;  // experts that may be chosen
  if constexpr (VALUES) {
    for (int e = threadIdx.x; e < 32 * PER; e += 32 * SEL_WARPS) {
      const float b = a.bias && e < a.E ? __ldg(a.bias + e) : 0.f;
      s_bias[e] = b > -INFINITY ? b : -INFINITY;  // NaN too: the expert's value is -inf
    }
    __syncthreads();
  }
  for (int t = blockIdx.x * SEL_WARPS + warp; t < a.T; t += gridDim.x * SEL_WARPS) {
    float v[PER];
    const int64_t row = (int64_t)t * a.stride + lane;
    if (a.type == STRATA_F32) {
#pragma unroll
      for (int j = 0; j < PER; ++j) v[j] = lane + 32 * j < a.E ? __ldg(static_cast<const float*>(a.logits) + row + 32 * j) : lowest;
    } else {
      uint16_t raw[PER];
#pragma unroll
      for (int j = 0; j < PER; ++j)  // 0xffff: NaN
        raw[j] = lane + 32 * j < a.E ? __ldg(static_cast<const uint16_t*>(a.logits) + row + 32 * j) : (uint16_t)0xffff;
#pragma unroll
      for (int j = 0; j < PER; ++j)
        v[j] = a.type == STRATA_BF16 ? __uint_as_float((uint32_t)raw[j] << 16) : __half2float(__ushort_as_half(raw[j]));
    }
    // masked logits as -inf (a comparison with NaN is false)
#pragma unroll
    for (int j = 0; j < PER; ++j) v[j] = v[j] > lowest ? fminf(v[j], FLT_MAX) : -INFINITY;

    // Values: logits, or with a bias scores + bias.  Without groups they stay in registers, with groups they go by
    // shared memory and only the kept groups' come back.
    float inv_z = 1.f, err = 0.f, m = 0.f;
    if (a.softmax) {
      m = v[0];
#pragma unroll
      for (int j = 1; j < PER; ++j) m = fmaxf(m, v[j]);
      m = warp_max_key(m);
      if (m == -INFINITY) m = 0.f;
    }
    if (a.softmax && (VALUES || !a.renorm)) {
      float z = 0.f;
      // an expert that its bias masks is no part of the softmax
      float mb = m;
      if (VALUES && a.bias) {
        mb = -INFINITY;
#pragma unroll
        for (int j = 0; j < PER; ++j)
          if (s_bias[lane + 32 * j] > -INFINITY) mb = fmaxf(mb, v[j]);
        mb = warp_max_key(mb);
        if (mb == -INFINITY) mb = 0.f;
        m = mb;
      }
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        const float e = VALUES && !(s_bias[lane + 32 * j] > -INFINITY) ? 0.f : ex2((v[j] - m) * LOG2E);
        z += e;
        if (VALUES && a.bias) v[j] = v[j] > -INFINITY ? e : -INFINITY;
      }
      z = warp_sum(z);
      inv_z = z > 0.f ? 1.f / z : 1.f;
      if (VALUES && a.bias) {
#pragma unroll
        for (int j = 0; j < PER; ++j)  // (a masked expert stays at -inf whatever its bias: -inf + inf would be a NaN)
          v[j] = v[j] > -INFINITY ? fmaf(v[j], inv_z, s_bias[lane + 32 * j]) : -INFINITY;
      }
      err = U32 * ERR_SOFTMAX * inv_z + 1e-37f;
    }
    if (VALUES && !a.softmax) {
      err = U32 * ERR_SIGMOID + 1e-37f;
      if (a.bias) {
#pragma unroll
        for (int j = 0; j < PER; ++j) v[j] = v[j] > -INFINITY ? sigmoid_fast(v[j]) + s_bias[lane + 32 * j] : -INFINITY;
      }
    }

    uint32_t key[PER];
    if (grouped) {
#pragma unroll
      for (int j = 0; j < PER; ++j) sc.val[lane + 33 * j] = v[j];
      __syncwarp();
      // each group's two largest, of the values with a bias, of the logits without (the same experts, and equal
      // scores are then known for what they are)
      const int g = lane / L;
      float k0 = -INFINITY, k1 = -INFINITY;
      if (g < a.G) {
        const int end = (g + 1) * a.size;
#pragma unroll 8
        for (int e = g * a.size + lane % L; e < end; e += L) {
          const float w = sc.val[e + (e >> 5)];
          k1 = fmaxf(k1, fminf(k0, w));
          k0 = fmaxf(k0, w);
        }
      }
      for (int o = 1; o < L; o <<= 1) {
        const float w0 = __shfl_xor_sync(0xffffffffu, k0, o), w1 = __shfl_xor_sync(0xffffffffu, k1, o);
        k1 = fmaxf(fminf(k0, w0), fmaxf(k1, w1));
        k0 = fmaxf(k0, w0);
      }
      float v0 = k0, v1 = k1;
      if (!a.bias) {
        if (k0 > -INFINITY) v0 = a.softmax ? ex2((k0 - m) * LOG2E) * inv_z : sigmoid_fast(k0);
        if (k1 > -INFINITY) v1 = a.softmax ? ex2((k1 - m) * LOG2E) * inv_z : sigmoid_fast(k1);
      }
      const bool two = a.group_sum == 2 && v1 > -INFINITY;
      // (a sum below the fp32 range is its lowest number, not the -inf of a group without a usable expert: sums that were cut
      // so are equal or nearly, and the groups are then told apart in 64 bits)
      const float gs = v0 > -INFINITY ? fmaxf(two ? v0 + v1 : v0, -FLT_MAX) : -INFINITY;
      int rank = 0;
#pragma unroll 4
      for (int h = 0; h < a.G; ++h) {
        const float o = __shfl_sync(0xffffffffu, gs, h * L);
        rank += (o > gs || (o == gs && h < g)) ? 1 : 0;
      }
      const bool mine = g < a.G && rank < a.keep;
      uint32_t in = __ballot_sync(0xffffffffu, mine);  // L bits a group
      // the scores' error: of two values and of their sum, none of them larger than `big`
      const float big = warp_max_key(gs > -INFINITY ? fmaxf(fabsf(gs), fmaxf(fabsf(v0), two ? fabsf(v1) : 0.f)) : 0.f);
      const float ge = 2.f * err + 3.f * U32 * big;
      // (a group without a usable expert is no rival, and none is pushed out by one)
      const float least = warp_min_key(mine && gs > -INFINITY ? gs : INFINITY);
      const float rival = warp_max_key(mine || g >= a.G ? -INFINITY : gs);
      if (rival > -INFINITY && !(least - rival > 2.f * ge)) {
        bool unsure = false;  // this kept group and one that is dropped are too near, and not equal
        for (int h = 0; h < a.G; ++h) {
          const float o = __shfl_sync(0xffffffffu, gs, h * L);
          const float o0 = __shfl_sync(0xffffffffu, k0, h * L), o1 = __shfl_sync(0xffffffffu, k1, h * L);
          const bool same = !a.bias && o0 == k0 && (a.group_sum == 1 || o1 == k1);
          if (mine && !(in >> (h * L) & 1u) && o > -INFINITY && !same && !(gs - o > 2.f * ge)) unsure = true;
        }
        if (__any_sync(0xffffffffu, unsure)) {
          bool sure;
          const uint32_t kept = groups_exact(a, t, sc, m, err, &sure);
          if (!sure) {
            const uint32_t usable = read_row(a, t, sc.l, &m);
            select_exact(a, t, sc.l, m, usable, sc.exact);
            continue;
          }
          in = __ballot_sync(0xffffffffu, g < a.G && (kept >> g & 1u));
        }
      }
      if ((in >> lane & 1u) && lane % L == 0) sc.kept[__popc(in & below) / L] = g;
      __syncwarp();
    }
    // the expert at place i of those that may be chosen
    const auto expert_at = [&](int i) {
      if (!grouped) return i;
      const int q = group_of(a, i);
      return sc.kept[q] * a.size + i - q * a.size;
    };
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      key[j] = MASKED;
      if (!grouped) {
        key[j] = value_key(v[j]);
      } else if (32 * j < total && lane + 32 * j < total) {
        const int e = expert_at(lane + 32 * j);
        key[j] = value_key(sc.val[e + (e >> 5)]);
      }
    }

    // candidates: every usable key not below the k-th largest of the lanes' largest (k lanes hold one at least), and
    // with a bias not surely below it.  The k-th largest by a bitonic sort of the 32.
    uint32_t tau = key[0];
#pragma unroll
    for (int j = 1; j < PER; ++j) tau = max(tau, key[j]);
#pragma unroll
    for (int n = 2; n <= 32; n <<= 1)
#pragma unroll
      for (int o = n >> 1; o; o >>= 1) {
        const uint32_t w = __shfl_xor_sync(0xffffffffu, tau, o);
        tau = (((lane & o) == 0) == ((lane & n) == 0)) ? max(tau, w) : min(tau, w);
      }
    tau = __shfl_sync(0xffffffffu, tau, a.k - 1);
    if (VALUES && a.bias && tau > MASKED) {
      const float f = key_logit(tau);
      if (f < INFINITY) tau = min(tau, value_key(f - 2.f * err - 4.f * U32 * fabsf(f)));
    }
    tau = max(tau, MASKED + 1u);
    uint32_t is = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      if (grouped && 32 * j >= total) break;
      if (key[j] >= tau) is |= 1u << j;
    }
    int pos = __popc(is);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int w = __shfl_up_sync(0xffffffffu, pos, o);
      if (lane >= o) pos += w;
    }
    int C = __shfl_sync(0xffffffffu, pos, 31);
    pos -= __popc(is);
    if (C <= CAND) {
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        if (grouped && 32 * j >= total) break;
        if (is >> j & 1) sc.cand[pos++] = (uint64_t)key[j] << 32 | (uint32_t)~expert_at(lane + 32 * j);
      }
      if (C < a.k) {
        // fewer usable experts than k: masked ones of the kept groups, lower ids first
#pragma unroll
        for (int j = 0; j < PER; ++j) {
          const int i = lane + 32 * j;
          const bool masked = i < total && key[j] == MASKED;
          const uint32_t bal = __ballot_sync(0xffffffffu, masked);
          const int at = C + __popc(bal & below);
          if (masked && at < a.k) sc.cand[at] = (uint64_t)MASKED << 32 | (uint32_t)~expert_at(i);
          C = min(a.k, C + __popc(bal));
        }
      }
      __syncwarp();
      for (int i = lane; i < C; i += 32) {
        const uint64_t me = sc.cand[i];
        int rank = 0;
#pragma unroll 4
        for (int q = 0; q < C; ++q) rank += sc.cand[q] > me ? 1 : 0;
        if (rank <= a.k) sc.sel[rank] = me;
      }
    } else if (VALUES && a.bias) {
      const uint32_t usable = read_row(a, t, sc.l, &m);
      select_exact(a, t, sc.l, m, usable, sc.exact);
      continue;
    } else {
      // a mass of equal logits: k rounds of the warp's largest (key, then lower id)
#pragma unroll 1
      for (int i = 0; i < a.k; ++i) {
        uint32_t bk = 0u, bj = 0u;
#pragma unroll
        for (int j = 0; j < PER; ++j)
          if (key[j] > bk) {
            bk = key[j];
            bj = j;
          }
        const uint32_t mx = __reduce_max_sync(0xffffffffu, bk);
        const uint32_t at = __reduce_min_sync(0xffffffffu, bk == mx ? lane + 32u * bj : 0xffffffffu);
#pragma unroll
        for (int j = 0; j < PER; ++j)
          if (at == (uint32_t)(lane + 32 * j)) key[j] = 0u;
        if (lane == 0) sc.sel[i] = (uint64_t)mx << 32 | (uint32_t)~expert_at((int)at);
      }
    }
    __syncwarp();
    if (VALUES && a.bias) {
      // neighbours in the order whose values fp32 cannot tell apart
      bool near = false;
      if (lane < a.k && lane + 1 < C) {
        const uint32_t p = cand_key(sc.sel[lane]), q = cand_key(sc.sel[lane + 1]);
        const float x = key_logit(p), y = key_logit(q);
        near = q > MASKED && too_near(x, y, err);
      }
      if (__any_sync(0xffffffffu, near)) order_exact(a, t, sc, C, near, err);
    }
    // weights: without groups or a bias the k largest softmax scores sum to k / E at least, above the clamp, and the
    // softmax's own sum divides out
    const bool has = lane < a.k;
    const uint64_t me = sc.sel[has ? lane : 0];
    float p = 0.f;
    if (has && cand_key(me) > MASKED) {
      const float x = fminf(load1(a.logits, row - lane + cand_id(me), a.type), FLT_MAX);
      const float e = expf(a.softmax ? x - m : -fabsf(x));
      // (the exponential of -|x|: that of a far negative logit's -x leaves fp32, and the score is then 0 too early)
      p = a.softmax ? e * inv_z : __fdividef(x < 0.f ? e : 1.f, 1.f + e);
    }
    const float sum = a.renorm ? fmaxf(warp_sum(p), SUM_MIN) : 1.f;
    if (has) {
      a.ids[(int64_t)t * a.k + lane] = cand_id(me);
      a.weights[(int64_t)t * a.k + lane] = __fdividef(p, sum) * a.scale;
    }
    __syncwarp();
  }
  griddep_launch_dependents();
}

template <bool VALUES, int PER>
cudaError_t launch_form(const SelectArgs& a, int grid, cudaStream_t s) {
  return launch_pdl(select_kernel<VALUES, PER>, grid, 32 * SEL_WARPS, 0, s, a);
}

}  // namespace

cudaError_t launch_select(const strata_select_t& sel, const void* logits, int T, const float* bias, int32_t* ids,
                          float* weights, cudaStream_t s) {
  const SelectArgs a{logits, sel.logits_stride, bias, ids, weights, T, sel.n_expert, sel.top_k,
                     sel.score == STRATA_SCORE_SOFTMAX, sel.n_group, sel.top_group, sel.group_sum, sel.renorm,
                     sel.logits_type, sel.scale, sel.n_expert / sel.n_group,
                     ((1 << 20) + sel.n_expert / sel.n_group - 1) / (sel.n_expert / sel.n_group)};
  const bool values = bias || sel.n_group > 1;
  // a warp takes ceil(T / what fits the GPU) tokens, so that all end together
  const int fit = 152 * SEL_CTAS * SEL_WARPS, turns = (T + fit - 1) / fit;
  const int warps = (T + turns - 1) / turns, grid = (warps + SEL_WARPS - 1) / SEL_WARPS;
  kernel_begin(KID_SELECT, s);
  const bool wide = sel.n_expert > 256;
  const cudaError_t err = values ? (wide ? launch_form<true, 16>(a, grid, s) : launch_form<true, 8>(a, grid, s))
                                 : (wide ? launch_form<false, 16>(a, grid, s) : launch_form<false, 8>(a, grid, s));
  kernel_end(KID_SELECT, s);
  return err;
}

}  // namespace strata
