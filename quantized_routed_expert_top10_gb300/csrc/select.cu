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

// A value's place in the choice as an unsigned number: larger values larger numbers (-0 as +0), a masked expert 1, one that
// does not exist or whose group is dropped 0.
__device__ __forceinline__ uint32_t value_key(float v) { return logit_key(v + 0.f); }

constexpr int CAND = 64;
struct SelectScratch {  // one per warp; the padded values (groups) or 64-bit values follow
  float l[EMAX];
  uint2 cand[CAND];     // key, id
  uint2 sel[STRATA_SELECT_K_MAX + 1];
};
// Distance of two groups' values in shared memory: lane / L is the group and the L lanes of a group read
// neighbouring values, so a distance of L modulo 32 puts the warp's 32 reads into 32 banks.
__host__ __device__ inline int group_lanes(int G) { return G > 16 ? 1 : G > 8 ? 2 : G > 4 ? 4 : G > 2 ? 8 : G > 1 ? 16 : 32; }
__host__ __device__ inline int group_pitch(int size, int G) { return size + ((group_lanes(G) - size) & 31); }
inline size_t select_warp_bytes(int E, int G, bool values) {
  if (!values) return sizeof(SelectScratch);
  const size_t groups = G > 1 ? sizeof(float) * G * group_pitch(E / G, G) : 0, exact = sizeof(double) * EMAX;
  return (sizeof(SelectScratch) + (groups > exact ? groups : exact) + 15) / 16 * 16;
}
static_assert(sizeof(SelectScratch) % 8 == 0, "64-bit values follow the scratch");

// Groups kept, where the fp32 scores do not decide: the groups' scores in 64 bits, from the two largest values of each
// (val: the values with a bias, the logits without).  Lane g < G scans group g.  *sure = false if a group's two largest
// cannot be told from its third.  z: the softmax's sum (without a bias any positive number: the order is the same).
__device__ __noinline__ uint32_t groups_exact(const SelectArgs& a, const float* l, const float* val, int size, int pitch,
                                              float m, double z, float err, bool* sure) {
  const int lane = threadIdx.x & 31;
  float v0 = -INFINITY, v1 = -INFINITY, v2 = -INFINITY;
  int e0 = 0, e1 = 0;
  if (lane < a.G)
    for (int i = 0; i < size; ++i) {
      const float v = val[lane * pitch + i];
      if (v > v0) {
        v2 = v1; v1 = v0; e1 = e0;
        v0 = v; e0 = lane * size + i;
      } else if (v > v1) {
        v2 = v1;
        v1 = v; e1 = lane * size + i;
      } else if (v > v2) {
        v2 = v;
      }
    }
  const float last = a.group_sum == 2 ? v1 : v0, behind = a.group_sum == 2 ? v2 : v1;
  const bool clear = !a.bias || behind == -INFINITY ||
                     last - behind > 2.f * (err + U32 * fmaxf(fabsf(last), fabsf(behind)));
  *sure = __all_sync(0xffffffffu, clear);
  double gs = -INFINITY;
  if (v0 > -INFINITY) gs = score_d(l[e0], a.softmax, m, z) + (a.bias ? (double)__ldg(a.bias + e0) : 0.0);
  if (a.group_sum == 2 && v1 > -INFINITY) gs += score_d(l[e1], a.softmax, m, z) + (a.bias ? (double)__ldg(a.bias + e1) : 0.0);
  int rank = 0;
  for (int g = 0; g < a.G; ++g) {
    const double o = __shfl_sync(0xffffffffu, gs, g);
    rank += (o > gs || (o == gs && g < lane)) ? 1 : 0;
  }
  return __ballot_sync(0xffffffffu, lane < a.G && rank < a.keep);
}

__device__ __forceinline__ uint32_t key_of_min(float v) { return __reduce_min_sync(0xffffffffu, value_key(v)); }
__device__ __forceinline__ uint32_t key_of_max(float v) { return __reduce_max_sync(0xffffffffu, value_key(v)); }

// One token per warp and turn.  VALUES: the choice goes by scores (a bias, or groups); otherwise by the logits alone.
// PER: experts of a lane (lane + 32 j), E <= 32 PER.
//
// The pass in fp32 knows how far its values may be off (err), and a choice that this could turn is made again in 64 bits:
// of the candidates' values, or of the groups' two largest; only where even that is not enough (a mass of near ties) of
// all.  64-bit arithmetic is slow on this GPU, and a token in about a thousand needs it.
template <bool VALUES, int PER>
__global__ void __launch_bounds__(32 * SEL_WARPS, 5) select_kernel(const __grid_constant__ SelectArgs a, int warp_bytes) {
  extern __shared__ __align__(16) char s_all[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  SelectScratch& sc = *reinterpret_cast<SelectScratch*>(s_all + warp * warp_bytes);
  float* const val = reinterpret_cast<float*>(&sc + 1);
  const float lowest = lowest_of(a.type);
  const uint32_t below = (1u << lane) - 1u;
  const int size = a.size, pitch = VALUES ? group_pitch(size, a.G) : 0, L = VALUES ? group_lanes(a.G) : 32;
  float b[PER];
  uint32_t open = 0;  // bit j: the expert exists and its bias does not mask it
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int e = lane + 32 * j;
    b[j] = VALUES && a.bias && e < a.E ? __ldg(a.bias + e) : 0.f;
    if (e < a.E && b[j] > -INFINITY) open |= 1u << j;
  }
  for (int t = blockIdx.x * SEL_WARPS + warp; t < a.T; t += gridDim.x * SEL_WARPS) {
    float l[PER];
    const int64_t row = (int64_t)t * a.stride + lane;
    if (a.type == STRATA_F32) {
#pragma unroll
      for (int j = 0; j < PER; ++j) l[j] = lane + 32 * j < a.E ? __ldg(static_cast<const float*>(a.logits) + row + 32 * j) : lowest;
    } else {
      uint16_t raw[PER];
#pragma unroll
      for (int j = 0; j < PER; ++j)
        raw[j] = lane + 32 * j < a.E ? __ldg(static_cast<const uint16_t*>(a.logits) + row + 32 * j) : (uint16_t)0;
#pragma unroll
      for (int j = 0; j < PER; ++j)
        l[j] = a.type == STRATA_BF16 ? __uint_as_float((uint32_t)raw[j] << 16) : __half2float(__ushort_as_half(raw[j]));
    }
    uint32_t usable = 0;
    float m = -FLT_MAX;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      // a comparison with NaN is false: such an expert is masked
      const bool ok = l[j] > lowest && (open >> j & 1);
      if (ok) usable |= 1u << j;
      l[j] = fminf(l[j], FLT_MAX);
      if (ok) m = fmaxf(m, l[j]);
      sc.l[lane + 32 * j] = l[j];
    }
    m = warp_max(m);

    // values, and the experts' places: the value with a bias, the logit (the score's order) without
    float inv_z = 1.f, err = 0.f;
    uint32_t key[PER];
    if constexpr (VALUES) {
      float v[PER];
      if (a.softmax) {
        float z = 0.f;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
          v[j] = usable >> j & 1 ? __expf(l[j] - m) : 0.f;
          z += v[j];
        }
        z = warp_sum(z);
        inv_z = z > 0.f ? 1.f / z : 1.f;
        err = U32 * ERR_SOFTMAX * inv_z + 1e-37f;
#pragma unroll
        for (int j = 0; j < PER; ++j) v[j] = fmaf(v[j], inv_z, b[j]);
      } else {
        err = U32 * ERR_SIGMOID + 1e-37f;
#pragma unroll
        for (int j = 0; j < PER; ++j) v[j] = __fdividef(1.f, 1.f + __expf(-l[j])) + b[j];
      }
      uint32_t in = 0xffffffffu;  // bit of a group's first lane: the group is kept
      if (a.G > 1) {
        // each group's two largest: of the values with a bias, of the logits without (the same experts, and
        // equal scores are then known for what they are)
#pragma unroll
        for (int j = 0; j < PER; ++j) {
          const int e = lane + 32 * j;
          if (e < a.E) val[e + group_of(a, e) * (pitch - size)] = !(usable >> j & 1) ? -INFINITY : a.bias ? v[j] : l[j];
        }
        __syncwarp();
        const int g = lane / L;
        float k0 = -INFINITY, k1 = -INFINITY;
        if (g < a.G) {
          const float* at = val + g * pitch;
#pragma unroll 8
          for (int i = lane % L; i < size; i += L) {
            const float w = at[i];
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
          v0 = k0 > -INFINITY ? (a.softmax ? __expf(k0 - m) * inv_z : __fdividef(1.f, 1.f + __expf(-k0))) : k0;
          v1 = k1 > -INFINITY ? (a.softmax ? __expf(k1 - m) * inv_z : __fdividef(1.f, 1.f + __expf(-k1))) : k1;
        }
        const bool two = a.group_sum == 2 && v1 > -INFINITY;
        const float gs = two ? v0 + v1 : v0;
        int rank = 0;
#pragma unroll 4
        for (int h = 0; h < a.G; ++h) {
          const float o = __shfl_sync(0xffffffffu, gs, h * L);
          rank += (o > gs || (o == gs && h < g)) ? 1 : 0;
        }
        const bool mine = g < a.G && rank < a.keep;
        in = __ballot_sync(0xffffffffu, mine);
        // the scores' error: of two values and of their sum, none of them larger than the largest score or value
        const float big = key_logit(key_of_max(gs > -INFINITY ? fmaxf(fabsf(gs), fmaxf(fabsf(v0), two ? fabsf(v1) : 0.f)) : 0.f));
        const float ge = 2.f * err + 3.f * U32 * big;
        // (a group without a usable expert is no rival, and none is pushed out by one)
        const float least = key_logit(key_of_min(mine && gs > -INFINITY ? gs : INFINITY));
        const float rival = key_logit(key_of_max(mine || g >= a.G ? -INFINITY : gs));
        if (rival > -INFINITY && !(least - rival > 2.f * ge)) {
          bool unsure = false;  // this kept group and one that is dropped are too near, and not equal
          for (int h = 0; h < a.G; ++h) {
            const float o = __shfl_sync(0xffffffffu, gs, h * L);
            const float o0 = __shfl_sync(0xffffffffu, k0, h * L), o1 = __shfl_sync(0xffffffffu, k1, h * L);
            const bool same = !a.bias && o0 == k0 && (a.group_sum == 1 || o1 == k1);
            if (mine && !(in >> (h * L) & 1u) && o > -INFINITY && !same && !(gs - o > 2.f * ge)) unsure = true;
          }
          if (__any_sync(0xffffffffu, unsure)) {
            const double z = a.softmax && a.bias ? softmax_sum_d(sc.l, usable, m) : 1.0;
            bool sure;
            const uint32_t kept = groups_exact(a, sc.l, val, size, pitch, m, z, err, &sure);
            if (!sure) {
              __syncwarp();
              select_exact(a, t, sc.l, m, usable, reinterpret_cast<double*>(val));
              continue;
            }
            in = __ballot_sync(0xffffffffu, g < a.G && (kept >> g & 1u));
          }
        }
      }
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        const int e = lane + 32 * j;
        const bool there = e < a.E && (a.G == 1 || (in >> (group_of(a, e) * L) & 1u));
        key[j] = !there ? 0u : !(usable >> j & 1) ? 1u : value_key(a.bias ? v[j] : l[j]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < PER; ++j)
        key[j] = lane + 32 * j >= a.E ? 0u : !(usable >> j & 1) ? 1u : value_key(l[j]);
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
        const uint32_t v = __shfl_xor_sync(0xffffffffu, tau, o);
        tau = (((lane & o) == 0) == ((lane & n) == 0)) ? max(tau, v) : min(tau, v);
      }
    tau = __shfl_sync(0xffffffffu, tau, a.k - 1);
    if (VALUES && a.bias && tau > 1u) {
      const float f = key_logit(tau);
      if (f < INFINITY) tau = min(tau, value_key(f - 2.f * err - 4.f * U32 * fabsf(f)));
    }
    const uint32_t thr = max(tau, 2u);
    uint32_t is = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j)
      if (key[j] >= thr) is |= 1u << j;
    int pos = __popc(is);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, pos, o);
      if (lane >= o) pos += v;
    }
    int C = __shfl_sync(0xffffffffu, pos, 31);
    pos -= __popc(is);
    if (C <= CAND) {
#pragma unroll
      for (int j = 0; j < PER; ++j)
        if (is >> j & 1) sc.cand[pos++] = make_uint2(key[j], (uint32_t)(lane + 32 * j));
      if (C < a.k) {
        // fewer usable experts than k: masked ones of the kept groups, lower ids first
#pragma unroll
        for (int j = 0; j < PER; ++j) {
          const uint32_t bal = __ballot_sync(0xffffffffu, key[j] == 1u);
          const int at = C + __popc(bal & below);
          if (key[j] == 1u && at < a.k) sc.cand[at] = make_uint2(1u, (uint32_t)(lane + 32 * j));
          C = min(a.k, C + __popc(bal));
        }
      }
      __syncwarp();
      for (int i = lane; i < C; i += 32) {
        const uint2 me = sc.cand[i];
        int rank = 0;
#pragma unroll 4
        for (int q = 0; q < C; ++q) {
          const uint2 o = sc.cand[q];
          rank += (o.x > me.x || (o.x == me.x && o.y < me.y)) ? 1 : 0;
        }
        if (rank <= a.k) sc.sel[rank] = me;
      }
    } else if (VALUES && a.bias) {
      __syncwarp();
      select_exact(a, t, sc.l, m, usable, reinterpret_cast<double*>(val));
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
        const uint32_t id = __reduce_min_sync(0xffffffffu, bk == mx ? lane + 32u * bj : 0xffffffffu);
#pragma unroll
        for (int j = 0; j < PER; ++j)
          if (id == (uint32_t)(lane + 32 * j)) key[j] = 0u;
        if (lane == 0) sc.sel[i] = make_uint2(mx, id);
      }
    }
    __syncwarp();
    if (VALUES && a.bias) {
      // neighbours in the order whose values fp32 cannot tell apart (the same logit and bias: a true tie)
      bool unsure = false;
      if (lane < a.k && lane + 1 < C) {
        const uint2 p = sc.sel[lane], q = sc.sel[lane + 1];
        if (q.x > 1u) {
          const float u = key_logit(p.x), v = key_logit(q.x);
          unsure = !(u - v > 2.f * err + U32 * (fabsf(u) + fabsf(v))) &&
                   !(sc.l[p.y] == sc.l[q.y] && __ldg(a.bias + p.y) == __ldg(a.bias + q.y));
        }
      }
      if (__any_sync(0xffffffffu, unsure)) {
        const double z = a.softmax ? softmax_sum_d(sc.l, usable, m) : 1.0;
        double mine[CAND / 32];
#pragma unroll
        for (int h = 0; h < CAND / 32; ++h) {
          mine[h] = -INFINITY;
          if (lane + 32 * h < C) {
            const uint2 c = sc.cand[lane + 32 * h];
            if (c.x > 1u) mine[h] = score_d(sc.l[c.y], a.softmax, m, z) + (double)__ldg(a.bias + c.y);
          }
        }
        int rank[CAND / 32] = {0, 0};
        for (int q = 0; q < C; ++q) {
          const double o = __shfl_sync(0xffffffffu, q < 32 ? mine[0] : mine[1], q & 31);
          const uint32_t oe = sc.cand[q].y;
#pragma unroll
          for (int h = 0; h < CAND / 32; ++h)
            if (lane + 32 * h < C) {
              const uint32_t e = sc.cand[lane + 32 * h].y;
              rank[h] += (o > mine[h] || (o == mine[h] && oe < e)) ? 1 : 0;
            }
        }
        __syncwarp();
#pragma unroll
        for (int h = 0; h < CAND / 32; ++h)
          if (lane + 32 * h < C && rank[h] < a.k) sc.sel[rank[h]] = sc.cand[lane + 32 * h];
        __syncwarp();
      }
    }
    // weights: without groups or a bias the k largest softmax scores sum to k / E at least, above the clamp, and the
    // softmax's own sum divides out
    const bool has = lane < a.k;
    const uint2 me = sc.sel[has ? lane : 0];
    float p = 0.f;
    if (has && me.x > 1u) {
      const float x = sc.l[me.y];
      p = a.softmax ? expf(x - m) : 1.f / (1.f + expf(-x));
    }
    if (a.softmax && (VALUES || !a.renorm)) {
      if constexpr (!VALUES) {
        float z = 0.f;
#pragma unroll
        for (int j = 0; j < PER; ++j) z += usable >> j & 1 ? __expf(sc.l[lane + 32 * j] - m) : 0.f;
        z = warp_sum(z);
        inv_z = z > 0.f ? 1.f / z : 1.f;
      }
      p *= inv_z;
    }
    const float sum = a.renorm ? fmaxf(warp_sum(p), SUM_MIN) : 1.f;
    if (has) {
      a.ids[(int64_t)t * a.k + lane] = (int)me.y;
      a.weights[(int64_t)t * a.k + lane] = p / sum * a.scale;
    }
    __syncwarp();
  }
}

template <bool VALUES, int PER>
void launch_form(const SelectArgs& a, int grid, int warp_bytes, cudaStream_t s) {
  select_kernel<VALUES, PER><<<grid, 32 * SEL_WARPS, SEL_WARPS * warp_bytes, s>>>(a, warp_bytes);
}

}  // namespace

cudaError_t launch_select(const strata_select_t& sel, const void* logits, int T, const float* bias, int32_t* ids,
                          float* weights, cudaStream_t s) {
  const SelectArgs a{logits, sel.logits_stride, bias, ids, weights, T, sel.n_expert, sel.top_k,
                     sel.score == STRATA_SCORE_SOFTMAX, sel.n_group, sel.top_group, sel.group_sum, sel.renorm,
                     sel.logits_type, sel.scale, sel.n_expert / sel.n_group,
                     ((1 << 20) + sel.n_expert / sel.n_group - 1) / (sel.n_expert / sel.n_group)};
  const bool values = bias || sel.n_group > 1;
  const int warp_bytes = (int)select_warp_bytes(sel.n_expert, sel.n_group, values);
  // a warp takes ceil(T / what fits the GPU) tokens, so that all end together
  const int fit = 152 * 5 * SEL_WARPS, turns = (T + fit - 1) / fit;
  const int warps = (T + turns - 1) / turns, grid = (warps + SEL_WARPS - 1) / SEL_WARPS;
  kernel_begin(KID_SELECT, s);
  if (values && sel.n_expert > 256) launch_form<true, 16>(a, grid, warp_bytes, s);
  else if (values) launch_form<true, 8>(a, grid, warp_bytes, s);
  else if (sel.n_expert > 256) launch_form<false, 16>(a, grid, warp_bytes, s);
  else launch_form<false, 8>(a, grid, warp_bytes, s);
  kernel_end(KID_SELECT, s);
  return cudaGetLastError();
}

}  // namespace strata
