// Elements of the three activation types (STRATA_F32, STRATA_BF16, STRATA_F16) at addresses and types known at run
// time: widened exactly to fp32 when read, rounded to nearest even when stored.
#pragma once
#include <cuda_bf16.h>

#include "ops_common.cuh"

namespace strata {

__device__ __forceinline__ float lowest_of(int type) {
  return type == STRATA_F32 ? -3.402823466e38f : type == STRATA_BF16 ? __uint_as_float(0xff7f0000u) : -65504.f;
}
__device__ __forceinline__ float load1(const void* p, int64_t i, int type) {
  if (type == STRATA_F32) return static_cast<const float*>(p)[i];
  if (type == STRATA_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  return __half2float(static_cast<const __half*>(p)[i]);
}
__device__ __forceinline__ void store1(void* p, int64_t i, int type, float v) {
  if (type == STRATA_F32) static_cast<float*>(p)[i] = v;
  else if (type == STRATA_BF16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else static_cast<__half*>(p)[i] = __float2half_rn(v);
}

// Eight consecutive elements on a 16-byte boundary, as read (one 16-byte piece of a 16-bit type, two of fp32).
struct Raw8 {
  uint4 lo, hi;
};
__device__ __forceinline__ Raw8 load8(const void* p, int64_t i, int type) {
  Raw8 r;
  if (type == STRATA_F32) {
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + i);
    r.lo = q[0];
    r.hi = q[1];
  } else {
    r.lo = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
    r.hi = make_uint4(0u, 0u, 0u, 0u);
  }
  return r;
}
__device__ __forceinline__ float2 widen2(uint32_t w, int type) {
  if (type == STRATA_BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
__device__ __forceinline__ void widen8(const Raw8& r, int type, float (&f)[8]) {
  if (type == STRATA_F32) {
    f[0] = __uint_as_float(r.lo.x); f[1] = __uint_as_float(r.lo.y);
    f[2] = __uint_as_float(r.lo.z); f[3] = __uint_as_float(r.lo.w);
    f[4] = __uint_as_float(r.hi.x); f[5] = __uint_as_float(r.hi.y);
    f[6] = __uint_as_float(r.hi.z); f[7] = __uint_as_float(r.hi.w);
  } else {
    const uint32_t w[4] = {r.lo.x, r.lo.y, r.lo.z, r.lo.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = widen2(w[i], type);
      f[2 * i] = v.x;
      f[2 * i + 1] = v.y;
    }
  }
}
__device__ __forceinline__ uint32_t narrow2(float a, float b, int type) {
  if (type == STRATA_BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void store8(void* p, int64_t i, int type, const float (&f)[8]) {
  if (type == STRATA_F32) {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    q[0] = make_float4(f[0], f[1], f[2], f[3]);
    q[1] = make_float4(f[4], f[5], f[6], f[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) =
        make_uint4(narrow2(f[0], f[1], type), narrow2(f[2], f[3], type), narrow2(f[4], f[5], type),
                   narrow2(f[6], f[7], type));
  }
}

}  // namespace strata
