// strata_moe_q4_experts: scratch, arguments and the kernel of the weights' format.
#include "q4_experts.cuh"

namespace strata {
namespace {

struct Scratch {
  size_t h, parts, total;
};
Scratch scratch_of(const strata_q4_experts_t& ex, int T) {
  const size_t pairs = (size_t)T * ex.top_k;
  Scratch s;
  s.h = 0;
  s.parts = align256(sizeof(float) * pairs * ex.down_q4.d_in);
  s.total = s.parts + align256(sizeof(float) * pairs * ex.gate_up_q4.d_in);
  return s;
}

// Part of the wait self-test: one CTA with copies on their way comes to a meeting of two.  words: 16 bytes of zeros, then the meeting's count.
// It must run out, and the copies be there afterwards (else ST_CORRUPT too).
__global__ void __launch_bounds__(q4x::THREADS) meet_selftest_kernel(char* words, unsigned long long limit_ns, int* status) {
  __shared__ uint4 slots[q4x::THREADS];
  const uint32_t slot = smem_u32(slots + threadIdx.x);
  slots[threadIdx.x] = make_uint4(~0u, ~0u, ~0u, ~0u);
  __syncthreads();
  q4::copy_async<16>(slot, words);
  q4::copy_commit();
  const bool met = q4x::meet(reinterpret_cast<unsigned*>(words + 16), 2, status, limit_ns);
  const uint4 v = q4::lds16(slot);
  if (met || (v.x | v.y | v.z | v.w)) set_status(status, ST_CORRUPT);
}

}  // namespace

cudaError_t launch_meet_selftest(char* words, unsigned long long limit_ns, int* status, cudaStream_t s) {
  STRATA_LAUNCH(KID_WAIT_SELFTEST, s, meet_selftest_kernel<<<1, q4x::THREADS, 0, s>>>(words, limit_ns, status));
  return cudaGetLastError();
}

size_t q4_experts_scratch(const strata_q4_experts_t& ex, int T) { return scratch_of(ex, T).total; }

cudaError_t launch_q4_experts(const strata_q4_experts_t& ex, const int32_t* ids, const float* weights, const void* x, int T, void* out,
                              char* scratch, unsigned* meet, int* status, cudaStream_t s) {
  const Scratch at = scratch_of(ex, T);
  const strata_q4_t &gu = ex.gate_up_q4, &dn = ex.down_q4;
  Q4ExpertArgs a{};
  a.ids = ids, a.weights = weights, a.x = x, a.out = out;
  a.h = (float*)(scratch + at.h), a.parts = (float*)(scratch + at.parts);
  a.meet = meet, a.status = status;
  a.x_stride = ex.x_stride, a.out_stride = ex.out_stride, a.x_type = ex.x_type, a.out_type = ex.out_type;
  a.base[0] = (const uint8_t*)ex.gate_up, a.base[1] = (const uint8_t*)ex.down;
  a.expert_stride[0] = ex.gate_up_stride, a.expert_stride[1] = ex.down_stride;
  a.slab[0] = q4::slab_bytes(gu.d_in, gu.group, gu.zeros != 0), a.slab[1] = q4::slab_bytes(dn.d_in, dn.group, dn.zeros != 0);
  a.T = T, a.k = ex.top_k, a.E = ex.n_expert;
  a.columns[0] = gu.d_in, a.columns[1] = dn.d_in;
  a.terms[0] = q4::terms_of(ex.x_type, true);
  a.terms[1] = q4::terms_of(STRATA_F32, true);  // the hidden values are fp32
  return gu.group == 32 ? launch_q4_experts_32(ex, a, s) : gu.group == 64 ? launch_q4_experts_64(ex, a, s) : launch_q4_experts_128(ex, a, s);
}

}  // namespace strata
