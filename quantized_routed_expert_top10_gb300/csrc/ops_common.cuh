// Shared by the operators of strata_moe_ops.h: kernel ids after the block's, launch helpers, launch entry points.
#pragma once
#include <atomic>

#include "common.cuh"
#include "strata_moe_ops.h"

namespace strata {

// Continues KernelId.
enum OpsKernelId : int {
  KID_SELECT = KID_COUNT, KID_NORM, KID_COMBINE_NORM, KID_ADAPTER_SHRINK, KID_ADAPTER_EXPAND, KID_ADAPTERS, KID_LINEAR,
  KID_Q4_EXPERTS, KID_PACK_Q4, KID_END
};

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
// CTAs of `threads` threads (a multiple of 32, up to 1,024) and smem dynamic bytes that an SM holds at once; asked once for
// each thread count, so a kernel's smem must go with its thread count.  At least 1.
template <auto* KERNEL>
int resident_ctas(int threads, size_t smem) {
  static std::atomic<int> known[33];
  std::atomic<int>& k = known[threads / 32];
  int n = k.load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, KERNEL, threads, smem) != cudaSuccess || n < 1) n = 1;
    k.store(n, std::memory_order_relaxed);
  }
  return n;
}

// Multiprocessors of the current device, asked once for each of the first 64.
inline cudaError_t sm_count(int* sms) {
  static std::atomic<int> known[64];
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  *sms = dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
  if (*sms) return cudaSuccess;
  err = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
  if (err == cudaSuccess && dev < 64) known[dev].store(*sms, std::memory_order_relaxed);
  return err;
}

// The operators of strata_moe_ops.h (arguments checked by ops_abi.cu).
cudaError_t launch_select(const strata_select_t& sel, const void* logits, int T, const float* bias, int32_t* ids,
                          float* weights, cudaStream_t s);
cudaError_t launch_norm(const strata_norm_t& nd, const void* x, int T, const float* gain, void* out, cudaStream_t s);
cudaError_t launch_combine_norm(const strata_combine_norm_t& cn, const void* parts, const float* part_weights,
                                const void* x, int T, const float* post_gain, const float* channel_gate,
                                const float* token_gate, const float* pre_gain, void* out, void* next, cudaStream_t s);
// v_terms: scratch for A_a x as bf16 terms, [3][T][rank].
cudaError_t launch_adapters(const strata_adapters_t& ad, const int32_t* seg_off, const int32_t* seg_adapter, int n_seg,
                            const void* x, int T, const void* base, void* y, uint16_t* v_terms, int* status,
                            cudaStream_t s);

cudaError_t launch_linear(const strata_linear_t& li, const void* x, int T, const float* bias, void* y, cudaStream_t s);
// scratch: q4_experts_scratch() bytes; meet: three words that are 0 before and after.
size_t q4_experts_scratch(const strata_q4_experts_t& ex, int T);
cudaError_t launch_q4_experts(const strata_q4_experts_t& ex, const int32_t* ids, const float* weights, const void* x, int T,
                              void* out, char* scratch, unsigned* meet, int* status, cudaStream_t s);

}  // namespace strata
