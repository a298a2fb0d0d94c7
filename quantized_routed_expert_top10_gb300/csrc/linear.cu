// strata_moe_linear: y = x W^T + bias of a few tokens, W 4-bit with group scales or bf16.
//
// One persistent kernel.  A unit is 16 rows of W (a slab) for one block of tokens (up to 24 term columns); S warps share it, each taking
// every S-th chunk of columns, and join their sums over shared memory.  The grid is units x blocks, so that a CTA lays out the terms of
// one block once, for all its units: at once where they fit beside the rings, else in panels of columns, unit by unit.  Where that is
// much work two CTAs, a cluster, do it together.
#include "q4_core.cuh"

namespace strata {
namespace {

using namespace q4;

struct LinearArgs {
  const void* x;
  const float* bias;
  void* y;
  int64_t x_stride, y_stride;
  int T, columns, rows, x_type, y_type;
  int tokens, terms;  // of a block
  int log_split;      // 2^this warps to a unit
  int panel;          // chunks whose activations lie in shared memory at once
  int row_stride;     // bytes between rows of terms
  int scale_stride;   // floats between tokens' scales
  int part_cols;      // term columns of a block, rounded up to whole tiles
};

// A warp's units, one after the other.
template <class W>
struct Units {
  const W& w;
  int unit, units, pass, member, lane;
  int whole, tail, stride;
  typename W::Cursor cursor;
  __device__ __forceinline__ bool next() {
    if (unit >= units || (whole == 0 && tail == 0)) return false;
    cursor = w.cursor(unit, member, lane);
    unit += pass;
    return true;
  }
};

// The units of this CTA for one block of tokens.
template <int NT, int WARPS, int DEPTH, bool PAIR, class W>
__device__ __forceinline__ void linear_block(const W& w, const LinearArgs& a, char* smem, int t0, int nt) {
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const int S = 1 << a.log_split, group = warp >> a.log_split, member = warp & (S - 1), n_group = WARPS >> a.log_split;
  constexpr int UNIT = ROWS * W::SLABS;
  const int units = (a.rows + UNIT - 1) / UNIT, chunks = (a.columns + W::COLUMNS - 1) / W::COLUMNS;
  const Share share(a.columns, W::COLUMNS, member, a.log_split);
  // the CTA's units lie gridDim.x apart, so that all CTAs have as many of them, or one more
  const int first = blockIdx.x, pass = gridDim.x * n_group;
  const int cols = nt * a.terms;

  float* part = reinterpret_cast<float*>(smem + WARPS * DEPTH * W::SLOT);
  const int part_step = a.part_cols * part_stride(W::SLABS);
  float* scale = part + WARPS * part_step;
  char* rows = reinterpret_cast<char*>(scale + a.tokens * a.scale_stride);
  Feed<W, DEPTH, Units<W>> feed(Units<W>{w, first + group * (int)gridDim.x, units, pass, member, lane, share.whole, share.tail, S * W::BYTES},
                                smem_u32(smem) + warp * (DEPTH * W::SLOT), lane);

  const int panel_steps = a.panel >> a.log_split;
  const bool panels = a.panel < chunks;
  for (int base = first; base < units; base += pass) {
    const int u = base + group * (int)gridDim.x;
    float acc[W::SLABS * NT][4] = {};
    for (int ch0 = 0, done = 0; ch0 < chunks; ch0 += a.panel, done += panel_steps) {
      if (panels || base == first) {  // activations of the panel
        const int c0 = ch0 * W::COLUMNS, c1 = min(c0 + a.panel * W::COLUMNS, (a.columns + BLOCK - 1) / BLOCK * BLOCK);
        const StageArgs to{static_cast<const char*>(a.x) + t0 * a.x_stride * (a.x_type == STRATA_F32 ? 4 : 2), a.x_stride, a.x_type, a.columns,
                           a.terms, rows, a.row_stride, scale, a.scale_stride, nullptr, 0, (int)(~blockIdx.x & 1)};
        if (PAIR) {
          cluster_meet();
          stage_rows<W::F16, true>(to, nt, c0, c1, (blockIdx.x & 1) * 2 * WARPS + (threadIdx.x >> 4), 4 * WARPS);
          cluster_meet();
        } else {
          __syncthreads();
          stage_rows<W::F16>(to, nt, c0, c1, threadIdx.x >> 4, 2 * WARPS);
          __syncthreads();
        }
      }
      uint32_t b[NT];
      uint2 cs[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) {  // columns behind the last read some row; their sums are not used
        b[t] = smem_u32(rows) + min(8 * t + (lane >> 2), cols - 1) * a.row_stride + (lane & 3) * 16 + member * 2 * W::COLUMNS;
        const int c = 8 * t + 2 * (lane & 3);
        cs[t].x = smem_u32(scale + min(c, cols - 1) / a.terms * a.scale_stride + member);
        cs[t].y = smem_u32(scale + min(c + 1, cols - 1) / a.terms * a.scale_stride + member);
      }
      if (u < units) {
        const int whole = min(panel_steps, share.whole - done);
        run_chunks<NT, W>(feed, whole, done <= share.whole && share.whole < done + panel_steps ? share.tail : 0, S, b, cs, acc);
      }
    }
    store_part<NT, W::SLABS>(part + warp * part_step, lane, acc);
    group_sync<WARPS>(group, S);
    const int row = lane % UNIT, n = u * UNIT + row;  // UNIT is 16 or 32
    if (u < units && n < a.rows) {
      const float bias = a.bias ? a.bias[n] : 0.f;
      for (int t = (member * 32 + lane) / UNIT; t < nt; t += S * 32 / UNIT) {
        const float v = sum_part<W::SLABS>(part + group * S * part_step, part_step, S, a.terms, t, row);
        store1(a.y, (t0 + t) * a.y_stride + n, a.y_type, v + bias);
      }
    }
    group_sync<WARPS>(group, S);
  }
  copy_wait<0>();
}

// TILES: of the largest block.  PAIR: two neighbouring CTAs, a cluster, lay out x for one another: each half of it, into both.
template <class W, int TILES, int WARPS, int DEPTH, bool PAIR>
__global__ void __launch_bounds__(32 * WARPS, 16 / WARPS) linear_kernel(W w, LinearArgs a) {
  extern __shared__ __align__(128) char smem[];
  griddep_wait();
  griddep_launch_dependents();
  for (int t0 = blockIdx.y * a.tokens; t0 < a.T; t0 += gridDim.y * a.tokens) {
    const int nt = min(a.tokens, a.T - t0), tiles = (nt * a.terms + 7) / 8;
    __syncthreads();
    if (TILES == 1 || tiles == 1) linear_block<1, WARPS, DEPTH, PAIR>(w, a, smem, t0, nt);
    else if (tiles == 2) linear_block<2, WARPS, DEPTH, PAIR>(w, a, smem, t0, nt);
    else linear_block<3, WARPS, DEPTH, PAIR>(w, a, smem, t0, nt);
  }
}

template <int TILES, int WARPS, int DEPTH, class W>
cudaError_t launch_tiles(const W& w, LinearArgs a, cudaStream_t s) {
  int sms = 0;
  cudaError_t err = sm_count(&sms);
  if (err != cudaSuccess) return err;
  const LinearPlan p = linear_plan({TILES, WARPS, DEPTH, W::SLOT, W::COLUMNS, W::SLABS}, a.T, a.columns, a.rows, a.terms, sms);
  a.tokens = p.tokens, a.log_split = p.log_split, a.panel = p.panel;
  a.row_stride = p.row_stride, a.scale_stride = p.scale_stride, a.part_cols = p.part_cols;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.grid_x, p.grid_y), cfg.blockDim = dim3(32 * WARPS), cfg.dynamicSmemBytes = p.bytes, cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2, attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr, cfg.numAttrs = p.pair ? 2 : 1;
  auto launch = [&](auto paired) {
    constexpr auto kernel = linear_kernel<W, TILES, WARPS, DEPTH, decltype(paired)::value>;
    const cudaError_t e = allow_smem<linear_kernel<W, TILES, WARPS, DEPTH, decltype(paired)::value>>(SMEM_MAX);
    return e != cudaSuccess ? e : cudaLaunchKernelEx(&cfg, kernel, w, a);
  };
  if constexpr (TILES > 1)
    if (p.pair) {
      STRATA_LAUNCH(KID_LINEAR, s, err = launch(std::true_type{}));
      return err;
    }
  STRATA_LAUNCH(KID_LINEAR, s, err = launch(std::false_type{}));
  return err;
}

// One tile: two CTAs of 8 warps an SM, one of which computes while the other lays out x or joins sums; more: one of 16, with more columns of x in
// shared memory and so fewer passes over the weights.
cudaError_t launch_bf16(const Bf16& w, LinearArgs a, cudaStream_t s) {
  a.terms = terms_of(a.x_type, false);
  return a.T * a.terms <= 8 ? launch_tiles<1, 8, 6>(w, a, s) : launch_tiles<TILES_MAX, 16, 3>(w, a, s);
}

// 4-bit weights, one tile: units of 32 rows where each CTA has 8 of them or more, one for each of its warps (131,072 rows, 27 of 16 rows a CTA: 38.2 us in
// units of 16, 36.9 in units of 32); of 16 where that would leave warps without work.
template <int GROUP, bool ZEROS, bool SCALE_F16>
cudaError_t launch_format(const uint8_t* p, int64_t slab, LinearArgs a, cudaStream_t s) {
  int sms = 0;
  cudaError_t err = sm_count(&sms);
  if (err != cudaSuccess) return err;
  a.terms = terms_of(a.x_type, true);
  const int slabs = (a.rows + ROWS - 1) / ROWS;
  const Q4<GROUP, ZEROS, SCALE_F16, 1> w{p, slab, slabs};
  if (a.T * a.terms > 8) return launch_tiles<TILES_MAX, 16, 3>(w, a, s);
  if (slabs / (2 * sms) >= 16) return launch_tiles<1, 8, 4>(Q4<GROUP, ZEROS, SCALE_F16, 2>{p, slab, slabs}, a, s);
  return launch_tiles<1, 8, 6>(w, a, s);
}

template <int GROUP>
cudaError_t launch_q4(const strata_linear_t& li, const LinearArgs& a, cudaStream_t s) {
  const strata_q4_t& q = li.q4;
  const uint8_t* p = (const uint8_t*)li.w;
  const int64_t slab = slab_bytes(q.d_in, q.group, q.zeros != 0);
  if (q.scale_type == STRATA_F16) return q.zeros ? launch_format<GROUP, true, true>(p, slab, a, s) : launch_format<GROUP, false, true>(p, slab, a, s);
  return q.zeros ? launch_format<GROUP, true, false>(p, slab, a, s) : launch_format<GROUP, false, false>(p, slab, a, s);
}

}  // namespace

cudaError_t launch_linear(const strata_linear_t& li, const void* x, int T, const float* bias, void* y, cudaStream_t s) {
  LinearArgs a{};
  a.x = x, a.bias = bias, a.y = y;
  a.x_stride = li.x_stride, a.y_stride = li.y_stride;
  a.T = T, a.columns = li.q4.d_in, a.rows = li.q4.n_out, a.x_type = li.x_type, a.y_type = li.y_type;
  if (li.weight == STRATA_W_BF16) return launch_bf16(Bf16{(const uint8_t*)li.w, li.w_stride, a.rows}, a, s);
  if (li.q4.group == 32) return launch_q4<32>(li, a, s);
  return li.q4.group == 64 ? launch_q4<64>(li, a, s) : launch_q4<128>(li, a, s);
}

}  // namespace strata
