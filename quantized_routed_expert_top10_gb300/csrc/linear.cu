// strata_moe_linear: y = x W^T + bias of a few tokens, W 4-bit with group scales or bf16.
//
// One persistent kernel.  A unit is 16 rows of W (a slab) for one block of tokens; S warps share it, each taking every S-th chunk of
// columns, and join their sums over shared memory.  The tokens' bf16 terms lie in shared memory for all warps of the CTA: all columns at
// once where they fit, else in panels.
#include "q4_core.cuh"

namespace strata {
namespace {

using namespace q4;

constexpr int DEPTH = 4;  // chunks that a warp's ring holds

struct LinearArgs {
  const void* x;
  const float* bias;
  void* y;
  int64_t x_stride, y_stride;
  int T, columns, rows, x_type, y_type;
  int tokens;      // of a block
  int split;       // warps to a unit
  int panel;       // chunks whose activations lie in shared memory at once, a multiple of split
  int row_stride;  // bytes between rows of terms
  int part_cols;   // term columns of a block, rounded up to whole tiles
};

template <int NT, class W>
__device__ __forceinline__ void linear_chunk(const W& w, uint32_t slot, int ch, uint32_t xs, int row_stride, int cols, uint32_t column0,
                                             int lane, float (&acc)[TILES_MAX][4]) {
  uint32_t rows[NT];
  float (&a)[NT][4] = reinterpret_cast<float (&)[NT][4]>(acc);
#pragma unroll
  for (int t = 0; t < NT; ++t)  // lanes behind the last column read some row; their sums are not used
    rows[t] = xs + min(8 * t + (lane >> 2), cols - 1) * row_stride + (lane & 3) * 16;
  chunk_products<NT>(w, slot, ch, rows, column0, lane, a);
}

template <class W>
__global__ void __launch_bounds__(THREADS, 1) linear_kernel(W w, LinearArgs a) {
  extern __shared__ __align__(128) char smem[];
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = a.split, group = warp / S, member = warp % S, n_group = WARPS / S;
  const int units = (a.rows + ROWS - 1) / ROWS, chunks = (a.columns + W::COLUMNS - 1) / W::COLUMNS;
  const int steps = (chunks + S - 1) / S;  // of a unit
  const int first = blockIdx.x * n_group, pass = gridDim.x * n_group;
  const int rounds = first < units ? (units - first + pass - 1) / pass : 0;
  const int terms = terms_of(a.x_type), blocks = (a.T + a.tokens - 1) / a.tokens;

  const uint32_t ring = smem_u32(smem) + warp * (DEPTH * W::SLOT);
  float* part = reinterpret_cast<float*>(smem + WARPS * DEPTH * W::SLOT);
  const int part_step = a.part_cols * PART_STRIDE;
  char* rows = reinterpret_cast<char*>(part + WARPS * part_step);
  const uint32_t xs = smem_u32(rows);

  // the chunks this warp will need, in the order of the loops below
  int l_round = 0, l_step = 0, l_block = 0, l_slot = 0;
  auto load_next = [&]() {
    if (l_block < blocks && rounds > 0) {
      const int u = first + group + l_round * pass, ch = member + l_step * S;
      if (u < units && ch < chunks) w.load(ring + l_slot * W::SLOT, u, ch, lane);
      if (++l_step == steps) {
        l_step = 0;
        if (++l_round == rounds) l_round = 0, ++l_block;
      }
    }
    l_slot = l_slot + 1 == DEPTH ? 0 : l_slot + 1;
    copy_commit();
  };
  for (int i = 0; i < DEPTH - 1; ++i) load_next();

  const int panel_steps = a.panel / S;
  const bool panels = a.panel < chunks;
  int slot = 0;
  for (int block = 0; block < blocks; ++block) {
    const int t0 = block * a.tokens, nt = min(a.tokens, a.T - t0), cols = nt * terms;
    for (int round = 0; round < rounds; ++round) {
      const int u = first + group + round * pass;
      float acc[TILES_MAX][4] = {};
      for (int step = 0; step < steps; ++step) {
        if (step % panel_steps == 0 && (panels || round == 0)) {  // activations of the next panel
          const int c0 = step * S * W::COLUMNS, c1 = min(c0 + a.panel * W::COLUMNS, (a.columns + BLOCK - 1) / BLOCK * BLOCK);
          const int eights = (c1 - c0) / 8;
          __syncthreads();
          for (int i = threadIdx.x; i < nt * eights; i += THREADS) {
            const int t = i / eights, c = (i - t * eights) * 8;
            stage8(a.x, (t0 + t) * a.x_stride, c0 + c, a.columns, a.x_type, terms, rows + t * terms * a.row_stride + c * 2,
                   a.row_stride);
          }
          __syncthreads();
        }
        copy_wait<DEPTH - 2>();
        load_next();  // into the slot of the step before
        const int ch = member + step * S;
        if (u < units && ch < chunks) {
          const uint32_t at = ring + slot * W::SLOT, column0 = (ch - step / panel_steps * a.panel) * W::COLUMNS;
          if (cols <= 8) linear_chunk<1>(w, at, ch, xs, a.row_stride, cols, column0, lane, acc);
          else if (cols <= 16) linear_chunk<2>(w, at, ch, xs, a.row_stride, cols, column0, lane, acc);
          else linear_chunk<3>(w, at, ch, xs, a.row_stride, cols, column0, lane, acc);
        }
        slot = slot + 1 == DEPTH ? 0 : slot + 1;
      }
      float* mine = part + warp * part_step;
      if (cols <= 8) store_part<1>(mine, lane, reinterpret_cast<float (&)[1][4]>(acc));
      else if (cols <= 16) store_part<2>(mine, lane, reinterpret_cast<float (&)[2][4]>(acc));
      else store_part<3>(mine, lane, acc);
      group_sync(group, S);
      if (u < units)
        for (int i = member * 32 + lane; i < nt * ROWS; i += S * 32) {
          const int t = i / ROWS, row = i % ROWS, n = u * ROWS + row;
          if (n < a.rows) {
            float v = sum_part(part + group * S * part_step, part_step, S, terms, t, row);
            if (a.bias) v += a.bias[n];
            store1(a.y, (t0 + t) * a.y_stride + n, a.y_type, v);
          }
        }
      group_sync(group, S);
    }
  }
  copy_wait<0>();
}

template <class W>
cudaError_t launch(const W& w, LinearArgs a, cudaStream_t s) {
  const int chunks = (a.columns + W::COLUMNS - 1) / W::COLUMNS, units = (a.rows + ROWS - 1) / ROWS;
  const int terms = terms_of(a.x_type);
  int sms = 0;
  cudaError_t err = sm_count(&sms);
  if (err != cudaSuccess) return err;
  a.tokens = 8 * TILES_MAX / terms < a.T ? 8 * TILES_MAX / terms : a.T;
  a.part_cols = (a.tokens * terms + 7) / 8 * 8;
  const size_t fixed = (size_t)WARPS * DEPTH * W::SLOT + sizeof(float) * WARPS * a.part_cols * PART_STRIDE;
  const size_t left = SMEM_MAX - fixed;
  // as many columns at once as fit; a panel is a whole number of the group's steps
  const int fit = (int)((left / (a.tokens * terms) - 64) / (2 * W::COLUMNS));  // chunks; 13 at least
  a.split = choose_split((units + sms - 1) / sms, chunks, fit);
  a.panel = (chunks + a.split - 1) / a.split * a.split;
  if (fit < a.panel) a.panel = fit / a.split * a.split;
  const int staged = a.panel * W::COLUMNS;
  a.row_stride = row_bytes(staged);
  const size_t smem = fixed + (size_t)a.tokens * terms * a.row_stride;
  err = allow_smem<linear_kernel<W>>(SMEM_MAX);
  if (err != cudaSuccess) return err;
  const int n_group = WARPS / a.split, ctas = (units + n_group - 1) / n_group;
  STRATA_LAUNCH(KID_LINEAR, s, err = launch_pdl(linear_kernel<W>, ctas < sms ? ctas : sms, THREADS, smem, s, w, a));
  return err;
}

template <int GROUP>
cudaError_t launch_q4(const strata_linear_t& li, const LinearArgs& a, cudaStream_t s) {
  const strata_q4_t& q = li.q4;
  const int64_t slab = slab_bytes(q.d_in, q.group, q.zeros != 0);
  const bool f16 = q.scale_type == STRATA_F16;
  if (q.zeros) return launch(Q4<GROUP, true>{(const uint8_t*)li.w, slab, q.d_in, f16}, a, s);
  return launch(Q4<GROUP, false>{(const uint8_t*)li.w, slab, q.d_in, f16}, a, s);
}

}  // namespace

cudaError_t launch_linear(const strata_linear_t& li, const void* x, int T, const float* bias, void* y, cudaStream_t s) {
  LinearArgs a{};
  a.x = x, a.bias = bias, a.y = y;
  a.x_stride = li.x_stride, a.y_stride = li.y_stride;
  a.T = T, a.columns = li.q4.d_in, a.rows = li.q4.n_out, a.x_type = li.x_type, a.y_type = li.y_type;
  if (li.weight == STRATA_W_BF16) return launch(Bf16{(const uint8_t*)li.w, li.w_stride, a.columns, a.rows}, a, s);
  if (li.q4.group == 32) return launch_q4<32>(li, a, s);
  return li.q4.group == 64 ? launch_q4<64>(li, a, s) : launch_q4<128>(li, a, s);
}

}  // namespace strata
