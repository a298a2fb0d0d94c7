// strata_moe_q4_experts: the routed experts of up to 64 tokens with 4-bit weights, after routing.
//
//   q4_gate_up   h[p] = silu(G_e x_t) * (U_e x_t) of every pair p = t * k + i with an expert
//   q4_down      parts[p] = D_e h[p]
//   q4_combine   out[t] = sum over i of w[t][i] * parts[t * k + i]
//
// Every CTA of the first two sorts the pairs by expert for itself (a count over at most 2,048 pairs), so that no launch and no exchange
// stands before the weights.  The units (16 rows of one expert: 8 of gate with the same 8 of up, or 16 of down) of all experts in use
// are dealt in equal contiguous stretches, one to each CTA; S warps share a unit.
#include "q4_core.cuh"

namespace strata {
namespace {

using namespace q4;

constexpr int DEPTH = 4;  // chunks that a warp's ring holds
constexpr int PAIRS_MAX = STRATA_Q4_EXPERTS_T_MAX * STRATA_Q4_EXPERTS_K_MAX;
static_assert(PAIRS_MAX < 65536 && STRATA_Q4_EXPERTS_E_MAX <= 2 * THREADS && PAIRS_MAX <= 4 * THREADS, "sorting of the pairs");

struct ExpertArgs {
  const int32_t* ids;
  const float* weights;
  const void* x;   // q4_gate_up: the tokens; q4_down: h
  float* to;       // h or parts, a row for each pair
  int* bad;        // 1: an id outside [-1, E) (written by q4_gate_up)
  int* status;
  int64_t x_stride;
  int T, k, E, x_type, terms;
  int columns, rows;  // of an expert's matrix; rows of `to`
  int tokens;         // of a block
  int row_stride, part_cols;
};

// The pairs by expert: expert[a], its pairs pair[off[a]] .. pair[off[a + 1] - 1], a < n.
struct Sorted {
  uint16_t *expert, *off, *pair;
  int n;
  bool bad;
};
__host__ __device__ constexpr int sorted_bytes(int E, int pairs) { return (4 * E + 2 * E + 2 * (E + 1) + 2 * pairs + 15) / 16 * 16; }

__device__ __forceinline__ Sorted sort_pairs(char* smem, const ExpertArgs& a) {
  __shared__ int warp_sum[WARPS];
  int* count = reinterpret_cast<int*>(smem);  // of expert e, then the first of its pairs
  Sorted s;
  s.expert = reinterpret_cast<uint16_t*>(count + a.E);
  s.off = s.expert + a.E;
  s.pair = s.off + a.E + 1;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, pairs = a.T * a.k;
  for (int e = tid; e < a.E; e += THREADS) count[e] = 0;
  __syncthreads();
  int id[4], rank[4];
  bool bad = false;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int p = tid + j * THREADS;
    id[j] = -1;
    if (p < pairs) {
      const int e = a.ids[p];
      bad |= e < -1 || e >= a.E;
      if (e >= 0 && e < a.E && a.weights[p] != 0.f) id[j] = e, rank[j] = atomicAdd(&count[e], 1);
    }
  }
  s.bad = __syncthreads_or(bad);
  // sums before expert e of its pairs (low half) and of the experts in use (high half); two experts a thread
  const int e0 = 2 * tid, c0 = e0 < a.E ? count[e0] : 0, c1 = e0 + 1 < a.E ? count[e0 + 1] : 0;
  const int mine = c0 + c1 + (((c0 > 0) + (c1 > 0)) << 16);
  int v = mine;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int up = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += up;
  }
  if (lane == 31) warp_sum[warp] = v;
  __syncthreads();
  int before = v - mine, all = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) before += warp_sum[w];
    all += warp_sum[w];
  }
  s.n = all >> 16;
  if (c0) s.expert[before >> 16] = e0, s.off[before >> 16] = before & 0xffff;
  if (e0 < a.E) count[e0] = before & 0xffff;
  before += c0 + ((c0 > 0) << 16);
  if (c1) s.expert[before >> 16] = e0 + 1, s.off[before >> 16] = before & 0xffff;
  if (e0 + 1 < a.E) count[e0 + 1] = before & 0xffff;
  if (tid == 0) s.off[s.n] = all & 0xffff;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < 4; ++j)  // the order within an expert does not matter: a pair's sums are its own column's
    if (id[j] >= 0) s.pair[count[id[j]] + rank[j]] = tid + j * THREADS;
  __syncthreads();
  return s;
}

template <int NT, class W>
__device__ __forceinline__ void expert_chunk(const W& w, uint32_t slot, int64_t s, int ch, uint32_t xs, int row_stride, int cols, int lane,
                                             float (&acc)[TILES_MAX][4]) {
  uint32_t rows[NT];
  float (&a)[NT][4] = reinterpret_cast<float (&)[NT][4]>(acc);
#pragma unroll
  for (int t = 0; t < NT; ++t)  // lanes behind the last column read some row; their sums are not used
    rows[t] = xs + min(8 * t + (lane >> 2), cols - 1) * row_stride + (lane & 3) * 16;
  chunk_products<NT>(w, slot, ch, rows, ch * W::COLUMNS, lane, a);
}

template <bool DOWN, class W>
__global__ void __launch_bounds__(THREADS, 1) experts_kernel(W w, int64_t expert_stride, ExpertArgs a) {
  extern __shared__ __align__(128) char smem[];
  if (!DOWN) griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t ring = smem_u32(smem) + warp * (DEPTH * W::SLOT);
  float* part = reinterpret_cast<float*>(smem + WARPS * DEPTH * W::SLOT);
  const int part_step = a.part_cols * PART_STRIDE;
  char* rows = reinterpret_cast<char*>(part + WARPS * part_step);
  const uint32_t xs = smem_u32(rows);
  const Sorted sorted = sort_pairs(rows + a.tokens * a.terms * a.row_stride, a);
  if (!DOWN && blockIdx.x == 0 && threadIdx.x == 0) {
    *a.bad = sorted.bad;
    if (sorted.bad) set_status(a.status, ST_CORRUPT);
  }
  if (sorted.bad) {
    if (DOWN) griddep_wait();  // its end has to mean the end of the kernels before it
    return;
  }

  const int slabs = DOWN ? a.rows / ROWS : a.rows / 8, chunks = (a.columns + CHUNK - 1) / CHUNK;
  const int units = sorted.n * slabs;
  const int u0 = (int)((int64_t)blockIdx.x * units / gridDim.x), u1 = (int)((int64_t)(blockIdx.x + 1) * units / gridDim.x);
  const int S = choose_split((units + gridDim.x - 1) / gridDim.x, chunks);
  const int group = warp / S, member = warp % S, n_group = WARPS / S;
  const int steps = (chunks + S - 1) / S;

  auto load = [&](uint32_t slot, int u, int ch) {
    const int e = u / slabs;
    W we = w;
    we.base += sorted.expert[e] * expert_stride;
    we.load(slot, u - e * slabs, ch, lane);
  };
  auto blocks_of = [&](int e) { return (sorted.off[e + 1] - sorted.off[e] + a.tokens - 1) / a.tokens; };
  // the chunks this warp will need, in the order of the loops below
  int l_begin = u0, l_end = u0, l_u = u0, l_step = 0, l_left = 0, l_slot = 0;  // an expert's stretch, its blocks left
  auto next_expert = [&]() {
    l_begin = l_u = l_end;
    if (l_begin < u1) {
      const int e = l_begin / slabs;
      l_end = min(u1, (e + 1) * slabs);
      l_left = blocks_of(e);
    }
  };
  next_expert();
  auto load_next = [&]() {
    if (l_begin < u1) {
      const int u = l_u + group, ch = member + l_step * S;
      if (u < l_end && ch < chunks) load(ring + l_slot * W::SLOT, u, ch);
      if (++l_step == steps) {
        l_step = 0;
        l_u += n_group;
        if (l_u >= l_end) {
          l_u = l_begin;
          if (--l_left == 0) next_expert();
        }
      }
    }
    l_slot = l_slot + 1 == DEPTH ? 0 : l_slot + 1;
    copy_commit();
  };
  for (int i = 0; i < DEPTH - 1; ++i) load_next();
  if (DOWN) griddep_wait();  // h

  int slot = 0;
  for (int begin = u0; begin < u1;) {
    const int e = begin / slabs, end = min(u1, (e + 1) * slabs), first = sorted.off[e], last = sorted.off[e + 1];
    for (int p0 = first; p0 < last; p0 += a.tokens) {
      const int np = min(a.tokens, last - p0), cols = np * a.terms, eights = a.columns / 8;
      __syncthreads();
      for (int i = threadIdx.x; i < np * eights; i += THREADS) {
        const int j = i / eights, c = (i - j * eights) * 8, p = sorted.pair[p0 + j];
        stage8(a.x, (DOWN ? p : p / a.k) * a.x_stride, c, a.columns, a.x_type, a.terms, rows + j * a.terms * a.row_stride + c * 2,
               a.row_stride);
      }
      __syncthreads();
      for (int base = begin; base < end; base += n_group) {
        const int u = base + group;
        float acc[TILES_MAX][4] = {};
        for (int step = 0; step < steps; ++step) {
          copy_wait<DEPTH - 2>();
          load_next();  // into the slot of the step before
          const int ch = member + step * S;
          if (u < end && ch < chunks) {
            const uint32_t at = ring + slot * W::SLOT;
            if (cols <= 8) expert_chunk<1>(w, at, u, ch, xs, a.row_stride, cols, lane, acc);
            else if (cols <= 16) expert_chunk<2>(w, at, u, ch, xs, a.row_stride, cols, lane, acc);
            else expert_chunk<3>(w, at, u, ch, xs, a.row_stride, cols, lane, acc);
          }
          slot = slot + 1 == DEPTH ? 0 : slot + 1;
        }
        float* mine = part + warp * part_step;
        if (cols <= 8) store_part<1>(mine, lane, reinterpret_cast<float (&)[1][4]>(acc));
        else if (cols <= 16) store_part<2>(mine, lane, reinterpret_cast<float (&)[2][4]>(acc));
        else store_part<3>(mine, lane, acc);
        group_sync(group, S);
        if (u < end) {
          const float* sums = part + group * S * part_step;
          const int at = (u - e * slabs) * (DOWN ? ROWS : 8);
          for (int i = member * 32 + lane; i < np * (DOWN ? ROWS : 8); i += S * 32) {
            const int j = DOWN ? i / ROWS : i / 8, row = DOWN ? i % ROWS : i % 8;
            float v = sum_part(sums, part_step, S, a.terms, j, row);
            if (!DOWN) v = silu_mul(v, sum_part(sums, part_step, S, a.terms, j, row + 8));
            a.to[(int64_t)sorted.pair[p0 + j] * a.rows + at + row] = v;
          }
        }
        group_sync(group, S);
      }
    }
    begin = end;
  }
  copy_wait<0>();
}

// Eight columns of a token a thread.
__global__ void __launch_bounds__(256) combine_kernel(const int32_t* ids, const float* weights, const float* parts, const int* bad, int T,
                                                      int k, int columns, int out_type, int64_t out_stride, void* out) {
  griddep_wait();
  griddep_launch_dependents();
  const int i = blockIdx.x * 256 + threadIdx.x, eights = columns / 8;
  if (i >= T * eights || *bad) return;
  const int t = i / eights, c = (i - t * eights) * 8;
  float sum[8] = {};
  for (int j = 0; j < k; ++j) {
    const int p = t * k + j;
    const float w = weights[p];
    if (ids[p] < 0 || w == 0.f) continue;
    float f[8];
    widen8(load8(parts, (int64_t)p * columns + c, STRATA_F32), STRATA_F32, f);
#pragma unroll
    for (int n = 0; n < 8; ++n) sum[n] = fmaf(w, f[n], sum[n]);
  }
  store8(out, t * out_stride + c, out_type, sum);
}

struct Scratch {
  size_t h, parts, total;
};
Scratch scratch_of(const strata_q4_experts_t& ex, int T) {
  const size_t pairs = (size_t)T * ex.top_k;
  Scratch s;
  s.h = 256;
  s.parts = s.h + align256(sizeof(float) * pairs * ex.down_q4.d_in);
  s.total = s.parts + align256(sizeof(float) * pairs * ex.gate_up_q4.d_in);
  return s;
}

template <bool DOWN, class W>
cudaError_t launch(const W& w, int64_t stride, ExpertArgs a, cudaStream_t s) {
  int sms = 0;
  cudaError_t err = sm_count(&sms);
  if (err != cudaSuccess) return err;
  const int sorted = sorted_bytes(a.E, a.T * a.k);
  a.row_stride = row_bytes(a.columns);
  // as many tokens at once as fit with their sums, of the pairs one expert can have
  const int most = a.T * a.k;
  auto bytes = [&](int tokens) {
    return (size_t)WARPS * DEPTH * W::SLOT + sizeof(float) * WARPS * ((tokens * a.terms + 7) / 8 * 8) * PART_STRIDE +
           (size_t)tokens * a.terms * a.row_stride + sorted;
  };
  a.tokens = 1;
  while (a.tokens < most && (a.tokens + 1) * a.terms <= 8 * TILES_MAX && bytes(a.tokens + 1) <= SMEM_MAX - 1024) ++a.tokens;
  a.part_cols = (a.tokens * a.terms + 7) / 8 * 8;
  err = allow_smem<experts_kernel<DOWN, W>>(SMEM_MAX - 1024);
  if (err != cudaSuccess) return err;
  STRATA_LAUNCH(DOWN ? KID_Q4_DOWN : KID_Q4_GATE_UP, s,
                err = launch_pdl(experts_kernel<DOWN, W>, sms, THREADS, bytes(a.tokens), s, w, stride, a));
  return err;
}

template <bool DOWN>
cudaError_t launch_format(const strata_q4_t& q, const void* w, int64_t stride, const ExpertArgs& a, cudaStream_t s) {
  const int64_t slab = slab_bytes(q.d_in, q.group, q.zeros != 0);
  const uint8_t* p = (const uint8_t*)w;
  const bool f16 = q.scale_type == STRATA_F16;
  if (q.group == 32)
    return q.zeros ? launch<DOWN>(Q4<32, true>{p, slab, q.d_in, f16}, stride, a, s)
                   : launch<DOWN>(Q4<32, false>{p, slab, q.d_in, f16}, stride, a, s);
  if (q.group == 64)
    return q.zeros ? launch<DOWN>(Q4<64, true>{p, slab, q.d_in, f16}, stride, a, s)
                   : launch<DOWN>(Q4<64, false>{p, slab, q.d_in, f16}, stride, a, s);
  return q.zeros ? launch<DOWN>(Q4<128, true>{p, slab, q.d_in, f16}, stride, a, s)
                 : launch<DOWN>(Q4<128, false>{p, slab, q.d_in, f16}, stride, a, s);
}

}  // namespace

size_t q4_experts_scratch(const strata_q4_experts_t& ex, int T) { return scratch_of(ex, T).total; }

cudaError_t launch_q4_experts(const strata_q4_experts_t& ex, const int32_t* ids, const float* weights, const void* x, int T, void* out,
                              char* scratch, int* status, cudaStream_t s) {
  const Scratch at = scratch_of(ex, T);
  const int d_model = ex.gate_up_q4.d_in, d_ff = ex.down_q4.d_in;
  float *h = (float*)(scratch + at.h), *parts = (float*)(scratch + at.parts);
  ExpertArgs a{};
  a.ids = ids, a.weights = weights, a.bad = (int*)scratch, a.status = status;
  a.T = T, a.k = ex.top_k, a.E = ex.n_expert;
  a.x = x, a.x_stride = ex.x_stride, a.x_type = ex.x_type, a.terms = terms_of(ex.x_type);
  a.to = h, a.columns = d_model, a.rows = d_ff;
  cudaError_t err = launch_format<false>(ex.gate_up_q4, ex.gate_up, ex.gate_up_stride, a, s);
  if (err != cudaSuccess) return err;
  a.x = h, a.x_stride = d_ff, a.x_type = STRATA_F32, a.terms = ex.out_type == STRATA_F32 ? 3 : 2;
  a.to = parts, a.columns = d_ff, a.rows = d_model;
  err = launch_format<true>(ex.down_q4, ex.down, ex.down_stride, a, s);
  if (err != cudaSuccess) return err;
  const int ctas = (T * (d_model / 8) + 255) / 256;
  STRATA_LAUNCH(KID_Q4_COMBINE, s,
                err = launch_pdl(combine_kernel, ctas, 256, 0, s, ids, weights, parts, a.bad, T, a.k, d_model, ex.out_type,
                                 ex.out_stride, out));
  return err;
}

}  // namespace strata
