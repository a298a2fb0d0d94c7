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
  int tokens;         // pairs of a block
  int resident;       // all tokens' (all pairs') terms lie in shared memory from the start, else a block's
  int staged;         // rows of x in shared memory at once
  int depth, row_stride, scale_stride, part_cols;
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
  if (pairs <= 32) {  // one warp, a pair a lane; an expert's first pair stands for it
    if (warp == 0) {
      const int e = lane < pairs ? a.ids[lane] : -1;
      const bool have = e >= 0 && e < a.E && a.weights[lane] != 0.f;
      const uint32_t same = __match_any_sync(0xffffffffu, have ? e : -1), before = (1u << lane) - 1u;
      const bool first = have && (same & before) == 0;
      const uint32_t firsts = __ballot_sync(0xffffffffu, first);
      const int count = first ? __popc(same) : 0;
      int off = count;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const int up = __shfl_up_sync(0xffffffffu, off, o);
        if (lane >= o) off += up;
      }
      off -= count;
      const int mine = __shfl_sync(0xffffffffu, off, __ffs(same) - 1);
      if (first) s.expert[__popc(firsts & before)] = e, s.off[__popc(firsts & before)] = off;
      if (have) s.pair[mine + __popc(same & before)] = lane;
      const int bad = __any_sync(0xffffffffu, lane < pairs && (e < -1 || e >= a.E));
      const int all = __popc(__ballot_sync(0xffffffffu, have));
      if (lane == 0) {
        warp_sum[0] = __popc(firsts), warp_sum[1] = bad;
        s.off[__popc(firsts)] = all;
      }
    }
    __syncthreads();
    s.n = warp_sum[0];
    s.bad = warp_sum[1];
    return s;
  }
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

// The units of a stretch u0 .. u1 - 1 in the order in which a CTA takes them: for each expert of the stretch, for each block of its pairs,
// its units, n_group at a time.  Walked by the copies, a ring ahead of the products.
template <class W>
struct Loader {
  const Sorted& sorted;
  const Share& share;
  int64_t expert_stride;
  int slabs, S, member, group, n_group, u1, tokens;
  int begin, end, blocks;  // the expert's stretch, its blocks left
  int u, left;             // this warp's unit, its chunks left
  const uint8_t* at;
  W w;                     // the expert's matrix, from the first unit's place
  const uint8_t* base;     // of expert 0

  // The next expert (true) or block with a unit for this warp, from the unit base on.
  __device__ __forceinline__ void expert() {
    begin = end;
    if (begin >= u1) return;
    const int e = begin / slabs;
    end = min(u1, (e + 1) * slabs);
    blocks = (sorted.off[e + 1] - sorted.off[e] + tokens - 1) / tokens;
    w.base = base + sorted.expert[e] * expert_stride - (int64_t)e * slabs * w.slab;
  }
  __device__ __forceinline__ void find(int from, int lane) {  // the first unit of this warp in the CTA's units from `from` on
    u = from + group;
    while (u >= end && begin < u1) {
      if (--blocks == 0) expert();
      u = begin + group;
    }
    left = begin < u1 ? share.whole + share.tail : 0;
    if (left) at = w.at(u, member, lane);
  }
  __device__ __forceinline__ void next(Ring& ring, int lane) {
    if (left) {
      const uint32_t slot = ring.next_fill();
      if (left == 1 && share.tail) w.load_tail(slot, at, u, 0, lane);
      else w.load(slot, at, u, 0, lane);
      at += S * W::BYTES;
      if (--left == 0) find(u - group + n_group, lane);
    }
    copy_commit();
  }
};

// The units begin .. end - 1 of one expert for np of its pairs (from position p0 of the sorted ones).
template <bool DOWN, int NT, class W>
__device__ __forceinline__ void expert_block(const W& w, const ExpertArgs& a, const Sorted& sorted, Loader<W>& loader, Ring& ring, float* part,
                                             const float* scale, const char* rows, int begin, int end, int first_unit, int p0, int np) {
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const int S = loader.S, group = loader.group, member = loader.member;
  const int part_step = a.part_cols * PART_STRIDE;
  uint32_t b0[NT];
  uint2 cs0[NT];
  auto row_of = [&](int j) {  // of pair j of the block among those in shared memory
    j = min(j, np - 1);       // columns behind the last read some row; their sums are not used
    return !a.resident ? j : DOWN ? p0 + j : sorted.pair[p0 + j] / a.k;
  };
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int c = 8 * t + (lane >> 2), j = c / a.terms;
    b0[t] = smem_u32(rows) + (row_of(j) * a.terms + (c - j * a.terms)) * a.row_stride + (lane & 3) * 16 + member * 2 * W::COLUMNS;
    const int c2 = 8 * t + 2 * (lane & 3);
    cs0[t].x = smem_u32(scale + row_of(c2 / a.terms) * a.scale_stride + member);
    cs0[t].y = smem_u32(scale + row_of((c2 + 1) / a.terms) * a.scale_stride + member);
  }
  for (int base = begin; base < end; base += loader.n_group) {
    const int u = base + group;
    float acc[NT][4] = {};
    if (u < end) {
      uint32_t b[NT];
      uint2 cs[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) b[t] = b0[t], cs[t] = cs0[t];
      run_chunks<NT>(w, ring, loader, loader.share.whole, loader.share.tail, S, b, cs, lane, acc);
    }
    store_part<NT>(part + warp * part_step, lane, acc);
    group_sync(group, S);
    if (u < end) {
      const float* sums = part + group * S * part_step;
      constexpr int OUT = DOWN ? ROWS : 8;
      for (int i = member * 32 + lane; i < np * OUT; i += S * 32) {
        const int j = i / OUT, row = i % OUT;
        float v = sum_part(sums, part_step, S, a.terms, j, row);
        if (!DOWN) v = silu_mul(v, sum_part(sums, part_step, S, a.terms, j, row + 8));
        a.to[(int64_t)sorted.pair[p0 + j] * a.rows + (u - first_unit) * OUT + row] = v;
      }
    }
    group_sync(group, S);
  }
}

template <bool DOWN, class W>
__global__ void __launch_bounds__(THREADS, 1) experts_kernel(W w, int64_t expert_stride, ExpertArgs a) {
  extern __shared__ __align__(128) char smem[];
  if (!DOWN) griddep_wait();
  griddep_launch_dependents();
  const int warp = warp_index(), lane = threadIdx.x & 31;
  float* part = reinterpret_cast<float*>(smem + WARPS * a.depth * W::SLOT);
  float* scale = part + WARPS * a.part_cols * PART_STRIDE;
  char* rows = reinterpret_cast<char*>(scale + a.staged * a.scale_stride);
  const Sorted sorted = sort_pairs(rows + a.staged * a.terms * a.row_stride, a);
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
  // 2^20 units at most (1,024 experts of 1,024 slabs): 32 bits hold their products with the grid
  const int u0 = (unsigned)(blockIdx.x * units) / gridDim.x, u1 = (unsigned)((blockIdx.x + 1) * units) / gridDim.x;
  const int S = choose_split((unsigned)(units + gridDim.x - 1) / gridDim.x, chunks);
  const Share share(a.columns, CHUNK, chunks, warp % S, S);
  Ring ring(smem_u32(smem) + warp * (a.depth * W::SLOT), a.depth, W::SLOT);
  Loader<W> loader{sorted, share, expert_stride, slabs, S, warp % S, warp / S, WARPS / S, u1, a.tokens, u0, u0, 0, 0, 0, nullptr, w, w.base};
  loader.expert();
  loader.find(u0, lane);
  for (int i = 0; i < a.depth - 1; ++i) loader.next(ring, lane);
  if (DOWN) griddep_wait();  // h

  // the terms of the block's rows: source(j) is row j of x
  auto stage = [&](int n, auto source) {
    const int half = threadIdx.x >> 4, halves = n < 2 * WARPS ? 2 * WARPS / n : 1;
    for (int j = half / halves; j < n; j += 2 * WARPS / halves) {
      if (half >= 2 * WARPS / halves * halves) break;
      stage_row<true>(a.x, source(j) * a.x_stride, a.x_type, a.columns, 0, a.columns, a.terms, rows + j * a.terms * a.row_stride,
                      a.row_stride, scale + j * a.scale_stride, half % halves, halves);
    }
  };
  if (a.resident && u0 < u1) {
    if (DOWN) stage(sorted.off[sorted.n], [&](int j) { return (int64_t)sorted.pair[j]; });
    else stage(a.T, [&](int j) { return (int64_t)j; });
    __syncthreads();
  }
  for (int begin = u0; begin < u1;) {
    const int e = begin / slabs, end = min(u1, (e + 1) * slabs), last = sorted.off[e + 1];
    for (int p0 = sorted.off[e]; p0 < last; p0 += a.tokens) {
      const int np = min(a.tokens, last - p0), tiles = (np * a.terms + 7) / 8;
      if (!a.resident) {
        __syncthreads();
        stage(np, [&](int j) { return (int64_t)(DOWN ? sorted.pair[p0 + j] : sorted.pair[p0 + j] / a.k); });
        __syncthreads();
      }
      if (tiles == 1) expert_block<DOWN, 1>(w, a, sorted, loader, ring, part, scale, rows, begin, end, e * slabs, p0, np);
      else if (tiles == 2) expert_block<DOWN, 2>(w, a, sorted, loader, ring, part, scale, rows, begin, end, e * slabs, p0, np);
      else expert_block<DOWN, 3>(w, a, sorted, loader, ring, part, scale, rows, begin, end, e * slabs, p0, np);
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
  const int sorted = sorted_bytes(a.E, a.T * a.k), most = DOWN ? a.T * a.k : a.T;
  a.row_stride = row_bytes(a.columns);
  a.scale_stride = ((a.columns + CHUNK - 1) / CHUNK + 3) / 4 * 4;
  a.depth = 4;
  a.tokens = 8 * TILES_MAX / a.terms < a.T * a.k ? 8 * TILES_MAX / a.terms : a.T * a.k;
  auto bytes = [&]() {
    a.part_cols = (a.tokens * a.terms + 7) / 8 * 8;
    return (size_t)WARPS * a.depth * W::SLOT + sizeof(float) * (WARPS * a.part_cols * PART_STRIDE + (size_t)a.staged * a.scale_stride) +
           (size_t)a.staged * a.terms * a.row_stride + sorted;
  };
  a.staged = most;
  a.resident = bytes() <= SMEM_MAX;
  if (!a.resident)  // as many of a block's as fit; one always does
    for (;; --a.tokens) {
      a.staged = a.tokens;
      if (bytes() <= SMEM_MAX) break;
    }
  err = allow_smem<experts_kernel<DOWN, W>>(SMEM_MAX);
  if (err != cudaSuccess) return err;
  STRATA_LAUNCH(DOWN ? KID_Q4_DOWN : KID_Q4_GATE_UP, s,
                err = launch_pdl(experts_kernel<DOWN, W>, sms, THREADS, bytes(), s, w, stride, a));
  return err;
}

template <bool DOWN, int GROUP>
cudaError_t launch_scales(const strata_q4_t& q, const uint8_t* p, int64_t slab, int64_t stride, const ExpertArgs& a, cudaStream_t s) {
  if (q.scale_type == STRATA_F16)
    return q.zeros ? launch<DOWN>(Q4<GROUP, true, true>{p, slab, q.d_in}, stride, a, s)
                   : launch<DOWN>(Q4<GROUP, false, true>{p, slab, q.d_in}, stride, a, s);
  return q.zeros ? launch<DOWN>(Q4<GROUP, true, false>{p, slab, q.d_in}, stride, a, s)
                 : launch<DOWN>(Q4<GROUP, false, false>{p, slab, q.d_in}, stride, a, s);
}

template <bool DOWN>
cudaError_t launch_format(const strata_q4_t& q, const void* w, int64_t stride, const ExpertArgs& a, cudaStream_t s) {
  const int64_t slab = slab_bytes(q.d_in, q.group, q.zeros != 0);
  const uint8_t* p = (const uint8_t*)w;
  if (q.group == 32) return launch_scales<DOWN, 32>(q, p, slab, stride, a, s);
  return q.group == 64 ? launch_scales<DOWN, 64>(q, p, slab, stride, a, s) : launch_scales<DOWN, 128>(q, p, slab, stride, a, s);
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
  a.x = x, a.x_stride = ex.x_stride, a.x_type = ex.x_type, a.terms = terms_of(ex.x_type, true);
  a.to = h, a.columns = d_model, a.rows = d_ff;
  cudaError_t err = launch_format<false>(ex.gate_up_q4, ex.gate_up, ex.gate_up_stride, a, s);
  if (err != cudaSuccess) return err;
  a.x = h, a.x_stride = d_ff, a.x_type = STRATA_F32;
  // one fp16 term (11 bits, an error of 2^-11 where the sum of many such is rounded to 8 bits) for a bf16 result, two for the others
  a.terms = ex.out_type == STRATA_BF16 ? 1 : 2;
 
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
