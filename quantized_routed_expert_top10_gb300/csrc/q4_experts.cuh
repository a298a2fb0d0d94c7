// strata_moe_q4_experts: the routed experts of up to 64 tokens with 4-bit weights, after routing, in one persistent kernel.
//
//   1. h[p] = silu(G_e x_t) * (U_e x_t) of every pair p = t * k + i with an expert
//   2. parts[p] = D_e h[p]
//   3. out[t] = sum over i of w[t][i] * parts[t * k + i], in the order of i
//
// Every CTA sorts the pairs by expert for itself (a count over at most 2,048 pairs), so that no launch and no exchange stands before the
// weights.  The units of step 1 (16 rows of one expert: 8 of gate with the same 8 of up) and then those of step 2 (16 rows of down) are dealt in
// equal contiguous stretches, one of each to a CTA; S warps share a unit.  All CTAs are resident (a cooperative launch) and meet between the
// steps; the copies of weights run ahead across the meeting, so step 2 finds its first chunks in shared memory.
#pragma once
#include "q4_core.cuh"

namespace strata {

struct Q4ExpertArgs {
  const int32_t* ids;
  const float* weights;
  const void* x;
  void* out;
  float *h, *parts;       // a row for each pair
  unsigned* meet;         // three words, 0 between calls: two meetings and the way out
  int* status;
  int64_t x_stride, out_stride;
  const uint8_t* base[2];  // packed matrices of expert 0 (gate and up; down)
  int64_t expert_stride[2];
  int64_t slab[2];         // bytes of 16 rows
  int T, k, E, x_type, out_type;
  int columns[2];          // d_model, d_ff
  int terms[2];
  int tokens[2];           // pairs of a block
  int resident;            // step 1: all tokens' terms lie in shared memory at once, else a block's
  int staged;              // rows of x or h in shared memory at once
  int row_stride, scale_stride, part_cols;
};

namespace q4x {

using namespace q4;

constexpr int WARPS = 8, THREADS = 32 * WARPS;  // two CTAs an SM, one of which computes while the other lays out x or joins sums
constexpr int DEPTH = 5;                        // chunks of a warp's ring
constexpr int PAIRS_MAX = STRATA_Q4_EXPERTS_T_MAX * STRATA_Q4_EXPERTS_K_MAX;
constexpr int PER_THREAD = PAIRS_MAX / THREADS, E_PER_THREAD = STRATA_Q4_EXPERTS_E_MAX / THREADS;
static_assert(PAIRS_MAX < 65536 && PAIRS_MAX % THREADS == 0 && STRATA_Q4_EXPERTS_E_MAX % THREADS == 0, "sorting of the pairs");

// The pairs by expert: expert[a], its pairs pair[off[a]] .. pair[off[a + 1] - 1], a < n.
struct Sorted {
  uint16_t *expert, *off, *pair;
  int n;
  bool bad;  // an id outside [-1, E)
};
__host__ __device__ constexpr int sorted_bytes(int E, int pairs) { return (4 * E + 2 * E + 2 * (E + 1) + 2 * pairs + 15) / 16 * 16; }

static __device__ __noinline__ Sorted sort_pairs(char* smem, const int32_t* ids, const float* weights, int pairs, int E) {
  __shared__ int warp_sum[WARPS];
  int* count = reinterpret_cast<int*>(smem);  // of expert e, then the first of its pairs
  Sorted s;
  s.expert = reinterpret_cast<uint16_t*>(count + E);
  s.off = s.expert + E;
  s.pair = s.off + E + 1;
  const int tid = threadIdx.x, lane = tid & 31, warp = warp_index();
  if (pairs <= 32) {  // one warp, a pair a lane; an expert's first pair stands for it
    if (warp == 0) {
      const int e = lane < pairs ? ids[lane] : -1;
      const float weight = lane < pairs ? weights[lane] : 0.f;
      const bool have = e >= 0 && e < E && weight != 0.f;
      const uint32_t same = __match_any_sync(0xffffffffu, have ? e : -1), before = (1u << lane) - 1u;
      const bool first = have && (same & before) == 0;
      const uint32_t firsts = __ballot_sync(0xffffffffu, first);
      const int count_here = first ? __popc(same) : 0;
      int off = count_here;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const int up = __shfl_up_sync(0xffffffffu, off, o);
        if (lane >= o) off += up;
      }
      off -= count_here;
      const int mine = __shfl_sync(0xffffffffu, off, __ffs(same) - 1);
      if (first) s.expert[__popc(firsts & before)] = e, s.off[__popc(firsts & before)] = off;
      if (have) s.pair[mine + __popc(same & before)] = lane;
      const int bad = __any_sync(0xffffffffu, lane < pairs && (e < -1 || e >= E));
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
  for (int e = tid; e < E; e += THREADS) count[e] = 0;
  __syncthreads();
  int id[PER_THREAD], rank[PER_THREAD];
  float weight[PER_THREAD];
#pragma unroll
  for (int j = 0; j < PER_THREAD; ++j) {
    const int p = tid + j * THREADS;
    id[j] = p < pairs ? ids[p] : -1;
    weight[j] = p < pairs ? weights[p] : 0.f;
  }
  bool bad = false;
#pragma unroll
  for (int j = 0; j < PER_THREAD; ++j) {
    bad |= id[j] < -1 || id[j] >= E;
    if (id[j] < 0 || id[j] >= E || weight[j] == 0.f) id[j] = -1;
    else rank[j] = atomicAdd(&count[id[j]], 1);
  }
  s.bad = __syncthreads_or(bad);
  // sums before each expert of the pairs (low half) and of the experts in use (high half); consecutive experts a thread
  const int e0 = E_PER_THREAD * tid;
  int c[E_PER_THREAD], mine = 0;
#pragma unroll
  for (int j = 0; j < E_PER_THREAD; ++j) {
    c[j] = e0 + j < E ? count[e0 + j] : 0;
    mine += c[j] + ((c[j] > 0) << 16);
  }
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
#pragma unroll
  for (int j = 0; j < E_PER_THREAD; ++j) {
    if (c[j]) s.expert[before >> 16] = e0 + j, s.off[before >> 16] = before & 0xffff;
    if (e0 + j < E) count[e0 + j] = before & 0xffff;
    before += c[j] + ((c[j] > 0) << 16);
  }
  if (tid == 0) s.off[s.n] = all & 0xffff;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < PER_THREAD; ++j)  // the order within an expert does not matter: a pair's sums are its own column's
    if (id[j] >= 0) s.pair[count[id[j]] + rank[j]] = tid + j * THREADS;
  __syncthreads();
  return s;
}

// A step's units as this CTA and this warp take them.
struct Step {
  const uint8_t* base;
  int64_t expert_stride, slab;
  int slabs, u0, u1;       // units of an expert, this CTA's stretch
  int log_split, n_group;  // warps to a unit, units at once
  int tokens;
  __device__ __forceinline__ Step(const Q4ExpertArgs& a, int i, int n_expert, int chunks) {
    base = a.base[i], expert_stride = a.expert_stride[i], slab = a.slab[i], tokens = a.tokens[i];
    slabs = i ? a.columns[0] / ROWS : a.columns[1] / 8;
    const unsigned units = n_expert * slabs, grid = gridDim.x;  // 2^20 units at most: 32 bits hold their products with the grid
    u0 = blockIdx.x * units / grid, u1 = (blockIdx.x + 1) * units / grid;
    log_split = 31 - __clz(choose_split(WARPS, (units + grid - 1) / grid, chunks, WARPS));
    n_group = WARPS >> log_split;
  }
};

// The chunks this warp will need, ahead of the products: for each expert of the stretch, for each block of its pairs, this warp's units,
// its chunks of each; then the same of the second step.
template <class W>
struct Loader {
  const Sorted& sorted;
  const Step& second;
  int warp, lane;
  const Step* step;
  Share share, share2;
  int tail_blocks, tail_blocks2;
  int begin, end, blocks, u, left;  // the expert's stretch, its blocks left; this warp's unit, its chunks left
  const uint8_t *expert_base, *at;
  int stride, group;  // bytes from a chunk of this warp to its next; which of the CTA's units at once is this warp's

  __device__ __forceinline__ void start() {
    group = warp >> step->log_split;
    stride = W::BYTES << step->log_split;
    next_expert();
    find(begin);
  }
  __device__ __forceinline__ void next_expert() {
    begin = end;
    if (begin >= step->u1) {
      if (step == &second) return;
      step = &second;
      share = share2, tail_blocks = tail_blocks2;
      group = warp >> step->log_split;
      stride = W::BYTES << step->log_split;
      begin = end = second.u0;
      if (begin >= second.u1) return;
    }
    const int e = begin / step->slabs;
    end = min(step->u1, (e + 1) * step->slabs);
    blocks = (sorted.off[e + 1] - sorted.off[e] + step->tokens - 1) / step->tokens;
    expert_base = step->base + sorted.expert[e] * step->expert_stride - (int64_t)e * step->slabs * step->slab;
  }
  __device__ __forceinline__ void find(int from) {  // this warp's first unit with chunks of its own, of the CTA's from `from` on
    u = from + group;
    while ((u >= end || share.whole + share.tail == 0) && begin < step->u1) {
      if (--blocks == 0 || share.whole + share.tail == 0) next_expert();
      u = begin + group;
    }
    left = begin < step->u1 ? share.whole + share.tail : 0;
    if (left) at = expert_base + u * step->slab + (warp & ((1 << step->log_split) - 1)) * W::BYTES + lane * 16;
  }
  template <class R>
  __device__ __forceinline__ void next(R& ring, int) {
    if (left) {
      const uint32_t slot = ring.next_fill();
      if (left == 1 && share.tail) W::load_tail(slot, at, tail_blocks, lane);
      else W::load(slot, at, lane);
      at += stride;
      if (--left == 0) find(u - group + step->n_group);
    }
    copy_commit();
  }
};

// All CTAs of the grid meet; false when the others did not come within the limit.
__device__ __forceinline__ bool meet(unsigned* count, int* status) {
  __syncthreads();
  bool late = false;
  if (threadIdx.x == 0) {
    __threadfence();
    atomicAdd(count, 1u);
    const unsigned long long t0 = globaltimer();
    for (unsigned i = 1;; ++i) {
      unsigned n;
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(n) : "l"(count) : "memory");
      if (n >= gridDim.x) break;
      if ((i & 1023u) == 0 && globaltimer() - t0 > kWaitLimitNs) {
        set_status(status, ST_TIMEOUT);
        late = true;
        break;
      }
    }
    __threadfence();
  }
  return !__syncthreads_or(late);
}

struct Shared {  // the CTA's dynamic shared memory behind the rings
  float *part, *scale;
  char* rows;
};

// The units begin .. end - 1 of the sorted expert whose first unit is `first`, for np of its pairs from sorted position p0.
template <bool DOWN, int NT, class W, class R>
__device__ __forceinline__ void expert_block(const W& w, const Q4ExpertArgs& a, const Sorted& sorted, const Step& step, Loader<W>& loader,
                                             const Share& share, R& ring, const Shared& sh, int begin, int end, int first, int p0, int np) {
  const int warp = warp_index(), lane = threadIdx.x & 31, terms = a.terms[DOWN];
  const int S = 1 << step.log_split, group = warp >> step.log_split, member = warp & (S - 1);
  const int part_step = a.part_cols * PART_STRIDE;
  uint32_t b0[NT];
  uint2 cs0[NT];
  auto row_of = [&](int j) {  // of pair j of the block among those in shared memory
    j = min(j, np - 1);       // columns behind the last read some row; their sums are not used
    return !DOWN && a.resident ? sorted.pair[p0 + j] / a.k : j;
  };
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int c = 8 * t + (lane >> 2), j = terms == 2 ? c >> 1 : c;
    b0[t] = smem_u32(sh.rows) + (row_of(j) * terms + c - j * terms) * a.row_stride + (lane & 3) * 16 + member * 2 * W::COLUMNS;
    const int c2 = 8 * t + 2 * (lane & 3);
    cs0[t].x = smem_u32(sh.scale + row_of(terms == 2 ? c2 >> 1 : c2) * a.scale_stride + member);
    cs0[t].y = smem_u32(sh.scale + row_of(terms == 2 ? c2 >> 1 : c2 + 1) * a.scale_stride + member);
  }
  for (int base = begin; base < end; base += step.n_group) {
    const int u = base + group;
    float acc[NT][4] = {};
    if (u < end) {
      uint32_t b[NT];
      uint2 cs[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) b[t] = b0[t], cs[t] = cs0[t];
      run_chunks<NT>(w, ring, loader, share.whole, share.tail, S, b, cs, lane, acc);
    }
    store_part<NT>(sh.part + warp * part_step, lane, acc);
    group_sync<WARPS>(group, S);
    if (u < end) {
      const float* sums = sh.part + group * S * part_step;
      constexpr int OUT = DOWN ? ROWS : 8;
      const int row_len = a.columns[!DOWN];
      float* to = (DOWN ? a.parts : a.h) + (u - first) * OUT;
      for (int i = member * 32 + lane; i < np * OUT; i += S * 32) {
        const int j = i / OUT, row = i % OUT;
        float v = sum_part(sums, part_step, S, terms, j, row);
        if (!DOWN) v = silu_mul(v, sum_part(sums, part_step, S, terms, j, row + 8));
        to[(int64_t)sorted.pair[p0 + j] * row_len + row] = v;
      }
    }
    group_sync<WARPS>(group, S);
  }
}

// Step 1 or 2 for this CTA's stretch.
template <bool DOWN, int TILES, class W, class R>
__device__ __forceinline__ void run_step(const W& w, const Q4ExpertArgs& a, const Sorted& sorted, const Step& step, Loader<W>& loader,
                                         const Share& share, R& ring, const Shared& sh) {
  // the terms of n rows; source(j) is row j's number in x or h
  auto stage = [&](int n, auto source) {
    const int half = threadIdx.x >> 4, halves = n < 2 * WARPS ? 2 * WARPS / n : 1, rows_at_once = 2 * WARPS / halves;
    if (half < rows_at_once * halves)
      for (int j = half / halves; j < n; j += rows_at_once)
        stage_row<true>(DOWN ? a.h : a.x, (int64_t)source(j) * (DOWN ? a.columns[1] : a.x_stride), DOWN ? STRATA_F32 : a.x_type,
                        a.columns[DOWN], 0, a.columns[DOWN], a.terms[DOWN], sh.rows + j * a.terms[DOWN] * a.row_stride, a.row_stride,
                        sh.scale + j * a.scale_stride, half % halves, halves);
  };
  if (!DOWN && a.resident && step.u0 < step.u1) {
    stage(a.T, [](int j) { return j; });
    __syncthreads();
  }
  for (int begin = step.u0; begin < step.u1;) {
    const int e = begin / step.slabs, first = e * step.slabs, end = min(step.u1, first + step.slabs), last = sorted.off[e + 1];
    for (int p0 = sorted.off[e]; p0 < last; p0 += step.tokens) {
      const int np = min(step.tokens, last - p0), tiles = (np * a.terms[DOWN] + 7) / 8;
      if (DOWN || !a.resident) {
        __syncthreads();
        stage(np, [&](int j) { return DOWN ? sorted.pair[p0 + j] : sorted.pair[p0 + j] / a.k; });
        __syncthreads();
      }
      if (TILES == 1 || tiles == 1) expert_block<DOWN, 1>(w, a, sorted, step, loader, share, ring, sh, begin, end, first, p0, np);
      else if (tiles == 2) expert_block<DOWN, 2>(w, a, sorted, step, loader, share, ring, sh, begin, end, first, p0, np);
      else expert_block<DOWN, 3>(w, a, sorted, step, loader, share, ring, sh, begin, end, first, p0, np);
    }
    begin = end;
  }
}

// Four columns of a token; the parts of up to 8 slots are asked for at once.
__device__ __forceinline__ void combine4(const Q4ExpertArgs& a, int i) {
  const int fours = a.columns[0] / 4, t = i / fours, c = (i - t * fours) * 4;
  float sum[4] = {};
  for (int j0 = 0; j0 < a.k; j0 += 8) {
    float w[8];
    float4 v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int p = t * a.k + j0 + j;
      const int id = j0 + j < a.k ? a.ids[p] : -1;
      const float weight = j0 + j < a.k ? a.weights[p] : 0.f;
      w[j] = id >= 0 ? weight : 0.f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (w[j] != 0.f) v[j] = __ldcg(reinterpret_cast<const float4*>(a.parts + (int64_t)(t * a.k + j0 + j) * a.columns[0] + c));
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (w[j] != 0.f) {
        sum[0] = fmaf(w[j], v[j].x, sum[0]);
        sum[1] = fmaf(w[j], v[j].y, sum[1]);
        sum[2] = fmaf(w[j], v[j].z, sum[2]);
        sum[3] = fmaf(w[j], v[j].w, sum[3]);
      }
  }
  const int64_t at = t * a.out_stride + c;
  if (a.out_type == STRATA_F32)
    *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = make_float4(sum[0], sum[1], sum[2], sum[3]);
  else
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) =
        make_uint2(narrow2(sum[0], sum[1], a.out_type), narrow2(sum[2], sum[3], a.out_type));
}

// TILES: of the largest block.
template <class W, int TILES>
__global__ void __launch_bounds__(THREADS, 2) experts_kernel(Q4ExpertArgs a) {
  extern __shared__ __align__(128) char smem[];
  const int warp = warp_index(), lane = threadIdx.x & 31;
  Shared sh;
  sh.part = reinterpret_cast<float*>(smem + WARPS * DEPTH * W::SLOT);
  sh.scale = sh.part + WARPS * a.part_cols * PART_STRIDE;
  sh.rows = reinterpret_cast<char*>(sh.scale + a.staged * a.scale_stride);
  const Sorted sorted = sort_pairs(sh.rows + a.staged * a.row_stride, a.ids, a.weights, a.T * a.k, a.E);
  if (sorted.bad) {  // the same in every CTA
    if (blockIdx.x == 0 && threadIdx.x == 0) set_status(a.status, ST_CORRUPT);
    return;
  }
  const int chunks1 = (a.columns[0] + CHUNK - 1) / CHUNK, chunks2 = (a.columns[1] + CHUNK - 1) / CHUNK;
  const Step step1(a, 0, sorted.n, chunks1), step2(a, 1, sorted.n, chunks2);
  const Share share1(a.columns[0], CHUNK, chunks1, warp & ((1 << step1.log_split) - 1), 1 << step1.log_split);
  const Share share2(a.columns[1], CHUNK, chunks2, warp & ((1 << step2.log_split) - 1), 1 << step2.log_split);
  Ring<DEPTH, W::SLOT> ring(smem_u32(smem) + warp * (DEPTH * W::SLOT));
  Loader<W> loader{sorted, step2, warp, lane, &step1, share1, share2, a.columns[0] % CHUNK / BLOCK, a.columns[1] % CHUNK / BLOCK,
                   step1.u0, step1.u0, 0, 0, 0, nullptr, nullptr};
  loader.start();
  for (int i = 0; i < DEPTH - 1; ++i) loader.next(ring, lane);

  W w1{nullptr, 0, a.columns[0]}, w2{nullptr, 0, a.columns[1]};
  run_step<false, TILES>(w1, a, sorted, step1, loader, share1, ring, sh);
  if (!meet(a.meet, a.status)) return;
  run_step<true, TILES>(w2, a, sorted, step2, loader, share2, ring, sh);
  copy_wait<0>();
  if (!meet(a.meet + 1, a.status)) return;
  for (int j = threadIdx.x;; j += THREADS) {  // 128 bytes of a row after the other to the CTAs
    const int i = ((j >> 3) * gridDim.x + blockIdx.x) * 8 + (j & 7);
    if (i >= a.T * (a.columns[0] / 4)) break;
    combine4(a, i);
  }
  if (threadIdx.x == 0 && atomicAdd(a.meet + 2, 1u) == gridDim.x - 1) {  // the last one out: nobody looks at them any more
    a.meet[0] = 0, a.meet[1] = 0;
    __threadfence();
    a.meet[2] = 0;
  }
}

template <class W, int TILES>
cudaError_t launch(Q4ExpertArgs a, cudaStream_t s) {
  int sms = 0;
  cudaError_t err = sm_count(&sms);
  if (err != cudaSuccess) return err;
  const int pairs = a.T * a.k, wide = a.columns[0] > a.columns[1] ? a.columns[0] : a.columns[1];
  a.row_stride = row_bytes(wide);
  a.scale_stride = ((wide + CHUNK - 1) / CHUNK + 3) / 4 * 4;
  // Two CTAs an SM if whole blocks fit, else one.
  auto plan = [&](size_t room) {
    for (int cols = 8 * TILES; cols >= 2; cols = cols > 8 ? cols - 8 : cols / 2) {
      a.part_cols = (cols + 7) / 8 * 8;
      for (int i = 0; i < 2; ++i) a.tokens[i] = cols / a.terms[i] < pairs ? cols / a.terms[i] : pairs;
      a.staged = cols;  // rows of terms
      const size_t bytes = (size_t)WARPS * DEPTH * W::SLOT + sizeof(float) * (WARPS * a.part_cols * PART_STRIDE + a.staged * a.scale_stride) +
                           (size_t)a.staged * a.row_stride + sorted_bytes(a.E, pairs);
      if (bytes <= room) return bytes;
    }
    return (size_t)0;
  };
  // All of one or two tokens from the start: the experts of a stretch read the same rows.
  int per_sm = 2;
  size_t smem = plan(SMEM_HALF);
  if (smem == 0 || a.staged < 8 * TILES) per_sm = 1, smem = plan(SMEM_MAX);
  a.resident = a.T <= 2 && a.T * a.terms[0] <= a.staged;
  err = allow_smem<experts_kernel<W, TILES>>(SMEM_MAX);
  if (err != cudaSuccess) return err;
  void* args[] = {&a};
  STRATA_LAUNCH(KID_Q4_EXPERTS, s,
                err = cudaLaunchCooperativeKernel((const void*)experts_kernel<W, TILES>, dim3(sms * per_sm), dim3(THREADS), args, smem, s));
  return err;
}

// The kernel of one format: blocks of a single tile where an expert has no more pairs than that on average, with fewer registers and
// half the sums' room; else of up to three tiles, with fewer passes over the weights.
template <int GROUP>
cudaError_t launch_group(const strata_q4_experts_t& ex, const Q4ExpertArgs& a, cudaStream_t s) {
  const strata_q4_t& q = ex.gate_up_q4;
  const int terms = a.terms[0] > a.terms[1] ? a.terms[0] : a.terms[1];
  const bool one = (int64_t)a.T * a.k * terms <= 8 * (int64_t)a.E || a.T * terms <= 8;
  const bool f16 = q.scale_type == STRATA_F16;
  if (one) {
    if (q.zeros) return f16 ? launch<Q4<GROUP, true, true>, 1>(a, s) : launch<Q4<GROUP, true, false>, 1>(a, s);
    return f16 ? launch<Q4<GROUP, false, true>, 1>(a, s) : launch<Q4<GROUP, false, false>, 1>(a, s);
  }
  if (q.zeros) return f16 ? launch<Q4<GROUP, true, true>, TILES_MAX>(a, s) : launch<Q4<GROUP, true, false>, TILES_MAX>(a, s);
  return f16 ? launch<Q4<GROUP, false, true>, TILES_MAX>(a, s) : launch<Q4<GROUP, false, false>, TILES_MAX>(a, s);
}

}  // namespace q4x

// One file for each group size.
cudaError_t launch_q4_experts_32(const strata_q4_experts_t& ex, const Q4ExpertArgs& a, cudaStream_t s);
cudaError_t launch_q4_experts_64(const strata_q4_experts_t& ex, const Q4ExpertArgs& a, cudaStream_t s);
cudaError_t launch_q4_experts_128(const strata_q4_experts_t& ex, const Q4ExpertArgs& a, cudaStream_t s);

}  // namespace strata
