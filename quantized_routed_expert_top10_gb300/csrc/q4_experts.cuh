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
//
// The stretches are equal in units, and a unit is passed over once for each block of its expert's pairs: an expert of many pairs keeps its few CTAs while the
// others wait at the meeting (64 tokens of 512 experts, by events after a flush of L2: 236 us with even lists, 656 with a hottest expert of 54 tokens and 235 in
// use, 980 to 1,016 with one more expert that all list; fp32 335 and 1,289).
//
// What bounds it: 64 tokens of 512 experts (1.03 GB in 209 us, 4.9 TB/s of 6.8) no pipe alone, see q4_core.cuh (issue in 57% of the cycles; a fifth of the
// warps' time at barriers, for windows, meetings and the stretch that holds an expert of two blocks); one token (26 MB in 22 us, 3.9 at the copy rate)
// a chain of latencies: launch 4 us, sort 1, first chunks 2, step 1 5, meeting 2, h 1.3, step 2 2.5, meeting 2, step 3 2.
// Three kernels with programmatic launches instead of the meetings took 30 us for one token.
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
  int slabs[2];            // units of an expert
  uint32_t slabs_inverse[2], grid_inverse, k_inverse;  // ceil(2^32 / n)
  int block[2];            // pairs whose columns one unit takes at once
  int rows[2];             // rows of x or h in shared memory at once
  int resident;            // step 1: the rows are all tokens', there from the start
  int staged[2];           // rows of terms
  int row_stride[2], scale_stride[2], part_cols[2];
  int sorted_at;           // bytes before the sorted pairs: rings, then a step's sums, scales and rows of terms
};

namespace q4x {

using namespace q4;

constexpr int WARPS = 8, THREADS = 32 * WARPS;  // two CTAs an SM, one of which computes while the other lays out x or joins sums
// chunks of a warp's ring: as many as leave room for 8 rows of 2,560 columns' terms (24 where blocks are larger, one CTA an SM)
constexpr int depth_of(int tiles, int slabs) { return slabs == 2 ? 3 : tiles == 1 ? 7 : 5; }
constexpr int PAIRS_MAX = STRATA_Q4_EXPERTS_T_MAX * STRATA_Q4_EXPERTS_K_MAX;
constexpr int SOME = 128, SOME_THREADS = 64;  // pairs that two warps sort while the others lay out x
static_assert(PAIRS_MAX < 65536 && PAIRS_MAX % THREADS == 0 && STRATA_Q4_EXPERTS_E_MAX % THREADS == 0, "sorting of the pairs");

// The pairs by expert: expert[a], its pairs pair[off[a]] .. pair[off[a + 1] - 1], a < n.
struct Sorted {
  int* count;  // of expert e, then the first of its pairs
  uint16_t *expert, *off, *pair;
};
__host__ __device__ constexpr int sorted_bytes(int E, int pairs) { return (4 * E + 2 * E + 2 * (E + 1) + 2 * pairs + 15) / 16 * 16; }

__device__ __forceinline__ Sorted sorted_at(char* smem, int E) {
  Sorted s;
  s.count = reinterpret_cast<int*>(smem);
  s.expert = reinterpret_cast<uint16_t*>(s.count + E);
  s.off = s.expert + E;
  s.pair = s.off + E + 1;
  return s;
}
// Up to 32 pairs, by one warp, a pair a lane; an expert's first pair stands for it.
__device__ __forceinline__ void sort_few(const Sorted& s, int2* found, const int32_t* ids, const float* weights, int pairs, int E) {
  const int lane = threadIdx.x & 31;
  const int e = lane < pairs ? ids[lane] : -1;
  const float weight = lane < pairs ? weights[lane] : 0.f;
  const bool have = e >= 0 && e < E && weight != 0.f;
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
  const int bad = __any_sync(0xffffffffu, lane < pairs && (e < -1 || e >= E));
  const int all = __popc(__ballot_sync(0xffffffffu, have));
  if (lane == 0) {
    s.off[__popc(firsts)] = all;
    *found = make_int2(__popc(firsts), bad);
  }
}
// Up to 128 pairs, by the CTA's first 64 threads: each looks through all pairs for its own expert, then for the experts that come before it (in the
// order in which their first pairs come).
static __device__ __noinline__ void sort_some(const Sorted& s, int2* found, int* scratch, const int32_t* ids, const float* weights, int pairs,
                                              int E) {
  constexpr int NONE = 1000;
  int *key = scratch, *lead = scratch + SOME;  // expert; its first pair
  const int tid = threadIdx.x;
  bool bad = false;
  for (int p = tid; p < SOME; p += SOME_THREADS) {
    const int e = p < pairs ? ids[p] : -1;
    const float weight = p < pairs ? weights[p] : 0.f;
    bad |= e < -1 || e >= E;
    key[p] = e >= 0 && e < E && weight != 0.f ? e : -1;
  }
  named_barrier(15, SOME_THREADS);
  if (__any_sync(0xffffffffu, bad) && (tid & 31) == 0) found->y = 1;  // 0 before the barrier
  int first[SOME / SOME_THREADS], rank[SOME / SOME_THREADS];
#pragma unroll
  for (int i = 0; i < SOME / SOME_THREADS; ++i) {
    const int p = tid + i * SOME_THREADS;
    first[i] = NONE, rank[i] = 0;
    if (i * SOME_THREADS >= pairs) break;
    const int mine = key[p];
    for (int q0 = 0; q0 < pairs; q0 += 4) {  // behind the last pair keys are -1
      const int4 k = *reinterpret_cast<const int4*>(key + q0);
      const int v[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (v[j] == mine && q0 + j <= p) {
          first[i] = min(first[i], q0 + j);
          rank[i] += q0 + j < p;
        }
    }
    if (mine < 0) first[i] = NONE;
  }
#pragma unroll
  for (int i = 0; i < SOME / SOME_THREADS; ++i) lead[tid + i * SOME_THREADS] = first[i];
  named_barrier(15, SOME_THREADS);
#pragma unroll
  for (int i = 0; i < SOME / SOME_THREADS; ++i) {
    const int p = tid + i * SOME_THREADS;
    if (i * SOME_THREADS >= pairs) break;
    int before = 0, experts = 0, all = 0, used = 0;
    for (int q0 = 0; q0 < pairs; q0 += 4) {
      const int4 k = *reinterpret_cast<const int4*>(lead + q0);
      const int v[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        before += v[j] < first[i];
        experts += v[j] == q0 + j && v[j] < first[i];
        all += v[j] != NONE;
        used += v[j] == q0 + j;
      }
    }
    if (first[i] != NONE) {
      s.pair[before + rank[i]] = p;
      if (first[i] == p) s.expert[experts] = key[p], s.off[experts] = before;
    }
    if (p == 0) s.off[used] = all, found->x = used;
  }
}
// Any number, by the whole CTA: counted, summed over all experts, dealt out.
static __device__ __noinline__ void sort_many(const Sorted& s, int2* found, const int32_t* ids, const float* weights, int pairs, int E) {
  __shared__ int warp_sum[WARPS];
  constexpr int N = THREADS, PER = PAIRS_MAX / N, E_PER = STRATA_Q4_EXPERTS_E_MAX / N;
  const int tid = threadIdx.x, lane = tid & 31, warp = warp_index();
  int id[PER], rank[PER];
  float weight[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int p = tid + j * N;
    id[j] = p < pairs ? ids[p] : -1;
    weight[j] = p < pairs ? weights[p] : 0.f;
  }
  for (int e = tid; e < E; e += N) s.count[e] = 0;
  __syncthreads();
  bool bad = false;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    bad |= id[j] < -1 || id[j] >= E;
    if (id[j] < 0 || id[j] >= E || weight[j] == 0.f) id[j] = -1;
    else rank[j] = atomicAdd(&s.count[id[j]], 1);
  }
  if (__any_sync(0xffffffffu, bad) && lane == 0) found->y = 1;  // 0 before
  __syncthreads();
  // sums before each expert of the pairs (low half) and of the experts in use (high half); consecutive experts a thread
  const int e0 = E_PER * tid;
  int c[E_PER], mine = 0;
#pragma unroll
  for (int j = 0; j < E_PER; ++j) {
    c[j] = e0 + j < E ? s.count[e0 + j] : 0;
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
#pragma unroll
  for (int j = 0; j < E_PER; ++j) {
    if (c[j]) s.expert[before >> 16] = e0 + j, s.off[before >> 16] = before & 0xffff;
    if (e0 + j < E) s.count[e0 + j] = before & 0xffff;
    before += c[j] + ((c[j] > 0) << 16);
  }
  if (tid == 0) {
    s.off[all >> 16] = all & 0xffff;
    found->x = all >> 16;
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < PER; ++j)  // the order within an expert does not matter: a pair's sums are its own column's
    if (id[j] >= 0) s.pair[s.count[id[j]] + rank[j]] = tid + j * N;
}

// A step's units as this CTA and this warp take them: of at most 2^20 (1,024 experts of 1,024) an equal contiguous stretch a CTA.
struct Step {
  const uint8_t* base;
  int64_t expert_stride, slab;
  int slabs, u0, u1;       // units of an expert, this CTA's stretch
  uint32_t slabs_inverse;
  int log_split, n_group;  // warps to a unit, units at once
  int block, rows;         // pairs a unit takes at once, rows in shared memory (any number where all tokens are there)
  __device__ __forceinline__ void set(const Q4ExpertArgs& a, int i, int n_expert) {
    base = a.base[i], expert_stride = a.expert_stride[i], slab = a.slab[i];
    slabs = a.slabs[i], slabs_inverse = a.slabs_inverse[i];
    block = a.block[i], rows = i == 0 && a.resident ? 1 << 30 : a.rows[i];
    const int units = n_expert * slabs, each = divide(units, a.grid_inverse), more = units - each * gridDim.x;
    u0 = each * blockIdx.x + min((int)blockIdx.x, more);
    u1 = u0 + each + ((int)blockIdx.x < more);
    log_split = 31 - __clz(choose_split(WARPS, each + (more > 0), (a.columns[i] + CHUNK - 1) / CHUNK, WARPS));
    n_group = WARPS >> log_split;
  }
};

// What is taken at once: units begin .. end - 1 for the sorted pairs p0 .. p1 - 1.  As many experts of the stretch as have room for their rows, or
// one expert for a block of its pairs after the other.
struct Window {
  int begin, end, p0, p1, last;  // last: of an expert taken in blocks
  __device__ __forceinline__ explicit Window(int u0) : begin(u0), end(u0), p0(0), p1(0), last(0) {}
  __device__ __forceinline__ bool next(const Step& step, const Sorted& sorted) {
    if (p1 < last) {
      p0 = p1, p1 = min(p0 + step.block, last);
      return true;
    }
    begin = end;
    if (begin >= step.u1) return false;
    int e = divide(begin, step.slabs_inverse);
    p0 = sorted.off[e], p1 = last = sorted.off[++e];
    if (p1 - p0 > step.block) {
      p1 = p0 + step.block;
    } else {
      for (; e * step.slabs < step.u1; ++e) {
        const int p2 = sorted.off[e + 1];
        if (p2 - p1 > step.block || p2 - p0 > step.rows) break;
        p1 = last = p2;
      }
    }
    end = min(step.u1, e * step.slabs);
    return true;
  }
};

// This warp's units, window after window, of the first step and then of the second.
template <class W>
struct Units {
  const Sorted& sorted;
  const Step *step, *second;
  int warp, lane;
  Share share, share2;
  Window window;
  int u, group, member;
  int whole, tail, stride;
  typename W::Cursor cursor;

  __device__ __forceinline__ Units(const Sorted& s, const Step& s1, const Step& s2, int w, int l, const Share& h1, const Share& h2)
      : sorted(s), step(&s1), second(&s2), warp(w), lane(l), share(h1), share2(h2), window(0) {
    enter();
  }
  __device__ __forceinline__ void enter() {
    group = warp >> step->log_split, member = warp & ((1 << step->log_split) - 1);
    whole = share.whole, tail = share.tail, stride = W::BYTES << step->log_split;
    window = Window(step->u0);
    u = step->u0;  // behind the empty window's end
  }
  __device__ __forceinline__ bool next() {
    while (u >= window.end || (whole == 0 && tail == 0)) {
      if ((whole == 0 && tail == 0) || !window.next(*step, sorted)) {
        if (step == second) return false;
        step = second, share = share2;
        enter();
      } else {
        u = window.begin + group;
      }
    }
    const int e = divide(u, step->slabs_inverse);
    cursor.at = step->base + sorted.expert[e] * step->expert_stride + (u - e * step->slabs) * (W::SLABS * step->slab) + member * W::BYTES + lane * 16;
    cursor.second = step->slab;
    u += step->n_group;
    return true;
  }
};
template <class W, int DEPTH>
using ExpertFeed = Feed<W, DEPTH, Units<W>>;

// `ctas` CTAs meet.  False (and ST_TIMEOUT) when the others did not come within the limit (the experts' kernel uses the library's; the wait self-test
// passes a short one): the kernel then returns, so copies still on their way to shared memory are waited for.
__device__ __forceinline__ bool meet(unsigned* count, unsigned ctas, int* status, unsigned long long limit_ns = kWaitLimitNs) {
  __syncthreads();
  bool late = false;
  if (threadIdx.x == 0) {
    __threadfence();
    atomicAdd(count, 1u);
    const unsigned long long t0 = globaltimer();
    for (unsigned i = 1;; ++i) {
      unsigned n;
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(n) : "l"(count) : "memory");
      if (n >= ctas) break;
      if ((i & 1023u) == 0 && globaltimer() - t0 > limit_ns) {
        set_status(status, ST_TIMEOUT);
        late = true;
        break;
      }
    }
    __threadfence();
  }
  if (!__syncthreads_or(late)) return true;
  copy_wait<0>();
  return false;
}

struct Shared {  // the CTA's dynamic shared memory behind the rings, in step 1 or 2
  float *part, *scale;
  char* rows;
  __device__ __forceinline__ Shared(const Q4ExpertArgs& a, char* behind, bool down, int slabs)
      : part(reinterpret_cast<float*>(behind)),
        scale(part + WARPS * a.part_cols[down] * part_stride(slabs)),
        rows(reinterpret_cast<char*>(scale + a.staged[down] * a.scale_stride[down])) {}
};

// Sums of unit u of the expert whose pairs in the window are lo .. lo + np - 1.
template <int NT, class W, class F>
__device__ __forceinline__ void unit_products(const Q4ExpertArgs& a, const Sorted& sorted, F& feed, const Share& share, const Shared& sh, bool down,
                                              int S, int member, int p0, int lo, int np) {
  const int warp = warp_index(), lane = feed.lane, shift = a.terms[down] - 1;  // one or two terms
  const int row_stride = a.row_stride[down], scale_stride = a.scale_stride[down];
  uint32_t b[NT];
  uint2 cs[NT];
  auto row_of = [&](int j) {  // of pair lo + j among those in shared memory
    j = min(j, np - 1);       // columns behind the last read some row; their sums are not used
    return !down && a.resident ? divide(sorted.pair[lo + j], a.k_inverse) : lo + j - p0;
  };
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int c = 8 * t + (lane >> 2), c2 = 8 * t + 2 * (lane & 3);
    b[t] = smem_u32(sh.rows) + ((row_of(c >> shift) << shift) + (c & shift)) * row_stride + (lane & 3) * 16 + member * 2 * W::COLUMNS;
    cs[t].x = smem_u32(sh.scale + row_of(c2 >> shift) * scale_stride + member);
    cs[t].y = smem_u32(sh.scale + row_of((c2 + 1) >> shift) * scale_stride + member);
  }
  float acc[W::SLABS * NT][4] = {};
  run_chunks<NT, W>(feed, share.whole, share.tail, S, b, cs, acc);
  store_part<NT, W::SLABS>(sh.part + warp * (a.part_cols[down] * part_stride(W::SLABS)), lane, acc);
}

// The terms of n rows of x or h by `halves` half warps, this one `half`: of all tokens, or of the sorted pairs from `pair` on.
__device__ __forceinline__ void stage(const Q4ExpertArgs& a, const Shared& sh, bool down, const uint16_t* pair, int n, int half, int halves) {
  const StageArgs to{down ? a.h : a.x, down ? a.columns[1] : a.x_stride, down ? STRATA_F32 : a.x_type, a.columns[down], a.terms[down],
                     sh.rows, a.row_stride[down], sh.scale, a.scale_stride[down], pair, down ? 0u : a.k_inverse, 0};
  stage_rows<true>(to, n, 0, a.columns[down], half, halves);
}

// Step 1 or 2 for this CTA's stretch: one code for both, so that the second finds its instructions at hand.
template <int TILES, class W, class F>
__device__ __forceinline__ void run_step(const Q4ExpertArgs& a, const Sorted& sorted, const Step& step, F& feed, const Share& share,
                                         const Shared& sh, bool down) {
  const int warp = warp_index(), lane = threadIdx.x & 31, terms = a.terms[down];
  const int S = 1 << step.log_split, group = warp >> step.log_split, member = warp & (S - 1);
  const int part_step = a.part_cols[down] * part_stride(W::SLABS);
  for (Window win(step.u0); win.next(step, sorted);) {
    if (down || !a.resident) {
      __syncthreads();
      stage(a, sh, down, sorted.pair + win.p0, win.p1 - win.p0, threadIdx.x >> 4, 2 * WARPS);
      __syncthreads();
    }
    for (int base = win.begin; base < win.end; base += step.n_group) {
      const int u = base + group;
      int e = 0, lo = 0, np = 0;
      if (u < win.end) {
        e = divide(u, step.slabs_inverse);
        lo = max((int)sorted.off[e], win.p0), np = min((int)sorted.off[e + 1], win.p1) - lo;
        const int tiles = (np * terms + 7) / 8;
        if (TILES == 1 || tiles == 1) unit_products<1, W>(a, sorted, feed, share, sh, down, S, member, win.p0, lo, np);
        else if (TILES == 2 || tiles == 2) unit_products<2, W>(a, sorted, feed, share, sh, down, S, member, win.p0, lo, np);
        else unit_products<TILES < 3 ? 1 : 3, W>(a, sorted, feed, share, sh, down, S, member, win.p0, lo, np);
      }
      group_sync<WARPS>(group, S);
      const int out = (down ? 4 : 3) + (W::SLABS == 2);  // 16 or 8 rows a slab
      const float* sums = sh.part + group * S * part_step;
      const int row_len = a.columns[!down];
      float* to = (down ? a.parts : a.h) + ((u - e * step.slabs) << out);
      for (int i = member * 32 + lane; i < np << out; i += S * 32) {
        const int j = i >> out, row = i & ((1 << out) - 1), at = down ? row : row + (row & 8);  // a slab's 8 rows of gate, then its 8 of up
        float v = sum_part<W::SLABS>(sums, part_step, S, terms, j, at);
        if (!down) v = silu_mul(v, sum_part<W::SLABS>(sums, part_step, S, terms, j, at + 8));
        to[(int64_t)sorted.pair[lo + j] * row_len + row] = v;
      }
      group_sync<WARPS>(group, S);
    }
  }
}

// Step 3: four columns of a token, its first 16 weights asked for before the parts are there.
constexpr int WEIGHTS = 16;
__device__ __forceinline__ void slot_weights(const Q4ExpertArgs& a, int t, int j0, float (&w)[WEIGHTS]) {
#pragma unroll
  for (int j = 0; j < WEIGHTS; ++j) {
    const int p = t * a.k + j0 + j;
    const int id = j0 + j < a.k ? a.ids[p] : -1;
    const float weight = j0 + j < a.k ? a.weights[p] : 0.f;
    w[j] = id >= 0 ? weight : 0.f;
  }
}
__device__ __forceinline__ void combine4(const Q4ExpertArgs& a, int t, int c, float (&w)[WEIGHTS]) {
  float sum[4] = {};
  for (int j0 = 0;;) {
    const float* parts = a.parts + (int64_t)(t * a.k + j0) * a.columns[0] + c;
    float4 v[WEIGHTS];
#pragma unroll
    for (int j = 0; j < WEIGHTS; ++j)
      if (w[j] != 0.f) v[j] = __ldcg(reinterpret_cast<const float4*>(parts + (int64_t)j * a.columns[0]));
#pragma unroll
    for (int j = 0; j < WEIGHTS; ++j)
      if (w[j] != 0.f) {
        sum[0] = fmaf(w[j], v[j].x, sum[0]);
        sum[1] = fmaf(w[j], v[j].y, sum[1]);
        sum[2] = fmaf(w[j], v[j].z, sum[2]);
        sum[3] = fmaf(w[j], v[j].w, sum[3]);
      }
    if ((j0 += WEIGHTS) >= a.k) break;
    slot_weights(a, t, j0, w);
  }
  const int64_t at = t * a.out_stride + c;
  if (a.out_type == STRATA_F32)
    *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = make_float4(sum[0], sum[1], sum[2], sum[3]);
  else
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) =
        make_uint2(narrow2(sum[0], sum[1], a.out_type), narrow2(sum[2], sum[3], a.out_type));
}

// TILES, TILES2: of the largest block of step 1 and of step 2.
template <class W, int TILES, int TILES2>
__global__ void __launch_bounds__(THREADS, 2) experts_kernel(Q4ExpertArgs a) {
  extern __shared__ __align__(128) char smem[];
  __shared__ int2 found;  // experts in use; an id outside [-1, E)
  __shared__ Step steps[2];
  constexpr int DEPTH = depth_of(TILES, W::SLABS);
  const int warp = warp_index(), lane = threadIdx.x & 31, pairs = a.T * a.k;
  const Shared sh(a, smem + WARPS * DEPTH * W::SLOT, false, W::SLABS), sh2(a, smem + WARPS * DEPTH * W::SLOT, true, W::SLABS);
  const Sorted sorted = sorted_at(smem + a.sorted_at, a.E);
  if (pairs <= 32) {
    if (warp == 0) {
      sort_few(sorted, &found, a.ids, a.weights, pairs, a.E);
      __syncwarp();
      if (lane < 2) steps[lane].set(a, lane, found.x);
    } else if (a.resident) {
      stage(a, sh, false, nullptr, a.T, (threadIdx.x >> 4) - 2, 2 * WARPS - 2);
    }
  } else {
    if (threadIdx.x == 0) found.y = 0;
    if (pairs <= SOME) {
      if (warp < SOME_THREADS / 32) {
        // (the units' sums are not in use yet)
        sort_some(sorted, &found, reinterpret_cast<int*>(sh.part), a.ids, a.weights, pairs, a.E);
        __syncwarp();
        if (threadIdx.x < 2) steps[threadIdx.x].set(a, threadIdx.x, found.x);
      } else if (a.resident) {
        stage(a, sh, false, nullptr, a.T, (threadIdx.x >> 4) - SOME_THREADS / 16, 2 * WARPS - SOME_THREADS / 16);
      }
    } else {
      sort_many(sorted, &found, a.ids, a.weights, pairs, a.E);
      if (threadIdx.x < 2) steps[threadIdx.x].set(a, threadIdx.x, found.x);
      if (a.resident) stage(a, sh, false, nullptr, a.T, threadIdx.x >> 4, 2 * WARPS);
    }
  }
  __syncthreads();
  if (found.y) {  // the same in every CTA
    if (blockIdx.x == 0 && threadIdx.x == 0) set_status(a.status, ST_CORRUPT);
    return;
  }
  const Step &step1 = steps[0], &step2 = steps[1];
  const Share share1(a.columns[0], CHUNK, warp & ((1 << step1.log_split) - 1), step1.log_split);
  const Share share2(a.columns[1], CHUNK, warp & ((1 << step2.log_split) - 1), step2.log_split);
  ExpertFeed<W, DEPTH> feed(Units<W>(sorted, step1, step2, warp, lane, share1, share2), smem_u32(smem) + warp * (DEPTH * W::SLOT), lane);

  run_step<TILES, W>(a, sorted, step1, feed, share1, sh, false);
  if (!meet(a.meet, gridDim.x, a.status)) return;
  run_step<TILES2, W>(a, sorted, step2, feed, share2, sh2, true);
  copy_wait<0>();
  const int fours = a.columns[0] / 4, items = a.T * fours;
  auto item_of = [&](int j) { return ((j >> 3) * gridDim.x + blockIdx.x) * 8 + (j & 7); };  // 128 bytes of fp32 after the other to the CTAs
  float weights[WEIGHTS];
  int item = item_of(threadIdx.x);
  if (item < items) slot_weights(a, item / fours, 0, weights);
  if (!meet(a.meet + 1, gridDim.x, a.status)) return;
  for (int j = threadIdx.x; item < items;) {
    combine4(a, item / fours, item % fours * 4, weights);
    item = item_of(j += THREADS);
    if (item < items) slot_weights(a, item / fours, 0, weights);
  }
  if (threadIdx.x == 0 && atomicAdd(a.meet + 2, 1u) == gridDim.x - 1) {  // the last one out: nobody looks at them any more
    a.meet[0] = 0, a.meet[1] = 0;
    __threadfence();
    a.meet[2] = 0;
  }
}

template <class W, int TILES, int TILES2>
cudaError_t launch(Q4ExpertArgs a, cudaStream_t s) {
  int sms = 0;
  cudaError_t err = sm_count(&sms);
  if (err != cudaSuccess) return err;
  constexpr int tiles[2] = {TILES, TILES2};
  constexpr size_t rings = (size_t)WARPS * depth_of(TILES, W::SLABS) * W::SLOT;
  const size_t sorted = sorted_bytes(a.E, a.T * a.k);
  size_t sums[2], row[2];  // bytes of the units' sums; of a row of terms and its scales
  for (int i = 0; i < 2; ++i) {
    a.row_stride[i] = row_bytes(a.columns[i]);
    a.scale_stride[i] = ((a.columns[i] + CHUNK - 1) / CHUNK + 3) / 4 * 4;
    a.part_cols[i] = 8 * tiles[i];
    sums[i] = sizeof(float) * WARPS * a.part_cols[i] * part_stride(W::SLABS);
    row[i] = a.row_stride[i] + sizeof(float) * a.scale_stride[i];
  }
  // two CTAs an SM where their rows of terms are half of a block's or more in both steps, else one
  int per_sm = 2;
  auto fit = [&](size_t room) {
    bool half = true;
    for (int i = 0; i < 2; ++i) {
      const size_t taken = rings + sums[i] + sorted, rows = room > taken ? (room - taken) / row[i] : 0;
      a.staged[i] = rows < 8u * tiles[i] ? (int)rows : 8 * tiles[i];
      half = half && a.staged[i] >= 4 * tiles[i];
    }
    return half;
  };
  if (!fit(SMEM_HALF)) per_sm = 1, fit(SMEM_MAX);
  for (int i = 0; i < 2; ++i) a.block[i] = a.rows[i] = a.staged[i] / a.terms[i];
  a.resident = a.T * a.terms[0] <= a.staged[0];
  if (a.resident) a.block[0] = 8 * TILES / a.terms[0];
  const size_t step1 = sums[0] + a.staged[0] * row[0], step2 = sums[1] + a.staged[1] * row[1];  // one after the other in the same place
  a.sorted_at = (int)(rings + (step1 > step2 ? step1 : step2));
  a.slabs[0] = a.columns[1] / (8 * W::SLABS), a.slabs[1] = a.columns[0] / (ROWS * W::SLABS);  // d_ff and d_model are multiples of 32
  for (int i = 0; i < 2; ++i) a.slabs_inverse[i] = inverse_of(a.slabs[i]);
  a.grid_inverse = inverse_of(sms * per_sm), a.k_inverse = inverse_of(a.k);
  err = allow_smem<experts_kernel<W, TILES, TILES2>>(SMEM_MAX);
  if (err != cudaSuccess) return err;
  void* args[] = {&a};
  STRATA_LAUNCH(KID_Q4_EXPERTS, s,
                err = cudaLaunchCooperativeKernel((const void*)experts_kernel<W, TILES, TILES2>, dim3(sms * per_sm), dim3(THREADS), args,
                                                  a.sorted_at + sorted, s));
  return err;
}

// The kernel of one format.  Blocks of a single tile of 8 columns in step 1 (two in step 2, where a pair has two), with a deeper ring, where an expert
// has two columns or fewer on average over both steps or where one block can hold all; else of up to three tiles.  An expert with more columns than a
// block is passed over again: 64 tokens, 10 of 512 experts and one more that all list, bf16 (2.1 columns on average) 1,043 us in single tiles, 980 in up
// to three; 16 tokens, 6 of 64, fp16 (2.25) 60 us either way.  Single tiles in units of 32 rows where a CTA will have 8 or more of them in step 1, of 16
// where that would leave warps without work: 64 tokens, 10 of 512 experts (75 units of 16 a CTA) 234 us in units of 16, 209 in units of 32.
template <int GROUP, bool ZEROS, bool SCALE_F16>
cudaError_t launch_format(const Q4ExpertArgs& a, cudaStream_t s) {
  int sms = 0;
  cudaError_t err = sm_count(&sms);
  if (err != cudaSuccess) return err;
  const bool one_block = a.T * a.terms[0] <= 8 && a.T * a.terms[1] <= 16;
  const int64_t pairs = a.T * a.k, used = pairs * a.E / (pairs + a.E);  // experts in use, about
  if (!one_block && pairs * (a.terms[0] + a.terms[1]) > 4 * a.E) return launch<Q4<GROUP, ZEROS, SCALE_F16>, TILES_MAX, TILES_MAX>(a, s);
  if (used * (a.columns[1] / 8) >= 16 * 2 * sms) return launch<Q4<GROUP, ZEROS, SCALE_F16, 2>, 1, 2>(a, s);
  return launch<Q4<GROUP, ZEROS, SCALE_F16>, 1, 2>(a, s);
}
template <int GROUP>
cudaError_t launch_group(const strata_q4_experts_t& ex, const Q4ExpertArgs& a, cudaStream_t s) {
  const bool f16 = ex.gate_up_q4.scale_type == STRATA_F16;
  if (ex.gate_up_q4.zeros) return f16 ? launch_format<GROUP, true, true>(a, s) : launch_format<GROUP, true, false>(a, s);
  return f16 ? launch_format<GROUP, false, true>(a, s) : launch_format<GROUP, false, false>(a, s);
}

}  // namespace q4x

// One file for each group size.
cudaError_t launch_q4_experts_32(const strata_q4_experts_t& ex, const Q4ExpertArgs& a, cudaStream_t s);
cudaError_t launch_q4_experts_64(const strata_q4_experts_t& ex, const Q4ExpertArgs& a, cudaStream_t s);
cudaError_t launch_q4_experts_128(const strata_q4_experts_t& ex, const Q4ExpertArgs& a, cudaStream_t s);

}  // namespace strata
