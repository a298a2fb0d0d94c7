// Sizes of strata_moe_linear's and strata_moe_q4_experts' tiles, and what a launch of strata_moe_linear lays out in shared memory.  Plain C++
// without CUDA, so that a test can walk it for any size without a GPU.
#pragma once
#include <cstddef>
#include <cstdint>

namespace strata {
namespace q4 {

constexpr int ROWS = 16, CHUNK = 128, BLOCK = 32;
constexpr int SMEM_MAX = 227 * 1024 - 256;   // dynamic; the rest holds the kernels' static words
constexpr int SMEM_HALF = 113 * 1024 - 256;  // of each of two CTAs an SM
constexpr int TILES_MAX = 3;                 // tiles of 8 term columns that a warp accumulates at once

// Bytes between rows of `columns` (a multiple of 32) terms in shared memory: 64 past a multiple of 128, so that the 16-byte
// operand loads of 8 lanes, 64 bytes of each of two rows, meet all banks once.
constexpr int row_bytes(int columns) { return (2 * columns) | 64; }
// Floats between two columns of a warp's sums: a unit's rows and 4 against bank conflicts.
constexpr int part_stride(int slabs) { return slabs * ROWS + 4; }

// Warps to a unit (16 rows x all chunks): the split with the fewest chunks one after the other, where a unit's end counts as one more
// and joining several warps' sums as another; equal: fewer warps a unit.
constexpr int choose_split(int warps, int units_of_cta, int chunks, int most) {
  int best = 1, cost = 1 << 30;
  for (int i = 0; 1 << i <= warps && 1 << i <= most; ++i) {  // 2^i warps a unit, warps / 2^i units at once
    const int rounds = (units_of_cta + (warps >> i) - 1) * (1 << i) / warps;
    const int c = rounds * (((chunks + (1 << i) - 1) >> i) + (i ? 2 : 1));
    if (c < cost) best = 1 << i, cost = c;
  }
  return best;
}

// A kernel of strata_moe_linear: its largest block's tiles, its warps and their rings' depth; of its weights the bytes of a chunk in the
// ring, the chunk's columns and a unit's slabs.
struct LinearKernel {
  int tiles, warps, depth, slot, columns, slabs;
};
struct LinearPlan {
  int tokens;        // of a block
  int part_cols;     // term columns of a block, rounded up to whole tiles
  int log_split;     // 2^this warps to a unit
  int panel;         // chunks whose activations lie in shared memory at once: all, or a multiple of the unit's warps and of CHUNK columns
  int row_stride;    // bytes between rows of terms
  int scale_stride;  // floats between tokens' scales
  int grid_x, grid_y;
  bool pair;         // two neighbouring CTAs lay out x for one another
  size_t bytes;      // of shared memory: rings, sums, scales, rows of terms
};

inline LinearPlan linear_plan(const LinearKernel& k, int T, int columns, int rows, int terms, int sms) {
  LinearPlan p{};
  const int chunks = (columns + k.columns - 1) / k.columns, units = (rows + ROWS * k.slabs - 1) / (ROWS * k.slabs);
  p.tokens = 8 * k.tiles / terms < T ? 8 * k.tiles / terms : T;
  p.part_cols = (p.tokens * terms + 7) / 8 * 8;
  const size_t fixed = (size_t)k.warps * k.depth * k.slot + sizeof(float) * k.warps * p.part_cols * part_stride(k.slabs);
  auto measure = [&]() {
    p.row_stride = row_bytes(p.panel * k.columns);
    p.scale_stride = (p.panel + 3) / 4 * 4;  // the rows behind the scales on 16-byte boundaries
    p.bytes = fixed + p.tokens * (sizeof(float) * p.scale_stride + (size_t)terms * p.row_stride);
  };
  // chunks of a block's terms and scales that fit beside the rings, with a row's padding
  const int fit = (int)((SMEM_MAX - fixed - (size_t)p.tokens * (terms * 64 + 16)) / (p.tokens * (terms * 2 * k.columns + sizeof(float))));
  p.panel = chunks;
  measure();
  const int per_sm = k.warps == 16 || p.bytes > SMEM_HALF ? 1 : 2;
  const int blocks = (T + p.tokens - 1) / p.tokens, ctas = sms * per_sm;
  p.grid_y = blocks < ctas ? blocks : ctas;
  const int most_x = ctas / p.grid_y;
  const int split = choose_split(k.warps, (units + most_x - 1) / most_x, chunks, fit);
  // a panel is a multiple of the unit's warps, whose chunks lie that far apart, and of CHUNK columns, which a half warp lays out at once: a panel that
  // ended inside of them would have it store into the next row
  const int step = split * k.columns < CHUNK ? CHUNK / k.columns : split;  // powers of two
  p.panel = (chunks + split - 1) / split * split;
  if (p.panel > fit) p.panel = fit / step * step;
  while (1 << p.log_split < split) ++p.log_split;
  measure();
  // where a half warp would lay out eight terms of chunks or more, and all of x at once, neighbouring CTAs share that (15 of them, 64 tokens to 10,240
  // bf16: 28.5 us alone, 24.9 in pairs); with fewer the two meetings cost more (5 of them, 4 tokens to 10,240: 9.6 and 9.9)
  const int most = units < most_x ? units : most_x, even = most & ~1;
  p.pair = k.tiles > 1 && p.panel >= chunks && even > 0 && (units + even - 1) / even == (units + most - 1) / most &&
           p.tokens * terms * ((columns + CHUNK - 1) / CHUNK) >= 8 * 2 * k.warps;
  p.grid_x = p.pair ? even : most;
  return p;
}

}  // namespace q4
}  // namespace strata
