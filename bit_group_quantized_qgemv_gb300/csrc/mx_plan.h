// mx_plan.h -- how a product with MXFP4 weights is cut into tiles (host only, no CUDA).
#pragma once

#include <atomic>
#include <initializer_list>

namespace qgemv {

constexpr int kMxRows = 128;      // weight rows of a tile
constexpr int kMxStep = 128;      // k of a stage
constexpr int kMxMinStages = 4, kMxMaxStages = 16;
constexpr int kMxRowSteps = 64;   // steps of fp16 rows that a block holds, at most
constexpr int kMxAccCols = 480;   // tensor memory of the accumulators (512 less the scales')
constexpr int kMxOut = 16;        // columns that results are written by
constexpr int kMxSplits[4] = {1, 2, 4, 8};
constexpr int kMxSmem = 227 * 1024 - 1024;  // dynamic shared memory (the rest is static)

// How many clusters of 1 << log2 blocks a kernel has at work at a time, each kernel's own table:
// asked once per size and device.  A question that fails is answered by 0 and asked again.
class MxClusterTable {
 public:
  template <typename Ask>  // ask(&n): whether n is the answer
  int get(int log2, int device, Ask ask) {
    std::atomic<int>& at = known_[log2][device & 63];
    const int known = at.load(std::memory_order_relaxed);
    if (known > 0) return known - 1;
    int n = 0;
    if (!ask(&n)) return 0;
    at.store(n + 1, std::memory_order_relaxed);
    return n;
  }

 private:
  std::atomic<int> known_[4][64] = {};  // one more than the answer
};

struct MxShape {
  long long M, N;
  int K;
  bool gated, fp16;    // two weights; fp16 rows of x
  int clusters[4];     // clusters of 1, 2, 4, 8 blocks that run at a time

  bool operator==(const MxShape& o) const {
    bool same = M == o.M && N == o.N && K == o.K && gated == o.gated && fp16 == o.fp16;
    for (int i = 0; i < 4; ++i) same = same && clusters[i] == o.clusters[i];
    return same;
  }
};

struct MxPlan {
  int cols;      // columns of a tile
  int tokens;    // rows of x of a tile
  int split;     // blocks that share K (a cluster)
  int stages;
  int row_tiles, tok_tiles;
  int row_steps; // steps of fp16 rows that a block holds
  bool pair;     // every other step's products into a second accumulator
  bool rows_first;  // tiles of rows change fastest
  int smem;      // dynamic shared memory of a block
};

inline int mx_stage_bytes(int w, int cols, bool fp16) {
  return w * kMxRows * kMxStep + (fp16 ? 0 : cols * kMxStep) + 512 * (w + (fp16 ? 0 : cols > 128 ? 2 : 1));
}

// Everything of a plan that follows from its columns and split; false where it does not
// fit a multiprocessor.
inline bool mx_fit(const MxShape& s, int cols, int split, MxPlan* p) {
  const int w = s.gated ? 2 : 1, steps = (s.K + kMxStep - 1) / kMxStep;
  p->cols = cols;
  p->tokens = s.fp16 ? static_cast<int>(s.M) : cols;
  p->split = split;
  p->row_tiles = static_cast<int>((s.N + kMxRows - 1) / kMxRows);
  p->tok_tiles = static_cast<int>((s.M + p->tokens - 1) / p->tokens);
  p->row_steps = s.fp16 ? (steps + split - 1) / split : 0;
  p->pair = !s.gated && 4 * cols <= kMxAccCols;
  // the smaller operand's tiles change fastest: blocks at work at a time share the larger's
  p->rows_first = 2 * s.M > w * s.N;
  if (split > steps || p->row_steps > kMxRowSteps || 2 * w * cols > kMxAccCols) return false;
  const int part = split > 1 ? w * ((p->tokens + split - 1) / split * split) * kMxRows * 4 : 0;
  const int out = s.fp16 || s.gated || split > 1 ? 0 : 2 * kMxOut * kMxRows * 4;
  const int other = 1024 + part + out + p->row_steps * (cols * kMxStep + 512);
  const int stage = mx_stage_bytes(w, cols, s.fp16);
  if (other > kMxSmem) return false;
  // Even, so that a stage is always filled and used by the same of two warps: a wait tells
  // a use of a stage from the one before it, not from two before.
  p->stages = (kMxSmem - other) / stage;
  p->stages = (p->stages > kMxMaxStages ? kMxMaxStages : p->stages) / 2 * 2;
  p->smem = other + p->stages * stage;
  return p->stages >= kMxMinStages;
}

// Clocks that a plan is expected to take.  A step of a tile is bound by shared memory (what
// the copies write, weights spread to bytes, and what the products read, x once for each
// weight), L2, the tensor core, or the waits and the issue of products; a tile by its steps
// or by the results of the one before.  The rates are fitted to 37 products of 9 to 8192 rows
// and 16 of 1 to 8 fp16 rows, each in all widths and splits, by themselves and in pairs: what
// this takes was the fastest or within 2% of it, but for three of the fp16 rows (7 to 11%).
inline double mx_cost(const MxShape& s, const MxPlan& p) {
  const int w = s.gated ? 2 : 1, steps = (s.K + kMxStep - 1) / kMxStep;
  int i = 0;
  while (kMxSplits[i] != p.split) ++i;
  const double tiles = static_cast<double>(p.row_tiles) * p.tok_tiles, clusters = s.clusters[i];
  const double rounds = static_cast<double>(static_cast<long long>((tiles + clusters - 1) / clusters));
  const int part = (steps + p.split - 1) / p.split;  // steps of a block
  double step, out, fill;
  if (s.fp16) {
    step = 420, out = 1200 + (p.split > 1 ? 1000 + 110 * i : 0), fill = 4800;
  } else {
    const double cols = p.cols;
    const double smem = w * kMxRows * 1.58 + (1 + w) * cols * 0.85, l2 = (w * 8704 + cols * 132) / 75;
    const double tensor = w * 4 * (cols / 2 > 32 + cols / 4 ? cols / 2 : 32 + cols / 4);
    step = p.pair ? 320 : 0;
    for (const double least : {smem, l2, tensor}) step = step > least ? step : least;
    out = 1800 + w * cols * (s.gated ? 23.5 : 19) + (p.split > 1 ? 1100 + 200 * i + w * cols * 66 : 0), fill = 6500;
  }
  return rounds * (part * step > out ? part * step : out) + out + fill;
}

// The plan that is expected to be fastest.  False: none fits (K too long for fp16 rows).
inline bool mx_plan(const MxShape& shape, MxPlan* best) {
  // fp16 rows: one tile of them, and the split that is best for eight, so that a row's
  // result does not depend on how many there are.
  MxShape s = shape;
  if (s.fp16) s.M = 8;
  double least = 0;
  bool any = false;
  for (int i = 0; i < 4; ++i) {
    if (s.clusters[i] < 1) continue;
    for (int cols = s.fp16 ? 32 : 16; cols <= (s.fp16 ? 32 : 240); cols += 16) {
      if (!s.fp16 && cols > 16 && cols - 16 >= s.M) break;  // wider than the rows there are
      MxPlan p;
      if (!mx_fit(s, cols, kMxSplits[i], &p)) continue;
      const double c = mx_cost(s, p);
      if (!any || c < least) least = c, *best = p, any = true;
    }
  }
  return any && (!s.fp16 || mx_fit(shape, 3 * shape.M <= 16 ? 16 : 32, best->split, best));
}

// Tiles of two blocks that share them (mx_pair.cu): 256 rows of weights (gated: 128 of each
// of the two), the columns half in each block.
struct MxPairPlan {
  int cols, stages;
  int row_tiles, tok_tiles;
  bool rows_first;
  bool two;      // every other step's products into a second accumulator
  int smem;
};

inline bool mx_pair_fit(const MxShape& s, int cols, MxPairPlan* p) {
  const int rows = s.gated ? 128 : 256;
  p->cols = cols;
  p->row_tiles = static_cast<int>((s.N + rows - 1) / rows);
  p->tok_tiles = static_cast<int>((s.M + cols - 1) / cols);
  p->rows_first = 2 * s.M > (s.gated ? 2 : 1) * s.N;
  const int other = 1024 + 2 * kMxOut * kMxRows * 4;
  const int stage = kMxRows * kMxStep + cols / 2 * kMxStep + 512 * (cols > 128 ? 3 : 2);
  p->stages = (kMxSmem - other) / stage;
  p->stages = (p->stages > kMxMaxStages ? kMxMaxStages : p->stages) / 2 * 2;
  p->two = 4 * cols <= kMxAccCols;
  p->smem = other + p->stages * stage;
  return cols % 32 == 0 && 2 * cols + 32 <= 512 && p->stages >= kMxMinStages;
}

inline double mx_pair_cost(const MxShape& s, const MxPairPlan& p) {
  const int steps = s.K / kMxStep;
  const double tiles = static_cast<double>(p.row_tiles) * p.tok_tiles, clusters = s.clusters[1];
  const double rounds = static_cast<double>(static_cast<long long>((tiles + clusters - 1) / clusters));
  const double tensor = 78 + 2.02 * p.cols, least = p.two ? 320 : 400, step = tensor > least ? tensor : least;
  const double per_tile = steps * step, out = 1500 + p.cols * (s.gated ? 33 : 15) * (p.two ? 1.25 : 1);
  return rounds * (per_tile > out ? per_tile : out) + out + 3400;
}

// The best of them; false: none (no clusters of two, or K is no whole number of steps).
inline bool mx_pair_plan(const MxShape& s, MxPairPlan* best, double* cost) {
  bool any = false;
  if (s.fp16 || s.clusters[1] < 1 || s.K % kMxStep != 0) return false;
  for (int cols = 32; cols <= 224; cols += 32) {
    if (cols > 32 && cols - 32 >= s.M) break;
    MxPairPlan p;
    if (!mx_pair_fit(s, cols, &p)) continue;
    const double c = mx_pair_cost(s, p);
    if (!any || c < *cost) *cost = c, *best = p, any = true;
  }
  return any;
}

}  // namespace qgemv
