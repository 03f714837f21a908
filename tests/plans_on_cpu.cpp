// Plans of products: reads "M N K gated fp16 c1 c2 c4 c8" lines, writes what mx_plan.h makes of them.
#include <cstdio>

#include "mx_plan.h"

int main() {
  qgemv::MxShape s{};
  int gated, fp16;
  while (std::scanf("%lld %lld %d %d %d %d %d %d %d", &s.M, &s.N, &s.K, &gated, &fp16, &s.clusters[0], &s.clusters[1],
                    &s.clusters[2], &s.clusters[3]) == 9) {
    s.gated = gated != 0;
    s.fp16 = fp16 != 0;
    qgemv::MxPlan p{};
    const bool ok = qgemv::mx_plan(s, &p);
    qgemv::MxPairPlan two{};
    double cost = 0;
    const bool pairs = qgemv::mx_pair_plan(s, &two, &cost);
    std::printf("%d %d %d %d %d %d %d %d %d %d %d ", ok, p.cols, p.tokens, p.split, p.stages, p.row_tiles, p.tok_tiles,
                p.row_steps, p.pair, p.rows_first, p.smem);
    std::printf("%d %d %d %d %d %d %d %d\n", pairs, pairs && ok && cost < qgemv::mx_cost(s, p), two.cols, two.stages,
                two.row_tiles, two.tok_tiles, two.smem, two.two);
  }
}
