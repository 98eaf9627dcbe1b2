// Test driver for csrc/chunk_plan.h: reads queries from stdin and prints the choice, one line each.
//   items blocks busiest longest line seg_cost -> 0 (equal parts of the line) or 1 (whole segments)
#include <cstdio>

#include "chunk_plan.h"

int main() {
  long long items;
  int blocks, busiest, longest, line, seg_cost;
  while (std::scanf("%lld %d %d %d %d %d", &items, &blocks, &busiest, &longest, &line, &seg_cost) == 6)
    std::printf("%d\n", sv::whole_segments(items, blocks, busiest, longest, line, seg_cost) ? 1 : 0);
  return 0;
}
