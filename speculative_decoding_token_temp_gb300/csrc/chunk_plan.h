// How the attention of chunks is shared out among its blocks: plain arithmetic, compiled into the
// plan's kernel and, on its own, into a CPU test.
#pragma once

#ifdef __CUDACC__
#define SV_PLAN __host__ __device__ __forceinline__
#else
#define SV_PLAN inline
#endif

namespace sv {

constexpr int kJoinCost = 9;     // the joining of cut segments (15 us), in tiles
constexpr int kPlanRounds = 64;  // segments a block whose lengths the plan adds up

// Do blocks take whole segments (true), sorted by length and dealt out to and fro, or equal parts of the line of tiles? Cut
// segments cost their beginning and end (seg_cost tiles) twice, and the joining; whole ones leave blocks with more and with less.
//   items     segments; longest: tiles of the longest
//   busiest   tiles of the busiest block, segments' ends among them, where there are at most kPlanRounds a block; 0: none
//   line      tiles of all segments, their ends among them
// Past kPlanRounds segments a block nothing is added up. Dealt out to and fro no block then gets more than the average and the
// longest segment: whole ones where that segment is shorter than what cuts cost, or an eighth of a block's share. Whole / cut,
// 8 kv heads of 64: 5000 rows of 64 heads a kv head from the beginning and 4 behind 10^6 tokens (a segment of 7814 tiles, a share
// of 1900) 12.8 / 3.3 ms, behind 100000 (783 of 1500) 3.1 / 2.3; 1250 rows behind 1-100 tokens and 256 behind 3000 (25 of 400:
// short segments are dear to cut) 0.44 / 0.54.
SV_PLAN bool whole_segments(long long items, int blocks, int busiest, int longest, int line, int seg_cost) {
  const int share = line / blocks, cuts = seg_cost + kJoinCost;
  if (items > (long long)kPlanRounds * blocks) return longest <= cuts || longest <= share / 8;
  return busiest > 0 && busiest <= share + cuts;
}

}  // namespace sv
