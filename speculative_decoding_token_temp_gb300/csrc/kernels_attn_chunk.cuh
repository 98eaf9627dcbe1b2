// Chunks of new tokens over the cache, on the fifth-generation tensor cores: what
// attn_prefix_kernel (its CHUNK form) works from.
//
// Rows of a sequence that fill 256-row blocks (whole tokens: 252 rows with 7 heads a kv head) make a dense product, so every sequence's keys
// and values are widened once per call into the workspace, as a shared prefix is, and read as
// 16-bit operands by all its row blocks: the prefix's tiles first, then the sequence's own, up
// to the last token that the row block sees.
//
// chunk_plan_kernel   one block: where each sequence's tiles stand in the widened memory, and
//                     the line of tiles, an entry a row block (the heads of an entry one after
//                     the other). The tiles behind a row block's last row are not on it.
// chunk_widen_kernel  keys to bf16, values to f16 relative to the tile's largest exponent. A
//                     token stored as NaN, or on a bad page, gets NaN keys and zero values: a
//                     row that does not see it has the weight 0 there, and 0 * NaN must not
//                     reach it. Where a tile's exponents differ by more than 20 (10 with fp32 queries), its values
//                     would lose places to tokens that a row may not even see: they are then
//                     widened without their exponents, and these join the scores one by one
//                     (`mixed`), as in attn_tc_kernel.
//
// The attention's blocks take whole segments (a row block at one kv head), sorted by length and
// dealt out to and fro, where the plan finds that even enough, and equal parts of the line
// otherwise. Queries come by TMA while the ends of the stretch before are worked on.
//
// fp32 queries are cut into three bf16 parts, exactly, and their weights into two f16 parts: five products where bf16 queries
// take two, one row tile of 128 a block (2 x 400 rows behind 1000 tokens, 32/8 heads of 128: 75 us, 1002 on the fp32 pipe).
//
// What bounds it: a tile of 256 rows x 128 tokens takes about 3000 clocks with either head_dim,
// and its MMAs 2048 at head_dim 128 and half of that at 64: the softmax warps' instructions (about
// 400 a warp and tile) and the chain scores, weights, values' sum. A segment's beginning and end
// are as long as 4 to 5 tiles. One prompt of 4096 tokens, 32/8 heads of 128: 127 us (plan 7, widening
// 9, attention 114, the empty joining 7; parts of them overlap), 1.08 PFLOP/s; 4 x 2048 rows behind
// 0-16384 tokens 767 us, 1.4 PFLOP/s.
#pragma once

#include "chunk_plan.h"
#include "kernels_attn_tc.cuh"

namespace sv {

constexpr int kPlanThreads = 1024;
constexpr int kWidenThreads = 256;
constexpr int kValueShift = 6;    // the largest value of a tile comes to at most 448 * 2^6
// Most that the exponents of a tile may differ by while they are left to its values: code * 2^(6 + e - largest) is exact in f16
// down to e = largest - 21, and a weight, which is then without them, is off by at most 2^-33 of the row's largest by itself, so by
// 2^-13 of it with them, for bf16 outputs. With fp32 queries 2^-23 of it.
constexpr int kValueSpread = 20, kValueSpread32 = 10;

// Row block rb of sequence b: its place on the line, its tiles (the prefix's and its own), the
// widened tile that is the sequence's first less the prefix's number of tiles.
struct ChunkEntry {
  int start, b, rb, nt;
  int w0, row0, rows, len;  // len -1: a bad kv_len
};

constexpr int kPlanBuckets = 1024;  // of lengths, one a thread of the plan

// The segment that block b of n takes in round r: to and fro, so that who got the longest of a round gets the shortest of the next.
__device__ __forceinline__ long long chunk_item(int r, int b, int n) { return (long long)r * n + (r & 1 ? n - 1 - b : b); }

struct ChunkHead {
  int entries;  // -1: cu is no prefix sum of the batch
  int line;     // the line's length
  int tiles;    // widened tiles, the prefix's among them
  int whole;    // blocks take whole segments (entry, head) instead of equal parts of the line
};

struct ChunkParams {
  ChunkHead* head;
  ChunkEntry* entry;
  int* order;          // [entries] the longest first
  int* first;          // [B] a sequence's first widened tile
  int blocks;          // of the attention
  const int32_t* pre_table;
  int pre_len, pre_tiles;
  int min_flat;        // sequences with fewer rows (times heads of a kv head) are left to attn_tc_kernel
};

// Exclusive prefix sum over the block's threads (a multiple of 32, at most 1024); `total` for all.
__device__ __forceinline__ int plan_scan(int x, int* s_warp, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kFull, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    const int y = s_warp[lane];
    int z = y;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(kFull, z, o);
      if (lane >= o) z += v;
    }
    s_warp[lane] = z;
  }
  __syncthreads();
  total = s_warp[31];
  return (warp > 0 ? s_warp[warp - 1] : 0) + incl - x;
}

__global__ void __launch_bounds__(kPlanThreads) chunk_plan_kernel(const __grid_constant__ AttnParams p, ChunkParams c) {
  __shared__ int s_warp[32], s_er[kPlanThreads], s_nrb[kPlanThreads];
  griddep_wait();
  griddep_launch();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, NR = p.block_rows;
  // cu first: only of a prefix sum do the sequences' row blocks fit where they are to stand
  bool bad_cu = false;
  if (p.cu != nullptr) {
    for (int b = tid; b < p.B; b += kPlanThreads) {
      const int lo = __ldg(p.cu + b), hi = __ldg(p.cu + b + 1);
      bad_cu |= lo < 0 || hi > p.total_draft || hi < lo || hi - lo > p.gamma || (b == 0 && lo != 0) || (b == p.B - 1 && hi != p.total_draft);
    }
  }
  if (__syncthreads_or(bad_cu)) {
    if (tid == 0) *c.head = ChunkHead{-1, 0, 0, 0};
    return;
  }
  uint32_t bits = 0;
  int entries = 0, tiles = c.pre_tiles;
  for (int b0 = 0; b0 < p.B; b0 += kPlanThreads) {
    const int b = b0 + tid;
    int nrb = 0, wt = 0;
    SeqInfo s{};
    if (b < p.B) {
      s = seq_info(p, b);
      if (s.bad) bits |= SPEC_DEV_OFFSETS;
      nrb = s.rows * p.G >= c.min_flat ? (s.rows * p.G - 1) / NR + 1 : 0;
      wt = nrb > 0 ? seq_ntiles(s) : 0;
    }
    int all_r, all_t;
    const int er = entries + plan_scan(nrb, s_warp, all_r), et = tiles + plan_scan(wt, s_warp, all_t);
    if (b < p.B) {
      c.first[b] = et;
      // the sequence's first entry, from which its others are made
      if (nrb > 0) c.entry[er] = ChunkEntry{0, b, 0, 0, et - c.pre_tiles, s.row0, s.rows, s.bad ? -1 : s.len};
    }
    entries += all_r;
    tiles += all_t;
    s_er[tid] = er;
    s_nrb[tid] = nrb;
    __syncthreads();
    // the sequences' row blocks: a warp a sequence, a lane a row block
    const int here = min(kPlanThreads, p.B - b0);
    for (int i = warp; i < here; i += kPlanThreads / 32) {
      const int n = s_nrb[i], at = s_er[i];
      if (n == 0) continue;
      const ChunkEntry first = c.entry[at];
      __syncwarp();
      const int len = max(first.len, 0);
      for (int rb = lane; rb < n; rb += 32) {
        const int last = (int)min((long long)first.rows, ((long long)(rb + 1) * NR - 1) / p.G + 1);  // rows up to the block's last
        const int sees = len - first.rows + last;
        ChunkEntry e = first;
        e.rb = rb;
        e.nt = max(1, c.pre_tiles + (sees > 0 ? (sees - 1) / kTile + 1 : 0));
        e.start = p.Hk * (e.nt + p.seg_cost);
        c.entry[at + rb] = e;
      }
    }
    __syncthreads();
  }
  // the line: the entries' lengths to where they begin
  int line = 0;
  for (int e0 = 0; e0 < entries; e0 += kPlanThreads) {
    const int e = e0 + tid, n = e < entries ? c.entry[e].start : 0;
    int all;
    const int at = line + plan_scan(n, s_warp, all);
    if (e < entries) c.entry[e].start = at;
    line += all;
  }
  // Whole segments, or equal parts of the line (whole_segments)? What the busiest block would get of whole ones, sorted by
  // length and dealt out to and fro, is added up here.
  __shared__ int s_hist[kPlanBuckets], s_most, s_long;
  if (tid == 0) s_most = 0, s_long = 1;
  for (int i = tid; i < kPlanBuckets; i += kPlanThreads) s_hist[i] = 0;
  __syncthreads();
  int longest = 1;
  for (int e = tid; e < entries; e += kPlanThreads) longest = max(longest, c.entry[e].nt);
  atomicMax(&s_long, longest);
  __syncthreads();
  const int unit = (s_long + kPlanBuckets - 1) / kPlanBuckets;  // tiles of a bucket
  for (int e = tid; e < entries; e += kPlanThreads) atomicAdd(&s_hist[kPlanBuckets - 1 - (c.entry[e].nt - 1) / unit], 1);
  __syncthreads();
  int all;
  const int count = s_hist[tid], at = plan_scan(count, s_warp, all);
  __syncthreads();
  s_hist[tid] = at;
  __syncthreads();
  for (int e = tid; e < entries; e += kPlanThreads) c.order[atomicAdd(&s_hist[kPlanBuckets - 1 - (c.entry[e].nt - 1) / unit], 1)] = e;
  __syncthreads();
  const long long items = (long long)entries * p.Hk;
  if (items <= (long long)kPlanRounds * c.blocks) {
    for (int b = tid; b < c.blocks; b += kPlanThreads) {
      int sum = 0;
      for (int r = 0; r < kPlanRounds; ++r) {
        const long long i = chunk_item(r, b, c.blocks);
        if (i >= items) break;
        sum += ((c.entry[c.order[i / p.Hk]].nt - 1) / unit + 1) * unit + p.seg_cost;  // (by its bucket: the same whatever the order within)
      }
      atomicMax(&s_most, sum);
    }
  }
  __syncthreads();
  if (tid == 0) {
    const bool even = whole_segments(items, c.blocks, s_most, s_long, line, p.seg_cost);
    *c.head = ChunkHead{entries, line, tiles, even ? 1 : 0};
  }
  if (bits) atomicOr(p.status, bits);
}

// The widened keys and values in the workspace: [kv head][tiles][128 tokens][D].
struct WideParams {
  uint16_t *k16, *v16;
  float* exp;  // prefix alone: [kv head][tile]: E, kSumShift more than the values are relative to (so the sums of 2^(x - m) are that much smaller)
  int tiles;
  // chunks
  float2* info;  // [kv head][tile]: E, and whether the tile is mixed
  int spread;    // of exponents, past which a tile is mixed
  float* ev;     // [kv head][tile][128]: a mixed tile's E, token by token
  int q_tma;     // bf16 queries come by TMA, whole tokens a load (any number of heads a kv head; rows and heads on the 16-byte grid)
  ChunkParams c;
};

// A unit is one tile of one kv head; the grid strides over them. The first 128 threads look the
// tokens up; then D / 8 lanes take a token, 8 codes and one 16-byte store of each operand a lane.
template <int D>
__global__ void __launch_bounds__(kWidenThreads) chunk_widen_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ WideParams w) {
  constexpr int L = D / 8, ROWS = kWidenThreads / L, STEPS = kTile / ROWS;
  __shared__ float s_max[4], s_min[4], s_ks[kTile], s_ev[kTile];
  __shared__ long long s_vec[kTile];
  griddep_wait();
  griddep_launch();
  const int tid = threadIdx.x, lane = tid & 31;
  const float nan = __int_as_float(0x7fffffff);
  const long long units = (long long)w.c.head->tiles * p.Hk;
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    const int wt = (int)(u / p.Hk), h = (int)(u - (long long)wt * p.Hk);
    const int32_t* pages = w.c.pre_table;
    int t0 = wt * kTile, len = w.c.pre_len;
    if (wt >= w.c.pre_tiles) {
      int lo = 0, hi = p.B;  // the last sequence whose tiles begin at or before this one (those without tiles share a place)
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (w.c.first[mid] <= wt)
          lo = mid;
        else
          hi = mid;
      }
      const SeqInfo s = seq_info(p, lo);
      pages = p.table + (long long)lo * p.pps;
      t0 = (wt - w.c.first[lo]) * kTile;
      len = s.len;
    }
    __syncthreads();  // (the unit before is done with the shared memory)
    if (tid < kTile) {
      const int t = t0 + tid;
      long long vec = -1;
      float ks = 0.f, ev = -1e30f;
      if (t < len) {
        const int page = __ldg(pages + (t >> p.page_shift));
        ks = nan;
        if ((unsigned)page < (unsigned)p.num_pages) {
          vec = (((long long)page * p.Hk + h) << p.page_shift) + (t & ((1 << p.page_shift) - 1));
          if (!in_idx(vec, ((long long)p.num_pages * p.Hk) << p.page_shift, p.status)) vec = -1;
        } else {
          atomicOr(p.status, SPEC_DEV_PAGE);
        }
        if (vec >= 0) {
          const unsigned kb = __ldg(p.k_exp + vec), vb = __ldg(p.v_exp + vec);
          if (kb != kNanExp && vb != kNanExp) {
            ks = exp_value(kb);
            ev = (float)((int)vb - kExpBias);
          }
        }
      }
      s_vec[tid] = vec;
      s_ks[tid] = ks;  // NaN: of a token that is not to be read as numbers
      s_ev[tid] = ev;
      float most = ev, least = ev < -200.f ? 1e30f : ev;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        most = fmaxf(most, __shfl_xor_sync(kFull, most, o));
        least = fminf(least, __shfl_xor_sync(kFull, least, o));
      }
      if (lane == 0) s_max[tid >> 5] = most, s_min[tid >> 5] = least;
    }
    __syncthreads();
    float e = fmaxf(fmaxf(s_max[0], s_max[1]), fmaxf(s_max[2], s_max[3]));
    const float least = fminf(fminf(s_min[0], s_min[1]), fminf(s_min[2], s_min[3]));
    if (e < -200.f) e = 0.f;  // no token with values
    const bool mixed = e - least > (float)w.spread;
    const long long at = (long long)h * w.tiles + wt;
    if (tid == 0) w.info[at] = make_float2(e + (float)kSumShift, mixed ? 1.f : 0.f);
    if (mixed && tid < kTile) w.ev[at * kTile + tid] = s_ev[tid] < -200.f ? 0.f : s_ev[tid] + (float)kSumShift;
    const int sub = tid % L, u0 = tid / L;
    uint2 kw[STEPS], vw[STEPS];
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const long long vec = s_vec[u0 + i * ROWS];
      kw[i] = vw[i] = make_uint2(0, 0);
      if (vec >= 0) {
        kw[i] = __ldg(reinterpret_cast<const uint2*>(p.k + vec * D) + sub);
        vw[i] = __ldg(reinterpret_cast<const uint2*>(p.v + vec * D) + sub);
      }
    }
    const long long row0 = at * kTile;
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const int r = u0 + i * ROWS;
      const uint32_t code = ((vw[i].x & 0x7f7f7f7fu) + 0x01010101u) | ((vw[i].y & 0x7f7f7f7fu) + 0x01010101u);
      const unsigned nans = __ballot_sync(kFull, (code & 0x80808080u) != 0) >> (lane / L * L) & (L == 32 ? ~0u : (1u << L) - 1);
      float ks = s_ks[r];
      const float ev = s_ev[r];
      if (nans) ks = nan;
      const float vs = ks != ks || ev < -200.f ? 0.f : ex2((mixed ? 0.f : ev - e) + (float)kValueShift);
      float x[8], y[8];
      codes4(kw[i].x, x);
      codes4(kw[i].y, x + 4);
      codes4(vw[i].x, y);
      codes4(vw[i].y, y + 4);
      uint32_t ok[4], ov[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * j] * ks, x[2 * j + 1] * ks);
        ok[j] = *reinterpret_cast<const uint32_t*>(&b);
        ov[j] = vs == 0.f ? 0u : half2_of(y[2 * j] * vs, y[2 * j + 1] * vs);
      }
      *reinterpret_cast<uint4*>(w.k16 + (row0 + r) * D + sub * 8) = make_uint4(ok[0], ok[1], ok[2], ok[3]);
      *reinterpret_cast<uint4*>(w.v16 + (row0 + r) * D + sub * 8) = make_uint4(ov[0], ov[1], ov[2], ov[3]);
    }
  }
}

// A stretch of a segment, with where its own tiles are: wide tile = tile + (tile < pre_tiles ? 0 : w0).
struct WideSeg : Seg {
  int w0;
};

// Block i's part of the line, its place: (entry, offset). By the first warp for the block.
__device__ __forceinline__ Part locate_chunk(const ChunkParams& c, int heads, Part& shared) {
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x, total = c.head->line, n = c.head->entries;
    Part r;
    if (c.head->whole) {  // the part: rounds
      const long long items = (long long)n * heads;
      const int full = (int)(items / gridDim.x);
      r.begin = 0;
      r.end = full + (chunk_item(full, blockIdx.x, gridDim.x) < items ? 1 : 0);
      r.total = total;
      r.ok = true;
      r.at = Place{0, 0};
      if (lane == 0) shared = r;
    } else {
      r.total = total;
      r.ok = n >= 0;
      r.begin = line_at(total, blockIdx.x, gridDim.x);
      r.end = line_at(total, blockIdx.x + 1, gridDim.x);
      int lo = 0, hi = max(n, 1);
      while (hi - lo > 1 && r.begin < total) {
        const int step = (hi - lo + 31) / 32, e = lo + lane * step;
        const unsigned in = __ballot_sync(kFull, e < hi && c.entry[e < hi ? e : lo].start <= r.begin);
        lo += (__popc(in) - 1) * step;  // (the first is among them)
        hi = min(hi, lo + step);
      }
      r.at.b = lo;
      r.at.off = r.begin < total ? r.begin - c.entry[lo].start : 0;
      if (lane == 0) shared = r;
    }
  }
  __syncthreads();
  return shared;
}

__device__ __forceinline__ WideSeg next_chunk(const AttnParams& p, const ChunkParams& c, Place& at, int& left) {
  const bool whole = c.head->whole;
  const long long item = whole ? chunk_item(at.b, blockIdx.x, gridDim.x) : 0;
  const int head = whole ? (int)(item % p.Hk) : 0;
  const ChunkEntry e = c.entry[whole ? c.order[item / p.Hk] : at.b];
  WideSeg g;
  g.row0 = e.row0, g.rows = e.rows, g.bad = e.len < 0, g.len = max(e.len, 0);
  g.nt = e.nt;
  g.f0 = e.rb * p.block_rows;
  g.pages = nullptr;
  g.w0 = e.w0;
  if (whole) {
    g.t0 = 0, g.n = e.nt, g.h = head;
    at.b += 1;
    left -= 1;
    return g;
  }
  const int line = e.nt + p.seg_cost, h = at.off / line, r = at.off - h * line, take = min(line - r, left);
  g.t0 = max(0, r - p.seg_cost);
  g.n = max(0, r + take - p.seg_cost - g.t0);
  g.h = h;
  at.off += take;
  left -= take;
  if (at.off >= p.Hk * line) {
    at.b += 1;
    at.off = 0;
  }
  return g;
}

}  // namespace sv
