// Attention of the rows of a verification round over the 8-bit paged cache: the work
// split, the joining of its parts, and the 32-bit kernel.
//
// Work split. Rows that share keys (the gamma_b + 1 rows of a sequence times the G query
// heads of a kv head) form row blocks of NR; a row block's keys, cut into tiles of 128
// tokens, are a segment. The segments of all sequences, heads and row blocks laid end to
// end are a line of tiles, of which every block of the grid takes an equal, contiguous
// stretch: long and short sequences, few and many, keep all SMs equally busy, and what a
// block reads does not depend on when it runs. A block that holds a whole segment writes
// its rows' output; the parts of a segment that is cut between blocks go to the workspace
// (running maximum, sum and weighted values of each row), and attn_merge_kernel joins them
// in order, so the result does not depend on timing.
//
// The shared prefix is one more sequence whose "rows" are all rows of the batch: one pass
// over its keys for the whole batch, whose normalised part and log-sum the pass over the
// sequences' own tokens joins in.
#pragma once

#include "kernels_kv.cuh"

namespace sv {

constexpr int kTile = 128;  // tokens of a tile
constexpr int kRowsS = 8;   // row block of the 32-bit kernel
constexpr int kNegInfBits = 0xff800000;

enum AttnMask : int { A_ALL = 0, A_CHAIN = 1, A_TREE = 2 };

struct AttnParams {
  const uint8_t *k, *v, *k_exp, *v_exp;
  int num_pages, page_shift, Hk, Hq, G;
  const void* q;
  long long q_row, q_head;  // strides in elements
  int B, gamma, total_draft, R;
  const int32_t* cu;
  const int32_t* table;
  int pps;
  const int32_t* kv_len;  // null: every sequence has fixed_len tokens
  int fixed_len;
  int mask;
  int skip_flat;            // sequences with at least so many rows (times G) are left out; 0: none
  int block_rows;           // flat rows of a row block where they are fewer than the kernel's; 0: as many
  int late_wait;            // the pass over the sequences' own tokens behind a prefix pass: see attn_tc_kernel
  int seg_cost;             // tiles that a segment's beginning and end count for
  float c;                  // scale * log2(e)
  float* part;              // the parts of cut segments: two slots a block
  struct CutRec* cut;       // what each block leaves for attn_merge_kernel
  const float *pre_o, *pre_lse;  // the prefix's part to join in (normalised values, log2 of the sum), or null
  float *dst_o, *dst_lse;        // the prefix pass: its part goes here instead of o and lse
  void* o;
  float* lse;
  uint32_t* status;
  uint64_t sees[SPEC_MAX_TREE_NODES];  // node j: bit i set when node i sees it (i == j or a descendant of j)
};

// The segment that begins in a block and goes on in others (parts = 0: none): blocks
// block .. block + parts - 1 hold it (`total`: the line's length).
struct CutRec {
  int parts, row0, rows, h, f0, bad, total;
};

struct SeqInfo {
  int row0, rows, len;
  bool bad;  // kv_len out of range: taken as 0, its rows are NaN
};

__device__ __forceinline__ SeqInfo seq_info(const AttnParams& p, int b) {
  SeqInfo s;
  if (p.cu != nullptr) {
    const int lo = __ldg(p.cu + b);
    s.row0 = lo + b;
    s.rows = __ldg(p.cu + b + 1) - lo + 1;
  } else {
    s.row0 = b * (p.gamma + 1);
    s.rows = p.gamma + 1;
  }
  s.len = p.kv_len != nullptr ? __ldg(p.kv_len + b) : p.fixed_len;
  s.bad = s.len < 0 || (long long)s.len > ((long long)p.pps << p.page_shift);
  if (s.bad) s.len = 0;
  return s;
}

__device__ __forceinline__ int seq_ntiles(const SeqInfo& s) { return s.len > 0 ? (s.len - 1) / kTile + 1 : 1; }

// Left to another pass (a batch of chunks that has both long and short ones).
__device__ __forceinline__ bool skipped(const AttnParams& p, const SeqInfo& s) { return p.skip_flat > 0 && s.rows * p.G >= p.skip_flat; }

// Tiles on the line of a sequence, over all its row blocks and kv heads.
template <int NR, bool SKIP = false>
__device__ __forceinline__ int seq_tiles(const AttnParams& p, const SeqInfo& s) {
  return SKIP && skipped(p, s) ? 0 : (s.rows * p.G + NR - 1) / NR * p.Hk * (seq_ntiles(s) + p.seg_cost);
}

// A place on the line of tiles: sequence b, tile `off` of it.
struct Place {
  int b, off;
};

// Block i's part of the line, as locate() finds it.
struct Part {
  int begin, end, total;
  bool ok;   // cu is a valid prefix sum (nothing else counts when it is not)
  Place at;  // where the part begins
};

// Where block i's part of a line of `total` tiles begins, of n blocks (the first total % n
// have one tile more). The host has seen to it that a line's length fits an int.
__device__ __forceinline__ int line_at(int total, int i, int n) { return total / n * i + min(i, total % n); }

// Warp-wide: the line's length, block i's part of it (of n), and the place where that
// begins. Each lane sums a stretch of sequences, the warp scans the sums, and the lane whose
// stretch holds the place walks to it.
template <int NR, bool SKIP = false>
__device__ __noinline__ Part locate(const AttnParams& p, int i, int n) {
  const int lane = threadIdx.x & 31, per = (p.B + 31) / 32, b0 = min(p.B, lane * per), b1 = min(p.B, b0 + per);
  int sum = 0;
  bool bad = false;
#pragma unroll 4
  for (int b = b0; b < b1; ++b) {
    if (p.cu != nullptr) {
      const int lo = __ldg(p.cu + b), hi = __ldg(p.cu + b + 1);
      if (lo < 0 || hi > p.total_draft || hi < lo || hi - lo > p.gamma || (b == 0 && lo != 0) ||
          (b == p.B - 1 && hi != p.total_draft)) {
        bad = true;
        continue;
      }
    }
    sum += seq_tiles<NR, SKIP>(p, seq_info(p, b));
  }
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kFull, incl, o);
    if (lane >= o) incl += y;
  }
  Part r;
  r.total = __shfl_sync(kFull, incl, 31);
  r.ok = !__any_sync(kFull, bad);
  r.begin = line_at(r.total, i, n);
  r.end = line_at(r.total, i + 1, n);
  const int excl = incl - sum;
  const bool here = r.ok && r.begin >= excl && r.begin < incl;
  int b = b0, off = r.begin - excl;
  if (here) {
#pragma unroll 1
    for (; b < b1 - 1; ++b) {
      const int t = seq_tiles<NR, SKIP>(p, seq_info(p, b));
      if (off < t) break;
      off -= t;
    }
  }
  const unsigned who = __ballot_sync(kFull, here);
  const int src = who ? __ffs(who) - 1 : 0;
  r.at.b = __shfl_sync(kFull, b, src);
  r.at.off = __shfl_sync(kFull, off, src);
  return r;
}

// The same for the whole block, by its first warp.
template <int NR>
__device__ __forceinline__ Part locate_block(const AttnParams& p, Part& shared) {
  if (threadIdx.x < 32) {
    const Part r = locate<NR>(p, blockIdx.x, gridDim.x);
    if (threadIdx.x == 0) shared = r;
  }
  __syncthreads();
  return shared;
}

// One segment's stretch that a block works on.
struct Seg {
  int row0, rows, len, h, f0;  // f0: first flat row (row * G + head within the group) of the row block
  int t0, n, nt;               // its tiles t0 .. t0 + n - 1 of nt
  const int32_t* pages;
  bool bad;
};

// The next stretch at `at` (advanced), at most `left` tiles of the line (reduced). It may
// be empty (n = 0): the block's part of the line ends among the tiles that only count.
template <int NR, bool SKIP = false>
__device__ __forceinline__ Seg next_seg(const AttnParams& p, Place& at, int& left) {
  Seg g;
  SeqInfo s = seq_info(p, at.b);
  if constexpr (SKIP) {
    while (skipped(p, s)) s = seq_info(p, ++at.b);  // (there is one that is not: its tiles are `left`)
  }
  g.row0 = s.row0, g.rows = s.rows, g.len = s.len, g.bad = s.bad;
  g.nt = seq_ntiles(s);
  const int nrb = (s.rows * p.G + NR - 1) / NR, line = g.nt + p.seg_cost;
  const int seg = at.off / line, r = at.off - seg * line;
  const int take = min(line - r, left);
  g.t0 = max(0, r - p.seg_cost);
  g.n = max(0, r + take - p.seg_cost - g.t0);
  g.h = seg / nrb;
  g.f0 = (seg - g.h * nrb) * NR;
  g.pages = p.table + (long long)at.b * p.pps;
  at.off += take;
  left -= take;
  if (at.off >= nrb * p.Hk * line) {
    at.b += 1;
    at.off = 0;
  }
  return g;
}

// Which of a segment's rows see one token t of its sequence: rows from `from` on, of these
// (in a tree) the ones whose bit stands in `nodes` (bit i - 1: row i). `sees` is
// AttnParams::sees in shared memory (lanes ask for different nodes).
struct Sight {
  int from;
  uint64_t nodes;
  __device__ __forceinline__ bool operator()(int row) const { return row >= from && ((nodes >> ((row - 1) & 63)) & 1); }
};

__device__ __forceinline__ Sight sight_of(int mask, const uint64_t* sees, int rows, int len, int t) {
  const int j = t - (len - rows);  // the round's row whose token it is
  Sight s{0, ~0ull};
  if (t >= len)
    s.from = 1 << 30;
  else if (mask != A_ALL && j >= 0) {
    s.from = j;
    if (mask == A_TREE && j > 0) s.nodes = sees[j - 1];
  }
  return s;
}

// ---------------------------------------------------------------------------
// The end of a row: weights of its values and of the prefix's part, and its log-sum.
struct Coef {
  float a, b, lse2;
};

__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// m, l: the row's reference and sum; pre: the log-sum of the prefix's part (-inf: none). The
// approximate functions are off by at most 2^-22 of their results.
__device__ __forceinline__ Coef row_coef(float pre, float m, float l, bool bad) {
  const float nan = __int_as_float(0x7fffffff), ninf = __int_as_float(kNegInfBits);
  Coef r{0.f, pre == ninf ? 0.f : 1.f, pre};
  if (l != 0.f) {
    const float own = m + lg2(l), mx = fmaxf(own, pre), e1 = ex2(own - mx), e2 = ex2(pre - mx), s = e1 + e2, is = rcp(s);
    r.a = e1 * is * rcp(l);
    r.b = pre == ninf ? 0.f : e2 * is;  // (never a NaN where there is no prefix: its part is then not there to be read)
    r.lse2 = mx + lg2(s);
  }
  if (bad) r.a = r.lse2 = nan;
  return r;
}

__device__ __forceinline__ void put(uint16_t* o, float x) {
  const __nv_bfloat16 h = __float2bfloat16_rn(x);
  *o = *reinterpret_cast<const uint16_t*>(&h);
}
__device__ __forceinline__ void put(float* o, float x) { *o = x; }

// Element d of row `idx` (row * Hq + head) of the output, or of the prefix pass's part.
template <typename E, int D>
__device__ __forceinline__ void store_out(const AttnParams& p, long long idx, int d, float x) {
  const long long at = idx * D + d;
  if (!in_idx(at, (long long)p.R * p.Hq * D, p.status)) return;
  if (p.dst_o != nullptr)
    p.dst_o[at] = x;
  else
    put(static_cast<E*>(p.o) + at, x);
}

// The same from the values' sum v under the row's weights.
template <typename E, int D>
__device__ __forceinline__ void finish(const AttnParams& p, long long idx, int d, float v, const Coef& r) {
  float x = v * r.a;
  if (p.pre_o != nullptr && r.b != 0.f) x += __ldcg(p.pre_o + idx * D + d) * r.b;
  store_out<E, D>(p, idx, d, x);
}

__device__ __forceinline__ void finish_lse(const AttnParams& p, long long idx, const Coef& r) {
  if (p.dst_o != nullptr)
    p.dst_lse[idx] = r.lse2;
  else if (p.lse != nullptr)
    p.lse[idx] = r.lse2 * 0.69314718055994530942f;
}

// What the values' sums are kept smaller by. Values may be as large as fp32 holds, so their
// sum under weights of up to 1, before it is divided by the weights', may not be: in the
// 32-bit kernel 2^20 tokens of the largest value stay in range, and the smallest (448 * 2^-100)
// keep 37 bits. The tensor-core kernels' weights hold the values' exponents.
template <typename E>
constexpr float kSumUnit = sizeof(E) == 4 ? 1048576.f : 1.f;

// A slot of the workspace: NR maxima, NR sums, NR x D values.
template <int NR, int D>
__device__ __forceinline__ float* slot_of(const AttnParams& p, int s) {
  return p.part + (long long)s * (NR * (D + 2));
}

// A cu that is no prefix sum of the batch: every row is NaN (by the first `threads` threads of each block).
template <typename E, int D>
__device__ __noinline__ void fill_nan(const AttnParams& p, int block, int blocks, int threads) {
  if (block == 0 && threadIdx.x == 0) atomicOr(p.status, SPEC_DEV_OFFSETS);
  const long long n = (long long)p.R * p.Hq * D;
  const float nan = __int_as_float(0x7fffffff);
  for (long long i = (long long)block * threads + threadIdx.x; i < n; i += (long long)blocks * threads) {
    put(static_cast<E*>(p.o) + i, nan);
    if (p.lse != nullptr && i % D == 0) p.lse[i / D] = nan;
  }
}

// What block `block` of `grid` leaves for attn_merge_kernel about a stretch g that ends the
// block's part of the line (at `end` of `total`).
__device__ __forceinline__ CutRec cut_rec(const Seg& g, int block, int grid, int end, int total) {
  CutRec r{0, g.row0, g.rows, g.h, g.f0, g.bad, total};
  if (g.t0 == 0 && g.n < g.nt) {
    const int last = end + (g.nt - g.n);
    int e = block + 1;
#pragma unroll 1
    while (e < grid && line_at(total, e, grid) < last) ++e;
    r.parts = e - block;
  }
  return r;
}

// ---------------------------------------------------------------------------
// Joins the parts of cut segments, in order: block x takes the segment that begins in block
// x of the attention kernel and goes on, block y 8 of its rows, one a warp. Bound by the
// latency of its loads, so they go out together: 6 us behind 304 blocks of 40 rows, 19 us behind
// 152 of 256 rows, 40 MB (one after another 9 and 21; a call of one token 10.9 -> 9.7 us).
constexpr int kMergeThreads = 256;

template <typename E, int D, int NR>
__global__ void __launch_bounds__(kMergeThreads) attn_merge_kernel(AttnParams p, int grid) {
  griddep_launch();  // (before the wait: the pass over the sequences' own tokens may begin beside the prefix pass)
  griddep_wait();
  const CutRec r = p.cut[blockIdx.x];
  const int i = blockIdx.x, lane = threadIdx.x & 31, c = blockIdx.y * 8 + (threadIdx.x >> 5), f = r.f0 + c;
  if (r.parts == 0 || c >= (p.block_rows > 0 ? p.block_rows : NR) || f >= r.rows * p.G) return;
  // part j: slot 2 i + 1 of the first block, slot 2 (i + j) of the others
  auto part_of = [&](int j) { return slot_of<NR, D>(p, j == 0 ? 2 * i + 1 : 2 * (i + j)); };
  const int some = r.total >= grid ? grid : r.total;  // blocks that have a part of the line
  auto holds = [&](int j) { return i + j < some; };
  // Everything that does not wait for the maxima is loaded at once: the first parts' values, which count only where their
  // sums do not vanish, and the prefix's part.
  constexpr int V = D / 32, kAhead = 4;
  const float ninf = __int_as_float(kNegInfBits);
  const long long idx = (long long)(r.row0 + f / p.G) * p.Hq + r.h * p.G + f % p.G;
  float ahead[kAhead][V], pre[V], pre_lse = ninf;
  auto load = [&](const float* s, float (&x)[V]) {
    if constexpr (V == 4) {
      const float4 y = *reinterpret_cast<const float4*>(s);
      x[0] = y.x, x[1] = y.y, x[2] = y.z, x[3] = y.w;
    } else {
      const float2 y = *reinterpret_cast<const float2*>(s);
      x[0] = y.x, x[1] = y.y;
    }
  };
  auto values = [&](int j) { return part_of(j) + 2 * NR + c * D + lane * V; };
  float mj = ninf, lj = 0.f;  // of part `lane`
  if (lane < r.parts && holds(lane)) {
    mj = part_of(lane)[c];
    lj = part_of(lane)[NR + c];
  }
#pragma unroll
  for (int j = 0; j < kAhead; ++j)
    if (j < r.parts && holds(j)) load(values(j), ahead[j]);
  if (p.pre_o != nullptr) {
    pre_lse = __ldcg(p.pre_lse + idx);
    load(p.pre_o + idx * D + lane * V, pre);
  }
  float m = mj;
  for (int j = lane + 32; j < r.parts; j += 32)
    if (holds(j)) m = fmaxf(m, part_of(j)[c]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
  const float mu = m == ninf ? 0.f : m;
  float l = 0.f, acc[V];
#pragma unroll
  for (int k = 0; k < V; ++k) acc[k] = 0.f;
  auto add = [&](float wt, const float (&x)[V]) {
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] = wt == 0.f ? acc[k] : acc[k] + wt * x[k];
  };
  for (int j0 = 0; j0 < r.parts; j0 += 32) {
    const int j = j0 + lane, cnt = min(32, r.parts - j0);
    if (j0 > 0) {
      lj = 0.f;
      if (j < r.parts && holds(j)) mj = part_of(j)[c], lj = part_of(j)[NR + c];
    }
    const float w = lj != 0.f ? exp2f(mj - mu) : 0.f;
    if (lj != 0.f) l += w * lj;
    if (j0 == 0) {
#pragma unroll
      for (int t = 0; t < kAhead; ++t) add(__shfl_sync(kFull, w, t), ahead[t]);
    }
#pragma unroll 4
    for (int t = j0 == 0 ? kAhead : 0; t < cnt; ++t) {
      const float wt = __shfl_sync(kFull, w, t);
      float x[V];
      if (wt != 0.f) load(values(j0 + t), x);
      add(wt, x);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(kFull, l, o);
  Coef co = row_coef(pre_lse, mu, l, r.bad != 0);
  co.a *= kSumUnit<E>;
#pragma unroll
  for (int k = 0; k < V; ++k) {
    float x = acc[k] * co.a;
    if (p.pre_o != nullptr && co.b != 0.f) x += pre[k] * co.b;
    store_out<E, D>(p, idx, lane * V + k, x);
  }
  if (lane == 0) finish_lse(p, idx, co);
}

// ---------------------------------------------------------------------------
// The 32-bit kernel: fp32 products and sums throughout, for fp32 queries (whose accuracy
// the tensor cores' 16-bit operands would lose). A block of 128 threads holds 8 rows; of a
// tile, a thread computes the scores of one token, then sums the values of 4 elements over
// its share of the tokens. Small calls are bound by the latency of one tile's steps (24 ragged
// sequences x 1-8 rows, head_dim 64, up to 600 tokens and a prefix of 100: 33 us in two passes
// and two joinings), large ones by the fp32 pipe.
template <typename E, int D>
__global__ void __launch_bounds__(128) attn_f32_kernel(AttnParams p) {
  constexpr int NR = kRowsS, KS = D + 16;  // a key's stride: 16 bytes more than its codes, so that 8 lanes hit all banks
  constexpr int NG = 128 / (D / 4);        // token groups of the values' sum
  __shared__ Part s_part;
  __shared__ __align__(16) float sq[NR][D];
  __shared__ __align__(16) uint8_t skv[kTile * KS + kTile * D];
  __shared__ __align__(16) float sp[kTile][NR];
  __shared__ float ss[NR][kTile + 4];
  __shared__ float sx[kTile];
  __shared__ int sbad[kTile];
  __shared__ float sm[NR], sl[NR], sf[NR];
  __shared__ uint64_t s_sees[SPEC_MAX_TREE_NODES];
  static_assert(sizeof(float) * NG * NR * D <= sizeof(skv), "the sums of the token groups fit where the tile was");
  uint8_t* sk = skv;
  uint8_t* svv = skv + kTile * KS;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const float ninf = __int_as_float(kNegInfBits), nan = __int_as_float(0x7fffffff);
  if (p.mask == A_TREE && tid < SPEC_MAX_TREE_NODES) s_sees[tid] = p.sees[tid];
  griddep_wait();
  griddep_launch();
  const Part line = locate_block<NR>(p, s_part);
  if (!line.ok) fill_nan<E, D>(p, blockIdx.x, gridDim.x, 128);
  Place at = line.at;
  int left = line.ok ? line.end - line.begin : 0;
  uint32_t bits = 0;
  if (tid == 0) p.cut[blockIdx.x].parts = 0;
  while (left > 0) {
    const Seg g = next_seg<NR>(p, at, left);
    if (g.n == 0) continue;
    if (left == 0 && tid == 0) p.cut[blockIdx.x] = cut_rec(g, blockIdx.x, gridDim.x, line.end, line.total);
    if (g.bad) bits |= SPEC_DEV_OFFSETS;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < NR * D / 128; ++k) {
      const int e = tid + k * 128, c = e / D, d = e % D, f = g.f0 + c;
      float x = 0.f;
      if (f < g.rows * p.G) {
        const long long a = (long long)(g.row0 + f / p.G) * p.q_row + (long long)(g.h * p.G + f % p.G) * p.q_head + d;
        if constexpr (sizeof(E) == 2)
          x = __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t*>(p.q) + a) << 16);
        else
          x = __ldg(static_cast<const float*>(p.q) + a);
      }
      // an infinite query's scores would be infinities, and -inf stands for a hidden token: the row is to be NaN
      x *= p.c;
      sq[c][d] = fabsf(x) <= 3.402823466e38f ? x : nan;
    }
    if (tid < NR) sm[tid] = ninf, sl[tid] = 0.f;
    float acc[NR][4];
#pragma unroll
    for (int c = 0; c < NR; ++c) acc[c][0] = acc[c][1] = acc[c][2] = acc[c][3] = 0.f;
    const int wi = tid % (D / 4), tg = tid / (D / 4);
    for (int tile = g.t0; tile < g.t0 + g.n; ++tile) {
      // A tile's loads: the page numbers, then what stands there, each all at once (one after another they were most of a
      // tile's time: 24 ragged sequences x up to 8 rows, head_dim 64, up to 600 tokens and a prefix of 100: 36.5 -> 35.3 us).
      constexpr int CH = D / 16, STEPS = CH < 4 ? CH : 4;
      const int t = tile * kTile + tid;
      auto place = [&](int tok) -> long long {  // of a token's vector: -1 past the end, -2 on a bad page
        if (tok >= g.len) return -1;
        const int page = __ldg(g.pages + (tok >> p.page_shift));
        return (unsigned)page < (unsigned)p.num_pages
                   ? (((long long)page * p.Hk + g.h) << p.page_shift) + (tok & ((1 << p.page_shift) - 1))
                   : -2;
      };
      sbad[tid] = 0;
      const long long own = place(t);
      if (own == -2) bits |= SPEC_DEV_PAGE;
      const unsigned kb = own >= 0 ? __ldg(p.k_exp + own) : 0u, vb = own >= 0 ? __ldg(p.v_exp + own) : 0u;
      __syncthreads();
#pragma unroll
      for (int e0 = 0; e0 < CH; e0 += STEPS) {
        long long vec[STEPS];
        uint4 kw[STEPS], vw[STEPS];
#pragma unroll
        for (int i = 0; i < STEPS; ++i) vec[i] = place(tile * kTile + (tid + (e0 + i) * 128) / CH);
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
          kw[i] = vw[i] = make_uint4(0, 0, 0, 0);
          if (vec[i] >= 0) {
            kw[i] = __ldg(reinterpret_cast<const uint4*>(p.k + vec[i] * D) + tid % CH);
            vw[i] = __ldg(reinterpret_cast<const uint4*>(p.v + vec[i] * D) + tid % CH);
          }
        }
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
          // NaN codes of values: zero, and the token marked (0 * NaN must not reach rows that do not see it)
          const int u = (tid + (e0 + i) * 128) / CH;
          uint32_t* w = &vw[i].x;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t mk = __vcmpeq4(w[k] & 0x7f7f7f7fu, 0x7f7f7f7fu);
            if (mk) sbad[u] = 1;
            w[k] &= ~mk;
          }
          *reinterpret_cast<uint4*>(sk + u * KS + tid % CH * 16) = kw[i];
          *reinterpret_cast<uint4*>(svv + u * D + tid % CH * 16) = vw[i];
        }
      }
      __syncthreads();
      {
        float ke = 0.f, ve = 0.f;
        if (own == -2 || sbad[tid]) {
          ke = nan;
        } else if (own >= 0) {
          ke = exp_value(kb);
          ve = exp_value(vb);
          if (ve != ve) ke = nan;
        }
        float s[NR];
#pragma unroll
        for (int c = 0; c < NR; ++c) s[c] = 0.f;
#pragma unroll 4
        for (int ch = 0; ch < D / 4; ++ch) {
          float x[4];
          codes4(*reinterpret_cast<const uint32_t*>(sk + tid * KS + ch * 4), x);
#pragma unroll
          for (int c = 0; c < NR; ++c) {
            const float4 y = *reinterpret_cast<const float4*>(&sq[c][ch * 4]);
            s[c] = fmaf(x[0], y.x, fmaf(x[1], y.y, fmaf(x[2], y.z, fmaf(x[3], y.w, s[c]))));
          }
        }
        const Sight sight = sight_of(p.mask, s_sees, g.rows, g.len, t);
#pragma unroll
        for (int c = 0; c < NR; ++c) ss[c][tid] = sight((g.f0 + c) / p.G) ? s[c] * ke : ninf;
        sx[tid] = ve * (1.f / kSumUnit<E>);
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < NR / 4; ++k) {
        const int c = warp * (NR / 4) + k;
        float x[4], mx = sm[c];
        const float m_old = mx;
#pragma unroll
        for (int u = 0; u < 4; ++u) mx = fmaxf(mx, x[u] = ss[c][u * 32 + lane]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
        const float mu = mx == ninf ? 0.f : mx;
        float sum = 0.f;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float e = exp2f(x[u] - mu);
          sum += e;
          sp[u * 32 + lane][c] = e == 0.f ? 0.f : e * sx[u * 32 + lane];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
        __syncwarp();
        if (lane == 0) {
          const float f = exp2f(m_old - mu);
          sf[c] = f;
          sl[c] = sl[c] * f + sum;
          sm[c] = mx;
        }
        __syncwarp();
      }
      __syncthreads();
#pragma unroll
      for (int c = 0; c < NR; ++c) {
        const float f = sf[c];
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[c][k] *= f;
      }
#pragma unroll 4
      for (int u = tg; u < kTile; u += NG) {
        float x[4];
        codes4(*reinterpret_cast<const uint32_t*>(svv + u * D + wi * 4), x);
        const float4 y0 = *reinterpret_cast<const float4*>(&sp[u][0]), y1 = *reinterpret_cast<const float4*>(&sp[u][4]);
        const float y[NR] = {y0.x, y0.y, y0.z, y0.w, y1.x, y1.y, y1.z, y1.w};
#pragma unroll
        for (int c = 0; c < NR; ++c) {
#pragma unroll
          for (int k = 0; k < 4; ++k) acc[c][k] = fmaf(y[c], x[k], acc[c][k]);
        }
      }
    }
    __syncthreads();
    float* red = reinterpret_cast<float*>(skv);
#pragma unroll
    for (int c = 0; c < NR; ++c)
      *reinterpret_cast<float4*>(red + ((tg * NR + c) * D + wi * 4)) = make_float4(acc[c][0], acc[c][1], acc[c][2], acc[c][3]);
    __syncthreads();
    const bool whole = g.n == g.nt;
    float* slot = whole ? nullptr : slot_of<NR, D>(p, 2 * blockIdx.x + (g.t0 == 0 ? 1 : 0));
    if (!whole && tid < NR) slot[tid] = sm[tid], slot[NR + tid] = sl[tid];
#pragma unroll
    for (int k2 = 0; k2 < NR * D / 128; ++k2) {
      const int e = tid + k2 * 128, c = e / D, d = e % D, f = g.f0 + c;
      float v = 0.f;
#pragma unroll
      for (int k = 0; k < NG; ++k) v += red[(k * NR + c) * D + d];
      if (!whole) {
        slot[2 * NR + e] = v;
      } else if (f < g.rows * p.G) {
        const long long idx = (long long)(g.row0 + f / p.G) * p.Hq + g.h * p.G + f % p.G;
        Coef r = row_coef(p.pre_o != nullptr ? __ldcg(p.pre_lse + idx) : ninf, sm[c] == ninf ? 0.f : sm[c], sl[c], g.bad);
        r.a *= kSumUnit<E>;
        finish<E, D>(p, idx, d, v, r);
        if (d == 0) finish_lse(p, idx, r);
      }
    }
  }
  if (bits) atomicOr(p.status, bits);
}

}  // namespace sv
