// Eviction: of each sequence and kv head the heaviest tokens within a budget, kept in their
// order and moved together.
//
// evict_select_kernel  one block a sequence and kv head finds which tokens stay. The weights
//                      as ordered 32-bit keys; the smallest key that stays by three counts of
//                      11, 11 and 10 bits, largest first; then one walk over the tokens in
//                      order: a token's new place is the number of those that stay before it.
//                      Of equal keys at the border the earliest stay, so that the result is
//                      one and the same however the counts are added.
// evict_move_kernel    moves keys, values, exponents and weights. In place a block walks its
//                      tokens from the front, every load of a step before its stores: a token's
//                      new place is never behind its old one, so a step's stores reach no later
//                      step's sources, and blocks that share a head take different bytes of
//                      its vectors. To other pages, every step has a block of its own.
//
// What bounds it: the move HBM, 64 sequences of 1000-8192 tokens x 8 heads of 128, at most 4096 kept,
// to other pages: 161 us for both kernels, of which the selection 24 (counts in shared memory, a
// barrier at each step); 5.8 TB/s over all. In place 216 us for 64 sequences of 8192 (a block waits for
// its loads at each step), 36 us for one (the chain of 16 steps). Few tokens: 8 us, two launches.
#pragma once

#include "kernels_kv.cuh"

namespace sv {

constexpr int kSelThreads = 512;
constexpr int kSelPer = 8;       // tokens of a thread and step
constexpr int kSelKeys = 16384;  // keys of a sequence's beginning that stay in shared memory

struct EvictParams {
  uint8_t *k, *v, *k_exp, *v_exp;
  float* mass;
  int num_pages, page_shift, Hk;
  int B, pps, new_pps;
  const int32_t *table, *new_table;  // the same in place
  const int32_t* kv_len;
  int budget, sinks, recent;
  int cached_keys;  // keys in shared memory (a multiple of 16)
  int wide;         // mass on the 16-byte grid
  int32_t *kept, *kv_len_out;
  uint32_t* status;
};

// Larger weights have larger keys; a NaN is below every number, and the zeros are equal.
__device__ __forceinline__ uint32_t mass_key(float x) {
  if (x != x) return 0u;
  const uint32_t b = __float_as_uint(x + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// The block's exclusive prefix sums of two counts packed in one number; `total` for all.
__device__ __forceinline__ unsigned long long block_scan(unsigned long long x, unsigned long long* s_warp, unsigned long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned long long incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long y = __shfl_up_sync(kFull, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();  // (the sums of a scan before are read)
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  unsigned long long before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kSelThreads / 32; ++w) {
    const unsigned long long y = s_warp[w];
    if (w < warp) before += y;
    all += y;
  }
  total = all;
  return before + incl - x;
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const __grid_constant__ EvictParams p) {
  extern __shared__ __align__(16) uint32_t s_key[];  // cached_keys
  __shared__ int s_hist[2048];
  __shared__ unsigned long long s_warp[kSelThreads / 32];
  __shared__ uint32_t s_digit;
  __shared__ int s_need;
  griddep_wait();
  griddep_launch();
  const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
  const int n = __ldg(p.kv_len + b), mask = (1 << p.page_shift) - 1;
  const int32_t* pages = p.table + (long long)b * p.pps;
  const int32_t* new_pages = p.new_table + (long long)b * p.new_pps;
  const bool moves = p.new_table != p.table;
  int32_t* kept = p.kept + ((long long)b * p.Hk + h) * p.budget;
  uint32_t bits = 0;
  if (n < 0 || (long long)n > ((long long)p.pps << p.page_shift)) {
    bits = SPEC_DEV_OFFSETS;
  } else {
    const int used = (n + mask) >> p.page_shift, fresh = moves ? (min(n, p.budget) + mask) >> p.page_shift : 0;
    bool bad = false;
    for (int i = tid; i < used; i += kSelThreads) bad |= (unsigned)__ldg(pages + i) >= (unsigned)p.num_pages;
    for (int i = tid; i < fresh; i += kSelThreads) bad |= (unsigned)__ldg(new_pages + i) >= (unsigned)p.num_pages;
    if (__syncthreads_or(bad)) bits = SPEC_DEV_PAGE;
  }
  const int stay = bits ? 0 : min(n, p.budget);
  if (tid == 0) {
    if (bits) atomicOr(p.status, bits);
    if (h == 0) p.kv_len_out[b] = bits ? (moves ? 0 : n) : stay;
  }
  if (bits || n <= p.budget) {
    for (int j = tid; j < p.budget; j += kSelThreads) kept[j] = j < stay ? j : -1;
    return;
  }
  const int lo = p.sinks, hi = n - p.recent, take = p.budget - p.sinks - p.recent;  // of the tokens lo .. hi - 1 `take` stay
  auto key_of = [&](int t) -> uint32_t {
    if (t < p.cached_keys) return s_key[t];
    const long long vec = (((long long)__ldg(pages + (t >> p.page_shift)) * p.Hk + h) << p.page_shift) + (t & mask);
    return mass_key(__ldcg(p.mass + vec));
  };
  // the weights of four neighbouring tokens at once (they share a page), all of a thread's on their way together
  const int upto = min(n, p.cached_keys);
  if (p.wide) {
#pragma unroll 4
    for (int t = tid * 4; t < upto; t += kSelThreads * 4) {
      const long long vec = (((long long)__ldg(pages + (t >> p.page_shift)) * p.Hk + h) << p.page_shift) + (t & mask);
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (in_idx(vec, ((long long)p.num_pages * p.Hk) << p.page_shift, p.status)) x = __ldcg(reinterpret_cast<const float4*>(p.mass + vec));
      *reinterpret_cast<uint4*>(s_key + t) = make_uint4(mass_key(x.x), mass_key(x.y), mass_key(x.z), mass_key(x.w));
    }
  } else {
    for (int t = tid; t < upto; t += kSelThreads) {
      const long long vec = (((long long)__ldg(pages + (t >> p.page_shift)) * p.Hk + h) << p.page_shift) + (t & mask);
      s_key[t] = in_idx(vec, ((long long)p.num_pages * p.Hk) << p.page_shift, p.status) ? mass_key(__ldcg(p.mass + vec)) : 0u;
    }
  }
  // the key of the last that stays: its digits from the top, among the keys that share the ones before
  uint32_t border = 0;
  int need = take;  // of the keys that share them, the largest that stay
  constexpr int kShift[3] = {21, 10, 0}, kBits[3] = {11, 11, 10};
  if (take > 0) {
#pragma unroll
    for (int r = 0; r < 3; ++r) {
      const int bins = 1 << kBits[r];
      for (int i = tid; i < bins; i += kSelThreads) s_hist[i] = 0;
      __syncthreads();
      for (int t = lo + tid; t < hi; t += kSelThreads) {
        const uint32_t key = key_of(t);
        if (r == 0 || key >> (kShift[r] + kBits[r]) == border >> (kShift[r] + kBits[r]))
          atomicAdd(&s_hist[(key >> kShift[r]) & (bins - 1)], 1);
      }
      __syncthreads();
      // from the largest digit down: the one that the count of `need` falls into
      constexpr int kMost = 2048 / kSelThreads;
      const int per = bins / kSelThreads;
      int c[kMost], sum = 0;
#pragma unroll
      for (int i = 0; i < kMost; ++i) {
        c[i] = i < per ? s_hist[bins - 1 - (tid * per + i)] : 0;
        sum += c[i];
      }
      unsigned long long all;
      int before = (int)block_scan((unsigned long long)sum, s_warp, all);
      if (before < need && need <= before + sum) {
#pragma unroll
        for (int i = 0; i < kMost; ++i) {
          if (before < need && need <= before + c[i]) {
            s_digit = (uint32_t)(bins - 1 - (tid * per + i));
            s_need = need - before;
          }
          before += c[i];
        }
      }
      __syncthreads();
      border |= s_digit << kShift[r];
      need = s_need;
    }
  }
  // the walk: (surely stays, equal to the border) before each token
  int sure = 0, equal = 0;
  for (int t0 = 0; t0 < n; t0 += kSelThreads * kSelPer) {
    uint32_t key[kSelPer];
    int cs = 0, ce = 0;
    const int first = t0 + tid * kSelPer;
#pragma unroll
    for (int i = 0; i < kSelPer; ++i) {
      const int t = first + i;
      key[i] = 0;
      const bool in = t >= lo && t < hi;
      if (in && take > 0) key[i] = key_of(t);
      const bool s = t < n && (!in || (take > 0 && key[i] > border)), e = in && take > 0 && key[i] == border;
      cs += s;
      ce += e;
    }
    unsigned long long all;
    const unsigned long long before = block_scan((unsigned long long)cs << 32 | (unsigned)ce, s_warp, all);
    int ns = sure + (int)(before >> 32), ne = equal + (int)(before & 0xffffffffu);
#pragma unroll
    for (int i = 0; i < kSelPer; ++i) {
      const int t = first + i;
      const bool in = t >= lo && t < hi;
      const bool s = t < n && (!in || (take > 0 && key[i] > border)), e = in && take > 0 && key[i] == border;
      if (s || (e && ne < need)) {
        const int j = ns + min(ne, need);
        if (in_idx(j, p.budget, p.status)) kept[j] = t;
      }
      ns += s;
      ne += e;
    }
    sure += (int)(all >> 32);
    equal += (int)(all & 0xffffffffu);
  }
}

// A block moves one kv head's tokens in steps of as many as it has threads (128 to other pages, 256 in place; 64 sequences
// to 8192 tokens, half kept, to other pages: 128 163 us, 256 175, 512 186): its threads look the step's places up,
// a token each, and move the tokens' exponents and weights; then D / 16 lanes a vector move the
// keys and the values. blockIdx.x = slice + slices * step: to other pages (PLACE false) every step
// has a block of its own; in place a block walks all of them, and `slices` blocks share a head's
// vectors, a piece each.
template <bool PLACE>
constexpr int kMoveStep = PLACE ? 256 : 128;

template <int D, bool PLACE>
__global__ void __launch_bounds__(kMoveStep<PLACE>) evict_move_kernel(const __grid_constant__ EvictParams p, int slices) {
  constexpr int LANES = D / 16, STEP = kMoveStep<PLACE>, U = LANES;  // U: vectors of a thread on their way
  __shared__ long long s_src[STEP], s_dst[STEP];
  griddep_wait();
  griddep_launch();
  const int h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x, mask = (1 << p.page_shift) - 1;
  const int32_t* pages = p.table + (long long)b * p.pps;
  const int32_t* new_pages = p.new_table + (long long)b * p.new_pps;
  const int32_t* kept = p.kept + ((long long)b * p.Hk + h) * p.budget;
  const long long places = ((long long)p.num_pages * p.Hk) << p.page_shift;
  auto place = [&](const int32_t* table, int t) -> long long {
    const long long vec = (((long long)__ldg(table + (t >> p.page_shift)) * p.Hk + h) << p.page_shift) + (t & mask);
    return in_idx(vec, places, p.status) ? vec : -1;
  };
  const int slice = PLACE ? blockIdx.x % slices : 0, lanes = PLACE ? LANES / slices : LANES;
  const int rows = STEP / lanes, row0 = tid / lanes, piece = slice * lanes + tid % lanes;
  for (int j0 = PLACE ? 0 : blockIdx.x * STEP; j0 < p.budget; j0 += PLACE ? STEP : p.budget) {
    const int j = j0 + tid, t = j < p.budget ? __ldcg(kept + j) : -1;
    long long src = -1, dst = -1;
    if (t >= 0 && !(PLACE && t == j)) {  // (in place: where it is already)
      src = place(pages, t);
      dst = place(new_pages, j);
      if (src < 0 || dst < 0) src = dst = -1;
    }
    s_src[tid] = src;
    s_dst[tid] = dst;
    if (__syncthreads_or(t >= 0) == 0) return;  // (past the last that stays)
    float w;
    uint8_t ke, ve;
    if (src >= 0 && slice == 0) {
      w = __ldcg(p.mass + src);
      ke = __ldcg(p.k_exp + src);
      ve = __ldcg(p.v_exp + src);
    }
    if (!PLACE && src >= 0) {
      p.mass[dst] = w;
      p.k_exp[dst] = ke;
      p.v_exp[dst] = ve;
    }
    // (with slices a step is fewer than U vectors of a thread)
    uint4 x[2][U];
    auto load = [&](int side) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = row0 + u * rows;
        const long long at = r < STEP ? s_src[r] : -1;
        if (at >= 0) x[side][u] = __ldcg(reinterpret_cast<const uint4*>((side ? p.v : p.k) + at * D) + piece);
      }
    };
    auto store = [&](int side) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = row0 + u * rows;
        const long long at = r < STEP ? s_dst[r] : -1;
        if (at >= 0) *(reinterpret_cast<uint4*>((side ? p.v : p.k) + at * D) + piece) = x[side][u];
      }
    };
    if (PLACE) {
      load(0);
      load(1);
      __syncthreads();  // every load of the step before its stores
      store(0);
      store(1);
      if (src >= 0 && slice == 0) {
        p.mass[dst] = w;
        p.k_exp[dst] = ke;
        p.v_exp[dst] = ve;
      }
      __syncthreads();  // (the places are read)
    } else {
      load(0);
      load(1);
      store(0);
      store(1);
    }
  }
}

}  // namespace sv
