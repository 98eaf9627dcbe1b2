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
#pragma once

#include "kernels_kv.cuh"

namespace sv {

constexpr int kSelThreads = 512;
constexpr int kSelPer = 8;       // tokens of a thread and step
constexpr int kSelKeys = 16384;  // keys of a sequence's beginning that stay in shared memory
constexpr int kMoveThreads = 256;
constexpr int kMoveUnroll = 8;

struct EvictParams {
  uint8_t *k, *v, *k_exp, *v_exp;
  float* mass;
  int num_pages, page_shift, Hk;
  int B, pps, new_pps;
  const int32_t *table, *new_table;  // the same in place
  const int32_t* kv_len;
  int budget, sinks, recent;
  int cached_keys;  // keys in shared memory
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
  extern __shared__ uint32_t s_key[];  // cached_keys
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
  for (int t = lo + tid; t < min(hi, p.cached_keys); t += kSelThreads) {
    const long long vec = (((long long)__ldg(pages + (t >> p.page_shift)) * p.Hk + h) << p.page_shift) + (t & mask);
    s_key[t] = in_idx(vec, ((long long)p.num_pages * p.Hk) << p.page_shift, p.status) ? mass_key(__ldcg(p.mass + vec)) : 0u;
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
      const int per = bins / kSelThreads;  // 4, 4, 2
      int c[4], sum = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        c[i] = i < per ? s_hist[bins - 1 - (tid * per + i)] : 0;
        sum += c[i];
      }
      unsigned long long all;
      int before = (int)block_scan((unsigned long long)sum, s_warp, all);
      if (before < need && need <= before + sum) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
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

// blockIdx.x = unit + units * step: units of a head are `slices` pieces of the vectors of the
// keys, as many of the values, and one for exponents and weights; a unit's blocks walk its
// tokens in steps, `steps` of them side by side (1 in place).
struct MoveSplit {
  int units, slices, steps;
};

template <int D>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const __grid_constant__ EvictParams p, MoveSplit m) {
  griddep_wait();
  griddep_launch();
  const int h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x, unit = blockIdx.x % m.units, mask = (1 << p.page_shift) - 1;
  const bool moves = p.new_table != p.table;
  const int32_t* pages = p.table + (long long)b * p.pps;
  const int32_t* new_pages = p.new_table + (long long)b * p.new_pps;
  const int32_t* kept = p.kept + ((long long)b * p.Hk + h) * p.budget;
  const long long places = ((long long)p.num_pages * p.Hk) << p.page_shift;
  auto place = [&](const int32_t* table, int t) -> long long {
    const long long vec = (((long long)__ldg(table + (t >> p.page_shift)) * p.Hk + h) << p.page_shift) + (t & mask);
    return in_idx(vec, places, p.status) ? vec : -1;
  };
  const bool vectors = unit < 2 * m.slices;
  const int lanes = vectors ? D / 16 / m.slices : 1, rows = kMoveThreads / lanes, piece = tid % lanes + (vectors ? unit % m.slices : 0) * lanes;
  uint8_t* const side = unit < m.slices ? p.k : p.v;
  const long long step = (long long)rows * kMoveUnroll;
  for (long long j0 = blockIdx.x / m.units * step; j0 < p.budget; j0 += m.steps * step) {
    int src[kMoveUnroll];
    bool some = false;
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      const long long j = j0 + u * rows + tid / lanes;
      src[u] = j < p.budget ? __ldcg(kept + j) : -1;
      some |= src[u] >= 0;
      if (!moves && src[u] == j) src[u] = -1;  // where it is already
    }
    if (__syncthreads_or(some) == 0) return;  // (past the last that stays)
    if (vectors) {
      uint4 x[kMoveUnroll];
#pragma unroll
      for (int u = 0; u < kMoveUnroll; ++u) {
        const long long at = src[u] >= 0 ? place(pages, src[u]) : -1;
        if (at >= 0) x[u] = __ldcg(reinterpret_cast<const uint4*>(side + at * D) + piece);
      }
      if (!moves) __syncthreads();
#pragma unroll
      for (int u = 0; u < kMoveUnroll; ++u) {
        const long long at = src[u] >= 0 ? place(new_pages, (int)j0 + u * rows + tid / lanes) : -1;
        if (at >= 0) *(reinterpret_cast<uint4*>(side + at * D) + piece) = x[u];
      }
    } else {
      float w[kMoveUnroll];
      uint8_t ke[kMoveUnroll], ve[kMoveUnroll];
#pragma unroll
      for (int u = 0; u < kMoveUnroll; ++u) {
        const long long at = src[u] >= 0 ? place(pages, src[u]) : -1;
        if (at >= 0) {
          w[u] = __ldcg(p.mass + at);
          ke[u] = __ldcg(p.k_exp + at);
          ve[u] = __ldcg(p.v_exp + at);
        }
      }
      if (!moves) __syncthreads();
#pragma unroll
      for (int u = 0; u < kMoveUnroll; ++u) {
        const long long at = src[u] >= 0 ? place(new_pages, (int)j0 + u * rows + tid / lanes) : -1;
        if (at >= 0) {
          p.mass[at] = w[u];
          p.k_exp[at] = ke[u];
          p.v_exp[at] = ve[u];
        }
      }
    }
  }
}

}  // namespace sv
