// Attention over the 8-bit cache on the fifth-generation tensor cores, for bf16 queries.
//
// A block holds up to NR rows (query rows times the query heads of one kv head) and walks
// 128-token tiles of their keys. Both products have the tokens or the head's elements on
// the 128-lane side, and the few rows on the other: S^T = K q^T (lanes = tokens) and
// O^T = V^T P^T (lanes = elements), so that few rows cost few columns instead of a
// 128-row tile that is mostly empty. Both run on the cache's codes as they are
// (kind::f8f6f4, e4m3 as the first operand): nothing is widened on the way, and a tile
// crosses shared memory once in and once out for each product. What is not 8 bits wide is
// split into 8-bit parts that stand side by side as columns of one MMA, and whose products
// are added:
//
//   queries  a bf16 query is, within its row's power of two, exactly the sum of two e4m3
//            parts (8 significant bits = 4 + 4; elements below 2^-8 of the row's largest
//            keep an absolute 2^-17 of it);
//   weights  a weight is rounded to f16, and every f16 number up to 2^15 is exactly the sum
//            of three e5m2 parts (each the rest of the ones before, scaled by 16 and 256 in
//            columns of its own: 11 bits are 3 + 4 + 4 with the rests' signs, and the last
//            part's smallest step is f16's, 2^-24). The largest weights of a row stand between
//            2^10 and 2^15: a weight keeps f16's 11 bits down to 2^-24 of the largest, then
//            an absolute 2^-35 of it. (e4m3 parts, whose range is short, end 2^-21 below the
//            largest; a long flat tail under one dominant token was lost there.)
//
//   Exponents: a key's is a factor of its token's scores, one lane's constant; a value's is
//   added to the score before the exponential (weights are 2^(x + e - m)), so that the
//   weighted values need no further scaling and no weight over- or underflows where values
//   differ much in size; the sum takes it out again (2^-e).
//
// Eight warps do the softmax: a thread is a token and half of the rows, whose weights sit
// in its registers. The maximum over tokens, which would cross lanes, is needed only when a weight
// would pass 2^15 (the first tile of a stretch, then rarely): the
// reference is not the maximum itself but anything that keeps the weights in range. One
// warp keeps rings of key and value tiles filled (a TMA load a page and operand; pages
// shorter than a tile make several), one issues the MMAs: the next tile's scores while this
// tile's weights are made. Two blocks share an SM, so that one's ends and waits are covered
// by the other.
//
// What bounds it: the cache's bytes where stretches are long (a tile, 32 KB of codes with
// head_dim 128, takes an SM 1270 clocks: 256 sequences x 1 row to 1-8192 tokens 328 us, 98 %
// of a copy's rate), else the instructions of a stretch's beginning and end, as many as three
// tiles': 64 x 6 rows to 6-4096 tokens 57 us (DRAM 66 %).
#pragma once

#include <cuda.h>

#include "kernels_attn.cuh"

namespace sv {

constexpr int kTcThreads = 320;        // eight softmax warps, one for copies, one for MMAs
constexpr int kTcSoft = 256;
constexpr int kSegRing = 8;            // more stretches than tiles can be in the rings
constexpr int kTcPollLimit = 1 << 18;  // bounded waits (SPEC_DEV_TIMEOUT): about a second
constexpr float kTop = 10.f;           // a fresh reference puts the largest weight at 2^10 ...
constexpr float kOver = 15.f;          // ... and is renewed when one would pass 2^15 (f16 and e5m2 end just below 2^16)
constexpr int kSumShift = 6;           // sums of 2^(x - m) are kept 2^6 smaller: values of exponent -100 leave them in range

template <int D, int NR>
struct TcShape {
  // Columns that the rows stand in: each half of the softmax warps has half of them, from a multiple of 8 on (a weights'
  // store and a load of tensor memory take 8); of 24 rows in 32 columns 4 a half are computed by the MMAs and read by none.
  static constexpr int NH = NR / 2, NC = 2 * ((NH + 7) / 8 * 8);
  static constexpr int kHalves = 128 / D;                    // token halves stacked on the lanes of O^T
  static constexpr int kNK = D == 64 ? 5 : NC <= 32 ? 3 : 2; // tiles of keys in the ring
  static constexpr int kNV = D == 64 ? 5 : 2;                // tiles of values
  static constexpr int kTileBytes = kTile * D;               // codes of one operand
  static constexpr int kChunk = kTile * 16;                  // 16 columns of the weights' parts: a 16-byte row a token
  static constexpr int kP = 3 * NC / 16 * kChunk;
  static constexpr int kQ = 2 * NC * D;                      // high and low parts of the queries
  // offsets from a 1024-byte boundary
  static constexpr int oK = 0;
  static constexpr int oV = oK + kNK * kTileBytes;
  static constexpr int oQ = oV + kNV * kTileBytes;
  static constexpr int oP = oQ + kQ;
  static constexpr int oE = oP + kP;                         // exponent bytes of a tile: keys', values'
  static constexpr int kSmem = oE + kNK * 2 * kTile + 1024;
  static constexpr uint64_t kLayoutD = D == 128 ? 2 : 4;     // descriptor: 128- or 64-byte swizzle
  // tensor memory: scores of the two parts, then the values' sums of the three
  static constexpr int cO = 2 * NC, cHalf = 3 * NC;
  static_assert(cO + kHalves * cHalf <= 256, "two blocks share the tensor memory");
  static_assert((kHalves == 2 ? NR * D * 4 : 0) + NR * D * 2 <= kP, "sums pass through the weights' memory");
  static_assert(kSmem <= 107 * 1024, "two blocks share the shared memory");
};

// ---- tcgen05 wrappers -------------------------------------------------------

// Shared-memory matrix descriptor without its address (low bits) and leading stride
// (bits 16-29): stride between groups of eight rows, swizzle (2: 128 bytes, 4: 64 bytes).
__host__ __device__ constexpr uint64_t mma_desc_hi(uint32_t sbo, uint64_t layout) {
  return (uint64_t)(sbo >> 4) << 32 | 1ull << 46 | layout << 61;
}
// Instruction descriptor: fp32 accumulator, e4m3 by e4m3 (or e5m2), M = 128.
__host__ __device__ constexpr uint32_t mma_idesc(int n, bool mn_major, bool b_e5m2) {
  return 1u << 4 | (b_e5m2 ? 1u << 10 : 0u) | (mn_major ? 3u << 15 : 0u) | (uint32_t)(n >> 3) << 17 | 8u << 24;
}
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_ld8(uint32_t a, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(a));
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool elect() {  // one lane of a converged warp
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r)::"memory");
  return r != 0;
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void bar_sync(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }
__device__ __forceinline__ bool bar_or(int id, int n, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
      "bar.red.or.pred p, %2, %3, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)v), "r"(id), "r"(n)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void tma_page(uint32_t dst, const CUtensorMap* map, int tok, int h, int page, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
          dst),
      "l"(map), "r"(0), "r"(tok), "r"(h), "r"(page), "r"(bar)
      : "memory");
}
// A bounded wait. Once one gives up, the block's later waits return at once: the loops run
// to their end (every address they form is in range whatever the data), and the status
// word says that the call's results are not to be used.
__device__ __noinline__ void tc_wait_long(uint32_t bar, unsigned parity, volatile int* gave_up, uint32_t* status) {
  for (int it = 0; !mbar_try_wait(bar, parity); ++it) {
    if (*gave_up) return;
    if (it == kTcPollLimit) {
      *gave_up = 1;
      atomicOr(status, SPEC_DEV_TIMEOUT);
      return;
    }
  }
}
__device__ __forceinline__ void tc_wait_one(uint32_t bar, unsigned parity, volatile int* gave_up, uint32_t* status) {
  if (!mbar_try_wait(bar, parity)) tc_wait_long(bar, parity, gave_up, status);
}
// The same by a whole warp, which goes on together (tensor-memory accesses and elections want it converged).
__device__ __forceinline__ void tc_wait(uint32_t bar, unsigned parity, volatile int* gave_up, uint32_t* status) {
  tc_wait_one(bar, parity, gave_up, status);
  __syncwarp();
}

// ---- arithmetic on pairs of floats ------------------------------------------
typedef unsigned long long f2;
__device__ __forceinline__ f2 pack(float a, float b) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack(f2 v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint32_t half2_of(float a, float b) {  // a in the low half
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
// Four f16 values rounded to e4m3 codes (in order from the low byte), and what those codes
// are as f16. The codes stay 16-bit registers until they are joined: a conversion packs its
// result beside another's, while a zero-extended one costs an instruction of its own.
__device__ __forceinline__ uint32_t narrow4(uint32_t h0, uint32_t h1) {
  uint32_t r;
  asm("{\n\t.reg .b16 a, b;\n\tcvt.rn.satfinite.e4m3x2.f16x2 a, %1;\n\tcvt.rn.satfinite.e4m3x2.f16x2 b, %2;\n\t"
      "mov.b32 %0, {a, b};\n\t}"
      : "=r"(r)
      : "r"(h0), "r"(h1));
  return r;
}
__device__ __forceinline__ uint32_t narrow4(uint32_t h0, uint32_t h1, uint32_t& w0, uint32_t& w1) {
  uint32_t r;
  asm("{\n\t.reg .b16 a, b;\n\tcvt.rn.satfinite.e4m3x2.f16x2 a, %3;\n\tcvt.rn.satfinite.e4m3x2.f16x2 b, %4;\n\t"
      "mov.b32 %0, {a, b};\n\tcvt.rn.f16x2.e4m3x2 %1, a;\n\tcvt.rn.f16x2.e4m3x2 %2, b;\n\t}"
      : "=r"(r), "=&r"(w0), "=r"(w1)
      : "r"(h0), "r"(h1));
  return r;
}
// The same to e5m2 codes.
__device__ __forceinline__ uint32_t narrow4_e5(uint32_t h0, uint32_t h1) {
  uint32_t r;
  asm("{\n\t.reg .b16 a, b;\n\tcvt.rn.satfinite.e5m2x2.f16x2 a, %1;\n\tcvt.rn.satfinite.e5m2x2.f16x2 b, %2;\n\t"
      "mov.b32 %0, {a, b};\n\t}"
      : "=r"(r)
      : "r"(h0), "r"(h1));
  return r;
}
__device__ __forceinline__ uint32_t narrow4_e5(uint32_t h0, uint32_t h1, uint32_t& w0, uint32_t& w1) {
  uint32_t r;
  asm("{\n\t.reg .b16 a, b;\n\tcvt.rn.satfinite.e5m2x2.f16x2 a, %3;\n\tcvt.rn.satfinite.e5m2x2.f16x2 b, %4;\n\t"
      "mov.b32 %0, {a, b};\n\tcvt.rn.f16x2.e5m2x2 %1, a;\n\tcvt.rn.f16x2.e5m2x2 %2, b;\n\t}"
      : "=r"(r), "=&r"(w0), "=r"(w1)
      : "r"(h0), "r"(h1));
  return r;
}
// 16 * (a - b) of f16 pairs: exact where b is a rounded to a part's 3 bits (the difference first: 16 a may pass f16's range)
__device__ __forceinline__ uint32_t rest16(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("{\n\t.reg .b32 t;\n\tsub.rn.f16x2 t, %1, %2;\n\tmul.rn.f16x2 %0, t, %3;\n\t}" : "=r"(r) : "r"(a), "r"(b), "r"(0x4c004c00u));
  return r;
}

__device__ __forceinline__ void tc_ld4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}
__device__ __forceinline__ void tc_st4(uint32_t a, const uint32_t (&r)[4]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%4], {%0,%1,%2,%3};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(a)
               : "memory");
}
// Four columns of the values' sums: the three parts' accumulators joined.
template <int NC>
__device__ __forceinline__ void tc_sum_parts(uint32_t at, float (&o)[4]) {
  uint32_t a[4], b[4], c[4];
  tc_ld4(at, a);
  tc_ld4(at + NC, b);
  tc_ld4(at + 2 * NC, c);
  tc_wait_ld();
#pragma unroll
  for (int j = 0; j < 4; ++j)
    o[j] = fmaf(fmaf(__uint_as_float(c[j]), 0.0625f, __uint_as_float(b[j])), 0.0625f, __uint_as_float(a[j]));
}

template <int D, int NR>
struct TcShared {
  using T = TcShape<D, NR>;
  uint64_t k_full[T::kNK], k_free[T::kNK], v_full[T::kNV], v_free[T::kNV], q_full, drained, s_full, s_free, p_full, o_done;
  uint64_t seg_full[kSegRing];
  Seg seg[kSegRing];                // the block's stretches, as the copying warp comes to them; n = 0: no more, -1: a bad cu
  uint32_t tmem;
  int gave_up;
  uint32_t bad_pages[T::kNK];
  uint64_t sees[SPEC_MAX_TREE_NODES];
  // Of a tile with masked places: the token's values hold a NaN code. Of the tile before as well: the second half of the
  // warps may still read that when the first half comes to this one, while the one before it is behind both (o_done).
  uint8_t nan_code[2][kTile];
  struct Rows {                     // of a stretch's rows
    alignas(16) float rq[NR];       // the factor of the scores: scale * log2(e) * the row's power of two
    alignas(16) int row[NR];        // query row of a flat row
    alignas(16) float neg_m[NR];    // the reference, negated
    alignas(16) int idx[NR];        // row * query heads + head, -1 past the last
  } rows[2];                        // the next stretch's queries are staged before this one's end
  alignas(16) float delta[NR];      // its last change, and 2^that
  alignas(16) float factor[NR];
  float red[4][NR];                 // of the warps of a token each: maxima of the columns
  alignas(16) float coef[2][NR];    // weights of a row's values and of the prefix's part
};

// Queries of a stretch staged for the scores' MMA: TPR threads a row find its power of two
// and write its two parts, rows of D bytes whose 16-byte chunks are exchanged as the swizzle
// has them. (Loops kept short: what runs once a stretch should not push the tiles' loop out
// of the instruction caches.)
template <int D, int NR>
__device__ __forceinline__ void stage_queries(const AttnParams& p, const Seg& g, typename TcShared<D, NR>::Rows& rows, uint8_t* q, int t) {
  constexpr int TPR = NR > 32 ? 4 : 8, E = D / TPR, NH = TcShape<D, NR>::NH, NC = TcShape<D, NR>::NC;
  const int c = t / TPR, part = t % TPR, f = g.f0 + c;
  if (c < NR) {  // (whole warps)
    const int i = f / p.G, hq = g.h * p.G + f - i * p.G, idx = (g.row0 + i) * p.Hq + hq;
    const bool here = f < g.rows * p.G;
    const uint16_t* src = static_cast<const uint16_t*>(p.q) + (long long)(g.row0 + i) * p.q_row + (long long)hq * p.q_head + part * E;
    const bool vec = ((uintptr_t)src & 15) == 0;
    uint4 x[E / 8];
#pragma unroll
    for (int k = 0; k < E / 8; ++k) x[k] = make_uint4(0, 0, 0, 0);
    if (here && vec) {
#pragma unroll
      for (int k = 0; k < E / 8; ++k) x[k] = __ldg(reinterpret_cast<const uint4*>(src) + k);
    } else if (here) {
#pragma unroll
      for (int k = 0; k < E / 8; ++k) {
        uint32_t* w = &x[k].x;
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = (uint32_t)__ldg(src + 8 * k + 2 * j) | (uint32_t)__ldg(src + 8 * k + 2 * j + 1) << 16;
      }
    }
    // the largest magnitude, by its bits (a NaN or an infinity is above every finite one)
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < E / 8; ++k)
      top = __vmaxu2(__vmaxu2(top, __vmaxu2(x[k].x & 0x7fff7fffu, x[k].y & 0x7fff7fffu)),
                     __vmaxu2(x[k].z & 0x7fff7fffu, x[k].w & 0x7fff7fffu));
    top = max(top & 0xffffu, top >> 16);
#pragma unroll
    for (int o = 1; o < TPR; o <<= 1) top = max(top, __shfl_xor_sync(kFull, top, o));
    const bool bad = top >= 0x7f80u;
    const int e = max((int)(top >> 7) - 127, -100) - 7;  // the largest element comes to [128, 256)
    const float inv = bad ? 0.f : __int_as_float((127 - e) << 23);
    if (part == 0) {
      rows.rq[c] = bad ? __int_as_float(0x7fffffff) : p.c * __int_as_float((e + 127) << 23);
      rows.row[c] = i;
      rows.idx[c] = here ? idx : -1;
      rows.neg_m[c] = 0.f;
    }
    const int rh = c < NH ? c : c - NH + NC / 2, rl = NC + rh;
#pragma unroll
    for (int k = 0; k < E / 8; ++k) {
      const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
      uint32_t hi[2], lo[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        // scaled to [0, 256) an element is exact in f16 (8 bits) down to 2^-17 of it
        uint32_t h[2], c1[2];
#pragma unroll
        for (int i2 = 0; i2 < 2; ++i2) {
          const uint32_t u = w[2 * j + i2];
          h[i2] = bad ? 0u : half2_of(__uint_as_float(u << 16) * inv, __uint_as_float(u & 0xffff0000u) * inv);
        }
        hi[j] = narrow4(h[0], h[1], c1[0], c1[1]);
#pragma unroll
        for (int i2 = 0; i2 < 2; ++i2) asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(h[i2]) : "r"(c1[i2]));
        lo[j] = narrow4(h[0], h[1]);
      }
      const int at = part * E + k * 8, chunk = at >> 4;
      const int ch_h = D == 128 ? chunk ^ (rh & 7) : chunk ^ ((rh >> 1) & 3);
      const int ch_l = D == 128 ? chunk ^ (rl & 7) : chunk ^ ((rl >> 1) & 3);
      *reinterpret_cast<uint2*>(q + rh * D + ch_h * 16 + (at & 15)) = make_uint2(hi[0], hi[1]);
      *reinterpret_cast<uint2*>(q + rl * D + ch_l * 16 + (at & 15)) = make_uint2(lo[0], lo[1]);
    }
  }
}

template <int D, int NR>
__global__ void __launch_bounds__(kTcThreads, 2)
attn_tc_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap map_k,
               const __grid_constant__ CUtensorMap map_v) {
  using T = TcShape<D, NR>;
  constexpr int NK = T::kNK, NV = T::kNV, kHalves = T::kHalves;
  extern __shared__ uint8_t dyn[];
  __shared__ TcShared<D, NR> sh;
  const uint32_t dyn_raw = (uint32_t)__cvta_generic_to_shared(dyn);
  const uint32_t base = (dyn_raw + 1023u) & ~1023u;
  uint8_t* const mem = dyn + (base - dyn_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto bar = [](const uint64_t& b) { return (uint32_t)__cvta_generic_to_shared(&b); };
  volatile int* gave_up = &sh.gave_up;

  if (tid == 0) {
    for (int i = 0; i < NK; ++i) {
      mbar_init(bar(sh.k_full[i]), 1);
      mbar_init(bar(sh.k_free[i]), 9);  // the scores' MMA, and the softmax warps (exponents)
    }
    for (int i = 0; i < NV; ++i) {
      mbar_init(bar(sh.v_full[i]), 1);
      mbar_init(bar(sh.v_free[i]), 1);
    }
    for (int i = 0; i < kSegRing; ++i) mbar_init(bar(sh.seg_full[i]), 1);
    mbar_init(bar(sh.q_full), kTcSoft);
    mbar_init(bar(sh.drained), 1);
    mbar_init(bar(sh.s_full), 1);
    mbar_init(bar(sh.s_free), 8);
    mbar_init(bar(sh.p_full), 8);
    mbar_init(bar(sh.o_done), 1);
    sh.gave_up = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (p.mask == A_TREE && tid < SPEC_MAX_TREE_NODES) sh.sees[tid] = p.sees[tid];
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 256;" ::"r"(
                     (uint32_t)__cvta_generic_to_shared(&sh.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    tc_before();
  }
  // Behind a prefix pass this one needs what that left only where rows are joined. It may begin
  // once the kernel before it has begun, and that one only after the prefix pass had waited for
  // everything before the call; so the wait for the prefix's part comes before the first join.
  if (!p.late_wait) griddep_wait();
  griddep_launch();
  __syncthreads();
  tc_after();
  const uint32_t tmem = sh.tmem;

  if (warp == 8) {
    // ---- the rings of tiles ----
    int gi = 0, ns = 0;
    uint32_t bits = 0;
    const Part line = locate<NR>(p, blockIdx.x, gridDim.x);
    Place at = line.at;
    int left = line.ok ? line.end - line.begin : 0;
    const int psz = 1 << p.page_shift, box = min(psz, kTile), np = kTile / box;
    const bool bulk = psz >= 64;
    if (lane == 0) p.cut[blockIdx.x].parts = 0;
    while (left > 0) {
      const Seg g = next_seg<NR>(p, at, left);
      if (g.n == 0) continue;
      if (g.bad) bits |= SPEC_DEV_OFFSETS;
      if (lane == 0) {
        if (left == 0) p.cut[blockIdx.x] = cut_rec(g, blockIdx.x, gridDim.x, line.end, line.total);
        // the stretch that had this place is read: its tiles left the rings before the ones in front of this one's came in
        sh.seg[ns % kSegRing] = g;
        mbar_arrive(bar(sh.seg_full[ns % kSegRing]));
      }
      ++ns;
      // the stretch's queries on their way to the L2 cache while the ones before are worked on
      for (int c = lane; c < NR && g.f0 + c < g.rows * p.G; c += 32) {
        const int f = g.f0 + c, i = f / p.G;
        const uint16_t* src = static_cast<const uint16_t*>(p.q) + (long long)(g.row0 + i) * p.q_row + (long long)(g.h * p.G + f - i * p.G) * p.q_head;
        asm volatile("prefetch.global.L2 [%0];" ::"l"(src));
        if (D == 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(src + 64));
      }
      auto page_of = [&](int tile) -> int {  // of this lane's part of a tile
        const int t = tile * kTile + lane * box;
        return lane < np && tile < g.t0 + g.n && t < g.len ? __ldg(g.pages + (t >> p.page_shift)) : -2;
      };
      // The exponents of a tile: by a bulk copy a page, or, where pages are small and that would be as many operations as the
      // codes take, by ordinary loads a tile ahead: lane l holds those of tokens 8 (l % 16) .. + 7, the keys' in the lower half
      // of the warp, the values' in the upper. (32 x 13 rows, head_dim 64, pages of 16: 36.4 -> 32.6 us; with pages of 64 the
      // warp would stand waiting for them: 256 x 1 row to 8192 330 -> 357 us.)
      const uint8_t* const exps = (lane < 16 ? p.k_exp : p.v_exp) + ((long long)g.h << p.page_shift);
      auto exps_of = [&](int tile, int page) -> uint2 {
        if (bulk) return make_uint2(0, 0);
        const int t = (lane & 15) * 8, mine = __shfl_sync(kFull, page, t / box);
        if ((unsigned)mine >= (unsigned)p.num_pages) return make_uint2(0, 0);
        return __ldcg(reinterpret_cast<const uint2*>(exps + (((long long)mine * p.Hk) << p.page_shift) + ((tile * kTile + t) & (psz - 1))));
      };
      int page = page_of(g.t0), next = page_of(g.t0 + 1);
      uint2 e = exps_of(g.t0, page);
      for (int k = 0; k < g.n; ++k, ++gi) {
        const int sk = gi % NK, sv = gi % NV, tile = g.t0 + k;
        const int after = page_of(tile + 2);
        const uint2 e_next = exps_of(tile + 1, next);
        const bool there = lane < np && tile * kTile + lane * box < g.len;
        const bool good = there && (unsigned)page < (unsigned)p.num_pages;
        const unsigned bad = __ballot_sync(kFull, there && !good), cnt = __popc(__ballot_sync(kFull, good));
        if (bad) bits |= SPEC_DEV_PAGE;
        const int tok = (tile * kTile + lane * box) & (psz - 1);
        const uint32_t bk = bar(sh.k_full[sk]), bv = bar(sh.v_full[sv]);
        if (gi >= NK) tc_wait(bar(sh.k_free[sk]), (gi / NK - 1) & 1, gave_up, p.status);
        if (good) tma_page(base + T::oK + sk * T::kTileBytes + lane * box * D, &map_k, tok, g.h, page, bk);
        if (!bulk) {
          *reinterpret_cast<uint2*>(mem + T::oE + sk * 2 * kTile + lane * 8) = e;
        } else if (good) {
          const long long vec = (((long long)page * p.Hk + g.h) << p.page_shift) + tok;
          bulk_copy(base + T::oE + sk * 2 * kTile + lane * box, p.k_exp + vec, box, bk);
          bulk_copy(base + T::oE + sk * 2 * kTile + kTile + lane * box, p.v_exp + vec, box, bk);
        }
        if (lane == 0) sh.bad_pages[sk] = bad;
        __syncwarp();
        if (lane == 0) mbar_expect_arrive(bk, cnt * (uint32_t)(box * (bulk ? D + 2 : D)));
        if (gi >= NV) tc_wait(bar(sh.v_free[sv]), (gi / NV - 1) & 1, gave_up, p.status);
        if (good) tma_page(base + T::oV + sv * T::kTileBytes + lane * box * D, &map_v, tok, g.h, page, bv);
        if (lane == 0) mbar_expect_arrive(bv, cnt * (uint32_t)(box * D));
        __syncwarp();
        page = next;
        next = after;
        e = e_next;
      }
    }
    if (lane == 0) {
      sh.seg[ns % kSegRing].n = line.ok ? 0 : -1;
      mbar_arrive(bar(sh.seg_full[ns % kSegRing]));
    }
    if (bits) atomicOr(p.status, bits);
    // no copy is left in flight when the block ends, even after a wait that gave up
    for (int i = 0; i < NK; ++i)
      for (int it = 0; gi > i && it < kTcPollLimit && !mbar_try_wait(bar(sh.k_full[i]), ((gi - 1 - i) / NK) & 1); ++it) {
      }
    for (int i = 0; i < NV; ++i)
      for (int it = 0; gi > i && it < kTcPollLimit && !mbar_try_wait(bar(sh.v_full[i]), ((gi - 1 - i) / NV) & 1); ++it) {
      }
  } else if (warp == 9) {
    // ---- the MMAs: scores of the next tile, then weighted values of this one ----
    // The whole warp walks the tiles, so that descriptors and addresses stay warp-uniform; one elected lane issues.
    constexpr uint32_t id_s = mma_idesc(2 * T::NC, false, false), id_o = mma_idesc(3 * T::NC, true, true);
    constexpr uint64_t hi_d = mma_desc_hi(8 * D, T::kLayoutD);                  // codes and queries: rows of D bytes
    constexpr uint64_t lbo_v = (uint64_t)(kTile / 2 * 64 >> 4) << 16;           // head_dim 64: to the second 64 tokens
    constexpr uint64_t hi_p = mma_desc_hi(T::kChunk, 0) | (uint64_t)(128 >> 4) << 16;  // weights: 8 tokens, then 16 columns on
    const uint32_t tm = __shfl_sync(kFull, tmem, 0);
    int gi = 0;
    for (int ns = 0;; ++ns) {
      tc_wait(bar(sh.seg_full[ns % kSegRing]), (ns / kSegRing) & 1, gave_up, p.status);
      const int n = __shfl_sync(kFull, *gave_up ? 0 : sh.seg[ns % kSegRing].n, 0);
      if (n <= 0) break;
      tc_wait(bar(sh.q_full), ns & 1, gave_up, p.status);
#pragma unroll 1
      for (int k = -1; k < n; ++k) {
        if (k + 1 < n) {
          const int i = gi + k + 1, st = i % NK;
          if (i > 0) tc_wait(bar(sh.s_free), (i - 1) & 1, gave_up, p.status);
          tc_wait(bar(sh.k_full[st]), (i / NK) & 1, gave_up, p.status);
          __syncwarp();
          tc_after();
          if (elect()) {
            const uint32_t a = (base + T::oK + st * T::kTileBytes) >> 4, b = (base + T::oQ) >> 4;
#pragma unroll
            for (int s = 0; s < D / 32; ++s) mma_f8(tm, hi_d | (a + s * 2), hi_d | (b + s * 2), id_s, s > 0);
            mma_commit(bar(sh.s_full));
            mma_commit(bar(sh.k_free[st]));
          }
          __syncwarp();
        }
        if (k < 0) continue;
        const int i = gi + k, st = i % NV;
        tc_wait(bar(sh.v_full[st]), (i / NV) & 1, gave_up, p.status);
        tc_wait(bar(sh.p_full), i & 1, gave_up, p.status);
        __syncwarp();
        tc_after();
        if (elect()) {
          const uint32_t a = (base + T::oV + st * T::kTileBytes) >> 4, b = (base + T::oP) >> 4, d = tm + T::cO;
          const uint32_t more = k > 0;
          // head_dim 64: 64 tokens' elements, then the next 64 tokens', make the 128 lanes; each half has its own weights
#pragma unroll
          for (int hf = 0; hf < kHalves; ++hf) {
#pragma unroll
            for (int s = 0; s < kTile / kHalves / 32; ++s)
              mma_f8(d + hf * T::cHalf, hi_d | lbo_v | (a + s * (32 * D >> 4)), hi_p | (b + hf * (1024 >> 4) + s * (512 >> 4)),
                     id_o, s > 0 ? 1u : more);
          }
          mma_commit(bar(sh.o_done));
          mma_commit(bar(sh.v_free[st]));
        }
        __syncwarp();
      }
      gi += n;
    }
    // no MMA is left in flight when the block ends, even after a wait that gave up
    if (elect()) mma_commit(bar(sh.drained));
    __syncwarp();
    for (int it = 0; it < kTcPollLimit && !mbar_try_wait(bar(sh.drained), 0); ++it) {
    }
  } else {
    // ---- softmax: thread = token (lane of S^T) and element (lane of O^T), half of the columns ----
    constexpr int NH = T::NH, NC = T::NC;
    constexpr float kSumScale = 1.f / (1 << kSumShift);
    const int t = tid & 127, wl = warp & 3, c0 = (warp >> 2) * NH, cc = (warp >> 2) * (NC / 2);  // its first row, first column
    const int half_bar = 2 + (warp >> 2);  // the columns' halves have references of their own and run on their own
    const uint32_t lanes = (uint32_t)(wl * 32) << 16;
    const uint32_t tS = tmem + lanes + cc, tO = tmem + lanes + T::cO + (kHalves == 2 && wl >= 2 ? T::cHalf : 0) + cc;
    uint8_t* const pw = mem + T::oP + t * 16;
    const float nan = __int_as_float(0x7fffffff), ninf = __int_as_float(kNegInfBits);
    int gi = 0;
    f2 l2[NH / 2];
    // Stretch ns's queries to the MMA warp, if it is one (false: no more stretches, also after a wait that gave up). The
    // buffer's last reader, the scores of the last tile of the stretch before, is done.
    auto begin = [&](int ns) -> bool {
      tc_wait(bar(sh.seg_full[ns % kSegRing]), (ns / kSegRing) & 1, gave_up, p.status);
      const Seg& g = sh.seg[ns % kSegRing];
      if (bar_or(1, kTcSoft, g.n <= 0 || *gave_up)) return false;  // (all threads alike)
      stage_queries<D, NR>(p, g, sh.rows[ns & 1], mem + T::oQ, tid);
      fence_async();
      mbar_arrive(bar(sh.q_full));
      return true;
    };
    bool more = begin(0);
    if (!more) {
      if (p.late_wait) griddep_wait();
      if (sh.seg[0].n < 0 && !*gave_up) fill_nan<uint16_t, D>(p, blockIdx.x, gridDim.x, kTcSoft);
    }
    bar_sync(1, kTcSoft);  // what was staged is seen by all
    for (int ns = 0; more; ++ns) {
      const Seg g = sh.seg[ns % kSegRing];
      auto& rows = sh.rows[ns & 1];
#pragma unroll
      for (int i = 0; i < NH / 2; ++i) l2[i] = 0ull;
      for (int k = 0; k < g.n; ++k, ++gi) {
        const int sk = gi % NK, tile = g.t0 + k, tok = tile * kTile + t;
        const bool first = k == 0;
        const bool masked = p.mask == A_ALL ? tile * kTile + kTile > g.len : tile * kTile + kTile - 1 > g.len - g.rows;
        tc_wait(bar(sh.k_full[sk]), (gi / NK) & 1, gave_up, p.status);
        const bool live = tok < g.len;
        const unsigned kb = mem[T::oE + sk * 2 * kTile + t], vb = mem[T::oE + sk * 2 * kTile + kTile + t];
        bool hurt = (sh.bad_pages[sk] >> (t >> min(p.page_shift, 7))) & 1;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(sh.k_free[sk]));
        hurt |= kb == kNanExp || vb == kNanExp;
        if (masked) {
          // what no row sees of this token's values is made zero, a NaN code too: 0 * NaN must not reach other rows;
          // the token is marked for the rows that see it
          const int sv = gi % NV;
          if (c0 == 0) {
            tc_wait(bar(sh.v_full[sv]), (gi / NV) & 1, gave_up, p.status);
            uint4* src = reinterpret_cast<uint4*>(mem + T::oV + sv * T::kTileBytes + t * D);
            uint32_t code = 0;
#pragma unroll
            for (int ch = 0; ch < D / 16; ++ch) {
              const uint4 v = src[(ch ^ t) & (D / 16 - 1)];
              code |= ((v.x & 0x7f7f7f7fu) + 0x01010101u) | ((v.y & 0x7f7f7f7fu) + 0x01010101u) |
                      ((v.z & 0x7f7f7f7fu) + 0x01010101u) | ((v.w & 0x7f7f7f7fu) + 0x01010101u);
            }
            const bool nan_here = code & 0x80808080u;
            if (!live || hurt || nan_here) {
#pragma unroll 1
              for (int ch = 0; ch < D / 16; ++ch) src[(ch ^ t) & (D / 16 - 1)] = make_uint4(0, 0, 0, 0);
            }
            sh.nan_code[gi & 1][t] = nan_here;
          }
          bar_sync(1, kTcSoft);
          hurt |= sh.nan_code[gi & 1][t] != 0;
        }
        const bool fine = live && !hurt;
        const float ks = !live ? 0.f : hurt ? nan : exp_value(kb);
        const float ev = fine ? (float)((int)vb - kExpBias) : 0.f;
        const float isv = fine ? __int_as_float((2 * kExpBias - (int)vb) << 23) * kSumScale : 1.f;
        const f2 ks2 = pack(ks, ks), ev2 = pack(ev, ev), isv2 = pack(isv, isv);
        uint32_t sight = ~0u;  // bit c: the row of column c0 + c sees this token
        if (masked) {
          const Sight sees = sight_of(p.mask, sh.sees, g.rows, g.len, tok);
          // rows come in order, G columns each: the first column that sees the token
          const int from = min(max((long long)sees.from * p.G - g.f0 - c0, 0ll), 32ll);
          sight = from >= 32 ? 0u : ~0u << from;
          if (p.mask == A_TREE && sees.nodes != ~0ull) {
#pragma unroll 1
            for (int c = 0; c < NH; ++c)
              if (!sees(rows.row[c0 + c])) sight &= ~(1u << c);
          }
        }
        // scores
        tc_wait(bar(sh.s_full), gi & 1, gave_up, p.status);
        tc_after();
        f2 x[NH / 2];
        float most = ninf;
        uint32_t hi[(NH + 7) / 8][8], lo[(NH + 7) / 8][8];
#pragma unroll
        for (int i = 0; i < NH / 8; ++i) {
          tc_ld8(tS + i * 8, hi[i]);
          tc_ld8(tS + NC + i * 8, lo[i]);
        }
        if (NH % 8) {
          tc_ld4(tS + NH / 8 * 8, reinterpret_cast<uint32_t(&)[4]>(hi[NH / 8]));
          tc_ld4(tS + NC + NH / 8 * 8, reinterpret_cast<uint32_t(&)[4]>(lo[NH / 8]));
        }
        tc_wait_ld();
#pragma unroll
        for (int c = 0; c < NH; c += 4) {
          const float4 rq = *reinterpret_cast<const float4*>(&rows.rq[c0 + c]);
          const float4 nm = *reinterpret_cast<const float4*>(&rows.neg_m[c0 + c]);
          const uint32_t *a = &hi[c / 8][c % 8], *b = &lo[c / 8][c % 8];
          const f2 s0 = add2(pack(__uint_as_float(a[0]), __uint_as_float(a[1])), pack(__uint_as_float(b[0]), __uint_as_float(b[1])));
          const f2 s1 = add2(pack(__uint_as_float(a[2]), __uint_as_float(a[3])), pack(__uint_as_float(b[2]), __uint_as_float(b[3])));
          f2 y0 = add2(fma2(mul2(s0, pack(rq.x, rq.y)), ks2, ev2), pack(nm.x, nm.y));
          f2 y1 = add2(fma2(mul2(s1, pack(rq.z, rq.w)), ks2, ev2), pack(nm.z, nm.w));
          float z[4];
          unpack(y0, z[0], z[1]);
          unpack(y1, z[2], z[3]);
          if (masked) {
#pragma unroll
            for (int q = 0; q < 4; ++q) z[q] = sight >> (c + q) & 1 ? z[q] : ninf;
            y0 = pack(z[0], z[1]);
            y1 = pack(z[2], z[3]);
          }
          most = fmaxf(most, fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3])));
          x[c / 2] = y0;
          x[c / 2 + 1] = y1;
        }
        tc_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(sh.s_free));
        if (bar_or(half_bar, 128, first || most > kOver)) {
          // new references: the maxima, over the warps' lanes, of the columns that need one
          uint32_t need = ~0u;
          if (!first) {
            need = 0;
#pragma unroll
            for (int c = 0; c < NH; c += 2) {
              float a, b;
              unpack(x[c / 2], a, b);
              need |= (a > kOver ? 1u << c : 0u) | (b > kOver ? 2u << c : 0u);
            }
            need = __reduce_or_sync(kFull, need);
          }
          float keep = ninf;
#pragma unroll
          for (int c = 0; c < NH; c += 2) {
            if (need >> c & 3u) {
              float a, b;
              unpack(x[c / 2], a, b);
              a = warp_max(a);
              b = warp_max(b);
              if (lane == c) keep = a;
              if (lane == c + 1) keep = b;
            }
          }
          if (lane < NH) sh.red[wl][c0 + lane] = keep;
          bar_sync(half_bar, 128);
          if (t < NH) {
            const int c = c0 + t;
            float d = 0.f;
            const float mx = fmaxf(fmaxf(sh.red[0][c], sh.red[1][c]), fmaxf(sh.red[2][c], sh.red[3][c]));
            if (mx != ninf && (first || mx > kTop)) d = mx - kTop;
            sh.delta[c] = -d;
            sh.factor[c] = first ? 1.f : ex2(-d);  // (nothing is summed yet: 0 times an infinity is no 0)
            rows.neg_m[c] -= d;
          }
          bar_sync(half_bar, 128);
          if (!first) {
            tc_wait(bar(sh.o_done), (gi - 1) & 1, gave_up, p.status);  // the accumulator holds the earlier tiles
            tc_after();
          }
#pragma unroll
          for (int c = 0; c < NH; c += 4) {
            const float4 d = *reinterpret_cast<const float4*>(&sh.delta[c0 + c]), f = *reinterpret_cast<const float4*>(&sh.factor[c0 + c]);
            x[c / 2] = add2(x[c / 2], pack(d.x, d.y));
            x[c / 2 + 1] = add2(x[c / 2 + 1], pack(d.z, d.w));
            l2[c / 2] = mul2(l2[c / 2], pack(f.x, f.y));
            l2[c / 2 + 1] = mul2(l2[c / 2 + 1], pack(f.z, f.w));
          }
          if (!first) {
#pragma unroll 1
            for (int c = 0; c < NH; c += 4) {
              const float4 f4 = *reinterpret_cast<const float4*>(&sh.factor[c0 + c]);
              const float f[4] = {f4.x, f4.y, f4.z, f4.w};
              if (f[0] == 1.f && f[1] == 1.f && f[2] == 1.f && f[3] == 1.f) continue;  // (the same for all threads of a warp)
              uint32_t o[3][4];
#pragma unroll
              for (int part = 0; part < 3; ++part) tc_ld4(tO + part * NC + c, o[part]);
              tc_wait_ld();
#pragma unroll
              for (int part = 0; part < 3; ++part) {
#pragma unroll
                for (int j = 0; j < 4; ++j) o[part][j] = __float_as_uint(__uint_as_float(o[part][j]) * f[j]);
                tc_st4(tO + part * NC + c, o[part]);
              }
            }
            tc_wait_st();
          }
          tc_before();
        }
        // weights (the buffer's last reader: the values' MMA of the tile before)
        if (gi > 0) tc_wait(bar(sh.o_done), (gi - 1) & 1, gave_up, p.status);
#pragma unroll
        for (int c = 0; c < NH; c += 8) {
          uint32_t part[3][2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            if (c + 4 * j >= NH) break;
            uint32_t h[2], w[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float a, b;
              f2& l = l2[c / 2 + 2 * j + i];
              unpack(x[c / 2 + 2 * j + i], a, b);
              a = ex2(a);
              b = ex2(b);
              l = fma2(pack(a, b), isv2, l);
              h[i] = half2_of(a, b);
            }
            part[0][j] = narrow4_e5(h[0], h[1], w[0], w[1]);
            h[0] = rest16(h[0], w[0]), h[1] = rest16(h[1], w[1]);
            part[1][j] = narrow4_e5(h[0], h[1], w[0], w[1]);
            part[2][j] = narrow4_e5(rest16(h[0], w[0]), rest16(h[1], w[1]));
          }
#pragma unroll
          for (int k3 = 0; k3 < 3; ++k3) {
            const int col = k3 * NC + cc + c;
            uint8_t* at = pw + (col >> 4) * T::kChunk + (col & 8);
            if (c + 4 < NH)
              *reinterpret_cast<uint2*>(at) = make_uint2(part[k3][0], part[k3][1]);
            else
              *reinterpret_cast<uint32_t*>(at) = part[k3][0];
          }
        }
        fence_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(sh.p_full));
      }
      // ---- the end of the stretch: the next one's queries first, so that its scores are computed meanwhile ----
      more = begin(ns + 1);
      const bool whole = g.n == g.nt, join = whole && p.pre_o != nullptr && t < D;
      const int d = t & (D - 1);
      if (p.late_wait) griddep_wait();
      float pre[NH];  // this element of the prefix's part, on its way while the sums are joined
#pragma unroll
      for (int c = 0; c < NH; ++c) {
        const int idx = rows.idx[c0 + c];
        pre[c] = join && idx >= 0 ? __ldcg(p.pre_o + (long long)idx * D + d) : 0.f;
      }
      tc_wait(bar(sh.o_done), (gi - 1) & 1, gave_up, p.status);
      tc_after();
      // the weights' memory, read by now: the second token half's sums with head_dim 64, then partial sums of the weights
      float* const half = reinterpret_cast<float*>(mem + T::oP) + c0 * D;
      float* const part = reinterpret_cast<float*>(mem + T::oP + (kHalves == 2 ? NR * D * 4 : 0));
      constexpr int kPer = D / 2;  // partial sums of a column: over the lanes first that share a place
#pragma unroll
      for (int c = 0; c < NH; c += 2) {
        float a, b;
        unpack(l2[c / 2], a, b);
#pragma unroll
        for (int o = 16; o >= kPer / 4; o >>= 1) {
          a += __shfl_xor_sync(kFull, a, o);
          b += __shfl_xor_sync(kFull, b, o);
        }
        if (lane < kPer / 4) {
          part[(c0 + c) * kPer + wl * (kPer / 4) + lane] = a;
          part[(c0 + c + 1) * kPer + wl * (kPer / 4) + lane] = b;
        }
      }
      float* slot = whole ? nullptr : slot_of<NR, D>(p, 2 * blockIdx.x + (g.t0 == 0 ? 1 : 0));
      bar_sync(1, kTcSoft);
      if (tid < 4 * NR) {  // (whole warps) four threads a column
        const int col = tid >> 2, idx = rows.idx[col];
        const float lse = whole && idx >= 0 && p.pre_o != nullptr ? __ldcg(p.pre_lse + idx) : ninf;
        float l = 0.f;
        const float m = (float)kSumShift - rows.neg_m[col];  // what sums and values, both scaled so, are relative to
#pragma unroll
        for (int i = 0; i < kPer / 4; ++i) l += part[col * kPer + ((i + col) * 4 & (kPer - 1)) + (tid & 3)];
        l += __shfl_xor_sync(kFull, l, 1);
        l += __shfl_xor_sync(kFull, l, 2);
        if ((tid & 3) != 0) {
        } else if (!whole) {
          slot[col] = l == 0.f ? ninf : m;  // a row that saw nothing has no reference
          slot[NR + col] = l;
        } else if (idx >= 0) {
          const Coef r = row_coef(lse, m, l, g.bad);
          sh.coef[0][col] = r.a * kSumScale;
          sh.coef[1][col] = r.b;
          finish_lse(p, idx, r);
        }
      }
      if (kHalves == 2 && t >= D) {
#pragma unroll 1
        for (int c = 0; c < NH; c += 4) {
          float o[4];
          tc_sum_parts<NC>(tO + c, o);
#pragma unroll
          for (int j = 0; j < 4; ++j) half[(c + j) * D + d] = o[j];
        }
      }
      bar_sync(1, kTcSoft);
      if (t < D && !whole) {
        slot += 2 * NR + c0 * D + d;
#pragma unroll 1
        for (int c = 0; c < NH; c += 4, slot += 4 * D) {
          float o[4];
          tc_sum_parts<NC>(tO + c, o);
#pragma unroll
          for (int j = 0; j < 4; ++j) slot[j * D] = (kHalves == 2 ? o[j] + half[(c + j) * D + d] : o[j]) * kSumScale;
        }
      } else if (t < D) {
#pragma unroll
        for (int c = 0; c < NH; c += 4) {
          const int4 i4 = *reinterpret_cast<const int4*>(&rows.idx[c0 + c]);
          if (i4.x < 0) break;  // (past the last row)
          const int idx[4] = {i4.x, i4.y, i4.z, i4.w};
          const float4 a4 = *reinterpret_cast<const float4*>(&sh.coef[0][c0 + c]);
          const float a[4] = {a4.x, a4.y, a4.z, a4.w};
          float o[4];
          tc_sum_parts<NC>(tO + c, o);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (kHalves == 2) o[j] += half[(c + j) * D + d];
            o[j] *= a[j];
          }
          if (p.pre_o != nullptr) {
            const float4 b4 = *reinterpret_cast<const float4*>(&sh.coef[1][c0 + c]);
            const float b[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (b[j] != 0.f) o[j] = fmaf(pre[c + j], b[j], o[j]);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (idx[j] >= 0) store_out<uint16_t, D>(p, idx[j], d, o[j]);
        }
      }
      tc_before();
      bar_sync(1, kTcSoft);
    }
  }
  if (p.late_wait) griddep_wait();  // (also of a block that joined nothing: no kernel of a call ends before the ones in front of it)
  tc_before();
  __syncthreads();
  if (warp == 9) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 256;" ::"r"(tmem));
  }
}

}  // namespace sv
