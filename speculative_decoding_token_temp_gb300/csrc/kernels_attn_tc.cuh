// Attention over the 8-bit cache on the fifth-generation tensor cores, for bf16 queries.
//
// A block holds up to NR rows (query rows times the query heads of one kv head) and walks
// 128-token tiles of their keys. Both products have the tokens or the head's elements on
// the 128-lane side, and the few rows on the other: S^T = K q^T (lanes = tokens) and
// O^T = V^T P^T (lanes = elements), so that few rows cost few columns instead of a
// 128-row tile that is mostly empty.
//
//   K q^T  runs on the codes as they are (kind::f8f6f4): a bf16 query is, within its row's
//          power of two, exactly the sum of two e4m3 numbers (8 significant bits = 4 + 4;
//          elements below 2^-8 of the row's largest keep an absolute 2^-18 of it), so the
//          query is staged twice, as its high and its low part side by side, and one MMA
//          gives both products. No rounding of keys or queries, and no work to widen keys.
//   V^T P^T runs in f16 (kind::f16): a value's code is exact in f16, and a weight's f16
//          (11 bits, down to 2^-30 of the row's largest) keeps long flat tails that 8 bits
//          would drop. The values are widened by the softmax warps as they pass.
//   Exponents: a key's is a factor of its token's scores, one lane's constant; a value's is
//          added to the score before the exponential (weights are 2^(x + e - m)), so that
//          the weighted values need no further scaling and no weight over- or underflows
//          where values differ much in size; the sum takes it out again (2^-e).
//
// Warps: two groups of four take the tiles in turn, each with its own scores, weights,
// widened values, accumulator and running maximum, so that one group's softmax runs while
// the other's products do; the groups' sums are joined at the end of a stretch. One warp
// keeps a ring of tiles filled (a TMA load a page and operand; pages shorter than a tile
// make several), one issues the MMAs as their operands become ready. A thread of a group
// is a token: its weights of all rows sit in its registers, and the maximum over tokens,
// which would cross lanes, is needed only when a score exceeds the reference by 2^14 (the
// first tile of a stretch, then rarely): the reference is not the maximum itself but
// anything that keeps the weights inside f16's range.
//
// What bounds it: the cache's bytes. A tile is 32 KB of codes (head_dim 128); three are in
// flight.
#pragma once

#include <cuda.h>

#include "kernels_attn.cuh"

namespace sv {

constexpr int kTcThreads = 320;
constexpr int kTcPollLimit = 1 << 22;  // bounded waits (SPEC_DEV_TIMEOUT)
constexpr float kTop = 6.f;            // a fresh reference puts the largest weight at 2^6 ...
constexpr float kOver = 14.f;          // ... and is renewed when one would pass 2^14 (f16 ends at 2^16)

template <int D>
struct TcShape {
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr int kTileBytes = kTile * D;                       // codes of one operand
  static constexpr int kV16 = D == 128 ? 32768 : 16384;              // widened values of a group
  static constexpr int kP = 16384;                                   // weights of a group: 128 tokens x 128 bytes
  static constexpr int kQ = 2 * 64 * D;                              // high and low parts of 64 rows
  // offsets from a 1024-byte boundary
  static constexpr int oV16 = 0;
  static constexpr int oP = oV16 + 2 * kV16;
  static constexpr int oQ = oP + 2 * kP;
  static constexpr int oK = oQ + kQ;
  static constexpr int oV = oK + kStages * kTileBytes;
  static constexpr int oE = oV + kStages * kTileBytes;               // exponent bytes: keys', values'
  static constexpr int kSmem = oE + kStages * 2 * kTile + 1024;
  static constexpr int kSwz = D == 128 ? 7 : 3;                      // 16-byte chunks of a row of codes, less one
  static constexpr uint64_t kLayoutD = D == 128 ? 2 : 4;             // descriptor: 128- or 64-byte swizzle
};

// ---- tcgen05 wrappers -------------------------------------------------------

// Shared-memory matrix descriptor: address, leading and stride byte offsets, swizzle.
__device__ __forceinline__ uint64_t mma_desc(uint32_t addr, uint32_t lbo, uint32_t sbo, uint64_t layout) {
  return (uint64_t)((addr & 0x3ffffu) >> 4) | (uint64_t)(lbo >> 4) << 16 | (uint64_t)(sbo >> 4) << 32 | 1ull << 46 |
         layout << 61;
}
// Instruction descriptor: fp32 accumulator, operand types 0 (e4m3 / f16), M = 128.
__host__ __device__ constexpr uint32_t mma_idesc(int n, bool mn_major) {
  return 1u << 4 | (mn_major ? 3u << 15 : 0u) | (uint32_t)(n >> 3) << 17 | 8u << 24;
}
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
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
__device__ __forceinline__ void tc_ld16(uint32_t a, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(a));
}
__device__ __forceinline__ void tc_st16(uint32_t a, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(a)
      : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool mbar_test(uint32_t bar, unsigned parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
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
__device__ __forceinline__ void tc_wait(uint32_t bar, unsigned parity, volatile int* gave_up, uint32_t* status) {
  if (mbar_try_wait(bar, parity)) return;
  for (int it = 0; !mbar_try_wait(bar, parity); ++it) {
    if (*gave_up) return;
    if (it == kTcPollLimit) {
      *gave_up = 1;
      atomicOr(status, SPEC_DEV_TIMEOUT);
      return;
    }
  }
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
__device__ __forceinline__ uint32_t widen2(uint32_t two) {  // two e4m3 codes (low 16 bits) as f16x2
  uint32_t r;
  asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(two));
  return r;
}

// Sums over a warp of 16 or 32 columns held by every lane: lane c (mod 16) gets column c's.
template <int N>
__device__ __forceinline__ float column_sums(float (&v)[N], int lane) {
  if constexpr (N == 16) {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] += __shfl_xor_sync(kFull, v[i], 16);
  }
#pragma unroll
  for (int o = N / 2; o >= 1; o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float send = up ? v[i] : v[i + o], keep = up ? v[i + o] : v[i];
      v[i] = keep + __shfl_xor_sync(kFull, send, o);
    }
  }
  return v[0];
}

template <int NR>
struct TcShared {
  LocateShared loc;
  uint64_t full[6], empty[6], q_full, drained, s_full[2], s_free[2], p_full[2], o_done[2];
  uint32_t tmem;
  int gave_up;
  uint32_t bad_pages[6];
  alignas(16) float rq[NR];          // a row's factor of the scores: scale * log2(e) * its power of two
  alignas(16) int row[NR];           // query row of a flat row
  alignas(16) float neg_m[2][NR];    // the groups' references, negated
  alignas(16) float delta[2][NR];
  float red[2][4][NR];               // of the groups' warps: maxima, then sums
  float wgt[2][NR];                  // a group's weight in the joined sum
  Coef coef[NR];
  long long idx[NR];
};

template <int D, int NR>
__global__ void __launch_bounds__(kTcThreads, 1)
attn_tc_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap map_k,
               const __grid_constant__ CUtensorMap map_v) {
  using T = TcShape<D>;
  constexpr int NST = T::kStages;
  constexpr int kHalves = D == 128 ? 1 : 2;  // token halves stacked on the lanes of O^T
  extern __shared__ uint8_t dyn[];
  __shared__ TcShared<NR> sh;
  const uint32_t dyn_raw = (uint32_t)__cvta_generic_to_shared(dyn);
  const uint32_t base = (dyn_raw + 1023u) & ~1023u;
  uint8_t* const mem = dyn + (base - dyn_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto bar = [](const uint64_t& b) { return (uint32_t)__cvta_generic_to_shared(&b); };
  volatile int* gave_up = &sh.gave_up;

  if (tid == 0) {
    for (int i = 0; i < NST; ++i) {
      mbar_init(bar(sh.full[i]), 1);
      mbar_init(bar(sh.empty[i]), 5);  // the scores' MMA and the four warps that widened the values
    }
    mbar_init(bar(sh.q_full), 256);
    mbar_init(bar(sh.drained), 1);
    for (int w = 0; w < 2; ++w) {
      mbar_init(bar(sh.s_full[w]), 1);
      mbar_init(bar(sh.s_free[w]), 4);
      mbar_init(bar(sh.p_full[w]), 4);
      mbar_init(bar(sh.o_done[w]), 1);
    }
    sh.gave_up = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     (uint32_t)__cvta_generic_to_shared(&sh.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    tc_before();
  }
  griddep_wait();
  griddep_launch();
  long long begin, end, total;
  const bool ok = locate<NR, kTcThreads>(p, sh.loc, blockIdx.x, blockIdx.x + 1, gridDim.x, &begin, &end, &total);
  tc_after();
  const uint32_t tmem = sh.tmem;
  if (!ok) {
    fill_nan<uint16_t, D>(p, blockIdx.x, gridDim.x);
    begin = end = 0;
  }
  const long long tiles = end - begin;

  if (warp == 8) {
    // ---- the ring of tiles ----
    Place at = sh.loc.at[0];
    long long left = tiles;
    unsigned gi = 0;
    uint32_t bits = 0;
    const int psz = 1 << p.page_shift, box = min(psz, kTile), np = kTile / box;
    while (left > 0) {
      const Seg g = next_seg<NR>(p, at, left);
      if (g.bad) bits |= SPEC_DEV_OFFSETS;
      auto page_of = [&](int tile) -> int {  // of this lane's part of a tile; -2: nothing there
        const int t = tile * kTile + lane * box;
        return lane < np && t < g.len ? __ldg(g.pages + (t >> p.page_shift)) : -2;
      };
      int page = page_of(g.t0);
      for (int k = 0; k < g.n; ++k, ++gi) {
        const int st = gi % NST, tile = g.t0 + k;
        const int next = k + 1 < g.n ? page_of(tile + 1) : -2;
        const bool there = lane < np && tile * kTile + lane * box < g.len;
        const bool good = there && (unsigned)page < (unsigned)p.num_pages;
        const unsigned bad = __ballot_sync(kFull, there && !good), cnt = __popc(__ballot_sync(kFull, good));
        if (bad) bits |= SPEC_DEV_PAGE;
        if (gi >= NST) tc_wait(bar(sh.empty[st]), (gi / NST - 1) & 1, gave_up, p.status);
        __syncwarp();
        if (lane == 0) {
          sh.bad_pages[st] = bad;
          mbar_expect_arrive(bar(sh.full[st]), cnt * (uint32_t)(box * (2 * D + 2)));
        }
        __syncwarp();
        if (good) {
          const int tok = (tile * kTile + lane * box) & (psz - 1);
          const uint32_t b = bar(sh.full[st]);
          tma_page(base + T::oK + st * T::kTileBytes + lane * box * D, &map_k, tok, g.h, page, b);
          tma_page(base + T::oV + st * T::kTileBytes + lane * box * D, &map_v, tok, g.h, page, b);
          const long long vec = (((long long)page * p.Hk + g.h) << p.page_shift) + tok;
          bulk_copy(base + T::oE + st * 2 * kTile + lane * box, p.k_exp + vec, box, b);
          bulk_copy(base + T::oE + st * 2 * kTile + kTile + lane * box, p.v_exp + vec, box, b);
        }
        page = next;
      }
    }
    if (bits) atomicOr(p.status, bits);
    // no copy is left in flight when the block ends, even after a wait that gave up
    for (int st = 0; st < NST; ++st)
      if (gi > (unsigned)st) {
        const unsigned uses = (gi - 1 - st) / NST;
        for (int it = 0; it < kTcPollLimit && !mbar_try_wait(bar(sh.full[st]), uses & 1); ++it) {
        }
      }
  } else if (warp == 9) {
    // ---- the MMAs, as their operands become ready ----
    if (lane == 0) {
      constexpr uint32_t id_s = mma_idesc(2 * NR, false), id_o = mma_idesc(NR, true);
      Place at = sh.loc.at[0];
      long long left = tiles;
      unsigned qi = 0, pi = 0, qseg = 0;
      int qk = 0, qn = 0;             // the scores' tile within its stretch
      Place pat = at;
      long long pleft = tiles;
      int pk = 0, pn = 0;             // the weights' tile within its stretch
      int idle = 0;
      while (pi < (unsigned)tiles && !*gave_up) {
        bool moved = false;
        if (qi < (unsigned)tiles) {
          if (qk == qn) {
            qn = next_seg<NR>(p, at, left).n;
            qk = 0;
            ++qseg;
          }
          const int st = qi % NST, w = qi & 1;
          const unsigned u = qi >> 1;
          if ((qk > 0 || mbar_test(bar(sh.q_full), (qseg - 1) & 1)) && (u == 0 || mbar_test(bar(sh.s_free[w]), (u - 1) & 1)) &&
              mbar_test(bar(sh.full[st]), (qi / NST) & 1)) {
            tc_after();
            const uint32_t a = base + T::oK + st * T::kTileBytes, b = base + T::oQ;
#pragma unroll
            for (int s = 0; s < D / 32; ++s)
              mma_f8(tmem + w * 256, mma_desc(a + s * 32, 16, 8 * D, T::kLayoutD), mma_desc(b + s * 32, 16, 8 * D, T::kLayoutD),
                     id_s, s > 0);
            mma_commit(bar(sh.s_full[w]));
            mma_commit(bar(sh.empty[st]));
            ++qi;
            ++qk;
            moved = true;
          }
        }
        if (pi < qi) {
          if (pk == pn) {
            pn = next_seg<NR>(p, pat, pleft).n;
            pk = 0;
          }
          const int w = pi & 1;
          if (mbar_test(bar(sh.p_full[w]), (pi >> 1) & 1)) {
            tc_after();
            const uint32_t a = base + T::oV16 + w * T::kV16, b = base + T::oP + w * T::kP;
#pragma unroll
            for (int hf = 0; hf < kHalves; ++hf) {
#pragma unroll
              for (int s = 0; s < kTile / kHalves / 16; ++s)
                mma_f16(tmem + w * 256 + 128 + hf * NR, mma_desc(a + s * 2048, T::kV16 / 2, 1024, 2),
                        mma_desc(b + hf * 8192 + s * 2048, 16, 1024, 2), id_o, s > 0 || pk >= 2);
            }
            mma_commit(bar(sh.o_done[w]));
            ++pi;
            ++pk;
            moved = true;
          }
        }
        if (moved) {
          idle = 0;
        } else if (++idle > (1 << 26)) {
          *gave_up = 1;
          atomicOr(p.status, SPEC_DEV_TIMEOUT);
        }
      }
      // no MMA is left in flight when the block ends, even after a wait that gave up
      mma_commit(bar(sh.drained));
      for (int it = 0; it < kTcPollLimit && !mbar_try_wait(bar(sh.drained), 0); ++it) {
      }
    }
    __syncwarp();
  } else {
    // ---- softmax: group w, thread = token (lane of S^T) and element (lane of O^T) ----
    const int w = warp >> 2, t = tid & 127, wl = warp & 3;
    const uint32_t lanes = (uint32_t)(wl * 32) << 16;
    const uint32_t tS = tmem + lanes + w * 256, tO = tmem + lanes + w * 256 + 128 + (kHalves == 2 && wl >= 2 ? NR : 0);
    uint8_t* const v16 = mem + T::oV16 + w * T::kV16;
    uint8_t* const pw = mem + T::oP + w * T::kP + t * 128;
    const float nan = __int_as_float(0x7fffffff), ninf = __int_as_float(kNegInfBits);
    Place at = sh.loc.at[0];
    long long left = tiles;
    unsigned gi = 0;
    f2 l2[NR / 2];
    while (left > 0) {
      const Seg g = next_seg<NR>(p, at, left);
      const int flat = g.rows * p.G;
      // the queries: four threads a row find its power of two and stage its two parts
      {
        const int c = tid >> 2, f = g.f0 + c, part = tid & 3;
        if (c < NR) {
          float x[D / 4];
          float m = 0.f;
          if (f < flat) {
            const uint16_t* src = static_cast<const uint16_t*>(p.q) + (long long)(g.row0 + f / p.G) * p.q_row +
                                  (long long)(g.h * p.G + f % p.G) * p.q_head + part * (D / 4);
            if (((uintptr_t)src & 15) == 0) {
#pragma unroll
              for (int i = 0; i < D / 32; ++i) {
                float y[8];
                load8<true>(src + i * 8, y);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[i * 8 + j] = y[j];
              }
            } else {
#pragma unroll
              for (int i = 0; i < D / 4; ++i) x[i] = __uint_as_float((uint32_t)__ldg(src + i) << 16);
            }
          } else {
#pragma unroll
            for (int i = 0; i < D / 4; ++i) x[i] = 0.f;
          }
          bool bad = false;
#pragma unroll
          for (int i = 0; i < D / 4; ++i) {
            m = fmaxf(m, fabsf(x[i]));
            bad |= !(fabsf(x[i]) <= 3.402823466e38f);
          }
          if (bad) m = __int_as_float(0x7f800000);
          m = fmaxf(m, __shfl_xor_sync(kFull, m, 1));
          m = fmaxf(m, __shfl_xor_sync(kFull, m, 2));
          bad = m == __int_as_float(0x7f800000);
          const int e = max((__float_as_int(m) >> 23) - 127, -100) - 7;  // the largest element comes to [128, 256)
          const float inv = __int_as_float((127 - e) << 23);
          if (part == 0) {
            sh.rq[c] = bad ? nan : p.c * __int_as_float((e + 127) << 23);
            sh.row[c] = f / p.G;
          }
#pragma unroll
          for (int i = 0; i < D / 64; ++i) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              float y[4], b[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) y[k] = bad ? 0.f : x[i * 16 + j * 4 + k] * inv;
              const uint32_t h0 = __nv_cvt_float2_to_fp8x2(make_float2(y[0], y[1]), __NV_SATFINITE, __NV_E4M3);
              const uint32_t h1 = __nv_cvt_float2_to_fp8x2(make_float2(y[2], y[3]), __NV_SATFINITE, __NV_E4M3);
              hi[j] = h0 | h1 << 16;
              codes4(hi[j], b);
              const uint32_t l0 = __nv_cvt_float2_to_fp8x2(make_float2(y[0] - b[0], y[1] - b[1]), __NV_SATFINITE, __NV_E4M3);
              const uint32_t l1 = __nv_cvt_float2_to_fp8x2(make_float2(y[2] - b[2], y[3] - b[3]), __NV_SATFINITE, __NV_E4M3);
              lo[j] = l0 | l1 << 16;
            }
            const int chunk = part * (D / 64) + i;
            // rows of D bytes, 16-byte chunks exchanged as the swizzle has them
            const int rl = NR + c;
            const int ch_h = D == 128 ? chunk ^ (c & 7) : chunk ^ ((c >> 1) & 3);
            const int ch_l = D == 128 ? chunk ^ (rl & 7) : chunk ^ ((rl >> 1) & 3);
            *reinterpret_cast<uint4*>(mem + T::oQ + c * D + ch_h * 16) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4*>(mem + T::oQ + rl * D + ch_l * 16) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          }
        }
        if (tid < 2 * NR) sh.neg_m[tid / NR][tid % NR] = 0.f;
        fence_async();
        mbar_arrive(bar(sh.q_full));
        bar_sync(3, 256);  // rq, row and the references are seen by both groups
      }
#pragma unroll
      for (int i = 0; i < NR / 2; ++i) l2[i] = 0ull;
      int mine = 0;  // tiles of this group in the stretch
      for (int k = 0; k < g.n; ++k, ++gi) {
        if ((int)(gi & 1) != w) continue;
        const int st = gi % NST, tile = g.t0 + k, tok = tile * kTile + t;
        const unsigned u = gi >> 1;
        const bool first = mine == 0;
        ++mine;
        const bool masked = p.mask == A_ALL ? tile * kTile + kTile > g.len : tile * kTile + kTile - 1 > g.len - g.rows;
        tc_wait(bar(sh.full[st]), (gi / NST) & 1, gave_up, p.status);
        const bool live = tok < g.len;
        bool hurt = live && ((sh.bad_pages[st] >> (t >> min(p.page_shift, 7))) & 1);
        const unsigned kb = mem[T::oE + st * 2 * kTile + t], vb = mem[T::oE + st * 2 * kTile + kTile + t];
        if (u > 0) tc_wait(bar(sh.o_done[w]), (u - 1) & 1, gave_up, p.status);
        // widen this token's values
        {
          const uint8_t* src = mem + T::oV + st * T::kTileBytes + t * D;
          const bool zero = !live || hurt;
#pragma unroll
          for (int ch = 0; ch < D / 16; ++ch) {
            uint4 v = *reinterpret_cast<const uint4*>(src + ((D == 128 ? ch ^ (t & 7) : ch ^ ((t >> 1) & 3)) * 16));
            if (masked) {
              // a NaN code must not reach rows that do not see the token (0 * NaN): its token is marked instead
              uint32_t* q = &v.x;
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const uint32_t mk = __vcmpeq4(q[j] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                if (live && mk) hurt = true;
                q[j] &= ~mk;
              }
            }
            if (zero) v = make_uint4(0, 0, 0, 0);
            const uint4 a = make_uint4(widen2(v.x), widen2(v.x >> 16), widen2(v.y), widen2(v.y >> 16));
            const uint4 b = make_uint4(widen2(v.z), widen2(v.z >> 16), widen2(v.w), widen2(v.w >> 16));
            uint8_t* dst;
            int r, c0;
            if constexpr (D == 128) {
              dst = v16 + (ch >> 2) * 16384 + t * 128;
              r = t & 7;
              c0 = (ch & 3) * 2;
            } else {
              dst = v16 + (t >> 6) * 8192 + (t & 63) * 128;
              r = t & 7;
              c0 = ch * 2;
            }
            *reinterpret_cast<uint4*>(dst + ((c0 ^ r) * 16)) = a;
            *reinterpret_cast<uint4*>(dst + (((c0 + 1) ^ r) * 16)) = b;
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(sh.empty[st]));
        hurt |= live && (kb == kNanExp || vb == kNanExp);
        const float ks = !live ? 0.f : hurt ? nan : exp_value(kb);
        const float ev = live && !hurt ? (float)((int)vb - kExpBias) : 0.f;
        const f2 ks2 = pack(ks, ks), ev2 = pack(ev, ev);
        const float isv = live && !hurt ? __int_as_float((2 * kExpBias - (int)vb) << 23) : 1.f;
        const f2 isv2 = pack(isv, isv);
        // scores
        tc_wait(bar(sh.s_full[w]), u & 1, gave_up, p.status);
        tc_after();
        f2 x[NR / 2];
        float most = ninf;
#pragma unroll
        for (int c = 0; c < NR; c += 16) {
          uint32_t hi[16], lo[16];
          tc_ld16(tS + c, hi);
          tc_ld16(tS + NR + c, lo);
          tc_wait_ld();
#pragma unroll
          for (int j = 0; j < 16; j += 4) {
            const float4 rq = *reinterpret_cast<const float4*>(&sh.rq[c + j]);
            const float4 nm = *reinterpret_cast<const float4*>(&sh.neg_m[w][c + j]);
            const f2 s0 = add2(pack(__uint_as_float(hi[j]), __uint_as_float(hi[j + 1])), pack(__uint_as_float(lo[j]), __uint_as_float(lo[j + 1])));
            const f2 s1 = add2(pack(__uint_as_float(hi[j + 2]), __uint_as_float(hi[j + 3])), pack(__uint_as_float(lo[j + 2]), __uint_as_float(lo[j + 3])));
            f2 y0 = add2(fma2(mul2(s0, pack(rq.x, rq.y)), ks2, ev2), pack(nm.x, nm.y));
            f2 y1 = add2(fma2(mul2(s1, pack(rq.z, rq.w)), ks2, ev2), pack(nm.z, nm.w));
            float z[4];
            unpack(y0, z[0], z[1]);
            unpack(y1, z[2], z[3]);
            if (masked) {
              const int4 rows = *reinterpret_cast<const int4*>(&sh.row[c + j]);
              const int ri[4] = {rows.x, rows.y, rows.z, rows.w};
#pragma unroll
              for (int q = 0; q < 4; ++q)
                if (!(live && ri[q] < g.rows && sees(p, ri[q], g.rows, g.len, tok))) z[q] = ninf;
              y0 = pack(z[0], z[1]);
              y1 = pack(z[2], z[3]);
            }
            most = fmaxf(most, fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3])));
            x[(c + j) / 2] = y0;
            x[(c + j) / 2 + 1] = y1;
          }
        }
        tc_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(sh.s_free[w]));
        if (bar_or(1 + w, 128, first || most > kOver)) {
          // a new reference: the maxima of the columns, of the warps, of the group
#pragma unroll
          for (int c = 0; c < NR; c += 16) {
            float keep = 0.f;
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
              float a, b;
              unpack(x[(c + j) / 2], a, b);
              a = warp_max(a);
              b = warp_max(b);
              if (lane == j) keep = a;
              if (lane == j + 1) keep = b;
            }
            if (lane < 16) sh.red[w][wl][c + lane] = keep;
          }
          bar_sync(1 + w, 128);
          if (t < NR) {
            const float mx = fmaxf(fmaxf(sh.red[w][0][t], sh.red[w][1][t]), fmaxf(sh.red[w][2][t], sh.red[w][3][t]));
            float d = 0.f;
            if (mx != ninf && (first || mx > kTop)) d = mx - kTop;
            sh.delta[w][t] = -d;
            sh.neg_m[w][t] -= d;
          }
          bar_sync(1 + w, 128);
#pragma unroll
          for (int c = 0; c < NR; c += 4) {
            const float4 d = *reinterpret_cast<const float4*>(&sh.delta[w][c]);
            x[c / 2] = add2(x[c / 2], pack(d.x, d.y));
            x[c / 2 + 1] = add2(x[c / 2 + 1], pack(d.z, d.w));
            if (!first) {
              l2[c / 2] = mul2(l2[c / 2], pack(ex2(d.x), ex2(d.y)));
              l2[c / 2 + 1] = mul2(l2[c / 2 + 1], pack(ex2(d.z), ex2(d.w)));
            }
          }
          if (!first) {  // o_done was waited for above: the accumulator holds the earlier tiles
            tc_after();
#pragma unroll 1
            for (int c = 0; c < NR; c += 16) {
              uint32_t o[16];
              tc_ld16(tO + c, o);
              tc_wait_ld();
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * ex2(sh.delta[w][c + j]));
              tc_st16(tO + c, o);
            }
            tc_wait_st();
            tc_before();
          }
        }
        // weights
#pragma unroll
        for (int c = 0; c < NR; c += 8) {
          uint32_t h[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float a, b;
            unpack(x[c / 2 + j], a, b);
            a = ex2(a);
            b = ex2(b);
            l2[c / 2 + j] = fma2(pack(a, b), isv2, l2[c / 2 + j]);
            h[j] = half2_of(a, b);
          }
          *reinterpret_cast<uint4*>(pw + (((c >> 3) ^ (t & 7)) * 16)) = make_uint4(h[0], h[1], h[2], h[3]);
        }
        fence_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(sh.p_full[w]));
      }
      // ---- the end of the stretch: the groups' sums joined ----
      if (mine > 0) {
        const unsigned u = ((gi - 1 - ((gi - 1 - w) & 1)) >> 1);  // this group's last use
        tc_wait(bar(sh.o_done[w]), u & 1, gave_up, p.status);
        tc_after();
      }
      {
        float l[NR];
#pragma unroll
        for (int i = 0; i < NR / 2; ++i) unpack(l2[i], l[2 * i], l[2 * i + 1]);
#pragma unroll
        for (int c = 0; c < NR; c += 16) {
          float v[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) v[j] = l[c + j];
          const float s = column_sums<16>(v, lane);
          if (lane < 16) sh.red[w][wl][c + lane] = s;
        }
      }
      const bool whole = g.n == g.nt;
      const int n_own = mine, n_other = g.n - mine;
      bar_sync(3, 256);
      float* slot = whole ? nullptr : slot_of<NR, D>(p, 2 * blockIdx.x + (g.t0 == 0 ? 1 : 0));
      if (tid < NR) {  // (threads of group 0)
        const int c = tid, f = g.f0 + c;
        const float m0 = n_own > 0 ? -sh.neg_m[0][c] : ninf, m1 = n_other > 0 ? -sh.neg_m[1][c] : ninf;
        const float l0 = sh.red[0][0][c] + sh.red[0][1][c] + sh.red[0][2][c] + sh.red[0][3][c];
        const float l1 = sh.red[1][0][c] + sh.red[1][1][c] + sh.red[1][2][c] + sh.red[1][3][c];
        // a group that saw nothing of a row has sum 0 and no reference of its own
        const bool h0 = n_own > 0 && l0 != 0.f, h1 = n_other > 0 && l1 != 0.f;
        const float m = fmaxf(h0 ? m0 : ninf, h1 ? m1 : ninf), mu = m == ninf ? 0.f : m;
        const float w0 = h0 ? exp2f(m0 - mu) : 0.f, w1 = h1 ? exp2f(m1 - mu) : 0.f;
        const float l = (h0 ? w0 * l0 : 0.f) + (h1 ? w1 * l1 : 0.f);
        sh.wgt[0][c] = w0;
        sh.wgt[1][c] = w1;
        const long long idx = (long long)(g.row0 + f / p.G) * p.Hq + g.h * p.G + f % p.G;
        sh.idx[c] = f < flat ? idx : -1;
        if (!whole) {
          slot[c] = mu;
          slot[NR + c] = l;
        } else if (f < flat) {
          const Coef r = row_coef(p, idx, mu, l, g.bad);
          sh.coef[c] = r;
          finish_lse(p, idx, r);
        }
      }
      bar_sync(3, 256);
      // values: every thread but the one that writes an element passes its sums through shared memory
      float* const box = reinterpret_cast<float*>(mem);  // widened values and weights, all read by now
      const int d = D == 128 ? t : t & 63;
      const int src = D == 128 ? w : w * 2 + (t >> 6);   // contribution number; 0 writes
      if (src != 0 && mine > 0) {
#pragma unroll 1
        for (int c = 0; c < NR; c += 16) {
          uint32_t o[16];
          tc_ld16(tO + c, o);
          tc_wait_ld();
#pragma unroll
          for (int j = 0; j < 16; ++j) box[((src - 1) * NR + c + j) * D + d] = __uint_as_float(o[j]);
        }
      }
      bar_sync(3, 256);
      if (src == 0) {
#pragma unroll 1
        for (int c = 0; c < NR; c += 16) {
          uint32_t o[16];
          if (n_own > 0) {
            tc_ld16(tO + c, o);
            tc_wait_ld();
          }
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const long long idx = sh.idx[c + j];
            if (whole && idx < 0) continue;
            const float w0 = sh.wgt[0][c + j], w1 = sh.wgt[1][c + j];
            float y = 0.f;
            if (w0 != 0.f) {
              float a = __uint_as_float(o[j]);
              if constexpr (kHalves == 2) a += box[(c + j) * D + d];
              y = a * w0;
            }
            if (w1 != 0.f) {
              float a = box[((kHalves - 1) * NR + c + j) * D + d];
              if constexpr (kHalves == 2) a += box[(2 * NR + c + j) * D + d];
              y += a * w1;
            }
            if (whole)
              finish<uint16_t, D>(p, idx, d, y, sh.coef[c + j]);
            else
              slot[2 * NR + (c + j) * D + d] = y;
          }
        }
      }
      tc_before();
      bar_sync(3, 256);
    }
  }
  tc_before();
  __syncthreads();
  if (warp == 9) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
}

}  // namespace sv
