// The shared prefix's part for many rows, on the fifth-generation tensor cores.
//
// Where the rows that share keys fill 128-row tiles, the product is a dense one and what
// bounds it is the tensor pipe, not the cache's bytes. So the prefix is widened once per
// call into the workspace (widen_kernel), and the attention reads 16-bit operands:
//
//   keys    bf16, exponent included: exact (4 significant bits, bf16's exponent range), and
//           bf16 queries times bf16 keys need no scaling at all;
//   values  f16, relative to the largest exponent of their 128 tokens (one number a tile
//           and head): code * 2^(6 + e - largest), exact down to 21 binades below the tile's
//           largest exponent; it joins the tile's scores before the exponential (as E), as
//           the exponents of single values do in attn_tc_kernel;
//   weights f16 (11 bits), kept in tensor memory where the scores were.
//
// A block holds 256 rows as two tiles of 128 and walks the keys in tiles of 128 tokens:
// S = Q K^T and O += P V, lanes = rows. Two threads share a row, half of a tile's tokens
// each, so maxima and sums need one other thread, and that only when the reference is
// renewed (a row's largest score passes it by 2^15). While one group makes weights, the tensor pipe sums the other's
// values and then computes its next scores: MMAs of one block run in the order they are
// issued, so a group's next scores may overwrite its weights without a wait.
//
// What bounds it: 256 rows x 128 tokens (head_dim 128) take 2850 clocks, of which the MMAs are
// 2048 at their nominal rate; the scores' read both operands from shared memory at its full
// rate, beside the copies into it. A softmax group's own work is 1300 clocks; 1110 (maxima
// from the loads of scores) left the time as it was. 9216 rows a kv head x 16384 tokens, 8 kv
// heads: 410 us, and 17 us to widen (34 MB read, 67 MB written, mostly to L2).
#pragma once

#include "kernels_attn_chunk.cuh"

#include <type_traits>

namespace sv {

constexpr int kRowsP = 256;         // rows of a block
constexpr float kFarP = 262144.f;   // scores further than this from a row's reference are counted from a score of its own (`far`)
constexpr int kPreThreads = 576;    // two softmax groups of eight warps, one warp for copies, one for MMAs
constexpr float kTopP = 8.f;        // a fresh reference puts a row's largest weight at 2^8 ...
constexpr float kOverP = 15.f;      // ... and is renewed when one would pass 2^15

// fp32 queries are three bf16 parts (24 bits), their weights two f16 parts (22 bits) side by side where the scores were; one
// row tile a block then.
template <int D, bool F32 = false>
struct PreShape {
  static constexpr int kGroups = F32 ? 1 : 2;            // row tiles
  static constexpr int kRows = kGroups * 128, kSoft = kGroups * 256, kThreads = kSoft + 64;
  static constexpr int kParts = F32 ? 3 : 1;             // of a query
  static constexpr int kAtoms = D / 64;                  // 64 16-bit elements: 128 bytes
  static constexpr int kTileBytes = kTile * D * 2;       // of 16-bit keys or values
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr int oQ = 0;                           // [row tile][part]
  static constexpr int oK = oQ + kGroups * kParts * 128 * D * 2;
  static constexpr int oV = oK + kStages * kTileBytes;
  static constexpr int kSmem = oV + kStages * kTileBytes + 1024;
  static constexpr int cS = 0, cO = 256;                 // columns of tensor memory: scores (and weights), values' sums
};

// One block a tile and kv head. Its first 128 threads look the tokens up; then D / 8 lanes
// take a token, 8 codes and one 16-byte store of each operand a lane.
template <int D>
__global__ void __launch_bounds__(256) widen_kernel(AttnParams p, WideParams w) {
  constexpr int L = D / 8, ROWS = 256 / L, STEPS = kTile / ROWS;
  __shared__ float s_max[4], s_ks[kTile], s_ev[kTile];
  __shared__ long long s_vec[kTile];
  griddep_wait();
  griddep_launch();
  const int tile = blockIdx.x, h = blockIdx.y, tid = threadIdx.x;
  const float nan = __int_as_float(0x7fffffff);
  if (tid < kTile) {
    const int t = tile * kTile + tid;
    long long vec = -1;
    float ks = 0.f, ev = -1e30f;
    if (t < p.fixed_len) {
      const int page = __ldg(p.table + (t >> p.page_shift));
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
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ev = fmaxf(ev, __shfl_xor_sync(kFull, ev, o));
    if ((tid & 31) == 0) s_max[tid >> 5] = ev;
  }
  __syncthreads();
  float e = fmaxf(fmaxf(s_max[0], s_max[1]), fmaxf(s_max[2], s_max[3]));
  if (e < -200.f) e = 0.f;  // no token with values
  if (tid == 0) w.exp[(long long)h * w.tiles + tile] = e + (float)kSumShift;
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
  const long long row0 = ((long long)h * w.tiles + tile) * kTile;
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    const int u = u0 + i * ROWS;
    const float ks = s_ks[u], ev = s_ev[u], vs = ks != ks ? nan : ev < -200.f ? 0.f : ex2(ev - e + (float)kValueShift);
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
      ov[j] = half2_of(y[2 * j] * vs, y[2 * j + 1] * vs);
    }
    *reinterpret_cast<uint4*>(w.k16 + (row0 + u) * D + sub * 8) = make_uint4(ok[0], ok[1], ok[2], ok[3]);
    *reinterpret_cast<uint4*>(w.v16 + (row0 + u) * D + sub * 8) = make_uint4(ov[0], ov[1], ov[2], ov[3]);
  }
}

__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {  // a in tensor memory
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void tc_ld32(uint32_t a, float* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
        "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]), "=f"(r[16]), "=f"(r[17]),
        "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]), "=f"(r[25]), "=f"(r[26]),
        "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
      : "r"(a));
}
__device__ __forceinline__ void tc_st16(uint32_t a, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(a)
      : "memory");
}
__device__ __forceinline__ void tma_rows(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

// 64 bytes of a row; whole sectors at once where they lie on the 32-byte grid (a warp's rows are far apart).
__device__ __forceinline__ void store64(void* p, const uint32_t (&y)[16]) {
  if (((uintptr_t)p & 31) == 0) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(static_cast<char*>(p) + 32 * i), "r"(y[8 * i]),
                   "r"(y[8 * i + 1]), "r"(y[8 * i + 2]), "r"(y[8 * i + 3]), "r"(y[8 * i + 4]), "r"(y[8 * i + 5]), "r"(y[8 * i + 6]),
                   "r"(y[8 * i + 7])
                   : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) static_cast<uint4*>(p)[i] = make_uint4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
  }
}

__device__ __forceinline__ void tma_queries(uint32_t dst, const CUtensorMap* map, int x, int head, int row, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(head), "r"(row), "r"(bar)
      : "memory");
}

template <int D, bool F32>
struct PreShared {
  using T = PreShape<D, F32>;
  Part line;
  uint64_t k_full[T::kStages], k_free[T::kStages], v_full[T::kStages], v_free[T::kStages];
  uint64_t q_full, q_free, drained, s_full[2], p_full[2], o_done[2];
  uint32_t tmem;
  int gave_up;
  float top[T::kGroups][2][128];  // of the halves of a row: the largest score, then the sum
};

// CHUNK: the rows of every sequence over the prefix and its own tokens, causal (kernels_attn_chunk.cuh);
// otherwise the rows of the whole batch over the prefix, whose part goes to dst_o and dst_lse.
template <int D, bool CHUNK, bool F32>
__global__ void __launch_bounds__((PreShape<D, F32>::kThreads), 1)
attn_prefix_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ WideParams wide,
                   const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                   const __grid_constant__ CUtensorMap map_q) {
  using T = PreShape<D, F32>;
  using E16 = std::conditional_t<F32, float, uint16_t>;  // queries and output
  static_assert(CHUNK || !F32, "the prefix pass takes bf16 queries");
  constexpr int NR = T::kRows, NST = T::kStages, kSoftThreads = T::kSoft, kCopyWarp = T::kSoft / 32, kMmaWarp = kCopyWarp + 1;
  extern __shared__ uint8_t dyn[];
  __shared__ PreShared<D, F32> sh;
  const uint32_t dyn_raw = (uint32_t)__cvta_generic_to_shared(dyn);
  const uint32_t base = (dyn_raw + 1023u) & ~1023u;
  uint8_t* const mem = dyn + (base - dyn_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto bar = [](const uint64_t& b) { return (uint32_t)__cvta_generic_to_shared(&b); };
  volatile int* gave_up = &sh.gave_up;

  if (tid == 0) {
    for (int i = 0; i < NST; ++i) {
      mbar_init(bar(sh.k_full[i]), 1);
      mbar_init(bar(sh.k_free[i]), 1);
      mbar_init(bar(sh.v_full[i]), 1);
      mbar_init(bar(sh.v_free[i]), 1);
    }
    mbar_init(bar(sh.q_full), CHUNK && wide.q_tma ? 1 : kSoftThreads);
    mbar_init(bar(sh.q_free), 1);
    mbar_init(bar(sh.drained), 1);
    for (int w = 0; w < 2; ++w) {
      mbar_init(bar(sh.s_full[w]), 1);
      mbar_init(bar(sh.p_full[w]), 8);
      mbar_init(bar(sh.o_done[w]), 1);
    }
    sh.gave_up = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     (uint32_t)__cvta_generic_to_shared(&sh.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    tc_before();
  }
  griddep_wait();
  griddep_launch();
  const Part line = CHUNK ? locate_chunk(wide.c, p.Hk, sh.line) : locate_block<NR>(p, sh.line);  // (the prefix: one dense sequence, no cu)
  tc_after();
  const uint32_t tmem = sh.tmem;
  Place at = line.at;
  int left = line.end - line.begin;
  const int group = CHUNK ? p.block_rows / T::kGroups : 128;  // rows of a group
  if (CHUNK && !line.ok) fill_nan<E16, D>(p, blockIdx.x, gridDim.x, T::kThreads);
  auto next = [&]() -> WideSeg {
    if constexpr (CHUNK) {
      return next_chunk(p, wide.c, at, left);
    } else {
      WideSeg g;
      static_cast<Seg&>(g) = next_seg<NR>(p, at, left);
      g.row0 = g.w0 = 0;  // (all rows of the batch)
      return g;
    }
  };
  auto wide_tile = [&](const WideSeg& g, int tile) { return CHUNK ? tile + (tile < wide.c.pre_tiles ? 0 : g.w0) : tile; };

  if (warp == kCopyWarp) {
    // ---- the rings of tiles ----
    if (lane == 0) {
      asm volatile("fence.proxy.async.global;" ::: "memory");  // the widened prefix was written with ordinary stores
      int gi = 0, nseg = 0;
      while (left > 0) {
        const WideSeg g = next();
        if (CHUNK && wide.q_tma && g.n > 0) {
          // the stretch's queries, as soon as the last scores of the one before are computed: while its ends are worked on
          const int groups = T::kGroups == 2 && g.rows * p.G - g.f0 > group ? 2 : 1;
          if (nseg > 0) tc_wait_one(bar(sh.q_free), (nseg - 1) & 1, gave_up, p.status);
          ++nseg;
          mbar_expect_arrive(bar(sh.q_full), groups * group * D * 2);
          for (int w = 0; w < groups; ++w)
#pragma unroll
            for (int a = 0; a < T::kAtoms; ++a)
              tma_queries(base + T::oQ + w * 128 * D * 2 + a * 16384, &map_q, a * 64, g.h * p.G, g.row0 + (g.f0 + w * group) / p.G, bar(sh.q_full));
        }
        for (int k = 0; k < g.n; ++k, ++gi) {
          const int st = gi % NST, row = (g.h * wide.tiles + wide_tile(g, g.t0 + k)) * kTile;
          const uint32_t bk = bar(sh.k_full[st]), bv = bar(sh.v_full[st]);
          if (gi >= NST) tc_wait_one(bar(sh.k_free[st]), (gi / NST - 1) & 1, gave_up, p.status);
          mbar_expect_arrive(bk, T::kTileBytes);
#pragma unroll
          for (int a = 0; a < T::kAtoms; ++a)
            tma_rows(base + T::oK + st * T::kTileBytes + a * 16384, &map_k, a * 64, row, bk);
          if (gi >= NST) tc_wait_one(bar(sh.v_free[st]), (gi / NST - 1) & 1, gave_up, p.status);
          mbar_expect_arrive(bv, T::kTileBytes);
#pragma unroll
          for (int a = 0; a < T::kAtoms; ++a)
            tma_rows(base + T::oV + st * T::kTileBytes + a * 16384, &map_v, a * 64, row, bv);
        }
      }
      // no copy is left in flight when the block ends, even after a wait that gave up
      for (int it = 0; nseg > 0 && it < kTcPollLimit && !mbar_try_wait(bar(sh.q_full), (nseg - 1) & 1); ++it) {
      }
      for (int i = 0; i < NST; ++i)
        for (int it = 0; gi > i && it < kTcPollLimit && !(mbar_try_wait(bar(sh.k_full[i]), ((gi - 1 - i) / NST) & 1) &&
                                                         mbar_try_wait(bar(sh.v_full[i]), ((gi - 1 - i) / NST) & 1)); ++it) {
        }
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // ---- the MMAs: of one group the values' sum of a tile and the next scores, then of the other ----
    constexpr uint32_t id_s = 1u << 4 | 1u << 7 | 1u << 10 | (128u >> 3) << 17 | 8u << 24;  // bf16 x bf16, K-major
    constexpr uint32_t id_o = 1u << 4 | 1u << 16 | (uint32_t)(D >> 3) << 17 | 8u << 24;      // f16 x f16, values token by token
    constexpr uint64_t hi = mma_desc_hi(1024, 2), lbo_v = (uint64_t)(16384 >> 4) << 16;
    const uint32_t tm = __shfl_sync(kFull, tmem, 0);
    int gi = 0, nseg = 0, done[2] = {0, 0};
    auto scores = [&](int w, int i) {
      const uint32_t b = (base + T::oK + (i % NST) * T::kTileBytes) >> 4;
#pragma unroll
      for (int part = T::kParts - 1; part >= 0; --part) {  // (the small parts first)
        const uint32_t a = (base + T::oQ + (w * T::kParts + part) * 128 * D * 2) >> 4;
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
          const uint32_t off = (uint32_t)((s >> 2) * 16384 + (s & 3) * 32) >> 4;
          mma_f16(tm + T::cS + w * 128, hi | (a + off), hi | (b + off), id_s, part < T::kParts - 1 || s > 0);
        }
      }
      mma_commit(bar(sh.s_full[w]));
    };
    while (left > 0) {
      const WideSeg g = next();
      const int n = __shfl_sync(kFull, g.n, 0), groups = __shfl_sync(kFull, T::kGroups == 2 && g.rows * p.G - g.f0 > group ? 2 : 1, 0);
      if (n == 0) continue;
      tc_wait(bar(sh.q_full), nseg & 1, gave_up, p.status);
      ++nseg;
      tc_wait(bar(sh.k_full[gi % NST]), (gi / NST) & 1, gave_up, p.status);
      __syncwarp();
      tc_after();
      if (elect()) {
        scores(0, gi);
        if (groups == 2) scores(1, gi);
        mma_commit(bar(sh.k_free[gi % NST]));
        if (CHUNK && n == 1) mma_commit(bar(sh.q_free));
      }
      __syncwarp();
      for (int k = 0; k < n; ++k, ++gi) {
        const int st = gi % NST;
        for (int w = 0; w < groups; ++w) {
          if (w == 0) {
            tc_wait(bar(sh.v_full[st]), (gi / NST) & 1, gave_up, p.status);
            if (k + 1 < n) tc_wait(bar(sh.k_full[(gi + 1) % NST]), ((gi + 1) / NST) & 1, gave_up, p.status);
          }
          // a group counts its own tiles: they differ where a stretch has one group
          tc_wait(bar(sh.p_full[w]), (w == 0 ? done[0]++ : done[1]++) & 1, gave_up, p.status);
          __syncwarp();
          tc_after();
          if (elect()) {
            const uint32_t b = (base + T::oV + st * T::kTileBytes) >> 4;
#pragma unroll
            for (int part = F32 ? 1 : 0; part >= 0; --part)
#pragma unroll
              for (int s = 0; s < kTile / 16; ++s)
                mma_f16_ts(tm + T::cO + w * 128, tm + T::cS + w * 128 + part * 64 + s * 8, hi | lbo_v | (b + s * (2048 >> 4)), id_o,
                           s > 0 || k > 0 || (F32 && part == 0));
            if (k + 1 < n)
              scores(w, gi + 1);
            else
              mma_commit(bar(sh.o_done[w]));
            if (w + 1 == groups) {
              mma_commit(bar(sh.v_free[st]));
              if (k + 1 < n) mma_commit(bar(sh.k_free[(gi + 1) % NST]));
              if (CHUNK && k + 2 == n) mma_commit(bar(sh.q_free));
            }
          }
          __syncwarp();
        }
      }
    }
    // no MMA is left in flight when the block ends, even after a wait that gave up
    if (elect()) mma_commit(bar(sh.drained));
    __syncwarp();
    for (int it = 0; it < kTcPollLimit && !mbar_try_wait(bar(sh.drained), 0); ++it) {
    }
  } else {
    // ---- softmax: group w, a row and half of a tile's tokens a thread ----
    const int w = warp >> 3, half = (warp >> 2) & 1, t = tid & 127, c = w * group + t;
    const int pair_bar = 1 + w * 4 + (warp & 3);  // the two warps that share 32 rows
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lanes + T::cS + w * 128, tO = tmem + lanes + T::cO + w * 128;
    const float nan = __int_as_float(0x7fffffff), ninf = __int_as_float(kNegInfBits);
    unsigned tiles_done = 0, ends = 0;
    if (tid == 0) p.cut[blockIdx.x].parts = 0;
    while (left > 0) {
      const WideSeg g = next();
      if (g.n == 0) continue;
      if (left == 0 && tid == 0) p.cut[blockIdx.x] = cut_rec(g, blockIdx.x, gridDim.x, line.end, line.total);
      const int f = g.f0 + c, flat = CHUNK && t >= group ? 0 : g.rows * p.G;  // (rows past the group's are none)
      // half of this thread's query row into shared memory, swizzled
      bool bad = false;  // a query that is no finite number
      if constexpr (F32) {
        // cut to bf16, what is left cut again, and again: exact (and what is no finite number leaves a NaN)
        uint8_t* const q = mem + T::oQ;
        const float* src = static_cast<const float*>(p.q) + (long long)(g.row0 + f / p.G) * p.q_row + (long long)(g.h * p.G + f % p.G) * p.q_head;
        const bool vec = ((uintptr_t)src & 15) == 0;
#pragma unroll 1
        for (int i8 = 0; i8 < D / 16; ++i8) {
          const int ch = half * (D / 16) + i8;
          Raw8<float> r{};
          if (f < flat) {
            if (vec)
              r.template load<true>(src + ch * 8);
            else
              r.template load<false>(src + ch * 8);
          }
          float x[8];
          r.floats(x);
#pragma unroll
          for (int part = 0; part < 3; ++part) {
            uint32_t y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t u = __float_as_uint(x[2 * i]) & 0xffff0000u, v = __float_as_uint(x[2 * i + 1]) & 0xffff0000u;
              y[i] = u >> 16 | v;
              x[2 * i] -= __uint_as_float(u);
              x[2 * i + 1] -= __uint_as_float(v);
            }
            *reinterpret_cast<uint4*>(q + part * 128 * D * 2 + (ch >> 3) * 16384 + t * 128 + (((ch & 7) ^ (t & 7)) * 16)) =
                make_uint4(y[0], y[1], y[2], y[3]);
          }
        }
        fence_async();
        mbar_arrive(bar(sh.q_full));
      } else if (!(CHUNK && wide.q_tma)) {
        uint8_t* const q = mem + T::oQ + w * 128 * D * 2;
        const uint16_t* src = static_cast<const uint16_t*>(p.q) + (long long)(g.row0 + f / p.G) * p.q_row +
                              (long long)(g.h * p.G + f % p.G) * p.q_head;
        const bool vec = ((uintptr_t)src & 15) == 0;
#pragma unroll
        for (int i8 = 0; i8 < D / 16; ++i8) {
          const int ch = half * (D / 16) + i8;
          uint32_t x[4] = {0, 0, 0, 0};
          if (f < flat) {
            if (vec) {
              const uint4 v = __ldg(reinterpret_cast<const uint4*>(src) + ch);
              x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                x[i] = (uint32_t)__ldg(src + ch * 8 + 2 * i) | (uint32_t)__ldg(src + ch * 8 + 2 * i + 1) << 16;
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) bad |= (x[i] & 0x7f80u) == 0x7f80u || (x[i] & 0x7f800000u) == 0x7f800000u;
          *reinterpret_cast<uint4*>(q + (ch >> 3) * 16384 + t * 128 + (((ch & 7) ^ (t & 7)) * 16)) = make_uint4(x[0], x[1], x[2], x[3]);
        }
        fence_async();
        mbar_arrive(bar(sh.q_full));
      }
      const bool have = g.rows * p.G - g.f0 > w * group;  // this group has rows
      // of the sequence's own tokens this row sees the first `own`
      const int own = CHUNK ? (f < flat ? g.len - g.rows + f / p.G + 1 : 0) : g.len, pre_tiles = CHUNK ? wide.c.pre_tiles : 0;
      // Weights are 2^((s - far) c + E - m). Of scores in the millions c s + E - m keeps no places: such a row's are counted from
      // the largest one, whose difference to others is exact.
      float m = 0.f, l = 0.f, far = 0.f;
      if (have) {
        for (int k = 0; k < g.n; ++k, ++tiles_done) {
          const int tile = g.t0 + k;
          int valid = own - tile * kTile - half * 64;
          if constexpr (CHUNK) valid = (tile < pre_tiles ? (f < flat ? wide.c.pre_len : 0) - tile * kTile : own - (tile - pre_tiles) * kTile) - half * 64;
          const long long info = (long long)g.h * wide.tiles + wide_tile(g, tile);
          float E;
          bool mixed = false;
          if constexpr (CHUNK) {
            const float2 e = __ldcg(wide.info + info);
            E = e.x;
            mixed = e.y != 0.f;
          } else {
            E = __ldcg(wide.exp + info);
          }
          tc_wait(bar(sh.s_full[w]), tiles_done & 1, gave_up, p.status);
          tc_after();
          float s[64];
          tc_ld32(tS + half * 64, s);
          tc_ld32(tS + half * 64 + 32, s + 32);
          tc_wait_ld();
          if (valid < 64) {
#pragma unroll
            for (int i = 0; i < 64; ++i)
              if (i >= valid) s[i] = ninf;
          }
          if (CHUNK && far != 0.f) {
#pragma unroll
            for (int i = 0; i < 64; ++i) s[i] -= far;
          }
          if (CHUNK && mixed) {  // the values' exponents join the scores
            const float inv = 1.f / p.c;
            const float* ev = wide.ev + info * kTile + half * 64;
#pragma unroll
            for (int i = 0; i < 64; ++i) s[i] = fmaf(__ldcg(ev + i), inv, s[i]);
            E = 0.f;
          }
          float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
          for (int i = 4; i < 64; i += 4)
#pragma unroll
            for (int j = 0; j < 4; ++j) mx[j] = fmaxf(mx[j], s[i + j]);
          float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
          // (the barrier also stands between both halves' loads and the weights that overwrite scores)
          if (bar_or(pair_bar, 64, k == 0 || fmaf(top, p.c, E - m) > kOverP)) {
            sh.top[w][half][t] = top;
            bar_sync(pair_bar, 64);
            top = fmaxf(top, sh.top[w][half ^ 1][t]);
            const float x = fmaf(top, p.c, E - m);
            const bool renew = top != ninf && (k == 0 || x > kOverP);
            float d = renew ? x - kTopP : 0.f, shift = 0.f;
            if (CHUNK && renew && fabsf(x) > kFarP) {
              shift = top;
              d = E - kTopP - m;
#pragma unroll
              for (int i = 0; i < 64; ++i) s[i] -= shift;
            }
            const float fac = ex2(CHUNK ? -fmaf(shift, p.c, d) : -d);
            m += d;
            far += shift;
            if (k > 0) {  // the tiles before are summed: the scores' barrier stands behind their MMAs
              l *= fac;
#pragma unroll 1
              for (int i = half * (D / 2); i < (half + 1) * (D / 2); i += 16) {
                uint32_t o[16];
                tc_ld8(tO + i, *reinterpret_cast<uint32_t(*)[8]>(o));
                tc_ld8(tO + i + 8, *reinterpret_cast<uint32_t(*)[8]>(o + 8));
                tc_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * fac);
                tc_st16(tO + i, o);
              }
            }
          }
          const float off = E - m;
          if (CHUNK && mixed) {
            const float* ev = wide.ev + info * kTile + half * 64;
#pragma unroll
            for (int i = 0; i < 64; ++i) l += ex2(fmaf(s[i], p.c, off) - __ldcg(ev + i));
          }
          const f2 c2 = pack(p.c, p.c), off2 = pack(off, off);
          f2 sum[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
          for (int i = 0; i < 64; i += 32) {
            uint32_t h[16], rest[16];
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
              float a, b;
              unpack(fma2(pack(s[i + j], s[i + j + 1]), c2, off2), a, b);
              a = ex2(a);
              b = ex2(b);
              sum[(j >> 1) & 3] = add2(sum[(j >> 1) & 3], pack(a, b));
              h[j / 2] = half2_of(a, b);
              if constexpr (F32) {
                const float2 r = __half22float2(*reinterpret_cast<const __half2*>(&h[j / 2]));
                rest[j / 2] = half2_of(a - r.x, b - r.y);
              }
            }
            tc_st16(tS + half * 32 + i / 2, h);
            if constexpr (F32) tc_st16(tS + 64 + half * 32 + i / 2, rest);
          }
          tc_wait_st();
          tc_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(sh.p_full[w]));
          float a, b;
          unpack(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), a, b);
          if (!(CHUNK && mixed)) l += (a + b) * ex2(-E);
        }
        // ---- the end of the stretch ----
        if (!CHUNK && bad) l = nan;
        if (CHUNK) m = fmaf(far, p.c, m);
        bar_sync(pair_bar, 64);  // the last maxima are read
        sh.top[w][half][t] = l;
        bar_sync(pair_bar, 64);
        l += sh.top[w][half ^ 1][t];
        if constexpr (CHUNK) {
          // Every score of a row that sees tokens of this stretch was -inf, as a hidden token's is: an infinite query met keys of
          // one sign (or scores passed fp32's range). That row is NaN; only one that sees none of the stretch has no part in it.
          const bool sees = f < flat && (g.t0 < pre_tiles || own > (g.t0 - pre_tiles) * kTile);
          if (sees && l == 0.f) l = nan;
        }
        tc_wait(bar(sh.o_done[w]), ends & 1, gave_up, p.status);
        ++ends;
        tc_after();
        const bool whole = g.n == g.nt;
        float* slot = whole ? nullptr : slot_of<NR, D>(p, 2 * blockIdx.x + (g.t0 == 0 ? 1 : 0));
        const long long idx = (long long)(g.row0 + f / p.G) * p.Hq + g.h * p.G + f % p.G;
        Coef r{};
        if (!whole) {
          if (half == 0 && (!CHUNK || t < group)) {
            slot[c] = CHUNK && l == 0.f ? ninf : m;  // a row that saw nothing has no reference
            slot[NR + c] = l;
          }
        } else if (f < flat) {
          r = row_coef(ninf, m, l, CHUNK && g.bad);
          if (half == 0) finish_lse(p, idx, r);
        }
        float* dst = whole ? (CHUNK ? nullptr : p.dst_o + idx * D) : slot + 2 * NR + c * D;
        const float scale = (whole ? r.a : 1.f / kSumUnit<E16>) * (1.f / (1 << (kValueShift + kSumShift)));
#pragma unroll 1
        for (int i = half * (D / 2); i < (half + 1) * (D / 2); i += 32) {
          float o[32];
          tc_ld32(tO + i, o);
          tc_wait_ld();
          if (F32 && whole) {
            if (f < flat && in_idx(idx, (long long)p.R * p.Hq, p.status)) {
#pragma unroll
              for (int j = 0; j < 32; j += 4)
                *reinterpret_cast<float4*>(static_cast<float*>(p.o) + idx * D + i + j) =
                    make_float4(o[j] * scale, o[j + 1] * scale, o[j + 2] * scale, o[j + 3] * scale);
            }
          } else if (CHUNK && whole) {
            if (f < flat && in_idx(idx, (long long)p.R * p.Hq, p.status)) {
              uint32_t y[16];
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(o[2 * j] * scale, o[2 * j + 1] * scale);
                y[j] = *reinterpret_cast<const uint32_t*>(&b);
              }
              store64(static_cast<uint16_t*>(p.o) + idx * D + i, y);
            }
          } else if (f < flat && in_idx(idx, (long long)p.R * p.Hq, p.status)) {
#pragma unroll
            for (int j = 0; j < 32; j += 4)
              *reinterpret_cast<float4*>(dst + i + j) = make_float4(o[j] * scale, o[j + 1] * scale, o[j + 2] * scale, o[j + 3] * scale);
          }
        }
        tc_before();
      }
      if (!(CHUNK && wide.q_tma)) bar_sync(9, kSoftThreads);  // both groups are done with the queries' memory
    }
  }
  tc_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
}

}  // namespace sv
