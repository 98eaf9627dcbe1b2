// The weight that cached tokens gather: for each token and kv head, the sum over a round's
// rows and the head's query heads of the softmax weights exp(scale * q . k - lse), from the
// log-sums that the attention has left.
//
// Only the keys are read. A warp takes 32 tokens, whose codes pass through a ring of its own in
// shared memory (nothing of it is shared between warps, so none waits for another), and are, widened
// to f16 (exact), the first operand of m16n8k16 MMAs; the queries, f16 in shared memory, are the
// second, 8 rows at a time. Which elements share a step of an MMA does not matter as long as both
// operands agree, so a lane takes 16 neighbouring codes of a token by one load. The sum over rows
// ends in the lanes that hold the token: no maxima, no second product, and the sum does not depend
// on what runs when.
//
// A bf16 query is, scaled by its row's power of two to below 2^15, exactly an f16 number down
// to 2^-39 of the row's largest element; an fp32 query is two of them (22 bits).
//
// Few rows leave it bound by the keys' bytes: 256 sequences x 1 row x 4 heads to 1-8192 tokens 186
// us, 6.2 TB/s. More rows are bound by the MMAs and the instructions around them, hardly side by
// side (12 warps an SM hold the widened codes; with half of the MMAs left out 50 us): 8 windows of 32 rows x 4 heads behind 2000-16384
// tokens 68 us, 300 TFLOP/s. Those would need the fifth-generation MMAs, whose scores come with
// tokens on the lanes as well; not built.
#pragma once

#include "kernels_attn.cuh"

namespace sv {

constexpr int kWeighThreads = 128;
constexpr int kWeighStages = 2;         // tiles of a warp on their way or worked on
constexpr int kWeighAllRows = 1 << 14;  // a sequence's rows are one row block on the line of tiles

struct WeighParams {
  AttnParams a;
  const float* lse;           // [R][Hq]
  const int32_t* n_accepted;  // [B]: rows 0..n_accepted[b] count; null: all
  float* mass;                // [num_pages][Hk][page_size]
  float keep, scale;
};

// four e4m3 codes as two pairs of f16
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=&r"(lo), "=r"(hi)
      : "r"(w));
}
__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// 16 bytes to shared memory, or zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool some) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(some ? 16 : 0) : "memory");
}

// FEW: no sequence has more than 8 rows (times heads of a kv head). Codes are then widened where an MMA takes them, and with
// half of the registers twice the warps fit an SM.
template <typename E, int D, bool FEW>
struct WeighShape {
  // Rows (query rows times heads of a kv head) at a time: the codes are read and widened again for each such number. 128 of
  // bf16 (35 KB at head_dim 128) leave room for the blocks that the registers allow: 8 windows of 32 rows x 4 heads 68 us,
  // with 64 at a time 73. fp32 queries are two parts, and 128 of them would cost a block an SM.
  static constexpr int kCols = FEW ? 8 : sizeof(E) == 2 ? 128 : 64;
  static constexpr int kRing = kWeighThreads * kWeighStages * D;  // bytes
  static constexpr int kParts = sizeof(E) == 2 ? 1 : 2;
  static constexpr int kStride = D + 8;  // halves of a row: neighbouring rows' 16-byte loads fall into different banks
};

// Columns c0 + at on of a segment's rows to columns `at` on of shared memory, two threads a column.
template <typename E, int D, bool FEW>
__device__ __forceinline__ void weigh_stage(const WeighParams& p, const Seg& g, int counted, int c0, int at, __half* q, float* rq, float* neg, int* lim) {
  using T = WeighShape<E, D, FEW>;
  const AttnParams& a = p.a;
  const int col = at + (threadIdx.x >> 1), part = threadIdx.x & 1, f = c0 + col, i = f / a.G;
  if (FEW && threadIdx.x >= 32) return;  // (whole warps)
  bool here = f < g.rows * a.G && i < counted;
  float x[D / 2];
#pragma unroll
  for (int k = 0; k < D / 2; ++k) x[k] = 0.f;
  float lse = 0.f;
  if (here) {
    const int hq = g.h * a.G + f - i * a.G;
    lse = __ldg(p.lse + (long long)(g.row0 + i) * a.Hq + hq);
    here = fabsf(lse) <= 3.402823466e38f;  // a row that sees nothing, or whose sum is no number, adds nothing
    const E* src = static_cast<const E*>(a.q) + (long long)(g.row0 + i) * a.q_row + (long long)hq * a.q_head + part * (D / 2);
    if (here) {
      if (((uintptr_t)src & 15) == 0) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          Raw8<E> r;
          r.template load<true>(src + 8 * k);
          r.floats(*reinterpret_cast<float(*)[8]>(x + 8 * k));
        }
      } else {
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          Raw8<E> r;
          r.template load<false>(src + 8 * k);
          r.floats(*reinterpret_cast<float(*)[8]>(x + 8 * k));
        }
      }
    }
  }
  uint32_t top = 0;
#pragma unroll
  for (int k = 0; k < D / 2; ++k) top = max(top, __float_as_uint(x[k]) & 0x7fffffffu);
  top = max(top, __shfl_xor_sync(kFull, top, 1));
  if (FEW && col >= T::kCols) return;
  const int e = max((int)(top >> 23) - 127, -100) - 14;  // the largest element comes to [2^14, 2^15)
  const float inv = __int_as_float((127 - e) << 23);
  uint32_t* dst = reinterpret_cast<uint32_t*>(q + col * T::kStride + part * (D / 2));
#pragma unroll
  for (int k = 0; k < D / 2; k += 2) {
    const float y0 = x[k] * inv, y1 = x[k + 1] * inv;
    const uint32_t hi = pack_f16(y0, y1);
    dst[k / 2] = hi;
    if constexpr (T::kParts == 2) {
      const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&hi));
      dst[T::kCols * T::kStride / 2 + k / 2] = pack_f16(y0 - h.x, y1 - h.y);
    }
  }
  if (part == 0) {
    rq[col] = here ? p.scale * __int_as_float((e + 127) << 23) : 0.f;
    neg[col] = here ? -lse : 0.f;
    lim[col] = here ? g.len - g.rows + i + 1 : 0;  // the row sees the tokens before this one
  }
}

// The weights of 8 NB columns from column 8 nt on, added to the sums of this lane's tokens tok, tok + 8, ...
// `codes(m, j)`: this lane's 16 codes of piece j of token tok + 8 m, as 4 words; `lo`, `hi`: the same widened, where they are
// kept (not FEW).
template <typename E, int D, bool FEW, int NB, typename F>
__device__ __forceinline__ void weigh_columns(const __half* s_q, const float* s_rq, const float* s_neg, const int* s_lim, int nt, F codes,
                                              const uint32_t (&lo)[4][D / 64][4], const uint32_t (&hi)[4][D / 64][4], const float (&ks)[4],
                                              int tok, float (&sum)[4]) {
  using T = WeighShape<E, D, FEW>;
  const int t4 = threadIdx.x & 3, g8 = (threadIdx.x & 31) >> 2;
  float acc[NB][2][4];
#pragma unroll
  for (int n = 0; n < NB; ++n)
#pragma unroll
    for (int m = 0; m < 2; ++m) acc[n][m][0] = acc[n][m][1] = acc[n][m][2] = acc[n][m][3] = 0.f;
#pragma unroll
  for (int part = T::kParts - 1; part >= 0; --part) {  // (the small parts first)
#pragma unroll
    for (int j = 0; j < D / 64; ++j) {
      uint32_t w[NB][8];
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        const uint4* q = reinterpret_cast<const uint4*>(s_q + (part * T::kCols + (nt + n) * 8 + g8) * T::kStride + t4 * 16) + j * 8;
        const uint4 q0 = q[0], q1 = q[1];
        w[n][0] = q0.x, w[n][1] = q0.y, w[n][2] = q0.z, w[n][3] = q0.w, w[n][4] = q1.x, w[n][5] = q1.y, w[n][6] = q1.z, w[n][7] = q1.w;
      }
      if constexpr (FEW) {
        const uint4 c[4] = {codes(0, j), codes(1, j), codes(2, j), codes(3, j)};
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          uint32_t l[4], h[4];
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const uint32_t x[4] = {c[m].x, c[m].y, c[m].z, c[m].w};
            widen4(x[s], l[m], h[m]);
          }
#pragma unroll
          for (int m = 0; m < 2; ++m) mma_16816(acc[0][m], l[2 * m], l[2 * m + 1], h[2 * m], h[2 * m + 1], w[0][2 * s], w[0][2 * s + 1]);
        }
      } else {
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
          for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int m = 0; m < 2; ++m)
              mma_16816(acc[n][m], lo[2 * m][j][s], lo[2 * m + 1][j][s], hi[2 * m][j][s], hi[2 * m + 1][j][s], w[n][2 * s], w[n][2 * s + 1]);
      }
    }
  }
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    const int col = (nt + n) * 8 + t4 * 2;
    const float2 rq = *reinterpret_cast<const float2*>(s_rq + col), neg = *reinterpret_cast<const float2*>(s_neg + col);
    const int2 lim = *reinterpret_cast<const int2*>(s_lim + col);
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const float* c = &acc[n][m >> 1][(m & 1) * 2];
      // the difference in natural units, where it is small, then in binary ones
      const float e0 = ex2(fmaf(c[0] * ks[m], rq.x, neg.x) * 1.4426950408889634f);
      const float e1 = ex2(fmaf(c[1] * ks[m], rq.y, neg.y) * 1.4426950408889634f);
      sum[m] += (tok + 8 * m < lim.x ? e0 : 0.f) + (tok + 8 * m < lim.y ? e1 : 0.f);
    }
  }
}

template <typename E, int D, bool FEW>
__global__ void __launch_bounds__(kWeighThreads, FEW ? (sizeof(E) == 2 ? 5 : 4) : 3) weigh_kernel(const __grid_constant__ WeighParams p) {
  using T = WeighShape<E, D, FEW>;
  constexpr int kCols = T::kCols;
  constexpr int CH = D / 64;  // 16-byte pieces of a token in a lane
  __shared__ Part s_part;
  __shared__ __align__(16) __half s_q[T::kParts * kCols * T::kStride];
  __shared__ __align__(16) float s_rq[kCols], s_neg[kCols];
  __shared__ __align__(16) int s_lim[kCols];
  __shared__ long long s_vec[kWeighThreads / 32][kWeighStages][32];
  extern __shared__ __align__(128) uint8_t s_ring[];  // [warp][stage][32 tokens][D]
  const AttnParams& a = p.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, t4 = lane & 3, g8 = lane >> 2;
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(s_ring) + warp * kWeighStages * (32 * D);
  griddep_wait();
  griddep_launch();
  const Part line = locate_block<kWeighAllRows>(a, s_part);
  uint32_t bits = line.ok ? 0 : SPEC_DEV_OFFSETS;
  Place at = line.at;
  int left = line.ok ? line.end - line.begin : 0;
  while (left > 0) {
    const int b = at.b;
    const Seg g = next_seg<kWeighAllRows>(a, at, left);
    if (g.n == 0) continue;
    int counted = g.rows;
    bool bad = g.bad;
    if (p.n_accepted != nullptr) {
      const int n = __ldg(p.n_accepted + b);
      bad |= n < 0 || n >= g.rows;
      counted = min(n + 1, g.rows);
    }
    if (bad) {
      bits |= SPEC_DEV_OFFSETS;
      continue;
    }
    const int ctx = g.len - g.rows;
    for (int c0 = 0; c0 == 0 || c0 < counted * a.G; c0 += kCols) {
      __syncthreads();
#pragma unroll 1
      for (int at_col = 0; at_col < (FEW ? 1 : min(kCols, counted * a.G - c0)); at_col += kWeighThreads / 2)
        weigh_stage<E, D, FEW>(p, g, counted, c0, at_col, s_q, s_rq, s_neg, s_lim);
      __syncthreads();
      const int tiles_n = min(kCols, counted * a.G - c0 + 7) / 8;  // of 8 columns
      // A warp's tiles pass through a ring of its own: the codes of tiles ahead are on their way to shared memory, and of the
      // next tile the exponents and the weights so far to registers.
      const int end = min(g.t0 + g.n, (g.len - warp * 32 + kTile - 1) / kTile);  // tiles that hold tokens of this warp's
      auto page_of = [&](int tile) -> int {
        const int t = tile * kTile + warp * 32 + lane;
        return tile < end && t < g.len ? __ldg(g.pages + (t >> a.page_shift)) : -1;
      };
      auto fetch = [&](int tile, int page) {
        const int t = tile * kTile + warp * 32 + lane, st = tile % kWeighStages;
        long long vec = -1;
        if (tile < end) {
          if (t < g.len) {
            if ((unsigned)page < (unsigned)a.num_pages)
              vec = (((long long)page * a.Hk + g.h) << a.page_shift) + (t & ((1 << a.page_shift) - 1));
            else
              bits |= SPEC_DEV_PAGE;
            if (vec >= 0 && !in_idx(vec, ((long long)a.num_pages * a.Hk) << a.page_shift, a.status)) vec = -1;
          }
          s_vec[warp][st][lane] = vec;
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            const int row = i * (512 / D) + lane / (D / 16), c = lane % (D / 16);
            const long long v = __shfl_sync(kFull, vec, row);
            const uint32_t dst = ring + st * (32 * D) + row * D + (D == 128 ? c ^ (row & 1) * 4 : c) * 16;
            copy16(dst, a.k + (v >= 0 ? v * D + c * 16 : 0), v >= 0);
          }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
      long long vec_next;
      unsigned exp_next = 0;
      float old_next = 0.f;
      auto peek = [&](int tile) {
        vec_next = tile < end ? s_vec[warp][tile % kWeighStages][lane] : -1;
        exp_next = vec_next >= 0 ? __ldg(a.k_exp + vec_next) : 0u;
        old_next = vec_next < 0 || (c0 == 0 && (tile * kTile + warp * 32 + lane >= ctx || p.keep == 0.f)) ? 0.f : p.mass[vec_next];
      };
      __syncwarp();  // (the stretch before is read)
#pragma unroll
      for (int i = 0; i < kWeighStages - 1; ++i) fetch(g.t0 + i, page_of(g.t0 + i));
      int page = page_of(g.t0 + kWeighStages - 1);
      peek(g.t0);  // (a lane reads the places that it wrote itself)
      for (int tile = g.t0; tile < end; ++tile) {
        const int tb = tile * kTile + warp * 32;
        const long long vec = vec_next;
        const float old = old_next, own_ks = exp_value(exp_next);
        fetch(tile + kWeighStages - 1, page);
        page = page_of(tile + kWeighStages);
        peek(tile + 1);
        asm volatile("cp.async.wait_group %0;" ::"n"(kWeighStages - 1) : "memory");
        __syncwarp();
        float ks[4], sum[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          ks[m] = __shfl_sync(kFull, own_ks, g8 + 8 * m);
          sum[m] = 0.f;
        }
        const uint8_t* const codes = s_ring + (warp * kWeighStages + tile % kWeighStages) * (32 * D);
        auto raw = [&](int m, int j) {
          const int row = g8 + 8 * m, c = 4 * j + t4;
          return *reinterpret_cast<const uint4*>(codes + row * D + (D == 128 ? c ^ (row & 1) * 4 : c) * 16);
        };
        uint32_t lo[4][CH][4], hi[4][CH][4];
        if constexpr (FEW) {
          weigh_columns<E, D, FEW, 1>(s_q, s_rq, s_neg, s_lim, 0, raw, lo, hi, ks, tb + g8, sum);
          __syncwarp();  // (the stage may be written again)
        } else {
#pragma unroll
          for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int j = 0; j < CH; ++j) {
              const uint4 x = raw(m, j);
              const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
              for (int s = 0; s < 4; ++s) widen4(w[s], lo[m][j][s], hi[m][j][s]);
            }
          __syncwarp();  // (the stage may be written again)
          // two groups of 8 columns at once where there are more (the MMAs of one wait for one another; columns past the last are zeros)
          if (tiles_n == 1) {
            weigh_columns<E, D, FEW, 1>(s_q, s_rq, s_neg, s_lim, 0, raw, lo, hi, ks, tb + g8, sum);
          } else {
#pragma unroll 1
            for (int nt = 0; nt < tiles_n; nt += 2) weigh_columns<E, D, FEW, 2>(s_q, s_rq, s_neg, s_lim, nt, raw, lo, hi, ks, tb + g8, sum);
          }
        }
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          sum[m] += __shfl_xor_sync(kFull, sum[m], 1);
          sum[m] += __shfl_xor_sync(kFull, sum[m], 2);
        }
        // lane l's token is in the lanes of l % 8: the sum of number l / 8
        float mine = 0.f;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const float x = __shfl_sync(kFull, sum[m], (lane & 7) * 4);
          if ((lane >> 3) == m) mine = x;
        }
        if (vec >= 0) p.mass[vec] = fmaf(c0 == 0 ? p.keep : 1.f, old, mine);
      }
    }
  }
  if (bits) atomicOr(a.status, bits);
}

}  // namespace sv
