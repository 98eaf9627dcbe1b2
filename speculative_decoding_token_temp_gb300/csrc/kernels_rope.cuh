// Queries and keys on their way from a projection to the attention: the norm of each head,
// the rotation by the row's positions, and, into the 8-bit cache, the quantising write.
//
//   y_d = x_d * w_d / sqrt(mean(x^2) + eps)
//   (y_a, y_b) <- (y_a cos t - y_b sin t, y_b cos t + y_a sin t),  t = position * frequency
//
// Angles. A pair's frequency is held as turns a position in units of 2^-64 turn. The product
// with a 32-bit position, modulo 2^64, is the angle reduced to one turn, exactly, for every
// position: an angle of 10^6 radians in fp32 would be off by 0.03. Its upper 32 bits go to
// sincospif as half turns (2^-32 of a turn, then fp32's own 2^-24 of the angle).
//
// All arithmetic is fp32 from the source's elements to the one rounding at the end: bf16 or
// fp32 out, or the cache's codes (of the fp32 key, which is not rounded to bf16 on the way).
#pragma once

#include "kernels_kv.cuh"

namespace sv {

constexpr int kRopeThreads = 256;

struct RopeParams {
  KvParams kv;  // the sources of keys and values; with a cache: the cache, the rows' places
  const void* q;
  long long q_row, q_head;
  void *q_out, *k_out;  // k_out: without a cache
  const void *q_w, *k_w;
  float eps;
  int norm;             // 0: no norms
  int rows, Hq, heads;  // heads: queries', keys' and, with a cache, values'
  const int32_t* pos;
  int axes;
  const uint64_t* step;
  const uint8_t* axis;
  int rot, interleaved;
};

__device__ __forceinline__ float elem(const uint16_t* p) { return __uint_as_float((uint32_t)__ldg(p) << 16); }
__device__ __forceinline__ float elem(const float* p) { return __ldg(p); }

// A block takes R rows. Its threads compute the rows' sines and cosines, once for all heads;
// then 8 / R warps a row walk the row's heads, D / 8 lanes a head and 8 elements a lane, U
// groups of heads on their way at once.
template <typename E, int D, bool CACHE, bool VEC, int R>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int L = D / 8, GRP = 32 / L, W = kRopeThreads / 32 / R, U = 16 / (int)sizeof(E) / 2;
  __shared__ float2 s_turn[R][D / 2];  // cosine, sine
  __shared__ __align__(16) float s_w[2][D];
  griddep_wait();
  griddep_launch();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, sub = lane % L, grp = lane / L;
  const int row0 = blockIdx.x * R, row = row0 + warp / W;
  const bool here = row < p.rows;
  const int Hk = p.kv.Hk;
  uint32_t bits = 0;

  auto source = [&](int h) -> const E* {
    const E* s;
    if (h < p.Hq)
      s = static_cast<const E*>(p.q) + (long long)row * p.q_row + (long long)h * p.q_head;
    else if (h < p.Hq + Hk)
      s = static_cast<const E*>(p.kv.src_k) + (long long)row * p.kv.k_row + (long long)(h - p.Hq) * p.kv.k_head;
    else
      s = static_cast<const E*>(p.kv.src_v) + (long long)row * p.kv.v_row + (long long)(h - p.Hq - Hk) * p.kv.v_head;
    return s + sub * 8;
  };
  Raw8<E> raw[U]{};
  auto load = [&](int g) {  // groups g, g + W, ...
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = (g + u * W) * GRP + grp;
      if (here && h < p.heads) raw[u].template load<VEC>(source(h));
    }
  };
  int g = warp % W;
  load(g);
  long long at = -1;
  if (CACHE && here) at = kv_place(p.kv, row, &bits);
  const int pairs = p.rot >> 1;
  for (int i = tid; i < R * pairs; i += kRopeThreads) {
    const int r = i / pairs, j = i - r * pairs;
    if (row0 + r < p.rows) {
      const int a = p.axis != nullptr ? min((int)__ldg(p.axis + j), p.axes - 1) : 0;
      const long long n = __ldg(p.pos + (long long)(row0 + r) * p.axes + a);
      const uint64_t turn = (uint64_t)n * __ldg(reinterpret_cast<const unsigned long long*>(p.step) + j);
      float s, c;
      sincospif((float)(int)(turn >> 32) * (1.f / 2147483648.f), &s, &c);
      s_turn[r][j] = make_float2(c, s);
    }
  }
  if (p.norm) {
    for (int i = tid; i < 2 * D; i += kRopeThreads) {
      const E* w = static_cast<const E*>(i < D ? p.q_w : p.k_w);
      s_w[i / D][i % D] = w != nullptr ? elem(w + i % D) : 1.f;
    }
  }
  __syncthreads();
  if (!here) return;

  // of this lane's elements: cosines, and sines with the sign that the element's partner gets
  const int half = p.rot >> 4;  // lanes of half of the rotated elements
  const bool turns = sub < 2 * half;
  const int partner = lane + (p.interleaved || !turns ? 0 : sub < half ? half : -half);
  float c[8], s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = 1.f, s[i] = 0.f;
  if (turns) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 t = s_turn[warp / W][p.interleaved ? sub * 4 + i / 2 : (sub < half ? sub : sub - half) * 8 + i];
      c[i] = t.x;
      s[i] = (p.interleaved ? (i & 1) == 0 : sub < half) ? -t.y : t.y;
    }
  }

  for (; g * GRP < p.heads; g += W * U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h0 = (g + u * W) * GRP, h = h0 + grp;
      if (h0 >= p.heads) break;  // (the whole warp)
      const bool is_q = h < p.Hq, is_v = h >= p.Hq + Hk;
      float x[8];
      raw[u].floats(x);
      if (p.norm) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
        if (!is_v) {
          const float f = __frsqrt_rn(fmaf(ss, 1.f / D, p.eps));
          const float4* w = reinterpret_cast<const float4*>(&s_w[is_q ? 0 : 1][sub * 8]);
          const float4 a = w[0], b = w[1];
          const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = x[i] * f * v[i];
        }
      }
      float y[8];
      if (p.interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = x[i ^ 1];
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = __shfl_sync(kFull, x[i], partner);
      }
      if (turns && !is_v) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = fmaf(x[i], c[i], y[i] * s[i]);
      }
      if (!CACHE) {
        if (h < p.heads) {
          E* to = is_q ? static_cast<E*>(p.q_out) + ((long long)row * p.Hq + h) * D
                       : static_cast<E*>(p.k_out) + ((long long)row * Hk + h - p.Hq) * D;
          store8(to + sub * 8, x);
        }
      } else {
        if (is_q) store8(static_cast<E*>(p.q_out) + ((long long)row * p.Hq + h) * D + sub * 8, x);
        if (h0 + GRP > p.Hq) {  // (the whole warp)
          uint32_t top = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
#pragma unroll
          for (int o = L / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(kFull, top, o));
          if (!is_q && h < p.heads && at >= 0) {
            const bool bad = top >= 0x7f800000u;
            const int e = top == 0 ? SPEC_KV_ZERO_EXP : vector_exp(top);
            const float inv = bad ? 0.f : __int_as_float((kExpBias - e) << 23);
            uint32_t w[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i] * inv, x[4 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
              const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i + 2] * inv, x[4 * i + 3] * inv), __NV_SATFINITE, __NV_E4M3);
              w[i] = bad ? 0u : lo | hi << 16;
            }
            const long long vec = at + ((long long)(is_v ? h - p.Hq - Hk : h - p.Hq) << p.kv.page_shift);
            if (in_idx(vec, ((long long)p.kv.num_pages * Hk) << p.kv.page_shift, p.kv.status)) {
              *reinterpret_cast<uint2*>((is_v ? p.kv.v : p.kv.k) + vec * D + sub * 8) = make_uint2(w[0], w[1]);
              if (sub == 0) (is_v ? p.kv.v_exp : p.kv.k_exp)[vec] = (uint8_t)(bad ? kNanExp : e + kExpBias);
            }
            if (bad) bits |= SPEC_DEV_NONFINITE;
          }
        }
      }
    }
    if ((g + W * U) * GRP < p.heads) load(g + W * U);
  }
  if (CACHE && bits) atomicOr(p.kv.status, bits);
}

}  // namespace sv
