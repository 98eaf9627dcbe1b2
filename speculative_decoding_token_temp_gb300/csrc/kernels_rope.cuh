// Queries and keys on their way from a projection to the attention: the norm of each head,
// the rotation by the row's positions, and, into the 8-bit cache, the quantising write.
//
//   y_d = x_d * w_d / sqrt(mean(x^2) + eps)
//   (y_a, y_b) <- (y_a cos t - y_b sin t, y_b cos t + y_a sin t),  t = position * frequency
//
// Angles. A pair's frequency is held as turns a position in units of 2^-64 turn. The product
// with a 32-bit position, modulo 2^64, is the angle reduced to one turn, exactly, for every
// position: an angle of 10^6 radians in fp32 would be off by 0.03. Less its nearest quarter turn it
// goes to sincospif as half turns of at most 1/4 (off by 2^-25 of that).
//
// A head's elements are rotated as f * (x_a * (w_a cos) + x_b * (w_b sin)), f = 1 / sqrt(...): the
// weights join the row's sines and cosines, once for all its heads, and what lanes exchange are
// the source's own elements, two bf16 in a register.
//
// All arithmetic is fp32 from the source's elements to the one rounding at the end: bf16 or
// fp32 out, or the cache's codes (of the fp32 key, which is not rounded to bf16 on the way).
//
// What bounds it: HBM where rows are many: 32768 rows of 32 + 8 heads of 128 in bf16, 110 us, 6.1 TB/s
// of the measured 6.8 (instructions issued in 70 % of cycles). 2304 rows into the cache, whose data
// is in L2: 13.6 us. A few rows: 4 us, the chain of loads, sines, barrier, exchange.
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
  int rows, Hq;
  const int32_t* pos;
  int axes;
  const uint64_t* step;
  const uint8_t* axis;
  int rot, interleaved;
};

__device__ __forceinline__ float elem(const uint16_t* p) { return __uint_as_float((uint32_t)__ldg(p) << 16); }
__device__ __forceinline__ float elem(const float* p) { return __ldg(p); }

__device__ __forceinline__ void load8(float (&x)[8], const float* p) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

// The elements of another lane (`from`), or zeros.
__device__ __forceinline__ Raw8<uint16_t> other(const Raw8<uint16_t>& r, int from, bool some) {
  const uint32_t x = __shfl_sync(kFull, r.w.x, from), y = __shfl_sync(kFull, r.w.y, from);
  const uint32_t z = __shfl_sync(kFull, r.w.z, from), w = __shfl_sync(kFull, r.w.w, from);
  Raw8<uint16_t> o;
  o.w = make_uint4(some ? x : 0u, some ? y : 0u, some ? z : 0u, some ? w : 0u);
  return o;
}
__device__ __forceinline__ Raw8<float> other(const Raw8<float>& r, int from, bool some) {
  Raw8<float> o;
  o.a = make_float4(__shfl_sync(kFull, r.a.x, from), __shfl_sync(kFull, r.a.y, from), __shfl_sync(kFull, r.a.z, from), __shfl_sync(kFull, r.a.w, from));
  o.b = make_float4(__shfl_sync(kFull, r.b.x, from), __shfl_sync(kFull, r.b.y, from), __shfl_sync(kFull, r.b.z, from), __shfl_sync(kFull, r.b.w, from));
  if (!some) o.a = o.b = make_float4(0.f, 0.f, 0.f, 0.f);
  return o;
}

// Heads h, h + STEP, ... of a row, of which `src` is this lane's part of the first.
template <bool VEC, int STEP, typename E, int U>
__device__ __forceinline__ void load_heads(Raw8<E> (&raw)[U], const E* src, long long stride, int h, int heads) {
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (h + u * STEP < heads) raw[u].template load<VEC>(src + u * STEP * stride);
}
// All heads of one kind, from those in `raw` on; whole warps (`grp`: which of a warp's heads is this lane's).
template <bool VEC, int STEP, typename E, int U, typename F>
__device__ __forceinline__ void walk_heads(Raw8<E> (&raw)[U], const E* src, long long stride, int h, int grp, int heads, F each) {
  for (; h - grp < heads; h += U * STEP) {
    Raw8<E> next[U]{};
    src += U * STEP * stride;
    load_heads<VEC, STEP>(next, src, stride, h + U * STEP, heads);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (h - grp + u * STEP < heads) each(raw[u], h + u * STEP);
#pragma unroll
    for (int u = 0; u < U; ++u) raw[u] = next[u];
  }
}

// A block takes R rows. Its threads compute the rows' sines and cosines, once for all heads;
// then 8 / R warps a row walk the queries' heads, the keys' and the values' (D / 8 lanes a head,
// 8 elements a lane, as many heads side by side as a warp holds). The next heads are on their
// way while the ones before are worked on, the first of each kind from the beginning.
template <typename E, int D, bool CACHE, bool VEC, int R>
__global__ void __launch_bounds__(kRopeThreads, sizeof(E) == 2 ? 4 : 3) rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int L = D / 8, GRP = 32 / L, W = kRopeThreads / 32 / R, U = 4 / (int)sizeof(E), STEP = W * GRP;
  __shared__ __align__(16) float s_cos[R][D / 2], s_sin[R][D / 2];
  __shared__ __align__(16) float s_w[2][D];
  griddep_wait();
  griddep_launch();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, sub = lane % L, grp = lane / L;
  const int row0 = blockIdx.x * R, row = row0 + warp / W, h0 = warp % W * GRP + grp;
  const bool here = row < p.rows;
  const int Hk = p.kv.Hk;
  uint32_t bits = 0;

  const E* const q = static_cast<const E*>(p.q) + (long long)row * p.q_row + h0 * p.q_head + sub * 8;
  const E* const k = static_cast<const E*>(p.kv.src_k) + (long long)row * p.kv.k_row + h0 * p.kv.k_head + sub * 8;
  Raw8<E> raw_q[U]{}, raw_k[U]{};
  if (here) {
    load_heads<VEC, STEP>(raw_q, q, p.q_head, h0, p.Hq);
    load_heads<VEC, STEP>(raw_k, k, p.kv.k_head, h0, Hk);
  }
  long long at = -1;
  if (CACHE && here) at = kv_place(p.kv, row, &bits);
  const int pairs = p.rot >> 1;
  for (int i = tid; i < R * pairs; i += kRopeThreads) {
    const int r = i / pairs, j = i - r * pairs;
    if (row0 + r < p.rows) {
      const int a = p.axis != nullptr ? min((int)__ldg(p.axis + j), p.axes - 1) : 0;
      const long long n = __ldg(p.pos + (long long)(row0 + r) * p.axes + a);
      const uint64_t turn = (uint64_t)n * __ldg(reinterpret_cast<const unsigned long long*>(p.step) + j);
      // the nearest quarter turn, and what is left of it as half turns of at most 1/4 (a small number keeps more places)
      const unsigned quarter = (unsigned)((turn + (1ull << 61)) >> 62);
      const long long rest = (long long)(turn - ((uint64_t)quarter << 62));
      float s, c;
      sincospif((float)rest * (1.f / 9223372036854775808.f), &s, &c);
      s_cos[r][j] = quarter & 1 ? (quarter & 2 ? s : -s) : (quarter & 2 ? -c : c);
      s_sin[r][j] = quarter & 1 ? (quarter & 2 ? -c : c) : (quarter & 2 ? -s : s);
    }
  }
  for (int i = tid; i < 2 * D; i += kRopeThreads) {
    const E* w = static_cast<const E*>(i < D ? p.q_w : p.k_w);
    s_w[i / D][i % D] = w != nullptr ? elem(w + i % D) : 1.f;
  }
  __syncthreads();
  if (!here) return;

  const int half = p.rot >> 4;  // lanes of half of the rotated elements
  const bool turns = sub < 2 * half;
  const int shift = p.interleaved || !turns ? 0 : sub < half ? half : -half;  // to the lane of this one's partners
  // of this lane's elements: weight times cosine, and the partner's weight times the sine with the sign that the partner gets
  float2 c[4], s[4];
  auto turn_by = [&](int side) {
    float w[8], z[8], ci[8], si[8];
    load8(w, s_w[side] + sub * 8);
    if (p.interleaved) {
#pragma unroll
      for (int i = 0; i < 8; ++i) z[i] = w[i ^ 1];
      if (turns) {
        const float4 a = *reinterpret_cast<const float4*>(&s_cos[warp / W][sub * 4]), b = *reinterpret_cast<const float4*>(&s_sin[warp / W][sub * 4]);
        ci[0] = ci[1] = a.x, ci[2] = ci[3] = a.y, ci[4] = ci[5] = a.z, ci[6] = ci[7] = a.w;
        si[0] = -(si[1] = b.x), si[2] = -(si[3] = b.y), si[4] = -(si[5] = b.z), si[6] = -(si[7] = b.w);
      }
    } else {
      load8(z, s_w[side] + (sub + shift) * 8);
      if (turns) {
        const int j = (sub < half ? sub : sub - half) * 8;
        load8(ci, &s_cos[warp / W][j]);
        load8(si, &s_sin[warp / W][j]);
        if (sub < half) {
#pragma unroll
          for (int i = 0; i < 8; ++i) si[i] = -si[i];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 a = make_float2(w[2 * i], w[2 * i + 1]), b = make_float2(z[2 * i], z[2 * i + 1]);
      c[i] = turns ? mul2(make_float2(ci[2 * i], ci[2 * i + 1]), a) : a;
      s[i] = turns ? mul2(make_float2(si[2 * i], si[2 * i + 1]), b) : make_float2(0.f, 0.f);
    }
  };
  auto turned = [&](const Raw8<E>& raw, float (&x)[8]) {
    raw.floats(x);
    float2* const x2 = reinterpret_cast<float2*>(x);
    float f = 1.f;
    if (p.norm) {
      float2 ss = mul2(x2[0], x2[0]);
#pragma unroll
      for (int i = 1; i < 4; ++i) ss = fma2(x2[i], x2[i], ss);
      float sum = ss.x + ss.y;
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
      const float v = fmaf(sum, 1.f / D, p.eps);
      f = rsqrtf(v);
      const float off = fmaf(-v * f, f, 1.f);  // one step of Newton's takes the function's two places
      f = fmaf(0.5f * f, v > 0.f && off < 1.f ? off : 0.f, f);
    }
    float y[8];
    if (p.interleaved) {
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = turns ? x[i ^ 1] : 0.f;
    } else {
      other(raw, lane + shift, turns).floats(y);
    }
    const float2* const y2 = reinterpret_cast<const float2*>(y);
#pragma unroll
    for (int i = 0; i < 4; ++i) x2[i] = mul2(fma2(x2[i], c[i], mul2(y2[i], s[i])), make_float2(f, f));
  };
  auto to_cache = [&](const float (&x)[8], int h, uint8_t* codes, uint8_t* exps) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(kFull, top, o));
    if (h >= Hk || at < 0) return;
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
    const long long vec = at + ((long long)h << p.kv.page_shift);
    if (in_idx(vec, ((long long)p.kv.num_pages * Hk) << p.kv.page_shift, p.kv.status)) {
      *reinterpret_cast<uint2*>(codes + vec * D + sub * 8) = make_uint2(w[0], w[1]);
      if (sub == 0) exps[vec] = (uint8_t)(bad ? kNanExp : e + kExpBias);
    }
    if (bad) bits |= SPEC_DEV_NONFINITE;
  };

  turn_by(0);
  E* const q_out = static_cast<E*>(p.q_out) + (long long)row * p.Hq * D + sub * 8;
  walk_heads<VEC, STEP>(raw_q, q, p.q_head, h0, grp, p.Hq, [&](const Raw8<E>& raw, int h) {
    float x[8];
    turned(raw, x);
    if (h < p.Hq) store8(q_out + h * D, x);
  });
  Raw8<E> raw_v[U]{};
  const E* const v = CACHE ? static_cast<const E*>(p.kv.src_v) + (long long)row * p.kv.v_row + h0 * p.kv.v_head + sub * 8 : nullptr;
  if (CACHE) load_heads<VEC, STEP>(raw_v, v, p.kv.v_head, h0, Hk);
  turn_by(1);
  E* const k_out = CACHE ? nullptr : static_cast<E*>(p.k_out) + (long long)row * Hk * D + sub * 8;
  walk_heads<VEC, STEP>(raw_k, k, p.kv.k_head, h0, grp, Hk, [&](const Raw8<E>& raw, int h) {
    float x[8];
    turned(raw, x);
    if (CACHE)
      to_cache(x, h, p.kv.k, p.kv.k_exp);
    else if (h < Hk)
      store8(k_out + h * D, x);
  });
  if (CACHE) {
    walk_heads<VEC, STEP>(raw_v, v, p.kv.v_head, h0, grp, Hk, [&](const Raw8<E>& raw, int h) {
      float x[8];
      raw.floats(x);
      to_cache(x, h, p.kv.v, p.kv.v_exp);
    });
    if (bits) atomicOr(p.kv.status, bits);
  }
}

}  // namespace sv
