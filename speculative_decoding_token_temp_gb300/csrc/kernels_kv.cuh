// The 8-bit paged key/value cache: quantising write (append) and read-back.
//
// Both move whole vectors (head_dim elements of one token at one kv head) between packed
// rows and their places in the pages; a group of head_dim / 8 lanes holds a vector, 8
// elements a lane, so that the bf16 side of a lane is one 16-byte access, its code side
// one 8-byte access, and the maximum of a vector is log2(head_dim / 8) shuffles.
//
// 32768 rows of 8 heads of 128 in bf16: append 41 us (4.9 TB/s), read 37 us (5.5 TB/s). The
// append issues instructions in 72 % of cycles (four vectors a lane on the way; two 47 us,
// eight 50), the read waits for its loads; neither is a limit by itself. A few hundred rows are
// one chain of dependent loads, position, page, data: 256 rows 2.5 us.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "kernels.cuh"
#include "spec_kv.h"

namespace sv {

constexpr float kE4m3Max = 448.f;
constexpr int kExpBias = 127;
constexpr int kNanExp = 255;  // the exponent byte of a vector that holds a NaN or an infinity

// 2^(byte - 127) for the bytes the append writes (1..247); NaN for kNanExp.
__device__ __forceinline__ float exp_value(unsigned byte) {
  return byte == (unsigned)kNanExp ? __int_as_float(0x7fffffff) : __int_as_float((int)byte << 23);
}

// The smallest e with m <= 448 * 2^e for a finite m > 0 (by its bits), at least SPEC_KV_MIN_EXP. With
// m = f * 2^k, f in [1, 2): 448 = 1.75 * 2^8, so e = k - 8, one more when f > 1.75. A
// subnormal m has k below the minimum whatever it is read as.
__device__ __forceinline__ int vector_exp(uint32_t bits) {
  const int b = (int)bits;
  const int e = (b >> 23) - 127 - 8 + ((b & 0x7fffff) > 0x600000 ? 1 : 0);
  return max(e, SPEC_KV_MIN_EXP);
}

// 8 consecutive elements, as they are in memory; VEC: their address is 16-byte aligned.
template <typename E>
struct Raw8;
template <>
struct Raw8<uint16_t> {
  uint4 w;
  template <bool VEC>
  __device__ __forceinline__ void load(const uint16_t* p) {
    if constexpr (VEC) {
      w = __ldg(reinterpret_cast<const uint4*>(p));
    } else {
      uint32_t x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = (uint32_t)__ldg(p + 2 * i) | (uint32_t)__ldg(p + 2 * i + 1) << 16;
      w = make_uint4(x[0], x[1], x[2], x[3]);
    }
  }
  // the largest magnitude among the lanes of a vector, by its bits as fp32's (a NaN or an
  // infinity is above every finite one)
  template <int L>
  __device__ __forceinline__ uint32_t top() const {
    constexpr uint32_t m = 0x7fff7fffu;
    uint32_t t = __vmaxu2(__vmaxu2(w.x & m, w.y & m), __vmaxu2(w.z & m, w.w & m));
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) t = __vmaxu2(t, __shfl_xor_sync(kFull, t, o));
    return max(t & 0xffff0000u, t << 16);
  }
  __device__ __forceinline__ void floats(float (&x)[8]) const {
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(v[i] << 16);
      x[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
    }
  }
};
template <>
struct Raw8<float> {
  float4 a, b;
  template <bool VEC>
  __device__ __forceinline__ void load(const float* p) {
    if constexpr (VEC) {
      a = __ldg(reinterpret_cast<const float4*>(p));
      b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    } else {
      a = make_float4(__ldg(p), __ldg(p + 1), __ldg(p + 2), __ldg(p + 3));
      b = make_float4(__ldg(p + 4), __ldg(p + 5), __ldg(p + 6), __ldg(p + 7));
    }
  }
  template <int L>
  __device__ __forceinline__ uint32_t top() const {
    const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t t = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) t = max(t, __float_as_uint(v[i]) & 0x7fffffffu);
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) t = max(t, __shfl_xor_sync(kFull, t, o));
    return t;
  }
  __device__ __forceinline__ void floats(float (&x)[8]) const {
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
};

__device__ __forceinline__ void store8(uint16_t* p, const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

// four e4m3 codes as floats (exact)
__device__ __forceinline__ void codes4(uint32_t w, float* x) {
  const __half2 a = __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xffffu), __NV_E4M3));
  const __half2 b = __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3));
  const float2 fa = __half22float2(a), fb = __half22float2(b);
  x[0] = fa.x, x[1] = fa.y, x[2] = fb.x, x[3] = fb.y;
}

struct KvParams {
  uint8_t *k, *v, *k_exp, *v_exp;
  int num_pages, page_shift, Hk;
  int rows, seqs, pps;
  const int32_t *table, *row_seq, *row_pos;
  const void *src_k, *src_v;              // append
  long long k_row, k_head, v_row, v_head; // strides of the sources in elements
  void *dst_k, *dst_v;                    // read; either may be null
  uint32_t* status;
};

// The place of row n: the index of its (page, head 0, slot) vector for heads strided by the
// page size, or -1 (left out) / -2 (bad, reported).
__device__ __forceinline__ long long kv_place(const KvParams& p, int n, uint32_t* bits) {
  const int pos = __ldg(p.row_pos + n);
  if (pos < 0) return -1;
  const int seq = __ldg(p.row_seq + n), page_i = pos >> p.page_shift;
  if ((unsigned)seq >= (unsigned)p.seqs || page_i >= p.pps) {
    *bits |= SPEC_DEV_OFFSETS;
    return -2;
  }
  const int page = __ldg(p.table + (long long)seq * p.pps + page_i);
  if ((unsigned)page >= (unsigned)p.num_pages) {
    *bits |= SPEC_DEV_PAGE;
    return -2;
  }
  const int size = 1 << p.page_shift;
  return (((long long)page * p.Hk) << p.page_shift) + (pos & (size - 1));
}

constexpr int kKvThreads = 256;
// vectors a lane group has on the way at once (64 bytes a lane of the append's source)
template <typename E>
constexpr int kKvUnroll = 16 / (int)sizeof(E) / 2;

// Both kernels: an item is `heads` heads of the key or the value side of a row (`split`
// items a side). A warp takes `per` (1..32) items in a row: its lanes look the places up,
// one item each (three dependent loads, once for all of them), then the warp moves the items
// one after the other, groups of D / 8 lanes a head each, so that neighbouring heads are
// read and written side by side.
struct KvSplit {
  int per, heads, split;
};
__device__ __forceinline__ long long kv_lookup(const KvParams& p, const KvSplit& k, int item, bool wanted, uint32_t* bits) {
  const int side = item / k.split;
  return side < p.rows * 2 && wanted ? kv_place(p, side >> 1, bits) : -1;
}

template <typename E, int D, bool VEC, int U>
__global__ void __launch_bounds__(kKvThreads, U == 1 ? 6 : 5) kv_append_kernel(KvParams p, KvSplit k) {
  constexpr int L = D / 8, GRP = 32 / L;  // lanes of a vector, vectors a warp holds at once
  griddep_wait();
  griddep_launch();
  const int lane = threadIdx.x & 31, sub = lane % L, grp = lane / L;
  const int items = p.rows * 2 * k.split, first = (blockIdx.x * (kKvThreads / 32) + (threadIdx.x >> 5)) * k.per;
  uint32_t bits = 0;
  const long long mine = lane < k.per ? kv_lookup(p, k, first + lane, true, &bits) : -1;
  const int n_items = min(k.per, items - first);
  for (int it = 0; it < n_items; ++it) {
    const int item = first + it, side = item / k.split, n = side >> 1, from = (item - side * k.split) * k.heads;
    const int to = min(p.Hk, from + k.heads);
    const bool is_v = side & 1;
    long long at = 0;
    if (U > 1 && (at = __shfl_sync(kFull, mine, it)) < 0) continue;
    const E* src = static_cast<const E*>(is_v ? p.src_v : p.src_k) + (long long)n * (is_v ? p.v_row : p.k_row) + sub * 8;
    const long long head = is_v ? p.v_head : p.k_head;
    for (int h0 = from + grp; h0 - grp < to; h0 += GRP * U) {
      Raw8<E> raw[U]{};
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (h0 + u * GRP < to) raw[u].template load<VEC>(src + (h0 + u * GRP) * head);
      // few rows: the source is on its way before the place is known (a row left out is read for nothing)
      if (U == 1 && (at = __shfl_sync(kFull, mine, it)) < 0) break;
      uint8_t* codes = (is_v ? p.v : p.k) + at * D + sub * 8;
      uint8_t* exps = (is_v ? p.v_exp : p.k_exp) + at;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = h0 + u * GRP;
        if (h - grp >= to) break;  // (the whole warp)
        const uint32_t top = raw[u].template top<L>();
        if (h >= to) continue;
        const bool bad = top >= 0x7f800000u;
        const int e = top == 0 ? SPEC_KV_ZERO_EXP : vector_exp(top);
        const float inv = bad ? 0.f : __int_as_float((kExpBias - e) << 23);  // 2^-e: e in [-100, 120]
        float x[8];
        raw[u].floats(x);
        uint32_t w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t a = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i] * inv, x[4 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
          const uint32_t b = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i + 2] * inv, x[4 * i + 3] * inv), __NV_SATFINITE, __NV_E4M3);
          w[i] = bad ? 0u : a | b << 16;
        }
        const long long vec = (long long)h << p.page_shift;
        if (!in_idx(at + vec, ((long long)p.num_pages * p.Hk) << p.page_shift, p.status)) continue;
        *reinterpret_cast<uint2*>(codes + vec * D) = make_uint2(w[0], w[1]);
        if (sub == 0) exps[vec] = (uint8_t)(bad ? kNanExp : e + kExpBias);
        if (bad) bits |= SPEC_DEV_NONFINITE;
      }
    }
  }
  if (bits) atomicOr(p.status, bits);
}

template <typename E, int D, int U>
__global__ void __launch_bounds__(kKvThreads) kv_read_kernel(KvParams p, KvSplit k) {
  constexpr int L = D / 8, GRP = 32 / L;
  griddep_wait();
  griddep_launch();
  const int lane = threadIdx.x & 31, sub = lane % L, grp = lane / L;
  const int items = p.rows * 2 * k.split, first = (blockIdx.x * (kKvThreads / 32) + (threadIdx.x >> 5)) * k.per;
  uint32_t bits = 0;
  const bool wanted = ((first + lane) / k.split & 1 ? p.dst_v : p.dst_k) != nullptr;
  const long long mine = lane < k.per ? kv_lookup(p, k, first + lane, wanted, &bits) : -1;
  const int n_items = min(k.per, items - first);
  for (int it = 0; it < n_items; ++it) {
    const int item = first + it, side = item / k.split, n = side >> 1, from = (item - side * k.split) * k.heads;
    const int to = min(p.Hk, from + k.heads);
    const bool is_v = side & 1;
    const long long at = __shfl_sync(kFull, mine, it);
    E* dst = static_cast<E*>(is_v ? p.dst_v : p.dst_k);
    if (dst == nullptr) continue;
    dst += (long long)n * p.Hk * D + sub * 8;
    const uint8_t* codes = (is_v ? p.v : p.k) + at * D + sub * 8;
    const uint8_t* exps = (is_v ? p.v_exp : p.k_exp) + at;
    for (int h0 = from + grp; h0 < to; h0 += GRP * U) {
      uint2 w[U];
      float s[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = h0 + u * GRP;
        const long long vec = (long long)h << p.page_shift;
        w[u] = make_uint2(0, 0);
        s[u] = at == -2 ? __int_as_float(0x7fffffff) : 0.f;
        if (at >= 0 && h < to && in_idx(at + vec, ((long long)p.num_pages * p.Hk) << p.page_shift, p.status)) {
          w[u] = *reinterpret_cast<const uint2*>(codes + vec * D);
          s[u] = exp_value(exps[vec]);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = h0 + u * GRP;
        if (h >= to) continue;
        float x[8];
        codes4(w[u].x, x);
        codes4(w[u].y, x + 4);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= s[u];
        store8(dst + (long long)h * D, x);
      }
    }
  }
  if (bits) atomicOr(p.status, bits);
}

}  // namespace sv
