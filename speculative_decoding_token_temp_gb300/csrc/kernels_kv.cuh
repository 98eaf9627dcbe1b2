// The 8-bit paged key/value cache: quantising write (append) and read-back.
//
// Both move whole vectors (head_dim elements of one token at one kv head) between packed
// rows and their places in the pages; a group of head_dim / 8 lanes holds a vector, 8
// elements a lane, so that the bf16 side of a lane is one 16-byte access, its code side
// one 8-byte access, and the maximum of a vector is log2(head_dim / 8) shuffles.
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

// The smallest e with m <= 448 * 2^e for a finite m > 0, at least SPEC_KV_MIN_EXP. With
// m = f * 2^k, f in [1, 2): 448 = 1.75 * 2^8, so e = k - 8, one more when f > 1.75. A
// subnormal m has k below the minimum whatever it is read as.
__device__ __forceinline__ int vector_exp(float m) {
  const int b = __float_as_int(m);
  const int e = (b >> 23) - 127 - 8 + ((b & 0x7fffff) > 0x600000 ? 1 : 0);
  return max(e, SPEC_KV_MIN_EXP);
}

// 8 consecutive elements as floats; VEC: their address is 16-byte aligned.
template <bool VEC>
__device__ __forceinline__ void load8(const uint16_t* p, float (&x)[8]) {
  uint32_t w[4];
  if constexpr (VEC) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = (uint32_t)__ldg(p + 2 * i) | (uint32_t)__ldg(p + 2 * i + 1) << 16;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
template <bool VEC>
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  if constexpr (VEC) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __ldg(p + i);
  }
}

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

// Append: vector j of the call is (row, k or v, head) with the head innermost, so that the
// lanes of a warp read neighbouring heads of one row (contiguous in a projection) and write
// whole vectors of D codes.
template <typename E, int D, bool VEC>
__global__ void __launch_bounds__(kKvThreads) kv_append_kernel(KvParams p) {
  constexpr int L = D / 8;  // lanes of a vector
  griddep_wait();
  const int lane = threadIdx.x % L;
  const long long total = (long long)p.rows * 2 * p.Hk;
  const long long step = (long long)gridDim.x * (kKvThreads / L);
  uint32_t bits = 0;
  for (long long j0 = (long long)blockIdx.x * (kKvThreads / L); j0 < total; j0 += step) {
    const long long j = j0 + threadIdx.x / L;
    const bool in = j < total;
    const int h = in ? (int)(j % p.Hk) : 0;
    const long long r2 = in ? j / p.Hk : 0;
    const bool is_v = r2 & 1;
    const int n = (int)(r2 >> 1);
    const long long at = in ? kv_place(p, n, &bits) : -1;
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 0.f;
    if (at >= 0) {
      const E* src = static_cast<const E*>(is_v ? p.src_v : p.src_k);
      load8<VEC>(src + (long long)n * (is_v ? p.v_row : p.k_row) + (long long)h * (is_v ? p.v_head : p.k_head) + lane * 8, x);
    }
    float m = 0.f;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      m = fmaxf(m, fabsf(x[i]));
      bad |= !(fabsf(x[i]) <= 3.402823466e38f);
    }
    if (bad) m = __int_as_float(0x7f800000);
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
    if (at < 0) continue;
    bad = m == __int_as_float(0x7f800000);
    const int e = m == 0.f ? SPEC_KV_ZERO_EXP : vector_exp(m);
    const float inv = __int_as_float((kExpBias - e) << 23);  // 2^-e: e in [-100, 120]
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t a = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i] * inv, x[4 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
      const uint32_t b = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i + 2] * inv, x[4 * i + 3] * inv), __NV_SATFINITE, __NV_E4M3);
      w[i] = bad ? 0u : a | b << 16;
    }
    const long long vec = at + ((long long)h << p.page_shift);
    if (!in_idx(vec, ((long long)p.num_pages * p.Hk) << p.page_shift, p.status)) continue;
    *reinterpret_cast<uint2*>((is_v ? p.v : p.k) + vec * D + lane * 8) = make_uint2(w[0], w[1]);
    if (lane == 0) (is_v ? p.v_exp : p.k_exp)[vec] = (uint8_t)(bad ? kNanExp : e + kExpBias);
    if (bad) bits |= SPEC_DEV_NONFINITE;
  }
  if (bits) atomicOr(p.status, bits);
}

// Read-back: the same split; a lane reads 8 codes and writes 8 numbers.
template <typename E, int D>
__global__ void __launch_bounds__(kKvThreads) kv_read_kernel(KvParams p) {
  constexpr int L = D / 8;
  griddep_wait();
  const int lane = threadIdx.x % L;
  const long long total = (long long)p.rows * 2 * p.Hk;
  const long long step = (long long)gridDim.x * (kKvThreads / L);
  uint32_t bits = 0;
  for (long long j = (long long)blockIdx.x * (kKvThreads / L) + threadIdx.x / L; j < total; j += step) {
    const int h = (int)(j % p.Hk);
    const long long r2 = j / p.Hk;
    const bool is_v = r2 & 1;
    const int n = (int)(r2 >> 1);
    E* dst = static_cast<E*>(is_v ? p.dst_v : p.dst_k);
    if (dst == nullptr) continue;
    const long long at = kv_place(p, n, &bits);
    float x[8];
    if (at >= 0) {
      const long long vec = at + ((long long)h << p.page_shift);
      if (!in_idx(vec, ((long long)p.num_pages * p.Hk) << p.page_shift, p.status)) continue;
      const uint2 w = *reinterpret_cast<const uint2*>((is_v ? p.v : p.k) + vec * D + lane * 8);
      const float s = exp_value((is_v ? p.v_exp : p.k_exp)[vec]);
      codes4(w.x, x);
      codes4(w.y, x + 4);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] *= s;
    } else {
      const float fill = at == -1 ? 0.f : __int_as_float(0x7fffffff);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = fill;
    }
    store8(dst + ((long long)n * p.Hk + h) * D + lane * 8, x);
  }
  if (bits) atomicOr(p.status, bits);
}

}  // namespace sv
