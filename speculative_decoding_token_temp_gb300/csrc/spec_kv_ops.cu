// Host entry points of the C ABI declared in include/spec_kv.h, around the attention: norms and
// rotation of queries and keys (with or without the cache's write), the weight that cached
// tokens gather, eviction. Argument checks and launches.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "kernels_evict.cuh"
#include "kernels_rope.cuh"
#include "kernels_weigh.cuh"
#include "kv_host.h"
#include "spec_kv.h"

namespace sv {
namespace {

spec_status check_rope(const spec_rope& r, const spec_head_norm& n, int head_dim, const int32_t* positions, size_t es) {
  if (r.rot_dim < 0 || r.rot_dim > head_dim || r.rot_dim % 16 != 0) return SPEC_ERR_INVALID_ARG;
  if (r.axes < 1 || r.axes > SPEC_ROPE_MAX_AXES) return SPEC_ERR_INVALID_ARG;
  if (r.rot_dim > 0 && (!r.step || !on(r.step, 8) || !positions || !on(positions, 4))) return SPEC_ERR_INVALID_ARG;
  if (isnan(n.eps) || isinf(n.eps)) return SPEC_ERR_INVALID_ARG;
  if (n.eps < 0.f && (n.q_weight || n.k_weight)) return SPEC_ERR_INVALID_ARG;
  if (!on(n.q_weight, es) || !on(n.k_weight, es)) return SPEC_ERR_INVALID_ARG;
  return SPEC_OK;
}

void fill_rope(RopeParams& p, const spec_rope& r, const spec_head_norm& n, const int32_t* positions) {
  p.q_w = n.q_weight;
  p.k_w = n.k_weight;
  p.norm = n.eps >= 0.f;
  p.eps = n.eps;
  p.pos = positions;
  p.axes = r.axes;
  p.step = r.step;
  p.axis = r.axis;
  p.rot = r.rot_dim;
  p.interleaved = r.interleaved != 0;
}

// Rows of a block: 8 (a warp a row, its sines and weights set up once for all heads) once that
// gives every SM a block, fewer below, down to all warps on one row. With the cache, 32/8 heads of
// 128 in bf16, 1 / 2 / 4 / 8 rows: 128 rows 4.2 / 5.2 / 7.2 / 10.0 us, 512 rows 7.3 / 6.7 / 7.3 /
// 10.1, 1024 rows 11.9 / 10.1 / 9.2 / 10.2, 2304 rows 24.3 / 18.3 / 14.1 / 12.9, 8192 rows 82.6 /
// 61.4 / 47.2 / 38.3. In fp32 8 are no better than 4 (4096 rows 49.6 / 39.6 / 39.3 / 42.9).
template <typename E, int D, bool CACHE, bool VEC, int R>
cudaError_t start_rope(const RopeParams& p, cudaStream_t s) {
  return start(rope_kernel<E, D, CACHE, VEC, R>, dim3((unsigned)cdiv(p.rows, R)), kRopeThreads, 0, s, p);
}
template <typename E, int D, bool CACHE, bool VEC>
cudaError_t launch_rope(const RopeParams& p, cudaStream_t s) {
  const long long rows = p.rows, sms = sm_count();
  if constexpr (VEC) {
    if (sizeof(E) == 2 && rows >= 8 * sms) return start_rope<E, D, CACHE, VEC, sizeof(E) == 2 ? 8 : 4>(p, s);
    if (2 * rows >= 3 * sms && rows < 3 * sms) return start_rope<E, D, CACHE, VEC, 2>(p, s);
  }
  return rows >= 3 * sms ? start_rope<E, D, CACHE, VEC, 4>(p, s) : start_rope<E, D, CACHE, VEC, 1>(p, s);
}
template <bool CACHE>
cudaError_t launch_rope(const RopeParams& p, spec_dtype dtype, int D, bool vec, cudaStream_t s) {
  if (dtype == SPEC_BF16) {
    if (D == 64) return vec ? launch_rope<uint16_t, 64, CACHE, true>(p, s) : launch_rope<uint16_t, 64, CACHE, false>(p, s);
    return vec ? launch_rope<uint16_t, 128, CACHE, true>(p, s) : launch_rope<uint16_t, 128, CACHE, false>(p, s);
  }
  if (D == 64) return vec ? launch_rope<float, 64, CACHE, true>(p, s) : launch_rope<float, 64, CACHE, false>(p, s);
  return vec ? launch_rope<float, 128, CACHE, true>(p, s) : launch_rope<float, 128, CACHE, false>(p, s);
}

template <typename E, int D, bool FEW>
cudaError_t launch_weigh(const WeighParams& p, long long line, cudaStream_t s) {
  static std::atomic<unsigned long long> done{0};
  static std::atomic<int> per_sm{0};
  constexpr int ring = WeighShape<E, D, FEW>::kRing;
  cudaError_t e = allow_smem(weigh_kernel<E, D, FEW>, done, ring);
  if (e != cudaSuccess) return e;
  int n = per_sm.load(std::memory_order_relaxed);
  if (n == 0) {
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, weigh_kernel<E, D, FEW>, kWeighThreads, ring);
    if (e != cudaSuccess || n < 1) return e != cudaSuccess ? e : cudaErrorInvalidConfiguration;
    per_sm.store(n, std::memory_order_relaxed);
  }
  const long long wave = (long long)n * sm_count();
  if (wave < 1) return cudaErrorInvalidConfiguration;
  return start(weigh_kernel<E, D, FEW>, dim3((unsigned)(line < wave ? line : wave)), kWeighThreads, ring, s, p);
}

template <typename E>
cudaError_t launch_weigh(const WeighParams& p, int D, long long line, cudaStream_t s) {
  if ((p.a.gamma + 1) * p.a.G <= 8) return D == 64 ? launch_weigh<E, 64, true>(p, line, s) : launch_weigh<E, 128, true>(p, line, s);
  return D == 64 ? launch_weigh<E, 64, false>(p, line, s) : launch_weigh<E, 128, false>(p, line, s);
}

template <int D>
cudaError_t launch_move(const EvictParams& p, cudaStream_t s) {
  const long long most = (long long)p.pps << p.page_shift, stay = most < p.budget ? most : p.budget;
  if (stay == 0) return cudaSuccess;
  if (p.new_table != p.table)
    return start(evict_move_kernel<D, false>, dim3((unsigned)cdiv(stay, kMoveStep<false>), (unsigned)p.Hk, (unsigned)p.B), kMoveStep<false>, 0, s, p,
                 1);
  int slices = 1;  // a block walks all tokens of its piece: narrower pieces, down to a sector, where there are few heads
  while (slices < D / 32 && (long long)slices * p.B * p.Hk < 2LL * sm_count()) slices *= 2;
  return start(evict_move_kernel<D, true>, dim3((unsigned)slices, (unsigned)p.Hk, (unsigned)p.B), kMoveStep<true>, 0, s, p, slices);
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" {

spec_status spec_qk_rope(int32_t rows, int32_t q_heads, int32_t k_heads, int32_t head_dim, spec_rope rope, spec_head_norm norm,
                         const int32_t* positions, spec_dtype dtype, const void* q, int64_t q_row_stride, int64_t q_head_stride,
                         const void* k, int64_t k_row_stride, int64_t k_head_stride, void* q_out, void* k_out,
                         spec_stream_t stream_) {
  const KvRange range("spec_qk_rope");
  if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_ERR_DTYPE;
  const size_t es = dtype == SPEC_BF16 ? 2 : 4;
  if (rows < 0 || rows > (1 << 22) || q_heads < 1 || q_heads > (1 << 14) || k_heads < 1 || k_heads > 256 ||
      (head_dim != 64 && head_dim != 128))
    return SPEC_ERR_INVALID_ARG;
  if (rows == 0) return SPEC_OK;
  const spec_status e = check_rope(rope, norm, head_dim, positions, es);
  if (e != SPEC_OK) return e;
  if (!q || !k || !on(q, es) || !on(k, es) || !q_out || !k_out || !on(q_out, 16) || !on(k_out, 16)) return SPEC_ERR_INVALID_ARG;
  if (q_row_stride < 0 || q_head_stride < 0 || k_row_stride < 0 || k_head_stride < 0) return SPEC_ERR_INVALID_ARG;
  RopeParams p;
  memset(&p, 0, sizeof(p));
  p.kv.Hk = k_heads;
  p.kv.src_k = k;
  p.kv.k_row = k_row_stride;
  p.kv.k_head = k_head_stride;
  p.q = q;
  p.q_row = q_row_stride;
  p.q_head = q_head_stride;
  p.q_out = q_out;
  p.k_out = k_out;
  p.rows = rows;
  p.Hq = q_heads;
  fill_rope(p, rope, norm, positions);
  const long long per = 16 / (long long)es;
  const bool vec = on(q, 16) && on(k, 16) && q_row_stride % per == 0 && q_head_stride % per == 0 && k_row_stride % per == 0 &&
                   k_head_stride % per == 0;
  const cudaError_t err = launch_rope<false>(p, dtype, head_dim, vec, reinterpret_cast<cudaStream_t>(stream_));
  return err == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

spec_status spec_qk_rope_append(spec_kv_cache c, spec_kv_rows r, int32_t q_heads, spec_rope rope, spec_head_norm norm,
                                const int32_t* positions, spec_dtype dtype, const void* q, int64_t q_row_stride,
                                int64_t q_head_stride, const void* k, int64_t k_row_stride, int64_t k_head_stride, const void* v,
                                int64_t v_row_stride, int64_t v_head_stride, void* q_out, uint32_t* device_status,
                                spec_stream_t stream_) {
  const KvRange range("spec_qk_rope_append");
  if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_ERR_DTYPE;
  spec_status e = check_cache(c);
  if (e != SPEC_OK) return e;
  if ((e = check_rows(r)) != SPEC_OK) return e;
  const size_t es = dtype == SPEC_BF16 ? 2 : 4;
  if (q_heads < 1 || q_heads > (1 << 14) || !device_status || !on(device_status, 4)) return SPEC_ERR_INVALID_ARG;
  if (r.rows == 0) return SPEC_OK;
  if ((e = check_rope(rope, norm, c.head_dim, positions, es)) != SPEC_OK) return e;
  if (!q || !k || !v || !on(q, es) || !on(k, es) || !on(v, es) || !q_out || !on(q_out, 16)) return SPEC_ERR_INVALID_ARG;
  if (q_row_stride < 0 || q_head_stride < 0 || k_row_stride < 0 || k_head_stride < 0 || v_row_stride < 0 || v_head_stride < 0)
    return SPEC_ERR_INVALID_ARG;
  RopeParams p;
  memset(&p, 0, sizeof(p));
  p.kv = kv_params(c, r, device_status);
  p.kv.src_k = k;
  p.kv.k_row = k_row_stride;
  p.kv.k_head = k_head_stride;
  p.kv.src_v = v;
  p.kv.v_row = v_row_stride;
  p.kv.v_head = v_head_stride;
  p.q = q;
  p.q_row = q_row_stride;
  p.q_head = q_head_stride;
  p.q_out = q_out;
  p.rows = r.rows;
  p.Hq = q_heads;
  fill_rope(p, rope, norm, positions);
  const long long per = 16 / (long long)es;
  const bool vec = on(q, 16) && on(k, 16) && on(v, 16) && q_row_stride % per == 0 && q_head_stride % per == 0 &&
                   k_row_stride % per == 0 && k_head_stride % per == 0 && v_row_stride % per == 0 && v_head_stride % per == 0;
  const cudaError_t err = launch_rope<true>(p, dtype, c.head_dim, vec, reinterpret_cast<cudaStream_t>(stream_));
  return err == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

spec_status spec_kv_weigh(spec_attn_batch g, spec_kv_cache c, spec_dtype dtype, const void* q, int64_t q_row_stride,
                          int64_t q_head_stride, const float* lse, const int32_t* n_accepted, float keep, float* mass,
                          uint32_t* device_status, spec_stream_t stream_) {
  const KvRange range("spec_kv_weigh");
  if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_ERR_DTYPE;
  const spec_status e = check_attn(g, c, SPEC_MAX_GAMMA);
  if (e != SPEC_OK) return e;
  if (g.parent != nullptr || g.prefix_len != 0 || !(keep >= 0.f) || isinf(keep)) return SPEC_ERR_INVALID_ARG;
  if (!device_status || !on(device_status, 4)) return SPEC_ERR_INVALID_ARG;
  if (g.B == 0) return SPEC_OK;
  const size_t es = dtype == SPEC_BF16 ? 2 : 4;
  if (!q || !on(q, es) || q_row_stride < 0 || q_head_stride < 0 || !lse || !on(lse, 4) || !mass || !on(mass, 4) || !on(n_accepted, 4))
    return SPEC_ERR_INVALID_ARG;
  if (!g.kv_len || !on(g.kv_len, 4) || !on(g.cu_draft, 4)) return SPEC_ERR_INVALID_ARG;
  if ((g.pages_per_seq > 0 && !g.page_table) || !on(g.page_table, 4)) return SPEC_ERR_INVALID_ARG;
  const long long tiles = cdiv((long long)g.pages_per_seq * c.page_size, kTile);
  const long long line = (long long)g.B * c.kv_heads * ((tiles > 1 ? tiles : 1) + 1);
  if (line > kMaxLine) return SPEC_ERR_INVALID_ARG;
  WeighParams p;
  p.a = attn_params(g, c, q, q_row_stride, q_head_stride, nullptr, nullptr, device_status, 1);
  p.lse = lse;
  p.n_accepted = n_accepted;
  p.mass = mass;
  p.keep = keep;
  p.scale = g.scale;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream_);
  const cudaError_t err = dtype == SPEC_BF16 ? launch_weigh<uint16_t>(p, c.head_dim, line, s) : launch_weigh<float>(p, c.head_dim, line, s);
  return err == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

spec_status spec_kv_evict(spec_evict_batch g, spec_kv_cache c, float* mass, int32_t* kept, int32_t* kv_len_out,
                          uint32_t* device_status, spec_stream_t stream_) {
  const KvRange range("spec_kv_evict");
  const spec_status e = check_cache(c);
  if (e != SPEC_OK) return e;
  if (g.B < 0 || g.B > 65535 || g.pages_per_seq < 0 || (long long)g.pages_per_seq * c.page_size > (1LL << 30)) return SPEC_ERR_INVALID_ARG;
  if (g.budget < 1 || g.budget > (1 << 30) || g.sinks < 0 || g.recent < 0 || (long long)g.sinks + g.recent > g.budget)
    return SPEC_ERR_INVALID_ARG;
  if (!device_status || !on(device_status, 4)) return SPEC_ERR_INVALID_ARG;
  if (g.B == 0) return SPEC_OK;
  if (!mass || !on(mass, 4) || !kept || !on(kept, 4) || !kv_len_out || !on(kv_len_out, 4) || !g.kv_len || !on(g.kv_len, 4) ||
      kv_len_out == g.kv_len)
    return SPEC_ERR_INVALID_ARG;
  if ((g.pages_per_seq > 0 && !g.page_table) || !on(g.page_table, 4) || !on(g.new_page_table, 4)) return SPEC_ERR_INVALID_ARG;
  EvictParams p;
  memset(&p, 0, sizeof(p));
  p.k = static_cast<uint8_t*>(c.k);
  p.v = static_cast<uint8_t*>(c.v);
  p.k_exp = c.k_exp;
  p.v_exp = c.v_exp;
  p.mass = mass;
  p.num_pages = c.num_pages;
  p.page_shift = page_shift_of(c.page_size);
  p.Hk = c.kv_heads;
  p.B = g.B;
  p.pps = p.new_pps = g.pages_per_seq;
  p.table = p.new_table = g.page_table;
  const long long most = (long long)g.pages_per_seq * c.page_size;  // tokens of a sequence
  if (g.new_page_table != nullptr && g.new_page_table != g.page_table) {
    p.new_table = g.new_page_table;
    p.new_pps = g.new_pages_per_seq;
    const long long stay = most < g.budget ? most : g.budget;
    if (g.new_pages_per_seq < 0 || (long long)g.new_pages_per_seq * c.page_size < stay) return SPEC_ERR_INVALID_ARG;
  }
  p.kv_len = g.kv_len;
  p.budget = g.budget;
  p.sinks = g.sinks;
  p.recent = g.recent;
  p.cached_keys = (int)(most < kSelKeys ? most : kSelKeys);
  p.wide = on(mass, 16);
  p.kept = kept;
  p.kv_len_out = kv_len_out;
  p.status = device_status;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream_);
  static std::atomic<unsigned long long> done{0};
  cudaError_t err = allow_smem(evict_select_kernel, done, kSelKeys * 4);
  if (err == cudaSuccess)
    err = start(evict_select_kernel, dim3((unsigned)p.Hk, (unsigned)p.B), kSelThreads, (size_t)p.cached_keys * 4, s, p);
  if (err == cudaSuccess) err = c.head_dim == 64 ? launch_move<64>(p, s) : launch_move<128>(p, s);
  return err == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // extern "C"
