// Host helpers of the cache's entry points (include/spec_kv.h): argument checks, launches.
#pragma once

#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "kernels_attn.cuh"
#include "kernels_kv.cuh"
#include "spec_kv.h"

#include <nvtx3/nvToolsExt.h>

#include <atomic>

namespace sv {
namespace {

struct KvRange {
  explicit KvRange(const char* name) { nvtxRangePushA(name); }
  ~KvRange() { nvtxRangePop(); }
  KvRange(const KvRange&) = delete;
  KvRange& operator=(const KvRange&) = delete;
};

inline long long cdiv(long long a, long long b) { return (a + b - 1) / b; }
inline size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }
inline bool on(const void* p, size_t n) { return ((uintptr_t)p % n) == 0; }

inline int page_shift_of(int page_size) {
  for (int s = 4; s <= 8; ++s)
    if (page_size == 1 << s) return s;
  return -1;
}

inline spec_status check_cache(const spec_kv_cache& c) {
  if (c.num_pages < 1 || page_shift_of(c.page_size) < 0 || c.kv_heads < 1 || c.kv_heads > 256 ||
      (c.head_dim != 64 && c.head_dim != 128))
    return SPEC_ERR_INVALID_ARG;
  if (!c.k || !c.v || !c.k_exp || !c.v_exp) return SPEC_ERR_INVALID_ARG;
  if (!on(c.k, 16) || !on(c.v, 16) || !on(c.k_exp, 16) || !on(c.v_exp, 16)) return SPEC_ERR_INVALID_ARG;
  return SPEC_OK;
}

inline spec_status check_rows(const spec_kv_rows& r) {
  if (r.rows < 0 || r.sequences < 0 || r.pages_per_seq < 0 || r.rows > (1 << 22)) return SPEC_ERR_INVALID_ARG;
  if (r.rows == 0) return SPEC_OK;
  if (!r.row_seq || !r.row_pos || (r.sequences > 0 && r.pages_per_seq > 0 && !r.page_table)) return SPEC_ERR_INVALID_ARG;
  if (!on(r.row_seq, 4) || !on(r.row_pos, 4) || !on(r.page_table, 4)) return SPEC_ERR_INVALID_ARG;
  return SPEC_OK;
}

inline int sm_count() {
  static std::atomic<int> known[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  const bool cached = dev >= 0 && dev < 64;
  int n = cached ? known[dev].load(std::memory_order_relaxed) : 0;
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    if (cached) known[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

// A launch with programmatic stream serialisation: the kernel may start while its
// predecessor drains, and waits for it before it touches memory.
template <typename... Args>
cudaError_t start(void (*kern)(Args...), dim3 grid, int threads, size_t smem, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

inline KvParams kv_params(const spec_kv_cache& c, const spec_kv_rows& r, uint32_t* status) {
  KvParams p;
  memset(&p, 0, sizeof(p));
  p.k = static_cast<uint8_t*>(c.k);
  p.v = static_cast<uint8_t*>(c.v);
  p.k_exp = c.k_exp;
  p.v_exp = c.v_exp;
  p.num_pages = c.num_pages;
  p.page_shift = page_shift_of(c.page_size);
  p.Hk = c.kv_heads;
  p.rows = r.rows;
  p.seqs = r.sequences;
  p.pps = r.pages_per_seq;
  p.table = r.page_table;
  p.row_seq = r.row_seq;
  p.row_pos = r.row_pos;
  p.status = status;
  return p;
}

constexpr long long kMaxLine = 1LL << 30;  // a line of tiles is counted in ints

inline long long rows_of(const spec_attn_batch& g) { return (long long)g.total_draft + g.B; }

inline spec_status check_attn(const spec_attn_batch& g, const spec_kv_cache& c, int max_gamma) {
  const spec_status e = check_cache(c);
  if (e != SPEC_OK) return e;
  if (g.B < 0 || g.gamma < 0 || g.gamma > max_gamma || g.total_draft < 0) return SPEC_ERR_INVALID_ARG;
  if (g.cu_draft == nullptr && (long long)g.B * g.gamma != g.total_draft) return SPEC_ERR_INVALID_ARG;
  if ((long long)g.total_draft > (long long)g.B * g.gamma) return SPEC_ERR_INVALID_ARG;
  if (g.q_heads < 1 || g.q_heads % c.kv_heads != 0 || g.q_heads / c.kv_heads > 64) return SPEC_ERR_INVALID_ARG;
  // flat rows (row * group + head) and row indices stay inside int
  if (rows_of(g) * g.q_heads > (1LL << 30)) return SPEC_ERR_INVALID_ARG;
  if (g.pages_per_seq < 0 || (long long)g.pages_per_seq * c.page_size > (1LL << 30)) return SPEC_ERR_INVALID_ARG;
  if (g.prefix_len < 0 || g.prefix_len > (1 << 30)) return SPEC_ERR_INVALID_ARG;
  if (!(g.scale > 0.f) || !isfinite(g.scale)) return SPEC_ERR_INVALID_ARG;
  if (g.parent != nullptr) {
    if (g.cu_draft != nullptr || g.gamma < 1 || g.gamma > SPEC_MAX_TREE_NODES) return SPEC_ERR_INVALID_ARG;
    for (int j = 0; j < g.gamma; ++j)
      if (g.parent[j] < -1 || g.parent[j] >= j) return SPEC_ERR_INVALID_ARG;
  }
  return SPEC_OK;
}

inline AttnParams attn_params(const spec_attn_batch& g, const spec_kv_cache& c, const void* q, int64_t q_row, int64_t q_head,
                       void* o, float* lse, uint32_t* status, int seg_cost) {
  AttnParams p;
  memset(&p, 0, sizeof(p));
  p.k = static_cast<const uint8_t*>(c.k);
  p.v = static_cast<const uint8_t*>(c.v);
  p.k_exp = c.k_exp;
  p.v_exp = c.v_exp;
  p.num_pages = c.num_pages;
  p.page_shift = page_shift_of(c.page_size);
  p.Hk = c.kv_heads;
  p.Hq = g.q_heads;
  p.G = g.q_heads / c.kv_heads;
  p.q = q;
  p.q_row = q_row;
  p.q_head = q_head;
  p.B = g.B;
  p.gamma = g.gamma;
  p.total_draft = g.total_draft;
  p.R = (int)rows_of(g);
  p.cu = g.cu_draft;
  p.table = g.page_table;
  p.pps = g.pages_per_seq;
  p.kv_len = g.kv_len;
  p.mask = g.parent != nullptr ? A_TREE : A_CHAIN;
  p.c = g.scale * 1.4426950408889634f;
  p.seg_cost = seg_cost;
  p.o = o;
  p.lse = lse;
  p.status = status;
  if (g.parent != nullptr)
    for (int i = 0; i < g.gamma; ++i)
      for (int j = i; j >= 0; j = g.parent[j]) p.sees[j] |= 1ull << i;
  return p;
}

// Lets a kernel use `bytes` of shared memory on the current device, once (`done`: a bit a device).
template <typename K>
cudaError_t allow_smem(K kern, std::atomic<unsigned long long>& done, int bytes) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

}  // namespace
}  // namespace sv
