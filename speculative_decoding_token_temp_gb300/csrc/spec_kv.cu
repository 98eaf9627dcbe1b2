// Host entry points of the C ABI declared in include/spec_kv.h: argument checks, workspace
// layout and launches of the cache's write and read-back and of the attention over it.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "kernels_attn.cuh"
#include "kernels_attn_prefix.cuh"
#include "kernels_attn_tc.cuh"
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

int page_shift_of(int page_size) {
  for (int s = 4; s <= 8; ++s)
    if (page_size == 1 << s) return s;
  return -1;
}

spec_status check_cache(const spec_kv_cache& c) {
  if (c.num_pages < 1 || page_shift_of(c.page_size) < 0 || c.kv_heads < 1 || c.kv_heads > 256 ||
      (c.head_dim != 64 && c.head_dim != 128))
    return SPEC_ERR_INVALID_ARG;
  if (!c.k || !c.v || !c.k_exp || !c.v_exp) return SPEC_ERR_INVALID_ARG;
  if (!on(c.k, 16) || !on(c.v, 16) || !on(c.k_exp, 16) || !on(c.v_exp, 16)) return SPEC_ERR_INVALID_ARG;
  return SPEC_OK;
}

spec_status check_rows(const spec_kv_rows& r) {
  if (r.rows < 0 || r.sequences < 0 || r.pages_per_seq < 0 || r.rows > (1 << 22)) return SPEC_ERR_INVALID_ARG;
  if (r.rows == 0) return SPEC_OK;
  if (!r.row_seq || !r.row_pos || (r.sequences > 0 && r.pages_per_seq > 0 && !r.page_table)) return SPEC_ERR_INVALID_ARG;
  if (!on(r.row_seq, 4) || !on(r.row_pos, 4) || !on(r.page_table, 4)) return SPEC_ERR_INVALID_ARG;
  return SPEC_OK;
}

int sm_count() {
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

KvParams kv_params(const spec_kv_cache& c, const spec_kv_rows& r, uint32_t* status) {
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

// The split of an append or a read: an item is one side of a row and as many of its heads as
// a warp has on the way at once (four steps of what it holds side by side), or only what it
// holds side by side where a row has no more heads, or where that many items do not fill half
// of the resident warps (64 an SM); then up to 16 items a warp, which spreads the lookups'
// latency over them. Append in bf16, one step / four: 8 heads of 128, 256 rows 3.7 / 4.1 us,
// 512 even, 2304 rows 8.2 / 5.8, 32768 rows 60 / 42; 2 heads (one step holds them) 32768 rows
// 16.4 / 19.7.
struct KvGrid {
  unsigned blocks;
  KvSplit k;
};
KvGrid kv_grid(const KvParams& p, int D, int unroll) {
  const long long warps = 64LL * (sm_count() > 0 ? sm_count() : 1), sides = 2LL * p.rows;
  const int side_by_side = 32 / (D / 8);
  KvGrid g;
  g.k.heads = side_by_side * unroll;
  if (p.Hk <= side_by_side || 2 * sides * cdiv(p.Hk, side_by_side) <= warps) g.k.heads = side_by_side;
  g.k.split = (int)cdiv(p.Hk, g.k.heads);
  const long long items = sides * g.k.split, per = cdiv(items, 2 * warps);
  g.k.per = (int)(per < 1 ? 1 : per > 16 ? 16 : per);
  g.blocks = (unsigned)cdiv(items, (long long)g.k.per * (kKvThreads / 32));
  return g;
}

template <typename E, int D, bool VEC>
cudaError_t launch_append(const KvParams& p, cudaStream_t s) {
  const KvGrid g = kv_grid(p, D, kKvUnroll<E>);
  return g.k.heads == 32 / (D / 8) ? start(kv_append_kernel<E, D, VEC, 1>, dim3(g.blocks), kKvThreads, 0, s, p, g.k)
                                   : start(kv_append_kernel<E, D, VEC, kKvUnroll<E>>, dim3(g.blocks), kKvThreads, 0, s, p, g.k);
}
template <typename E, int D>
cudaError_t launch_append(const KvParams& p, bool vec, cudaStream_t s) {
  return vec ? launch_append<E, D, true>(p, s) : launch_append<E, D, false>(p, s);
}

template <typename E, int D>
cudaError_t launch_read(const KvParams& p, cudaStream_t s) {
  const KvGrid g = kv_grid(p, D, 4);
  return g.k.heads == 32 / (D / 8) ? start(kv_read_kernel<E, D, 1>, dim3(g.blocks), kKvThreads, 0, s, p, g.k)
                                   : start(kv_read_kernel<E, D, 4>, dim3(g.blocks), kKvThreads, 0, s, p, g.k);
}

// ---------------------------------------------------------------------------
// attention

constexpr int kMaxGridS = 1024;  // largest grid of the 32-bit kernel (its workspace is sized for it)

// tiles that a segment's beginning and end count for on the line of tiles (the tensor-core kernel, 3 / 4 / 5: 64 x 6 rows
// 57.5 / 57.6 / 58.0 us, 256 x 1 row to 8192 327.7 / 328.6 / 330.7, 2304 rows behind 16384 541.1 / 539.5 / 540.6)
constexpr int kSegCostT = 4, kSegCostS = 1, kSegCostP = 2;
constexpr long long kMaxLine = 1LL << 30;  // a line of tiles is counted in ints
constexpr int kMaxGridP = 160;   // of attn_prefix_kernel (one block an SM)
// The prefix is widened and computed in 128-row tiles where that pays for the widening: from
// this many row-tiles of keys on (rows that share keys x tiles x kv heads). Below, the 48- or
// 32-row blocks of attn_tc_kernel do it. Whole calls, 8 kv heads, narrow / wide: head_dim 128,
// 288 rows x 2000 tokens 34 / 43 us, 1152 x 2000 51 / 57, 576 x 8192 66 / 69, 1152 x 8192
// 105 / 83; head_dim 64, 576 x 2000 34.5 / 35.6, 1152 x 2000 51 / 47, 576 x 8192 64 / 51.
constexpr long long kWideWork128 = 300000, kWideWork64 = 75000;
constexpr int kMaxGridT = 512;   // of the tensor-core kernel (two blocks an SM)

struct AttnLayout {
  int nr, pre_nr;      // rows of a row block, of the two passes
  long long grid;      // blocks of the pass over the sequences' tokens, at most
  long long pre_grid;  // of the prefix pass
  long long line;      // the longer pass's line of tiles, at most
  bool wide;           // the prefix widened and computed by attn_prefix_kernel
  long long tiles;     // of the prefix
  size_t part, cut, pre_part, pre_cut, pre_o, pre_lse, k16, v16, exp, total;
};

long long rows_of(const spec_attn_batch& g) { return (long long)g.total_draft + g.B; }

// Rows of a row block of the tensor-core kernel, for `flat` rows that share keys: as few
// blocks as hold them, each as small as that allows in steps of 8 from 16 on (what a softmax
// thread does is in proportion: 64 x 6 rows x 4 heads in blocks of 24 57 us, of 32 61; 256 x
// 9 x 4 in blocks of 40 80 us, of 48 91). A block's accumulators take 5 columns of tensor
// memory a row, 8 with head_dim 64, of 256 a group.
int tc_rows(long long flat, int head_dim) {
  const long long per = cdiv(flat, cdiv(flat, head_dim == 64 ? 32 : 48));
  return per <= 16 ? 16 : (int)(cdiv(per, 8) * 8);
}

AttnLayout attn_layout(const spec_attn_batch& g, const spec_kv_cache& c, spec_dtype dtype) {
  AttnLayout L;
  const int G = g.q_heads / c.kv_heads;
  const bool tc = dtype == SPEC_BF16;
  const long long cap = tc ? kMaxGridT : kMaxGridS;
  L.nr = tc ? tc_rows((long long)(g.gamma + 1) * G, c.head_dim) : kRowsS;
  const long long flat = rows_of(g) * G;
  L.tiles = cdiv(g.prefix_len, kTile);
  L.wide = tc && flat >= 128 && flat * L.tiles * c.kv_heads >= (c.head_dim == 64 ? kWideWork64 : kWideWork128);
  L.pre_nr = L.wide ? kRowsP : tc && flat > 0 ? tc_rows(flat, c.head_dim) : kRowsS;
  const long long most_tiles = cdiv((long long)g.pages_per_seq * c.page_size, kTile);
  const long long nt = most_tiles > 1 ? most_tiles : 1;
  const int more = tc ? kSegCostT : kSegCostS;  // a block for every tile of the line at most
  const long long own = (long long)g.B * cdiv((long long)(g.gamma + 1) * G, L.nr) * c.kv_heads * (nt + more);
  const long long pre = g.prefix_len > 0 ? cdiv(rows_of(g) * G, L.pre_nr) * c.kv_heads * (cdiv(g.prefix_len, kTile) + more) : 0;
  L.line = own > pre ? own : pre;
  L.grid = own < cap ? own : cap;
  const long long pre_cap = L.wide ? kMaxGridP : cap;
  L.pre_grid = pre < pre_cap ? pre : pre_cap;
  // each pass has parts and records of its own: the second may begin before the first has ended
  size_t off = 0;
  L.part = off;
  off = up256(off + sizeof(float) * (size_t)(2 * L.grid * L.nr) * (c.head_dim + 2));
  L.cut = off;
  off = up256(off + sizeof(CutRec) * (size_t)L.grid);
  L.pre_part = off;
  off = up256(off + sizeof(float) * (size_t)(2 * L.pre_grid * L.pre_nr) * (c.head_dim + 2));
  L.pre_cut = off;
  off = up256(off + sizeof(CutRec) * (size_t)L.pre_grid);
  L.pre_o = off;
  if (g.prefix_len > 0) off = up256(off + sizeof(float) * (size_t)rows_of(g) * g.q_heads * c.head_dim);
  L.pre_lse = off;
  if (g.prefix_len > 0) off = up256(off + sizeof(float) * (size_t)rows_of(g) * g.q_heads);
  const size_t wide_bytes = L.wide ? (size_t)2 * c.kv_heads * L.tiles * kTile * c.head_dim : 0;
  L.k16 = off;
  off = up256(off + wide_bytes);
  L.v16 = off;
  off = up256(off + wide_bytes);
  L.exp = off;
  if (L.wide) off = up256(off + sizeof(float) * (size_t)c.kv_heads * L.tiles);
  L.total = off;
  return L;
}

spec_status check_attn(const spec_attn_batch& g, const spec_kv_cache& c) {
  const spec_status e = check_cache(c);
  if (e != SPEC_OK) return e;
  if (g.B < 0 || g.gamma < 0 || g.gamma > SPEC_MAX_GAMMA || g.total_draft < 0) return SPEC_ERR_INVALID_ARG;
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

AttnParams attn_params(const spec_attn_batch& g, const spec_kv_cache& c, const void* q, int64_t q_row, int64_t q_head,
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

// The prefix as one sequence whose rows are all rows of the batch.
AttnParams prefix_params(const AttnParams& own, const spec_attn_batch& g, const spec_kv_cache& c, float* pre_o,
                         float* pre_lse) {
  AttnParams p = own;
  p.B = 1;
  p.gamma = own.R - 1;
  p.total_draft = own.R - 1;
  p.cu = nullptr;
  p.table = g.prefix_table;
  p.pps = (int)cdiv(g.prefix_len, c.page_size);
  p.kv_len = nullptr;
  p.fixed_len = g.prefix_len;
  p.mask = A_ALL;
  p.late_wait = 0;
  p.dst_o = pre_o;
  p.dst_lse = pre_lse;
  return p;
}

template <typename E, int D, int NR>
cudaError_t launch_merge(const AttnParams& p, int grid, cudaStream_t s) {
  if (grid < 2) return cudaSuccess;
  return start(attn_merge_kernel<E, D, NR>, dim3((unsigned)grid, cdiv(NR, 8)), kMergeThreads, 0, s, p, grid);
}

// One wave of the 32-bit kernel on the current device.
template <typename E, int D>
long long f32_wave() {
  static std::atomic<int> per_sm{0};
  int n = per_sm.load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, attn_f32_kernel<E, D>, 128, 0) != cudaSuccess || n < 1) return 0;
    per_sm.store(n, std::memory_order_relaxed);
  }
  const long long w = (long long)n * sm_count();
  return w < kMaxGridS ? w : kMaxGridS;
}

template <typename E, int D>
cudaError_t pass_f32(const AttnParams& p, long long grid, cudaStream_t s) {
  const long long wave = f32_wave<E, D>();
  if (wave < 1) return cudaErrorInvalidConfiguration;
  const int n = (int)(grid < wave ? grid : wave);
  const cudaError_t e = start(attn_f32_kernel<E, D>, dim3((unsigned)n), 128, 0, s, p);
  return e != cudaSuccess ? e : launch_merge<E, D, kRowsS>(p, n, s);
}

// The cache's codes of one operand as a tensor of pages: a TMA load takes one page's tokens
// of one kv head (at most a tile of them), its rows swizzled as the MMAs read them.
typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                             const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static std::atomic<EncodeFn> known{nullptr};
  EncodeFn f = known.load(std::memory_order_acquire);
  if (f == nullptr) {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult how;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &how) != cudaSuccess ||
        how != cudaDriverEntryPointSuccess)
      return nullptr;
    f = reinterpret_cast<EncodeFn>(ptr);
    known.store(f, std::memory_order_release);
  }
  return f;
}

bool page_map(CUtensorMap* m, const void* codes, const spec_kv_cache& c) {
  const EncodeFn f = encode_fn();
  if (f == nullptr) return false;
  const cuuint64_t D = (cuuint64_t)c.head_dim, S = (cuuint64_t)c.page_size, H = (cuuint64_t)c.kv_heads;
  const cuuint64_t dims[4] = {D, S, H, (cuuint64_t)c.num_pages};
  const cuuint64_t strides[3] = {D, S * D, H * S * D};
  const cuuint32_t box[4] = {(cuuint32_t)D, (cuuint32_t)(S < kTile ? S : kTile), 1, 1};
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  return f(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(codes), dims, strides, box, ones,
           CU_TENSOR_MAP_INTERLEAVE_NONE, c.head_dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Maps {
  CUtensorMap k, v;
};

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

template <int D, int NR>
cudaError_t pass_tc(const AttnParams& p, long long grid, const Maps& m, cudaStream_t s) {
  auto kern = attn_tc_kernel<D, NR>;
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = allow_smem(kern, done, TcShape<D, NR>::kSmem);
  if (e != cudaSuccess) return e;
  const long long sms = sm_count();
  if (sms < 1) return cudaErrorInvalidConfiguration;
  const int n = (int)(grid < 2 * sms ? grid : 2 * sms);
  e = start(kern, dim3((unsigned)n), kTcThreads, TcShape<D, NR>::kSmem, s, p, m.k, m.v);
  return e != cudaSuccess ? e : launch_merge<uint16_t, D, NR>(p, n, s);
}

template <int D>
cudaError_t pass_tc_nr(int nr, const AttnParams& p, long long grid, const Maps& m, cudaStream_t s) {
  if (nr == 16) return pass_tc<D, 16>(p, grid, m, s);
  if (nr == 24) return pass_tc<D, 24>(p, grid, m, s);
  if constexpr (D == 128) {
    if (nr == 40) return pass_tc<D, 40>(p, grid, m, s);
    if (nr == 48) return pass_tc<D, 48>(p, grid, m, s);
  }
  return pass_tc<D, 32>(p, grid, m, s);
}

// The widened prefix: 16-bit rows of head_dim elements, loaded 64 elements by a tile of tokens.
bool wide_map(CUtensorMap* m, void* base, const spec_kv_cache& c, long long rows, CUtensorMapDataType type) {
  const EncodeFn f = encode_fn();
  if (f == nullptr) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)c.head_dim, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)c.head_dim * 2};
  const cuuint32_t box[2] = {64, kTile};
  const cuuint32_t ones[2] = {1, 1};
  return f(m, type, 2, base, dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t pass_prefix(const AttnParams& p, const spec_kv_cache& c, const AttnLayout& L, char* ws, cudaStream_t s) {
  WideParams w;
  w.k16 = reinterpret_cast<uint16_t*>(ws + L.k16);
  w.v16 = reinterpret_cast<uint16_t*>(ws + L.v16);
  w.exp = reinterpret_cast<float*>(ws + L.exp);
  w.tiles = (int)L.tiles;
  Maps m;
  const long long rows = L.tiles * kTile * c.kv_heads;
  if (!wide_map(&m.k, w.k16, c, rows, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16) ||
      !wide_map(&m.v, w.v16, c, rows, CU_TENSOR_MAP_DATA_TYPE_FLOAT16))
    return cudaErrorInvalidValue;
  cudaError_t e = start(widen_kernel<D>, dim3((unsigned)L.tiles, (unsigned)c.kv_heads), 256, 0, s, p, w);
  if (e != cudaSuccess) return e;
  auto kern = attn_prefix_kernel<D>;
  static std::atomic<unsigned long long> done{0};
  if ((e = allow_smem(kern, done, PreShape<D>::kSmem)) != cudaSuccess) return e;
  const long long sms = sm_count();
  if (sms < 1) return cudaErrorInvalidConfiguration;
  const int n = (int)(L.pre_grid < sms ? L.pre_grid : sms);
  e = start(kern, dim3((unsigned)n), kPreThreads, PreShape<D>::kSmem, s, p, w, m.k, m.v);
  return e != cudaSuccess ? e : launch_merge<uint16_t, D, kRowsP>(p, n, s);
}

// One pass over keys: fp32 queries on the 32-bit kernel, bf16 queries on the tensor cores.
cudaError_t attn_pass(spec_dtype dtype, int D, int nr, const AttnParams& p, long long grid, const Maps& m, cudaStream_t s) {
  if (dtype == SPEC_F32) return D == 64 ? pass_f32<float, 64>(p, grid, s) : pass_f32<float, 128>(p, grid, s);
  return D == 64 ? pass_tc_nr<64>(nr, p, grid, m, s) : pass_tc_nr<128>(nr, p, grid, m, s);
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" {

spec_status spec_kv_append(spec_kv_cache c, spec_kv_rows r, spec_dtype dtype, const void* k, int64_t k_row_stride,
                           int64_t k_head_stride, const void* v, int64_t v_row_stride, int64_t v_head_stride,
                           uint32_t* device_status, spec_stream_t stream_) {
  const KvRange range("spec_kv_append");
  if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_ERR_DTYPE;
  spec_status e = check_cache(c);
  if (e != SPEC_OK) return e;
  if ((e = check_rows(r)) != SPEC_OK) return e;
  if (!device_status || !on(device_status, 4)) return SPEC_ERR_INVALID_ARG;
  if (r.rows == 0) return SPEC_OK;
  const size_t es = dtype == SPEC_BF16 ? 2 : 4;
  if (!k || !v || !on(k, es) || !on(v, es)) return SPEC_ERR_INVALID_ARG;
  if (k_row_stride < 0 || k_head_stride < 0 || v_row_stride < 0 || v_head_stride < 0) return SPEC_ERR_INVALID_ARG;
  KvParams p = kv_params(c, r, device_status);
  p.src_k = k;
  p.src_v = v;
  p.k_row = k_row_stride;
  p.k_head = k_head_stride;
  p.v_row = v_row_stride;
  p.v_head = v_head_stride;
  const long long per = 16 / (long long)es;
  const bool vec = on(k, 16) && on(v, 16) && k_row_stride % per == 0 && k_head_stride % per == 0 &&
                   v_row_stride % per == 0 && v_head_stride % per == 0;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream_);
  cudaError_t err;
  if (dtype == SPEC_BF16)
    err = c.head_dim == 64 ? launch_append<uint16_t, 64>(p, vec, s) : launch_append<uint16_t, 128>(p, vec, s);
  else
    err = c.head_dim == 64 ? launch_append<float, 64>(p, vec, s) : launch_append<float, 128>(p, vec, s);
  return err == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

spec_status spec_kv_read(spec_kv_cache c, spec_kv_rows r, spec_dtype dtype, void* k_out, void* v_out,
                         uint32_t* device_status, spec_stream_t stream_) {
  const KvRange range("spec_kv_read");
  if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_ERR_DTYPE;
  spec_status e = check_cache(c);
  if (e != SPEC_OK) return e;
  if ((e = check_rows(r)) != SPEC_OK) return e;
  if (!device_status || !on(device_status, 4) || !on(k_out, 16) || !on(v_out, 16)) return SPEC_ERR_INVALID_ARG;
  if (r.rows == 0 || (!k_out && !v_out)) return SPEC_OK;
  KvParams p = kv_params(c, r, device_status);
  p.dst_k = k_out;
  p.dst_v = v_out;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream_);
  cudaError_t err;
  if (dtype == SPEC_BF16)
    err = c.head_dim == 64 ? launch_read<uint16_t, 64>(p, s) : launch_read<uint16_t, 128>(p, s);
  else
    err = c.head_dim == 64 ? launch_read<float, 64>(p, s) : launch_read<float, 128>(p, s);
  return err == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

size_t spec_attention_workspace_bytes(spec_attn_batch g, spec_kv_cache c, spec_dtype dtype) {
  if ((dtype != SPEC_F32 && dtype != SPEC_BF16) || check_attn(g, c) != SPEC_OK) return 0;
  const AttnLayout L = attn_layout(g, c, dtype);
  return L.line <= kMaxLine ? L.total : 0;
}

spec_status spec_attention(spec_attn_batch g, spec_kv_cache c, spec_dtype dtype, const void* q, int64_t q_row_stride,
                           int64_t q_head_stride, void* o, float* lse, uint32_t* device_status, void* workspace,
                           size_t workspace_bytes, spec_stream_t stream_) {
  const KvRange range("spec_attention");
  if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_ERR_DTYPE;
  const spec_status e = check_attn(g, c);
  if (e != SPEC_OK) return e;
  if (!device_status || !on(device_status, 4)) return SPEC_ERR_INVALID_ARG;
  if (g.B == 0) return SPEC_OK;
  const size_t es = dtype == SPEC_BF16 ? 2 : 4;
  if (!q || !o || !on(q, es) || !on(o, 16) || !on(lse, 4) || q_row_stride < 0 || q_head_stride < 0)
    return SPEC_ERR_INVALID_ARG;
  if (!g.kv_len || !on(g.kv_len, 4) || !on(g.cu_draft, 4)) return SPEC_ERR_INVALID_ARG;
  if ((g.pages_per_seq > 0 && !g.page_table) || !on(g.page_table, 4)) return SPEC_ERR_INVALID_ARG;
  if ((g.prefix_len > 0 && !g.prefix_table) || !on(g.prefix_table, 4)) return SPEC_ERR_INVALID_ARG;
  const AttnLayout L = attn_layout(g, c, dtype);
  if (L.line > kMaxLine) return SPEC_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < L.total || !on(workspace, 256)) return SPEC_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream_);
  AttnParams p = attn_params(g, c, q, q_row_stride, q_head_stride, o, lse, device_status,
                             dtype == SPEC_BF16 ? kSegCostT : kSegCostS);
  p.part = reinterpret_cast<float*>(ws + L.part);
  p.cut = reinterpret_cast<CutRec*>(ws + L.cut);
  Maps maps;
  memset(&maps, 0, sizeof(maps));
  if (dtype == SPEC_BF16 && (!page_map(&maps.k, c.k, c) || !page_map(&maps.v, c.v, c))) return SPEC_ERR_CUDA;
  cudaError_t err = cudaSuccess;
  if (g.prefix_len > 0) {
    float* pre_o = reinterpret_cast<float*>(ws + L.pre_o);
    float* pre_lse = reinterpret_cast<float*>(ws + L.pre_lse);
    AttnParams pp = prefix_params(p, g, c, pre_o, pre_lse);
    pp.part = reinterpret_cast<float*>(ws + L.pre_part);
    pp.cut = reinterpret_cast<CutRec*>(ws + L.pre_cut);
    if (L.wide) pp.seg_cost = kSegCostP;
    if (L.wide)
      err = c.head_dim == 64 ? pass_prefix<64>(pp, c, L, ws, s) : pass_prefix<128>(pp, c, L, ws, s);
    else
      err = attn_pass(dtype, c.head_dim, L.pre_nr, pp, L.pre_grid, maps, s);
    if (err != cudaSuccess) return SPEC_ERR_CUDA;
    p.pre_o = pre_o;
    p.pre_lse = pre_lse;
    p.late_wait = 1;
  }
  err = attn_pass(dtype, c.head_dim, L.nr, p, L.grid, maps, s);
  return err == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // extern "C"
