/*
 * spec_kv.h -- C ABI of the 8-bit paged key/value cache and of the attention that scores
 * drafted tokens over it (GB300, sm_103a). Part of libspecverify.so; the conventions of
 * spec_verify.h hold (device pointers unless marked host, caller-owned buffers, no
 * allocation, asynchronous on the caller's stream, sticky device status word, no traps).
 *
 * A verification round ([SpS], "the target scores the last gamma+1 positions") runs the
 * target over gamma_b + 1 tokens per sequence. Around its attention stand three calls:
 *
 *   spec_kv_append   quantises the tokens' keys and values as it writes them to the cache
 *   spec_attention   the softmax attention of the gamma_b + 1 rows (a chain of drafts, or
 *                    a draft tree) over the cache, with or without a prefix that every
 *                    sequence of the batch shares and whose part is computed once for all
 *   spec_kv_read     cached tokens read back as numbers
 *
 * Cache format. A vector of head_dim elements x (the key or the value of one token at one
 * kv head) is held as head_dim e4m3 codes c and one exponent byte: x ~ c * 2^(byte - 127).
 * The exponent e is the smallest whole number with max|x| <= 448 * 2^e (448 is the code's
 * largest value), at least -100, and -60 for a vector of zeros; each code is x * 2^-e
 * rounded to nearest, ties to even. e4m3 is a floating-point code, so a scale between two
 * powers of two would not make it finer; a power of two makes the scaling exact, the
 * exponent one byte, and reading back exact in bf16 and fp32. A vector with a NaN or an
 * infinity is stored as zero codes under exponent byte 255, which reads back as NaN
 * (SPEC_DEV_NONFINITE is set).
 */
#ifndef SPEC_KV_H
#define SPEC_KV_H

#include "spec_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A page number outside [0, num_pages) where a token was to be read or written. */
#define SPEC_DEV_PAGE 64u

#define SPEC_KV_MIN_EXP (-100) /* the smallest exponent e the append writes */
#define SPEC_KV_ZERO_EXP (-60) /* the exponent of a vector of zeros */

/* The cache: pages of page_size tokens, a page's tokens of one kv head contiguous. */
typedef struct {
  void* k;        /* device [num_pages][kv_heads][page_size][head_dim] e4m3 codes, 16-byte aligned */
  void* v;        /* the same */
  uint8_t* k_exp; /* device [num_pages][kv_heads][page_size] exponent bytes, 16-byte aligned */
  uint8_t* v_exp; /* the same */
  int32_t num_pages;
  int32_t page_size; /* 16, 32, 64, 128 or 256 */
  int32_t kv_heads;  /* 1..256 */
  int32_t head_dim;  /* 64 or 128 */
} spec_kv_cache;

/* Where rows of an append or a read stand in the cache: row n is position row_pos[n] of
 * sequence row_seq[n], whose tokens p are in page page_table[row_seq[n]][p / page_size].
 * A negative row_pos leaves the row out: it is not written; it is read as zeros. (After
 * the verification of a tree, the nodes of the accepted path are appended at their
 * positions and the others left out.) */
typedef struct {
  int32_t rows; /* 0..2^22 */
  int32_t sequences;
  int32_t pages_per_seq;
  const int32_t* page_table; /* device [sequences][pages_per_seq] */
  const int32_t* row_seq;    /* device [rows] */
  const int32_t* row_pos;    /* device [rows] */
} spec_kv_rows;

/*
 * Writes rows' keys and values to the cache, quantised as above.
 *   k, v: [rows][kv_heads][head_dim] of dtype with the strides given (in elements; the
 *   head_dim elements of one vector are contiguous), e.g. slices of one fused projection.
 * A row with row_seq outside [0, sequences) or row_pos at or past pages_per_seq *
 * page_size sets SPEC_DEV_OFFSETS, one on a page outside the cache SPEC_DEV_PAGE; neither
 * is written. Two rows of one call must not name the same place.
 */
spec_status spec_kv_append(spec_kv_cache c, spec_kv_rows r, spec_dtype dtype, const void* k, int64_t k_row_stride,
                           int64_t k_head_stride, const void* v, int64_t v_row_stride, int64_t v_head_stride,
                           uint32_t* device_status, spec_stream_t stream);

/*
 * Reads rows back: k_out, v_out [rows][kv_heads][head_dim] of dtype, contiguous (either
 * may be NULL). Bad rows set the status bits of spec_kv_append and are NaN.
 */
spec_status spec_kv_read(spec_kv_cache c, spec_kv_rows r, spec_dtype dtype, void* k_out, void* v_out,
                         uint32_t* device_status, spec_stream_t stream);

/* The batch of an attention call. Rows (queries) are laid out as the target rows of
 * spec_verify.h: sequence b has gamma_b + 1 rows from row cu_draft[b] + b on. */
typedef struct {
  int32_t B;               /* sequences, >= 0 */
  int32_t gamma;           /* dense: drafts per sequence; packed: an upper bound; 0 = one token per sequence */
  int32_t total_draft;     /* sum of gamma_b */
  const int32_t* cu_draft; /* device [B+1]; NULL = dense */
  int32_t q_heads;         /* a multiple of the cache's kv_heads, at most 64 of them per kv head */
  int32_t pages_per_seq;
  const int32_t* page_table; /* device [B][pages_per_seq] */
  const int32_t* kv_len;     /* device [B]: tokens the cache holds of sequence b, this round's rows among them
                                (the last gamma_b + 1 of them) and without the shared prefix */
  int32_t prefix_len;          /* tokens of the shared prefix; 0 = none */
  const int32_t* prefix_table; /* device [ceil(prefix_len / page_size)]: its pages */
  const int32_t* parent;       /* HOST [gamma] or NULL: a draft tree as in spec_verify_tree (dense batches, gamma =
                                  its nodes): row 0 is the last context token, row j + 1 is node j */
  float scale;                 /* factor of the scores before the softmax, finite and > 0 */
} spec_attn_batch;

/* Bytes of scratch memory spec_attention needs (0 for an invalid geometry or dtype, or one
 * whose work, counted in 128-token tiles of all sequences at their longest, passes 2^30;
 * spec_attention refuses those with SPEC_ERR_INVALID_ARG). For bf16 queries, where many rows
 * share a long prefix, it holds that prefix in 16 bits: 4 bytes for each element of its keys
 * (4.3 GB for 2^20 tokens at 8 kv heads of 128). */
size_t spec_attention_workspace_bytes(spec_attn_batch g, spec_kv_cache c, spec_dtype dtype);

/*
 * Attention of every row over the shared prefix, its sequence's context and this round's
 * rows that it sees: with G = q_heads / kv_heads, row i of sequence b and query head h,
 *   o = sum_t softmax_t(scale * q . k_t) v_t,
 * over the prefix, the first kv_len[b] - (gamma_b + 1) tokens of the sequence, and of the
 * round's rows those up to i (chain) or i's ancestors and i itself (tree), with the
 * cached k, v of kv head h / G. A row that sees nothing (kv_len 0, or shorter than the
 * round, and no prefix) is zeros with lse = -inf.
 *
 *   q [total_draft + B][q_heads][head_dim] of dtype with the strides given (in elements);
 *   o [total_draft + B][q_heads][head_dim] of dtype, contiguous
 *   lse [total_draft + B][q_heads] fp32 or NULL: ln sum_t exp(scale * q . k_t)
 *
 * Accuracy. Scores, sums and lse are fp32. With bf16 queries a query's element is held to
 * 2^-17 of its row's largest, and a weight enters the values' sum with 11 bits down to 2^-24
 * of the row's largest weight (each times the token's 2^exponent) and to 2^-35 of that below.
 * Where many rows share a long prefix these are 2^-22 and 2^-33, and its values are exact
 * down to 2^-21 of the largest exponent among 128 tokens. The exponents of the values that a
 * row sees may differ by 100: past that the weight of a token of the smaller ones may be lost.
 *
 * What no row sees does not matter: unwritten places, pages past kv_len, NaN codes or
 * exponents of tokens that a row's mask hides. A row that sees a token stored as NaN (or
 * has a NaN or infinite query) is NaN.
 * Data errors: a kv_len outside [0, pages_per_seq * page_size] makes its sequence's rows
 * NaN and sets SPEC_DEV_OFFSETS; a page outside the cache makes the rows that see it NaN
 * and sets SPEC_DEV_PAGE; a cu_draft that is no prefix sum of counts 0..gamma up to
 * total_draft sets SPEC_DEV_OFFSETS and makes every row NaN.
 */
spec_status spec_attention(spec_attn_batch g, spec_kv_cache c, spec_dtype dtype, const void* q, int64_t q_row_stride,
                           int64_t q_head_stride, void* o, float* lse, uint32_t* device_status, void* workspace,
                           size_t workspace_bytes, spec_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_KV_H */
