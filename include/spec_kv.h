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
 * and around these what a target's layer and a long context need besides:
 *
 *   spec_qk_rope, spec_qk_rope_append   the norms of each head and the rotation by positions,
 *                    on the way from the projection to the attention, the second with the
 *                    cache's write in the same pass
 *   spec_attention_chunk   spec_attention for more rows a sequence: prompts, pieces of them
 *   spec_kv_weigh    the softmax weight that each cached token has gathered
 *   spec_kv_evict    cuts sequences to a budget of tokens, the heaviest kept
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

/* ---- chunks of new tokens ---------------------------------------------------- */

#define SPEC_MAX_CHUNK_GAMMA ((1 << 20) - 1) /* rows of a sequence in one spec_attention_chunk call, less one */

/*
 * spec_attention for chunks: the same rows, masks (chains only: parent NULL), prefix,
 * outputs, accuracy and data errors, with gamma up to SPEC_MAX_CHUNK_GAMMA. Row i of a
 * sequence of n_b = gamma_b + 1 rows sees the prefix, the first kv_len[b] - n_b tokens and
 * the chunk's own up to i; a packed batch may mix prompts with single tokens. Where fp32
 * queries' rows are many, their 24 bits enter the scores and a weight enters the values' sum
 * with 22 bits down to 2^-32 of the row's largest weight. Where rows are many, exponents of 128 neighbouring
 * tokens that differ by at most 20 (10 with fp32 queries) do not count in a weight's size: one of a token
 * of the larger exponents is then right to 2^-13 (2^-23) of the row's largest, each times its 2^exponent.
 *
 * Workspace. Long chunks are computed from keys and values widened to 16 bits: 4 bytes for each
 * element of the keys that the page table and the prefix have room for, not what kv_len says is
 * there (8.6 GB for 64 sequences of up to 32768 tokens at 8 kv heads of 128). Where that passes 32 GB, or
 * the tables' 128-token tiles times kv heads 2^23, the call takes smaller row blocks that read the
 * cache itself, several times slower; fp32 queries' choice counts the tables' tiles too.
 *
 * How much one call takes: its row blocks (of 256 rows times heads of a kv head, 128 with fp32
 * queries), each counted with the 128-token tiles of the page table that it may see (in a packed
 * batch of several sequences: all of them) and four more, over all kv heads, come to at most
 * 2^31 - 2^25. Past that the call is refused (SPEC_ERR_INVALID_ARG, a size of 0). A prompt of
 * 2^20 rows from the beginning at 32 query and 8 kv heads is a quarter of it, half with fp32 queries.
 */
size_t spec_attention_chunk_workspace_bytes(spec_attn_batch g, spec_kv_cache c, spec_dtype dtype);
spec_status spec_attention_chunk(spec_attn_batch g, spec_kv_cache c, spec_dtype dtype, const void* q, int64_t q_row_stride,
                                 int64_t q_head_stride, void* o, float* lse, uint32_t* device_status, void* workspace,
                                 size_t workspace_bytes, spec_stream_t stream);

/* ---- norms and rotation of queries and keys ---------------------------------- */

#define SPEC_ROPE_MAX_AXES 4

/* How heads are rotated. Pair j of a head (elements j and j + rot_dim / 2, or 2 j and
 * 2 j + 1 when interleaved) turns by position * step[j], where the position is the one of
 * the row's `axes` that axis[j] names. step is in units of 2^-64 turn, modulo one turn:
 * round(frequency / (2 pi) * 2^64); the angle is then right to 2^-32 of a turn for every
 * 32-bit position. */
typedef struct {
  int32_t rot_dim;      /* leading elements of a head that rotate: a multiple of 16, 0..head_dim */
  int32_t axes;         /* positions of a row, 1..SPEC_ROPE_MAX_AXES */
  int32_t interleaved;
  const uint64_t* step; /* device [rot_dim / 2] */
  const uint8_t* axis;  /* device [rot_dim / 2], or NULL: all of the first axis (a number past the last is the last) */
} spec_rope;

/* The norm of each head before the rotation: x * weight / sqrt(mean(x^2) + eps), over the
 * head's elements (whose squares' sum has to be in fp32's range). */
typedef struct {
  const void* q_weight; /* device [head_dim] of the call's dtype, or NULL: ones */
  const void* k_weight; /* the same */
  float eps;            /* negative: no norms (weights NULL) */
} spec_head_norm;

/*
 * Queries and keys normed and rotated: q_out [rows][q_heads][head_dim], k_out
 * [rows][k_heads][head_dim] of dtype, contiguous and 16-byte aligned, from rows with the
 * strides given (in elements). positions: device [rows][axes]. fp32 arithmetic, one rounding
 * at the end. The outputs must not overlap the inputs.
 */
spec_status spec_qk_rope(int32_t rows, int32_t q_heads, int32_t k_heads, int32_t head_dim, spec_rope rope, spec_head_norm norm,
                         const int32_t* positions, spec_dtype dtype, const void* q, int64_t q_row_stride, int64_t q_head_stride,
                         const void* k, int64_t k_row_stride, int64_t k_head_stride, void* q_out, void* k_out,
                         spec_stream_t stream);

/*
 * The same with the cache's write: the rotated keys and the values go to the cache as by
 * spec_kv_append (whose rules hold for r and the status word), quantised from their fp32
 * values; the queries to q_out. Rows left out of the cache still give their queries.
 */
spec_status spec_qk_rope_append(spec_kv_cache c, spec_kv_rows r, int32_t q_heads, spec_rope rope, spec_head_norm norm,
                                const int32_t* positions, spec_dtype dtype, const void* q, int64_t q_row_stride,
                                int64_t q_head_stride, const void* k, int64_t k_row_stride, int64_t k_head_stride, const void* v,
                                int64_t v_row_stride, int64_t v_head_stride, void* q_out, uint32_t* device_status,
                                spec_stream_t stream);

/* ---- eviction ---------------------------------------------------------------- */

/*
 * The weight that cached tokens gather. For every cached token t of sequence b and kv head h
 *   mass = keep * mass + sum_i sum_{heads of the group} exp(scale * q_i . k_t - lse_i)
 * over the rows i that see t (a chain, as in spec_attention; g.parent NULL, g.prefix_len 0).
 * The round's own tokens, the last gamma_b + 1, begin anew: their old mass counts as 0, and
 * with keep = 0 no old mass is read. What else mass holds is left as it is.
 *   lse [total_draft + B][q_heads] fp32 of spec_attention or spec_attention_chunk (with a
 *     shared prefix: its lse has the prefix in it). A row whose lse is not finite adds nothing.
 *   n_accepted [B] or NULL: only rows 0..n_accepted[b] count (what a verification accepted)
 *   mass [num_pages][kv_heads][page_size] fp32, 4-byte aligned
 * gamma at most SPEC_MAX_GAMMA: of a long chunk, pass its last rows. No two sequences may
 * share a page that holds a token of theirs. fp32 sums over queries held to 22 bits of
 * their row's largest element; results do not depend on timing.
 * Data errors: a bad kv_len or n_accepted (outside 0..gamma_b) sets SPEC_DEV_OFFSETS and
 * leaves its sequence out; tokens on pages outside the cache are left out (SPEC_DEV_PAGE); a
 * bad cu_draft sets SPEC_DEV_OFFSETS and leaves all out.
 */
spec_status spec_kv_weigh(spec_attn_batch g, spec_kv_cache c, spec_dtype dtype, const void* q, int64_t q_row_stride,
                          int64_t q_head_stride, const float* lse, const int32_t* n_accepted, float keep, float* mass,
                          uint32_t* device_status, spec_stream_t stream);

typedef struct {
  int32_t B; /* sequences, 0..65535 */
  int32_t pages_per_seq;
  const int32_t* page_table;     /* device [B][pages_per_seq] */
  const int32_t* kv_len;         /* device [B] */
  int32_t new_pages_per_seq;
  const int32_t* new_page_table; /* device [B][new_pages_per_seq]: pages that the kept tokens go to, none of them among
                                    the sequences' own; NULL (or page_table itself): in place */
  int32_t budget;                /* tokens of a sequence that stay at most, >= 1 */
  int32_t sinks, recent;         /* the first and the last tokens that stay in any case, sinks + recent <= budget */
} spec_evict_batch;

/*
 * Cuts every sequence of more than `budget` tokens to `budget`. At each kv head stay the first
 * `sinks`, the last `recent` and, of those between, the ones of the largest mass (of equal ones
 * the earliest; a NaN is lighter than every number). They keep their order: place j of the
 * sequence at that head is then the token that was at kept[b][h][j], with its key, value,
 * exponents and mass. To other pages shorter sequences are copied whole.
 *   kept device [B][kv_heads][budget]: old places, ascending; -1 past the last
 *   kv_len_out device [B] (not kv_len itself): min(kv_len, budget)
 * A sequence's pages must be its own. Rotated keys hold their positions, so attention over
 * what stays goes on as before; later tokens keep the positions they would have had.
 * Data errors: a bad kv_len sets SPEC_DEV_OFFSETS, a page outside the cache SPEC_DEV_PAGE; the
 * sequence is left as it was, its row of kept is -1, its kv_len_out kv_len (0 with other pages).
 */
spec_status spec_kv_evict(spec_evict_batch g, spec_kv_cache c, float* mass, int32_t* kept, int32_t* kv_len_out,
                          uint32_t* device_status, spec_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_KV_H */
