/*
 * paged_attention.h -- the paged cache that a top-K's indices point into, and
 * attention over it, on AMD Instinct MI355X (gfx950).
 *
 * One serving step of sparse attention: paged_layout gives new tokens their
 * pages and slots, paged_append / latent_append write them, topk_ragged
 * chooses positions from the indexer's scores, and paged_attention /
 * latent_attention read the chosen positions (or all of them).
 * latent_prefill attends a chunk of new tokens over its context.
 *
 * Conventions, as in topk_ragged.h:
 *   - All data pointers are DEVICE pointers owned by the caller.  The library
 *     never allocates device memory, never synchronises and never issues a
 *     host memset, so calls can be captured in a hipGraph and replayed.
 *   - Every call is asynchronous on `stream`; the device is the stream's.
 *   - Return values are topk_status codes; topk_ragged_last_error() has the
 *     text of the last failing call on the thread.
 *   - Strides count elements.  Workspaces are 16-byte aligned, hold nothing
 *     between launches (no initialisation) and must not be shared by launches
 *     that may overlap: give each stream, and each captured graph, its own.
 *     A size holds for the arguments it was asked for and for the same ones
 *     with fewer rows (num_rows; num_tokens, num_seqs), a narrower table, fewer
 *     chosen positions or a smaller context: one workspace for a server's
 *     largest step serves its others.  Sizes are host arithmetic; no call
 *     checks them, as no call is told the workspace's.
 *   - Outputs do not overlap inputs, and the cache is not written while it is
 *     read.
 *
 * The cache: a pool of num_pages pages of page_size tokens.  Position p of
 * sequence s lies in page block_table[s, p / page_size] at offset
 * p % page_size.  A page outside [0, num_pages) is no page: its tokens are
 * left out of attention as if they were masked, and appends to slots outside
 * the pool are dropped.  What a left-out token's place holds (NaN and
 * infinity included) has no effect.
 *
 * Rows: lengths[r] is how many positions row r sees, as topk_ragged's
 * lengths ([batch, next_n] row-major for multi-token steps: row b*next_n + j
 * belongs to sequence b).  A length outside [0, table_width * page_size] is
 * clamped into it (and to 2^30).  A row that sees nothing gets zeros and a log-sum-exp of
 * -inf.
 */
#ifndef PAGED_ATTENTION_H
#define PAGED_ATTENTION_H

#include "topk_ragged.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  PAGED_BF16 = 0,
  PAGED_FP16 = 1,
  PAGED_E4M3 = 2 /* 8-bit OCP e4m3 with a scale: value = stored * scale (caches only) */
} paged_dtype;

/* Rope dimensions at the end of a latent vector, and the expanded form's
 * per-head sizes: keys of 128 + 64, values of 128. */
#define PAGED_ROPE_DIM 64
#define PAGED_HEAD_DIM 128

/*
 * paged_layout -- block tables and slot maps of one step from request lengths.
 *
 *   lengths      int32 [num_seqs], tokens of each sequence after the step,
 *                clamped to [0, table_width * page_size] and to 2^30.
 *   new_tokens   int32 [num_seqs], how many of them are new, clamped to
 *                [0, length].
 *   free_pages   int32 [num_free], pages to hand out, in order.
 *   block_table  int32, row s at block_table + s * table_stride, updated in
 *                place: entries [ceil((length - new) / page_size),
 *                ceil(length / page_size)) get the next free pages (-1 once
 *                they run out); all others are left as they were.
 *   starts       int32 [num_seqs + 1], receives the exclusive prefix sum of
 *                the new tokens; sums stop at 2^31 - 1.
 *   slots        int32 [capacity]: token t (of sequence s, the tokens of a
 *                sequence in order) gets page * page_size + offset, or -1
 *                where its table entry is negative or its slot would pass
 *                2^31 - 1.  Past the last token: -1.
 *   row_lengths  int32 [capacity]: position + 1, the length that topk_ragged
 *                and the attention take for the token's row.  Past: 0.
 *   row_seqs     int32 [capacity]: the token's sequence.  Past: -1.
 *   pages        int32 [1]: pages that the step needs; more than num_free
 *                means that the free list ran out.
 *
 * Tokens past `capacity` are not written; starts and the table are whole
 * all the same.  num_seqs = 0 fills the outputs with their padding.
 */
int paged_layout(const int32_t* lengths, const int32_t* new_tokens, int32_t num_seqs, const int32_t* free_pages,
                 int32_t num_free, int32_t* block_table, int64_t table_stride, int32_t table_width,
                 int32_t page_size, int32_t capacity, int32_t* starts, int32_t* slots, int32_t* row_lengths,
                 int32_t* row_seqs, int32_t* pages, hipStream_t stream);

/* One part of an append: rows of `width` elements at src + t * src_stride go
 * to column 0 of the token's place in dst, whose rows are dst_token_stride
 * apart inside a page and pages dst_page_stride apart.  A part is made of
 * heads of head_width elements (width divides into them): dst heads are
 * dst_head_stride apart.  scales: NULL (1), or fp32, one for each head. */
typedef struct {
  const void* src;
  void* dst;
  const float* scales;
  int64_t src_stride;
  int64_t dst_page_stride, dst_token_stride, dst_head_stride;
  int32_t width, head_width;
} paged_part;

/*
 * paged_append -- writes new tokens into the cache, all parts in one launch
 * (keys and values, or a latent vector and its rope part).
 *
 *   slots   int32 [num_tokens]; outside [0, num_pages * page_size) a token is
 *           dropped.  No slot may occur twice.
 *   parts   num_parts of them, 1 or 2, in host memory.
 *   dtype   of the sources, PAGED_BF16 or PAGED_FP16; store: the same, or
 *           PAGED_E4M3: round(x / scale) to nearest even, magnitudes above
 *           448 stored as 448, NaN as NaN.
 */
int paged_append(const int32_t* slots, int32_t num_tokens, const paged_part* parts, int32_t num_parts,
                 int32_t page_size, int32_t num_pages, paged_dtype dtype, paged_dtype store, hipStream_t stream);

/*
 * paged_attention -- attention of single tokens over a paged cache of keys
 * and values: out = softmax(softmax_scale * q K^T) V for each row and head.
 *
 *   q            [num_rows, num_heads, head_dim], row and head strides given;
 *                head h reads key-value head h / (num_heads / num_kv_heads).
 *   k, v         caches with the same strides; v_scales multiplies the output,
 *                k_scales the scores (fp32 [num_kv_heads] or NULL; only with
 *                PAGED_E4M3).
 *   chosen       NULL: each row reads [0, lengths[r]).  Otherwise int32
 *                [num_rows, num_chosen], row r at chosen + r * chosen_stride:
 *                the positions it reads; entries outside [0, lengths[r]) are
 *                left out, so topk_ragged's output can be given as it is.  A
 *                position that occurs twice counts twice.
 *   out          [num_rows, num_heads, head_dim], contiguous, of q's type.
 *   lse          fp32 [num_rows, num_heads], or NULL: the natural logarithm
 *                of the softmax's sum.
 *   workspace    paged_attention_workspace_size() bytes; NULL when that is 0.
 *
 * head_dim is 64 or 128.  The last dimension of q, k, v and the cache is
 * contiguous, all their other strides and their pointers are multiples of 16
 * bytes, and no stride is negative.
 */
typedef struct {
  const void* q;
  const void* k;
  const void* v;             /* paged_attention only */
  const float* k_scales;     /* paged_attention: [num_kv_heads]; latent: [1] */
  const float* v_scales;     /* paged_attention: [num_kv_heads] */
  const int32_t* block_table;
  const int32_t* lengths;
  const int32_t* chosen;
  void* out;
  float* lse;
  int64_t q_row_stride, q_head_stride;
  int64_t page_stride, token_stride, head_stride;
  int64_t table_stride;
  int64_t chosen_stride;
  int32_t num_rows, next_n;
  int32_t num_heads, num_kv_heads;
  int32_t head_dim;          /* latent: the latent vector without its rope part */
  int32_t page_size, num_pages, table_width;
  int32_t num_chosen;
  float softmax_scale;       /* its product with log2(e) finite */
  paged_dtype dtype, store;
  int32_t max_splits;        /* 0: the library's rule; else at most this many parts a row (1 to 128) */
} paged_attention_args;

int paged_attention_workspace_size(const paged_attention_args* args, hipStream_t stream, size_t* bytes);
int paged_attention(const paged_attention_args* args, void* workspace, hipStream_t stream);

/*
 * latent_attention -- the absorbed form: every head reads one shared latent
 * vector a token, keys c[0 .. head_dim + 64), values c[0 .. head_dim):
 * out = softmax(softmax_scale * q c^T) c.  Arguments as for paged_attention
 * with k the cache [num_pages, page_size, head_dim + 64], v, v_scales and
 * num_kv_heads ignored, q [num_rows, num_heads, head_dim + 64] and out
 * [num_rows, num_heads, head_dim].  head_dim is 256 or 512.
 */
int latent_attention_workspace_size(const paged_attention_args* args, hipStream_t stream, size_t* bytes);
int latent_attention(const paged_attention_args* args, void* workspace, hipStream_t stream);

/*
 * latent_prefill -- the expanded form for chunks of new tokens: head h has
 * the keys [w_k[h] c, c_rope] and the values w_v[h] c, c the latent vectors of
 * the sequence's whole context in the paged cache (the new tokens' included).
 *
 *   q              [num_tokens, num_heads, 192]: 128 for w_k c, 64 rope.
 *   starts         int32 [num_seqs + 1]: sequence s owns tokens
 *                  [starts[s], starts[s + 1]), starts[0] >= 0, ascending.
 *                  Tokens outside every sequence are left as they were.
 *   lengths        int32 [num_seqs], the context after the chunk: token j of
 *                  a chunk of n sees positions [0, length - n + j].
 *   w_k, w_v       [num_heads, 128, latent_dim] contiguous, of q's type.
 *   context_tokens the most that the lengths add up to (each clamped to
 *                  [0, table_width * page_size]).  A sequence that does not
 *                  fit gets NaN in out and lse.
 *   out, lse       [num_tokens, num_heads, 128] and [num_tokens, num_heads].
 *   workspace      latent_prefill_workspace_size() bytes: the expanded keys
 *                  and values, 514 bytes a token and head and 256 more of a
 *                  sequence's first 1024 tokens, and the partial outputs of
 *                  split contexts.
 *
 * Values are kept in q's type; in fp16 one past 65504 is an infinity for the
 * rows that see it.  Keys are kept to fp16's 11 bits at any size, those of a
 * sequence's first 1024 tokens to twice as many.  A row whose weight lies on one
 * key behind those has a log-sum-exp off by up to 2^-11 softmax_scale sum |q k|;
 * with many keys alike in weight it is within 1e-6.
 */
typedef struct {
  const void* q;
  const void* cache;
  const float* scale;        /* fp32 [1] or NULL; only with PAGED_E4M3 */
  const void* w_k;
  const void* w_v;
  const int32_t* block_table;
  const int32_t* starts;
  const int32_t* lengths;
  void* out;
  float* lse;
  int64_t q_row_stride, q_head_stride;
  int64_t page_stride, token_stride;
  int64_t table_stride;
  int64_t context_tokens;
  int32_t num_tokens, num_seqs, num_heads;
  int32_t latent_dim;        /* 256 or 512 */
  int32_t page_size, num_pages, table_width;
  float softmax_scale;       /* its product with log2(e) finite */
  paged_dtype dtype, store;
} latent_prefill_args;

int latent_prefill_workspace_size(const latent_prefill_args* args, hipStream_t stream, size_t* bytes);
int latent_prefill(const latent_prefill_args* args, void* workspace, hipStream_t stream);

/* Arithmetic that the kernels share with the host (testing only; host
 * pointers).  paged_debug_place: the element offset of position pos in the
 * pool, or -1 where table_row holds no page in [0, num_pages) for it.
 * paged_debug_split: out[0] parts of out[1] positions for a row of n, at most
 * `most` parts, none meant to be shorter than `least`, multiples of `unit`. */
int64_t paged_debug_place(const int32_t* table_row, int32_t page_size, int32_t num_pages, int64_t page_stride,
                          int64_t token_stride, int32_t pos);
void paged_debug_split(int32_t n, int32_t most, int32_t least, int32_t unit, int32_t out[2]);

#ifdef __cplusplus
}
#endif

#endif /* PAGED_ATTENTION_H */
