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
 *   pages        int32 [1]: pages that the step needs; more than the free
 *                list has means that it ran out.  (It has num_free, or the
 *                `count` of paged_free, whose list is padded with -1.)
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
 * Sequences that share pages.  paged_fork makes the rows of a new batch go on
 * from those of the last one, paged_copy copies their last pages, paged_free
 * finds what no row holds, paged_compact moves pages together.  A row of
 * length n holds the first ceil(n / page_size) entries of its table row; pages
 * that several rows hold lie at the same place in each (as paged_fork leaves
 * them).
 *
 * paged_fork -- block table of a new batch: row i goes on from row parents[i]
 * (samples of one prompt, beams, a prefix that is in the cache; a row that
 * nothing goes on from is given up).
 *
 *   block_table, lengths   of the last batch, num_seqs rows; lengths are
 *                clamped to [0, table_width * page_size] and to 2^30.
 *   parents      int32 [num_rows]; outside [0, num_seqs): an empty row.
 *   keep         NULL, or int32 [num_rows]: row i keeps the first keep[i]
 *                tokens (clamped to [0, the parent's length]).
 *   free_pages   int32 [num_free], pages to hand out, in order.
 *   out_table    int32, row i at out_table + i * out_stride, table_width
 *                entries: the parent's for the tokens kept, then -1.  A last
 *                page that is not full, as row i will write to it, is the
 *                parent's only if no other row of the new batch holds that
 *                page full and no row before i holds it too; else the next
 *                free page (-1 once they run out).
 *   out_lengths  int32 [num_rows], the tokens kept.
 *   src, dst, tokens   int32 [num_rows]: for a row with a new last page that
 *                page's number before and now and how many of its tokens count,
 *                as paged_copy takes them; -1, -1, 0 for all others.
 *   pages        int32 [1]: pages that the call needs; more than the free
 *                list has (as for paged_layout) means that it ran out.
 *
 * The outputs overlap neither the inputs nor one another (refused).  A table
 * entry below 0 is no page: it is passed on, never copied.
 */
int paged_fork(const int32_t* block_table, int64_t table_stride, int32_t table_width, const int32_t* lengths,
               int32_t num_seqs, const int32_t* parents, const int32_t* keep, int32_t num_rows,
               const int32_t* free_pages, int32_t num_free, int32_t page_size, int32_t* out_table,
               int64_t out_stride, int32_t* out_lengths, int32_t* src, int32_t* dst, int32_t* tokens, int32_t* pages,
               hipStream_t stream);

/* One cache of a copy, strides in bytes: page p at data + p * page_stride, its
 * `tokens` tokens token_stride apart, each `outer` rows of `width` bytes
 * outer_stride apart (a cache without tokens: tokens = 1). */
typedef struct {
  void* data;
  int64_t page_stride, token_stride, outer_stride;
  int32_t tokens, outer, width;
} paged_pages;

/*
 * paged_copy -- pages src[i] to pages dst[i] of every cache, in one launch for
 * each PAGED_COPY_CACHES of them.
 *
 *   src, dst   int32 [num_pairs]; a pair with either outside [0, num_pages),
 *              or with both alike, is left out.  No page is the dst of two
 *              pairs, or of one and the src of another.
 *   tokens     NULL: whole pages.  Else int32 [num_pairs]: the first tokens[i]
 *              tokens of pair i's page, clamped to [0, the cache's].
 *   caches     num_caches of them, in host memory.
 */
#define PAGED_COPY_CACHES 32
int paged_copy(const int32_t* src, const int32_t* dst, const int32_t* tokens, int32_t num_pairs,
               const paged_pages* caches, int32_t num_caches, int32_t num_pages, hipStream_t stream);

/*
 * paged_free -- the pages that no row holds, from the block table alone: rows
 * that ended have length 0.
 *
 *   free_pages   int32 [num_pages], receives them in ascending order, -1 past
 *                the last.
 *   refs         int32 [num_pages], receives how many table entries hold each.
 *   count        int32 [1], receives how many are free.
 *   workspace    paged_free_workspace_size() bytes.
 *
 * Entries outside [0, num_pages) are no pages.
 */
int paged_free_workspace_size(int32_t num_pages, size_t* bytes);
int paged_free(const int32_t* block_table, int64_t table_stride, int32_t table_width, const int32_t* lengths,
               int32_t num_seqs, int32_t page_size, int32_t num_pages, int32_t* free_pages, int32_t* refs,
               int32_t* count, void* workspace, hipStream_t stream);

/*
 * paged_compact -- moves held pages to free ones with lower numbers: the k-th
 * held page from `limit` on goes to the k-th free page below it, for as long as
 * there are both.  limit -1: the number of held pages, so that they end up as
 * the first of the pool.
 *
 *   out_table    int32, row s at out_table + s * out_stride: the table with the
 *                pages' new numbers; may be block_table itself, with its
 *                stride.  Entries past a row's tokens are passed on.
 *   src, dst     int32 [num_pages / 2]: the moves, as paged_copy takes them, -1
 *                past the last.  A page that moves is no dst.
 *   moves, live  int32 [1]: how many pages move, and how many are held.
 *   workspace    paged_compact_workspace_size() bytes.
 */
int paged_compact_workspace_size(int32_t num_pages, size_t* bytes);
int paged_compact(const int32_t* block_table, int64_t table_stride, int32_t table_width, const int32_t* lengths,
                  int32_t num_seqs, int32_t page_size, int32_t num_pages, int32_t limit, int32_t* out_table,
                  int64_t out_stride, int32_t* src, int32_t* dst, int32_t* moves, int32_t* live, void* workspace,
                  hipStream_t stream);

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
 * paged_prefix_attention -- paged_attention of sequences that share their first
 * positions (samples of one prompt, requests behind one system prompt): what is
 * shared is read once for a group instead of once for each sequence.
 *
 *   group_starts  int32 [num_groups + 1], ascending: sequences
 *                 [group_starts[g], group_starts[g + 1]) are group g.  (A
 *                 sequence is a row of the block table: next_n rows of q.)
 *   shared        int32 [num_groups]: how many first positions the group's
 *                 sequences share, clamped to [0, table_width * page_size].
 *                 Their table entries for these are alike; those of the first
 *                 one that takes part are read.
 *
 * A sequence with a row shorter than that takes no part and is attended whole,
 * by itself, as is one that no group holds.  args->chosen is NULL; max_splits
 * holds for the shared and for the own positions of a row, at most 32 parts
 * each.  num_groups = 0 is paged_attention.  A workspace's size holds for any
 * other number of groups too, none among them, if it was asked for with one or more.
 */
int paged_prefix_attention_workspace_size(const paged_attention_args* args, int32_t num_groups, hipStream_t stream,
                                          size_t* bytes);
int paged_prefix_attention(const paged_attention_args* args, const int32_t* group_starts, const int32_t* shared,
                           int32_t num_groups, void* workspace, hipStream_t stream);

/*
 * Attention over pages that a cheap score chooses.  paged_bounds keeps, for each
 * page and key-value head, the largest and the smallest value of every key dim
 * in 8 bits; paged_block_select scores a row's pages by what no key between the
 * bounds can pass and takes the best; paged_block_attention reads those.
 *
 * paged_bounds -- bounds of the pages that hold new tokens, from all their
 * tokens in the cache:  with hi_d, lo_d the largest and smallest key value of
 * dim d over a page's tokens and s = max_d max(|hi_d|, |lo_d|) * (1 / 127),
 *   bounds[page, head] = [ceil(hi_d / s) .., floor(lo_d / s) ..], scales = s
 * (in fp32, 1 / 127 rounded first; clamped to [-127, 127], so that a key may lie
 * outside by 2^-23 of the largest magnitude, 2^-10 where s is subnormal; all zeros
 * where s is 0, as it is for zeros alone).  NaN is passed over, infinities count
 * as the type's largest value.  The scale of an e4m3 cache is not part of it: it
 * multiplies all of a head's scores.
 *
 *   k            the key cache, as for paged_attention.
 *   starts       int32 [num_seqs + 1], as paged_layout gives them: sequence s
 *                has starts[s + 1] - starts[s] new tokens, its last ones.
 *   lengths      int32 [num_seqs], tokens after the step.
 *   num_tokens   the most new tokens there are, paged_layout's capacity; tokens
 *                past it were not written: they count in no bounds, and pages
 *                that hold no other new tokens are left as they were.
 *   bounds       int8 [num_pages, num_kv_heads, 2, head_dim], page and head
 *                strides given (in bytes), 16-byte aligned.
 *   scales       fp32 [num_pages, num_kv_heads], rows scales_stride apart.
 *
 * A page that holds new tokens belongs to one sequence.
 */
typedef struct {
  const void* k;
  const int32_t* block_table;
  const int32_t* starts;
  const int32_t* lengths;
  void* bounds;
  float* scales;
  int64_t page_stride, token_stride, head_stride;
  int64_t bounds_page_stride, bounds_head_stride, scales_stride;
  int64_t table_stride;
  int32_t num_seqs, num_tokens;
  int32_t num_kv_heads, head_dim;
  int32_t page_size, num_pages, table_width;
  paged_dtype store;
} paged_bounds_args;

int paged_bounds(const paged_bounds_args* args, hipStream_t stream);

/*
 * paged_block_select -- for each row and key-value head the num_blocks pages
 * (blocks of its sequence, 0 for the first page_size positions) with the
 * largest scores, ascending, -1 past the last, as topk_ragged gives positions.
 * Block b's score is
 *   max over the heads h of the key-value head:
 *     (float)(sum_d max(Q_hd B_d, Q_hd b_d)) * s_h * s_b
 * with B, b the block's bounds and s_b their scale, s_h = max_d |q_hd| * (1 / 127) and
 * Q_hd = q_hd / s_h rounded to nearest even: whole numbers but for the scales,
 * so that equal inputs give equal choices everywhere.  Ties go to the lower
 * block.  Blocks [0, first) and the last `last` of the row come before all
 * others, blocks without a page after all others.  NaN in q counts as 0 and an
 * infinity as the type's largest value; a score past fp32's range counts as its
 * largest (smallest) finite number, one that is NaN (by its scale) as the smallest.
 *
 *   q            [num_rows, num_heads, head_dim], strides multiples of 16 bytes.
 *   lengths      int32 [num_rows]: row r has ceil(lengths[r] / page_size)
 *                blocks.
 *   blocks       int32 [num_rows, num_kv_heads, num_blocks], contiguous.
 *   workspace    paged_block_select_workspace_size() bytes; NULL when that is 0.
 *
 * first + last is at most num_blocks; table_width is at most 32768.
 */
typedef struct {
  const void* q;
  const void* bounds;
  const float* scales;
  const int32_t* block_table;
  const int32_t* lengths;
  int32_t* blocks;
  int64_t q_row_stride, q_head_stride;
  int64_t bounds_page_stride, bounds_head_stride, scales_stride;
  int64_t table_stride;
  int32_t num_rows, next_n;
  int32_t num_heads, num_kv_heads, head_dim;
  int32_t page_size, num_pages, table_width;
  int32_t num_blocks, first, last;
  paged_dtype dtype;
} paged_select_args;

int paged_block_select_workspace_size(const paged_select_args* args, hipStream_t stream, size_t* bytes);
int paged_block_select(const paged_select_args* args, void* workspace, hipStream_t stream);

/*
 * paged_block_attention -- paged_attention over chosen blocks (pages of the
 * row's sequence), chosen for each row and key-value head: blocks int32
 * [num_rows, num_kv_heads, num_blocks], strides given, as paged_block_select
 * gives them.  The row reads the positions of those blocks below its length;
 * blocks outside it are left out, one that occurs twice counts twice.
 * args->chosen is NULL.  num_blocks * page_size is at most 2^30.
 */
int paged_block_attention_workspace_size(const paged_attention_args* args, int32_t num_blocks, hipStream_t stream,
                                         size_t* bytes);
int paged_block_attention(const paged_attention_args* args, const int32_t* blocks, int64_t blocks_row_stride,
                          int64_t blocks_head_stride, int32_t num_blocks, void* workspace, hipStream_t stream);

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
