// Launch parameters shared by the host side and the kernels of the paged
// cache (layout, append, attention, latent attention, latent prefill).  Not
// part of the public ABI.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#include "paged_attention.h"

namespace rrt {

// Defined beside topk_ragged's host code: sets the thread's error text and
// returns code; the stream's device with its CU count.
int set_error(int code, const char* msg);
int device_of_stream(hipStream_t stream, int* dev, int* num_cus);

// ---------------------------------------------------------------------------
// Arithmetic that host and kernels must agree on
// ---------------------------------------------------------------------------

#define RRT_HD __host__ __device__ __forceinline__

RRT_HD int32_t clamp_to(int32_t x, int64_t most) {
  return x < 0 ? 0 : (int64_t)x > most ? (int32_t)most : x;
}

// Longest context a table row can hold; at most 2^30 positions, so that sums
// of a position and a tile stay in int32.
constexpr int32_t kMostTokens = 1 << 30;
RRT_HD int64_t table_tokens(int32_t width, int32_t page_size) {
  const int64_t n = (int64_t)width * page_size;
  return n > kMostTokens ? kMostTokens : n;
}

// x / d for 0 <= x < 2^31 by one multiplication: with s = ceil(log2 d) and
// m = ceil(2^(31 + s) / d) < 2^32, x m / 2^(31 + s) exceeds x / d by less than
// x / 2^(31 + s) < 1 / d, so its floor is the quotient's.
struct Divisor {
  uint32_t mul, shift, by;
};
inline Divisor divisor_of(int32_t d) {
  uint32_t s = 0;
  while ((1ull << s) < (uint64_t)d) ++s;
  return {(uint32_t)(((1ull << (31 + s)) + (uint64_t)d - 1) / (uint64_t)d), s, (uint32_t)d};
}
RRT_HD uint32_t divide(uint32_t x, const Divisor& d) { return (uint32_t)(((uint64_t)x * d.mul) >> 31 >> d.shift); }

// Place of position pos in the pool, in elements, or -1 where the table holds
// no page of it.  The caller keeps 0 <= pos < table_width * page_size.
RRT_HD int64_t locate(const int32_t* table_row, int32_t page_size, int32_t num_pages, int64_t page_stride,
                      int64_t token_stride, int32_t pos) {
  const uint32_t j = (uint32_t)pos / (uint32_t)page_size;
  const int32_t page = table_row[j];
  if ((uint32_t)page >= (uint32_t)num_pages) return -1;
  return (int64_t)page * page_stride + (int64_t)((uint32_t)pos - j * (uint32_t)page_size) * token_stride;
}

// How a row of n positions is split: `parts` parts of `chunk` positions (the
// last one shorter), chunk a multiple of `unit`, parts <= most and no part
// shorter than `least` positions except where n itself is (n = 0: one empty
// part).  A function of the row's own length, so a ragged batch's short rows
// are not cut into parts that are too small to be worth a join.  n is at most
// kMostTokens.
struct Split {
  int32_t parts, chunk;
};
RRT_HD Split split_of(int32_t n, int32_t most, int32_t least, int32_t unit) {
  // 32 bits are enough, and a 64-bit division is a hundred instructions.
  uint32_t parts = (uint32_t)n / (uint32_t)least;
  if (parts > (uint32_t)most) parts = (uint32_t)most;
  if (parts < 1) parts = 1;
  const uint32_t per = ((uint32_t)n + parts - 1) / parts;
  uint32_t chunk = (per + (uint32_t)unit - 1) / (uint32_t)unit * (uint32_t)unit;
  if (chunk < (uint32_t)unit) chunk = (uint32_t)unit;
  parts = ((uint32_t)n + chunk - 1) / chunk;
  return {parts < 1 ? 1 : (int32_t)parts, (int32_t)chunk};
}

// ---------------------------------------------------------------------------
// Kernel parameters
// ---------------------------------------------------------------------------

constexpr int kLayoutBlock = 1024;  // threads of a workgroup of paged_layout
constexpr int kAppendBlock = 256;   // and of paged_append

struct LayoutParams {
  const int32_t* lengths;
  const int32_t* new_tokens;
  const int32_t* free_pages;
  int32_t* table;
  int32_t *starts, *slots, *row_lengths, *row_seqs, *pages;
  int64_t table_stride;
  int32_t num_seqs, num_free, table_width, page_size, capacity;
};

struct AppendParams {
  const int32_t* slots;
  paged_part part[2];
  int32_t chunks[2];  // work items per token of each part
  int32_t num_tokens, page_size;
  int64_t num_slots;
};

struct AttnParams {
  paged_attention_args a;
  float* part_out;     // [rows, heads, most, head_dim], unnormalised
  float2* part_stat;   // [rows, heads, most]: maximum (base-2 logarithm) and sum
  float scale_log2;    // softmax_scale * log2(e)
  int32_t most;        // parts a row is split into, at most
  int32_t least;       // fewest positions of a part
  int32_t unit;        // a part's positions are a multiple of this
  int32_t groups;      // units of work along the rows: sequences, or rows
  int32_t group_rows;  // rows of a group: next_n, or 1
  int32_t col_tiles;   // column tiles of a key-value head
  Divisor page;        // by page_size
};

// The expanded form works on tiles of kCtxTile context tokens; a sequence
// has ceil(length / kCtxTile) of them, after those of the sequences before it.
constexpr int32_t kCtxTile = 64;
constexpr int32_t kExactTiles = 16;  // of a sequence, whose keys are kept in two parts

struct PrefillParams {
  latent_prefill_args a;
  char* keys;       // [heads][capacity] key tiles, fragment order (128 dims, 16 KB), in fp16
  char* lows;       // [heads][low_tiles], as keys: what their rounding left, of each sequence's first tiles
  char* ropes;      // [capacity] rope tiles, fragment order (8 KB), in fp16
  char* values;     // [heads][capacity] value tiles, fragment order (16 KB)
  uint64_t* valid;  // [capacity]: which of a tile's tokens are in the cache
  uint32_t* flags;  // [heads][capacity]: low half 1 where a value is not finite, high half where a key's power is not 0
  uint32_t* rope_flags;  // [capacity]: where a rope part's power is not 0, a half for 32 tokens each
  int16_t* key_exps;     // [heads][capacity][64]: a flagged tile's keys are kept times 2^-this
  int16_t* rope_exps;    // [capacity][64]: rope parts are kept times 2^-this
  float* part_out;    // split contexts: [rows][heads][parts][128], not divided by the sum,
  float2* part_stat;  // and (maximum, sum) of each
  float scale_log2;
  int32_t parts;      // of a row tile's context, at most
  int32_t capacity;   // tiles of the workspace
  int32_t low_tiles;  // of second parts: kExactTiles a sequence, or every tile if those are fewer
  int32_t row_tiles;  // query tiles of a head that the grid covers
};

// Where the second parts of a tile (the local-th of sequence seq) lie among
// those of a head.
RRT_HD int32_t low_tile(const PrefillParams& p, int32_t seq, int32_t local, int32_t tile) {
  return p.low_tiles < p.capacity ? seq * kExactTiles + local : tile;
}

// Kernel lookup: nullptr if there is no such instance.
const void* layout_kernel_ptr();
const void* append_kernel_ptr(int dtype, int store, bool wide);
const void* attn_kernel_ptr(int dtype, int store, int head_dim, bool chosen, int rows, int tiles);
const void* latent_kernel_ptr(int dtype, int store, int head_dim, bool chosen, int heads);
const void* join_kernel_ptr(int dtype, int head_dim, bool many);
const void* expand_kernel_ptr(int dtype, int store, int latent_dim);
const void* prefill_kernel_ptr(int dtype);
const void* prefill_join_kernel_ptr(int dtype);
int prefill_rows();       // query rows of a workgroup
int prefill_join_rows();  // and of one of the join

}  // namespace rrt
