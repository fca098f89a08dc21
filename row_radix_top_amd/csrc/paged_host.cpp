// Host side of the paged-cache entry points: argument checks, how rows are
// split, and the launches.  No allocation, no memset and no synchronisation.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstring>

#include "paged_host.hpp"

namespace {

// ---------------------------------------------------------------------------
// Attention
// ---------------------------------------------------------------------------

constexpr float kLog2e = 1.44269504088896340736f;

// A part's fewest positions and the unit its length is rounded to: four
// wavefronts take 32 tokens each.
constexpr int32_t kUnit = 128;
constexpr int32_t kLeast = 256, kLeastChosen = 512;
constexpr int32_t kMostParts = 128;
// The latent kernel's: tiles of 64 tokens, one workgroup on a CU.
constexpr int32_t kLatentUnit = 64;
constexpr int32_t kLatentLeast = 128;

// How many parts the longest row gets, at most; units: workgroups of an
// unsplit launch.  Times in us for 1, 2, 4, 8 and 16 parts at 256 CUs:
//   4 x 8 units of 8192 positions        83   49   31   29   29
//   8 units of 32768                    311  164   88   49   31 (32: 30)
//   16 x 8 ragged, 4000 to 16384        225  152  152  142  144
//   64 x 8 ragged, 1 to 32768           895  800  755  752  767
//   64 x 8 of 16384                     801  814  801  782  778
//   256 x 8 ragged, 500 to 4096         482  479  489  522  607
//   25 x 4 of 2048 chosen                27   25   26   27   27
//   40 x 4 of 2048 chosen                31   40   37   34   34
//   4 x 4 of 512 chosen                  14   19   18   18   18
// So: two workgroups a CU; four parts at least where rows may differ in length
// (the longest one ends the launch); where all are alike no more than one a CU,
// and a second launch only for parts of 512.
//
// The latent kernel takes a CU for itself, so that a workgroup too many is
// another round.  1, 2, 3, 4, 5 and 8 parts, 128 heads in units of 64:
//   80 units of 2048 chosen              92   61   52   69   69   75
//   200 units of 2048 chosen             98  119  131  144  149  201
//   40 units of 8192                    217  118   86   68   58   45 (12: 43, 13: 59)
//   80 units ragged, 1 to 16384         601  318  223  179  159  166
//   128 units ragged, 1 to 16384        604  329  238  212  213  229
//   256 units ragged, 1 to 8192         312  239  245  257  281  334
//   256 units ragged, 1 to 1024          53   64   82   97  105  169
// So: what fits one round where rows are alike or that is four parts or more;
// otherwise four or, of many units, two, none below 1024 positions.  One row of
// 256 positions takes 13 us in one part and 16 in two, one of 512 20 and 17.
int64_t parts_for(bool latent, bool chosen, int64_t units, int64_t longest, int64_t cus) {
  if (latent) {
    if (longest < 512) return 1;
    const int64_t once = std::max<int64_t>(1, cus / units);
    if (chosen || once >= 4) return once;
    return std::max(once, std::min<int64_t>(units * 8 <= cus * 5 ? 4 : 2, longest / 1024));
  }
  if (chosen) return std::max<int64_t>(1, cus / units);
  return std::max<int64_t>(4, ceil_div(2 * cus, units));
}

int check_attention(const paged_attention_args* a, bool latent) {
  REQUIRE(a != nullptr, "null args");
  if (int rc = check_types(a->dtype, a->store)) return rc;
  REQUIRE(a->num_rows >= 0, "num_rows must be >= 0");
  REQUIRE(a->next_n >= 1 && a->num_rows % a->next_n == 0, "next_n must be >= 1 and divide num_rows");
  REQUIRE(a->num_heads >= 1, "num_heads must be >= 1");
  if (latent) {
    REQUIRE(a->head_dim == 256 || a->head_dim == 512, "head_dim of the latent vector must be 256 or 512");
  } else {
    REQUIRE(a->head_dim == 64 || a->head_dim == 128, "head_dim must be 64 or 128");
    REQUIRE(a->num_kv_heads >= 1 && a->num_heads % a->num_kv_heads == 0, "num_kv_heads must be >= 1 and divide num_heads");
  }
  REQUIRE(a->page_size >= 1, "page_size must be >= 1");
  REQUIRE(a->table_width >= 1, "table_width must be >= 1");
  REQUIRE(a->max_splits >= 0 && a->max_splits <= kMostParts, "max_splits must be in [0, 128]");
  REQUIRE(a->chosen == nullptr || (a->num_chosen >= 1 && a->num_chosen <= rrt::kMostTokens),
          "num_chosen must be in [1, 2^30]");
  REQUIRE(std::isfinite(a->softmax_scale * kLog2e), "softmax_scale times log2(e) must be finite");
  if (a->num_rows == 0) return TOPK_OK;
  REQUIRE(a->num_pages >= 1, "num_pages must be >= 1");
  REQUIRE((int64_t)a->num_rows * a->num_heads <= INT32_MAX, "num_rows * num_heads must be below 2^31");
  REQUIRE(a->q != nullptr && a->k != nullptr && a->block_table != nullptr && a->lengths != nullptr && a->out != nullptr,
          "null q, k, block_table, lengths or out");
  REQUIRE(latent || a->v != nullptr, "null v");
  const int64_t sz = a->store == PAGED_E4M3 ? 1 : 2;
  REQUIRE(a->q_row_stride >= 0 && a->q_head_stride >= 0 && a->page_stride >= 0 && a->token_stride >= 0 &&
              a->head_stride >= 0 && a->table_stride >= 0 && a->chosen_stride >= 0,
          "strides must be >= 0");
  REQUIRE(aligned(a->q, 16) && a->q_row_stride % 8 == 0 && a->q_head_stride % 8 == 0,
          "q and its strides must be multiples of 16 bytes");
  REQUIRE(aligned(a->k, 16) && (latent || aligned(a->v, 16)) && a->page_stride * sz % 16 == 0 &&
              a->token_stride * sz % 16 == 0 && (latent || a->head_stride * sz % 16 == 0),
          "the cache and its strides must be multiples of 16 bytes");
  REQUIRE(aligned(a->out, 16), "out must be 16-byte aligned");
  REQUIRE(aligned(a->block_table, 4) && aligned(a->lengths, 4) && aligned(a->chosen, 4) && aligned(a->lse, 4) &&
              aligned(a->k_scales, 4) && aligned(a->v_scales, 4),
          "block_table, lengths, chosen, lse and scales must be 4-byte aligned");
  REQUIRE(a->store == PAGED_E4M3 || (a->k_scales == nullptr && a->v_scales == nullptr),
          "scales belong to an e4m3 cache");
  return TOPK_OK;
}

struct AttnPlan {
  rrt::AttnParams p;
  int threads;
  const void* fn;
  int64_t grid;
  size_t bytes;
};

// reserve: NULL, or receives the bytes of workspace that this launch or one of
// fewer rows may use.
// blocks: a->chosen holds blocks, this far apart for key-value heads (else NULL).
int plan_attention(const paged_attention_args* a, bool latent, hipStream_t stream, AttnPlan* out,
                   size_t* reserve = nullptr, const int64_t* blocks = nullptr) {
  if (int rc = check_attention(a, latent)) return rc;
  std::memset(out, 0, sizeof(*out));
  if (reserve != nullptr) *reserve = 0;
  if (a->num_rows == 0) return TOPK_OK;
  int dev = 0, cus = 0;
  if (int rc = rrt::device_of_stream(stream, &dev, &cus)) return rc;
  rrt::AttnParams& p = out->p;
  p.a = *a;
  p.scale_log2 = a->softmax_scale * kLog2e;
  p.page = rrt::divisor_of(a->page_size);
  out->threads = latent ? 512 : 256;
  const bool chosen = a->chosen != nullptr;
  int64_t units = 0;
  if (latent) {
    const int heads = a->num_heads <= 32 ? 32 : 64;
    p.unit = kLatentUnit;
    p.least = kLatentLeast;
    p.group_rows = 1;
    p.col_tiles = (int32_t)ceil_div(a->num_heads, heads);
    p.groups = a->num_rows;
    units = (int64_t)p.groups * p.col_tiles;
    out->fn = rrt::latent_kernel_ptr(a->dtype, a->store, a->head_dim, chosen, heads);
  } else {
    p.unit = kUnit;
    p.least = chosen ? kLeastChosen : kLeast;
    // Rows of a sequence read its cache together unless each has its own
    // chosen positions.
    p.group_rows = chosen ? 1 : a->next_n;
    const int64_t columns = (int64_t)p.group_rows * (a->num_heads / a->num_kv_heads);
    const int tiles = columns > 16 ? 2 : 1;
    p.col_tiles = (int32_t)ceil_div(columns, 16 * tiles);
    p.groups = a->num_rows / p.group_rows;
    units = (int64_t)p.groups * a->num_kv_heads * p.col_tiles;
    const int mode = blocks != nullptr ? rrt::kBlocks : chosen ? rrt::kChosen : p.group_rows > 1 ? rrt::kManyRows : rrt::kOneRow;
    p.chosen_head_stride = blocks != nullptr ? *blocks : 0;
    out->fn = rrt::attn_kernel_ptr(a->dtype, a->store, a->head_dim, mode, tiles);
  }
  const int64_t longest = chosen ? a->num_chosen : rrt::table_tokens(a->table_width, a->page_size);
  const int64_t each = units / p.groups;
  auto most_for = [&](int64_t groups) {
    const int64_t most = a->max_splits > 0 ? a->max_splits : parts_for(latent, chosen, groups * each, longest, cus);
    return std::max<int64_t>(1, std::min<int64_t>({most, (int64_t)kMostParts, longest / p.least}));
  };
  auto bytes_for = [&](int64_t groups) -> size_t {
    const int64_t most = most_for(groups);
    if (most == 1) return 0;
    return (size_t)(groups * p.group_rows) * a->num_heads * most * (a->head_dim * sizeof(float) + sizeof(float2));
  };
  p.most = (int32_t)most_for(p.groups);
  out->grid = ceil_div((int64_t)p.groups * p.most, 8) * 8 * each;  // see work_of
  out->bytes = bytes_for(p.groups);
  if (reserve == nullptr) return TOPK_OK;
  // Fewer rows may be split into more parts each.  Past two units a CU the rules
  // give every number of rows as many parts, and more rows need more.
  *reserve = out->bytes;
  for (int64_t g = std::min<int64_t>(p.groups - 1, 2 * (int64_t)cus / each + 1); g > 0; --g)
    *reserve = std::max(*reserve, bytes_for(g));
  return TOPK_OK;
}

int run_attention(const paged_attention_args* a, bool latent, void* workspace, hipStream_t stream,
                  const int64_t* blocks = nullptr) {
  AttnPlan plan;
  if (int rc = plan_attention(a, latent, stream, &plan, nullptr, blocks)) return rc;
  if (a->num_rows == 0) return TOPK_OK;
  if (plan.bytes > 0) {
    if (workspace == nullptr) {
      char buf[96];
      std::snprintf(buf, sizeof(buf), "this launch needs a workspace of %zu bytes", plan.bytes);
      return set_error(TOPK_EWORKSPACE, buf);
    }
    REQUIRE(aligned(workspace, 16), "workspace must be 16-byte aligned");
    plan.p.part_out = static_cast<float*>(workspace);
    plan.p.part_stat =
        reinterpret_cast<float2*>(plan.p.part_out + (int64_t)a->num_rows * a->num_heads * plan.p.most * a->head_dim);
  }
  const char* name = latent ? "latent_attention" : blocks != nullptr ? "paged_block_attention" : "paged_attention";
  if (int rc = launch(plan.fn, plan.grid, plan.threads, &plan.p, stream, name)) return rc;
  if (plan.p.most == 1) return TOPK_OK;
  const bool many = plan.p.most > 4;
  const int64_t outputs = (int64_t)a->num_rows * a->num_heads;
  return launch(rrt::join_kernel_ptr(a->dtype, a->head_dim, many), many ? outputs : ceil_div(outputs, 4), 256, &plan.p,
                stream, "join of split rows");
}

// ---------------------------------------------------------------------------
// Shared prefixes
// ---------------------------------------------------------------------------

// Parts of a row's shared positions and of its own, at most: a join's wavefront
// has a lane for each.
constexpr int32_t kMostSharedParts = 32, kMostOwnParts = 32;

struct PrefixPlan {
  rrt::AttnParams p;
  const void *shared_fn, *own_fn;
  int64_t shared_grid, own_grid;
  size_t bytes;
};

int plan_prefix(const paged_attention_args* a, const int32_t* group_starts, const int32_t* shared, int32_t num_groups,
                hipStream_t stream, PrefixPlan* out, size_t* reserve = nullptr) {
  if (int rc = check_attention(a, false)) return rc;
  REQUIRE(a->chosen == nullptr, "chosen must be NULL");
  REQUIRE(group_starts != nullptr && shared != nullptr, "null group_starts or shared");
  REQUIRE(aligned(group_starts, 4) && aligned(shared, 4), "group_starts and shared must be 4-byte aligned");
  std::memset(out, 0, sizeof(*out));
  if (reserve != nullptr) *reserve = 0;
  if (a->num_rows == 0) return TOPK_OK;
  int dev = 0, cus = 0;
  if (int rc = rrt::device_of_stream(stream, &dev, &cus)) return rc;
  rrt::AttnParams& p = out->p;
  p.a = *a;
  p.scale_log2 = a->softmax_scale * kLog2e;
  p.page = rrt::divisor_of(a->page_size);
  p.group_starts = group_starts;
  p.shared = shared;
  p.num_groups = num_groups;
  const int32_t per = a->num_heads / a->num_kv_heads;
  const int64_t seqs = a->num_rows / a->next_n, all = (int64_t)a->num_rows * per;
  const int64_t longest = rrt::table_tokens(a->table_width, a->page_size);

  // Both kinds of positions are shared out to as many workgroups as run at once; how,
  // the kernels find out from the lengths.  A part's number is bounded by what that gives a
  // batch of rows alike, and by four times that where one may be longer.
  p.workgroups = 2 * cus;
  auto limited = [&](int64_t parts, int64_t least, int32_t most) {
    if (a->max_splits > 0) parts = a->max_splits;
    return (int32_t)std::max<int64_t>(1, std::min<int64_t>({parts, (int64_t)most, ceil_div(longest, least)}));
  };

  // The shared part: wavefronts along the columns as far as a group has them.
  const int64_t each = ceil_div(all, num_groups);
  const int waves = each > 64 ? 4 : each > 32 ? 2 : 1;
  // (One wavefront a column's tile: tiles of 128 tokens, whose workgroups have a CU's
  // LDS to themselves.)
  auto shared_workgroups = [&](int waves) { return waves == 1 ? cus : 2 * cus; };
  p.shared_workgroups = shared_workgroups(waves);
  auto shared_parts = [&](int64_t seqs, int waves, bool one) {
    const int64_t units = ceil_div(seqs * a->next_n * per, 32 * waves) * a->num_kv_heads;
    return limited(ceil_div(shared_workgroups(waves), units) * (one ? 1 : 4), 256, kMostSharedParts);
  };
  // Tiles of columns: no more than this, as every group that has any begins one.
  const int64_t col_tiles = all <= num_groups ? all : (all - num_groups) / (32 * waves) + num_groups;
  p.shared_unit = rrt::prefix_unit(waves);
  p.shared_most = shared_parts(seqs, waves, num_groups == 1);
  // Sixteen tokens of one page, their bytes within 31 bits.
  const bool p16 = a->page_size % 16 == 0 && a->token_stride < (1 << 26);
  out->shared_fn = rrt::prefix_kernel_ptr(a->dtype, a->store, a->head_dim, waves, p16);
  // One workgroup makes the plan.  Parts times tiles times heads are at most
  // `workgroups` and one more for each tile and head; every group's rounds up to
  // eight.
  out->shared_grid = 1 + 8 * (ceil_div(p.shared_workgroups + col_tiles * a->num_kv_heads, 8) + col_tiles);

  // The rows' own.
  const int64_t columns = (int64_t)a->next_n * per;
  const int tiles = columns > 16 ? 2 : 1;
  p.unit = kUnit;
  p.least = kLeast;
  p.group_rows = a->next_n;
  p.col_tiles = (int32_t)ceil_div(columns, 16 * tiles);
  p.groups = (int32_t)seqs;
  const int64_t inner = (int64_t)a->num_kv_heads * p.col_tiles;
  auto own_parts = [&](int64_t seqs) { return limited(ceil_div(p.workgroups, seqs * inner) * 4, kLeast, kMostOwnParts); };
  p.most = own_parts(seqs);
  p.pitch = p.shared_most + p.most;
  out->own_fn = rrt::attn_kernel_ptr(a->dtype, a->store, a->head_dim, a->next_n > 1 ? rrt::kOwnManyRows : rrt::kOwnOneRow, tiles);
  auto items_for = [&](int64_t seqs) { return seqs + ceil_div(p.workgroups, inner); };
  out->own_grid = ceil_div(items_for(seqs), 8) * 8 * inner;
  const size_t part_bytes = a->head_dim * sizeof(float) + sizeof(float2);
  auto bytes_for = [&](int64_t seqs, int64_t pitch) {
    return (size_t)(seqs * a->next_n * a->num_heads * pitch) * part_bytes + sizeof(rrt::PrefixPlanned) +
           (size_t)ceil_div(seqs, 4) * 16 + (size_t)items_for(seqs) * sizeof(rrt::PrefixItem);
  };
  out->bytes = bytes_for(seqs, p.pitch);
  if (reserve == nullptr) return TOPK_OK;
  // Fewer rows, or as many in fewer groups, may be split into more parts each.
  // Past two units a CU the rules give every number of rows as many parts.
  *reserve = out->bytes;
  for (int w : {1, 2, 4}) {
    *reserve = std::max(*reserve, bytes_for(seqs, shared_parts(seqs, w, false) + own_parts(seqs)));
    for (int64_t n = std::min<int64_t>(seqs, 64 * w * (int64_t)cus + 1); n > 0; --n)
      *reserve = std::max(*reserve, bytes_for(n, shared_parts(n, w, false) + own_parts(n)));
  }
  return TOPK_OK;
}

// The arguments of paged_attention over the tokens of num_blocks chosen blocks.
int block_args(const paged_attention_args* a, const int32_t* blocks, int64_t row_stride, int64_t head_stride,
               int32_t num_blocks, paged_attention_args* out) {
  REQUIRE(a != nullptr, "null args");
  REQUIRE(a->chosen == nullptr, "blocks are chosen in place of positions: chosen must be NULL");
  REQUIRE(a->page_size >= 1, "page_size must be >= 1");
  REQUIRE(num_blocks >= 1 && (int64_t)num_blocks * a->page_size <= rrt::kMostTokens,
          "num_blocks must be >= 1, num_blocks * page_size at most 2^30");
  REQUIRE(row_stride >= 0 && head_stride >= 0, "strides must be >= 0");
  REQUIRE(aligned(blocks, 4), "blocks must be 4-byte aligned");
  REQUIRE(blocks != nullptr || a->num_rows <= 0, "null blocks");
  *out = *a;
  // Any address stands for the blocks where there are no rows.
  out->chosen = blocks != nullptr ? blocks : reinterpret_cast<const int32_t*>(16);
  out->chosen_stride = row_stride;
  out->num_chosen = num_blocks * a->page_size;
  return TOPK_OK;
}

// ---------------------------------------------------------------------------
// Bounds and the choice of blocks
// ---------------------------------------------------------------------------

int check_bounds(const paged_bounds_args* a) {
  REQUIRE(a != nullptr, "null args");
  REQUIRE(a->store == PAGED_BF16 || a->store == PAGED_FP16 || a->store == PAGED_E4M3,
          "store must be PAGED_BF16, PAGED_FP16 or PAGED_E4M3");
  REQUIRE(a->num_seqs >= 0, "num_seqs must be >= 0");
  REQUIRE(a->num_tokens >= 0, "num_tokens must be >= 0");
  REQUIRE(a->num_kv_heads >= 1, "num_kv_heads must be >= 1");
  REQUIRE(a->head_dim == 64 || a->head_dim == 128, "head_dim must be 64 or 128");
  REQUIRE(a->page_size >= 1, "page_size must be >= 1");
  REQUIRE(a->table_width >= 1, "table_width must be >= 1");
  if (a->num_seqs == 0 || a->num_tokens == 0) return TOPK_OK;
  REQUIRE(a->num_pages >= 1, "num_pages must be >= 1");
  REQUIRE(a->k != nullptr && a->block_table != nullptr && a->starts != nullptr && a->lengths != nullptr &&
              a->bounds != nullptr && a->scales != nullptr,
          "null k, block_table, starts, lengths, bounds or scales");
  const int64_t sz = a->store == PAGED_E4M3 ? 1 : 2;
  REQUIRE(a->page_stride >= 0 && a->token_stride >= 0 && a->head_stride >= 0 && a->bounds_page_stride >= 0 &&
              a->bounds_head_stride >= 0 && a->scales_stride >= 0 && a->table_stride >= 0,
          "strides must be >= 0");
  REQUIRE(aligned(a->k, 16) && a->page_stride * sz % 16 == 0 && a->token_stride * sz % 16 == 0 &&
              a->head_stride * sz % 16 == 0,
          "the cache and its strides must be multiples of 16 bytes");
  REQUIRE(aligned(a->bounds, 16) && a->bounds_page_stride % 16 == 0 && a->bounds_head_stride % 16 == 0,
          "bounds and their strides must be multiples of 16 bytes");
  REQUIRE(aligned(a->block_table, 4) && aligned(a->starts, 4) && aligned(a->lengths, 4) && aligned(a->scales, 4),
          "block_table, starts, lengths and scales must be 4-byte aligned");
  return TOPK_OK;
}

int check_select(const paged_select_args* a) {
  REQUIRE(a != nullptr, "null args");
  if (int rc = check_types(a->dtype, a->dtype)) return rc;
  REQUIRE(a->num_rows >= 0, "num_rows must be >= 0");
  REQUIRE(a->next_n >= 1 && a->num_rows % a->next_n == 0, "next_n must be >= 1 and divide num_rows");
  REQUIRE(a->num_heads >= 1, "num_heads must be >= 1");
  REQUIRE(a->num_kv_heads >= 1 && a->num_heads % a->num_kv_heads == 0, "num_kv_heads must be >= 1 and divide num_heads");
  REQUIRE(a->head_dim == 64 || a->head_dim == 128, "head_dim must be 64 or 128");
  REQUIRE(a->page_size >= 1, "page_size must be >= 1");
  REQUIRE(a->table_width >= 1 && a->table_width <= rrt::kMostBlocks, "table_width must be in [1, 32768]");
  REQUIRE(a->first >= 0 && a->last >= 0 && a->num_blocks >= 1 && (int64_t)a->first + a->last <= a->num_blocks,
          "num_blocks must be >= 1 and first + last, both >= 0, at most num_blocks");
  if (a->num_rows == 0) return TOPK_OK;
  REQUIRE(a->num_pages >= 1, "num_pages must be >= 1");
  REQUIRE((int64_t)a->num_rows * a->num_heads <= INT32_MAX, "num_rows * num_heads must be below 2^31");
  REQUIRE(a->q != nullptr && a->bounds != nullptr && a->scales != nullptr && a->block_table != nullptr &&
              a->lengths != nullptr && a->blocks != nullptr,
          "null q, bounds, scales, block_table, lengths or blocks");
  REQUIRE(a->q_row_stride >= 0 && a->q_head_stride >= 0 && a->bounds_page_stride >= 0 && a->bounds_head_stride >= 0 &&
              a->scales_stride >= 0 && a->table_stride >= 0,
          "strides must be >= 0");
  REQUIRE(aligned(a->q, 16) && a->q_row_stride % 8 == 0 && a->q_head_stride % 8 == 0,
          "q and its strides must be multiples of 16 bytes");
  REQUIRE(aligned(a->bounds, 16) && a->bounds_page_stride % 16 == 0 && a->bounds_head_stride % 16 == 0,
          "bounds and their strides must be multiples of 16 bytes");
  REQUIRE(aligned(a->scales, 4) && aligned(a->block_table, 4) && aligned(a->lengths, 4) && aligned(a->blocks, 4),
          "scales, block_table, lengths and blocks must be 4-byte aligned");
  return TOPK_OK;
}

struct SelectPlan {
  rrt::SelectParams p;
  int tiles, block;
  bool split;
  int64_t grid;
  size_t lds, bytes;
};

constexpr int32_t kFusedBlocks = 4096;       // what one wavefront picks from
constexpr size_t kFusedLds = 128 * 1024;

int plan_select(const paged_select_args* a, hipStream_t stream, SelectPlan* out, size_t* reserve = nullptr) {
  if (int rc = check_select(a)) return rc;
  std::memset(out, 0, sizeof(*out));
  if (reserve != nullptr) *reserve = 0;
  if (a->num_rows == 0) return TOPK_OK;
  int dev = 0, cus = 0;
  if (int rc = rrt::device_of_stream(stream, &dev, &cus)) return rc;
  rrt::SelectParams& p = out->p;
  p.a = *a;
  p.page = rrt::divisor_of(a->page_size);
  p.pitch = (int32_t)ceil_div(a->table_width, 16) * 16;
  const int32_t per = a->num_heads / a->num_kv_heads;
  p.hp2 = 1;
  while (p.hp2 < per && p.hp2 < 16) p.hp2 *= 2;
  const int64_t row_bytes = (int64_t)p.pitch * 4, seqs = a->num_rows / a->next_n;
  const int64_t tile_rows = per <= 16 ? 16 / p.hp2 : 1;  // rows of a sixteen
  const int64_t fit = a->table_width <= kFusedBlocks ? (int64_t)kFusedLds / row_bytes : 0;
  out->tiles = 1;
  out->block = rrt::kBlocksBlock;
  if (per > 16) {
    out->tiles = per <= 32 ? 2 : 4;
  } else {
    while (out->tiles < 4 && tile_rows * out->tiles < a->next_n && (fit == 0 || tile_rows * out->tiles * 2 <= fit))
      out->tiles *= 2;
  }
  p.unit_rows = (int32_t)std::min<int64_t>(per <= 16 ? tile_rows * out->tiles : 1, fit > 0 ? fit : INT32_MAX);
  p.seq_units = (int32_t)ceil_div(a->next_n, p.unit_rows);
  const int64_t units = seqs * p.seq_units * a->num_kv_heads;
  out->split = fit == 0 || (a->table_width > 512 && units * 2 <= cus);
  if (out->split) {
    // Parts of 128 blocks and more, 64 a wavefront's turn, two workgroups a CU.
    const int64_t tiles = p.pitch / 16, most = std::max<int64_t>(1, std::min<int64_t>(tiles / 8, ceil_div(2 * cus, units)));
    p.part_tiles = (int32_t)ceil_div(ceil_div(tiles, most), 4) * 4;
    p.parts = (int32_t)ceil_div(tiles, p.part_tiles);
    out->bytes = (size_t)a->num_rows * a->num_kv_heads * row_bytes;
  } else {
    p.parts = 1;
    out->lds = (size_t)row_bytes * p.unit_rows;
    // One to a CU, so that nothing else hides its waits: eight wavefronts.  us with four and
    // with eight of them, 32 heads on 4, rows of one sequence that share a workgroup:
    //   16 x 32 rows of 4096 blocks, 4 x 256 of 4096        141   92, 259  171
    //   64 rows alone of 1024 (64 heads on 8), of 4096       32   41, 106  136
    // (Rows that share one would take eight below that size too: 16 x 32 of 512 29  23, of
    // 2048 66  47.)
    if (out->lds > kFusedLds / 2) out->block = rrt::kSelectBlock;
  }
  out->grid = units * p.parts;
  if (reserve == nullptr) return TOPK_OK;
  // Fewer rows or a narrower table may be split where these are not: half a CU
  // each, of rows that fit kFusedLds.
  *reserve = out->split ? out->bytes
                        : std::min<size_t>((size_t)a->num_rows * a->num_kv_heads * row_bytes, (size_t)cus / 2 * kFusedLds);
  return TOPK_OK;
}

// ---------------------------------------------------------------------------
// Latent prefill
// ---------------------------------------------------------------------------

int check_prefill(const latent_prefill_args* a) {
  REQUIRE(a != nullptr, "null args");
  if (int rc = check_types(a->dtype, a->store)) return rc;
  REQUIRE(a->num_tokens >= 0, "num_tokens must be >= 0");
  REQUIRE(a->num_seqs >= 0, "num_seqs must be >= 0");
  REQUIRE(a->num_heads >= 1, "num_heads must be >= 1");
  REQUIRE(a->latent_dim == 256 || a->latent_dim == 512, "latent_dim must be 256 or 512");
  REQUIRE(a->page_size >= 1, "page_size must be >= 1");
  REQUIRE(a->table_width >= 1, "table_width must be >= 1");
  REQUIRE(a->context_tokens >= 0 && a->context_tokens <= rrt::kMostTokens, "context_tokens must be in [0, 2^30]");
  REQUIRE(std::isfinite(a->softmax_scale * kLog2e), "softmax_scale times log2(e) must be finite");
  if (a->num_tokens == 0 || a->num_seqs == 0) return TOPK_OK;
  REQUIRE(a->num_pages >= 1, "num_pages must be >= 1");
  REQUIRE(a->q != nullptr && a->cache != nullptr && a->w_k != nullptr && a->w_v != nullptr &&
              a->block_table != nullptr && a->starts != nullptr && a->lengths != nullptr && a->out != nullptr,
          "null q, cache, w_k, w_v, block_table, starts, lengths or out");
  const int64_t sz = a->store == PAGED_E4M3 ? 1 : 2;
  REQUIRE(a->q_row_stride >= 0 && a->q_head_stride >= 0 && a->page_stride >= 0 && a->token_stride >= 0 &&
              a->table_stride >= 0,
          "strides must be >= 0");
  REQUIRE(aligned(a->q, 16) && a->q_row_stride % 8 == 0 && a->q_head_stride % 8 == 0,
          "q and its strides must be multiples of 16 bytes");
  REQUIRE(aligned(a->cache, 16) && a->page_stride * sz % 16 == 0 && a->token_stride * sz % 16 == 0,
          "the cache and its strides must be multiples of 16 bytes");
  REQUIRE(aligned(a->w_k, 16) && aligned(a->w_v, 16), "w_k and w_v must be aligned to 16 bytes");
  REQUIRE(aligned(a->out, 16), "out must be 16-byte aligned");
  REQUIRE(aligned(a->block_table, 4) && aligned(a->starts, 4) && aligned(a->lengths, 4) && aligned(a->lse, 4) &&
              aligned(a->scale, 4),
          "block_table, starts, lengths, lse and scale must be 4-byte aligned");
  REQUIRE(a->store == PAGED_E4M3 || a->scale == nullptr, "scale belongs to an e4m3 cache");
  return TOPK_OK;
}

struct PrefillPlan {
  rrt::PrefillParams p;
  size_t low_at, rope_at, value_at, valid_at, flag_at, rope_flag_at, key_exp_at, rope_exp_at, part_at,
      stat_at, bytes;
};

int plan_prefill(const latent_prefill_args* a, hipStream_t stream, PrefillPlan* out, size_t* reserve = nullptr) {
  if (int rc = check_prefill(a)) return rc;
  std::memset(out, 0, sizeof(*out));
  if (reserve != nullptr) *reserve = 0;
  if (a->num_tokens == 0 || a->num_seqs == 0) return TOPK_OK;
  rrt::PrefillParams& p = out->p;
  p.a = *a;
  p.scale_log2 = a->softmax_scale * kLog2e;
  // Each sequence rounds up to whole tiles.
  const int64_t capacity = a->context_tokens / rrt::kCtxTile + a->num_seqs;
  const int64_t row_tiles = a->num_tokens / rrt::prefill_rows() + a->num_seqs;
  REQUIRE(capacity <= INT32_MAX && row_tiles <= INT32_MAX, "too many tokens and sequences for one launch");
  p.capacity = (int32_t)capacity;
  p.row_tiles = (int32_t)row_tiles;
  const size_t tiles = (size_t)capacity, heads = (size_t)a->num_heads;
  const size_t tile_bytes = (size_t)rrt::kCtxTile * PAGED_HEAD_DIM * 2;
  out->low_at = heads * tiles * tile_bytes;
  p.low_tiles = (int32_t)std::min<int64_t>(capacity, (int64_t)rrt::kExactTiles * a->num_seqs);
  out->rope_at = out->low_at + heads * (size_t)p.low_tiles * tile_bytes;
  out->value_at = out->rope_at + tiles * rrt::kCtxTile * PAGED_ROPE_DIM * 2;
  out->valid_at = out->value_at + heads * tiles * tile_bytes;
  out->flag_at = out->valid_at + tiles * sizeof(uint64_t);
  out->rope_flag_at = out->flag_at + heads * tiles * sizeof(uint32_t);
  out->key_exp_at = (out->rope_flag_at + tiles * sizeof(uint32_t) + 15) / 16 * 16;
  out->rope_exp_at = out->key_exp_at + heads * tiles * rrt::kCtxTile * sizeof(int16_t);
  out->part_at = out->rope_exp_at + tiles * rrt::kCtxTile * sizeof(int16_t);
  // Few row tiles: their contexts are shared out, as far as two workgroups a
  // CU go, and joined by a third launch.  us without, in parts of 1024 tokens
  // and of 256: 1 sequence of 8192, 34 rows x 8 heads 201, 66, 56; 1071 x 16 236,
  // 178, 178; 4 of 500 to 1500, 201 x 8 68, 57, 46; 1 of 1024, 5 x 16 48, 39, 33.
  // A part more than fits (3 sequences, 1782 x 24): 256, 263.
  // Rows are counted as if they filled their tiles, since how many sequences are
  // more than padding is not known here.  64 sequences of a row each are split
  // although their tiles fill the chip (8 heads, 4096 tokens: 1050 us, 1025 in one
  // part; 256 of up to 4096, 4 heads: 1240, 1135; 16 of 8192: 535, 568).
  const int64_t longest = std::min<int64_t>(a->context_tokens, rrt::table_tokens(a->table_width, a->page_size));
  int dev = 0, cus = 0;
  if (longest >= 512)
    if (int rc = rrt::device_of_stream(stream, &dev, &cus)) return rc;
  auto parts_for = [&](int64_t tokens) -> int64_t {
    const int64_t units = ceil_div(tokens, rrt::prefill_rows()) * a->num_heads;
    return std::max<int64_t>(1, std::min<int64_t>({2 * cus / units, longest / 256, 16}));
  };
  auto splits_for = [&](int64_t tokens) -> size_t {
    const int64_t parts = parts_for(tokens);
    return parts == 1 ? 0 : (size_t)tokens * heads * (size_t)parts;
  };
  p.parts = (int32_t)parts_for(a->num_tokens);
  constexpr size_t kSplitBytes = PAGED_HEAD_DIM * sizeof(float) + sizeof(float2);
  const size_t splits = splits_for(a->num_tokens);
  out->stat_at = out->part_at + splits * PAGED_HEAD_DIM * sizeof(float);
  out->bytes = out->part_at + splits * kSplitBytes;
  if (reserve == nullptr) return TOPK_OK;
  // Fewer rows may be split into more parts each: the most rows of each number
  // of row tiles, as far as any are split.
  *reserve = out->bytes;
  for (int64_t rows = rrt::prefill_rows(); rows < a->num_tokens && parts_for(rows) > 1; rows += rrt::prefill_rows())
    *reserve = std::max(*reserve, out->part_at + splits_for(rows) * kSplitBytes);
  return TOPK_OK;
}

}  // namespace

extern "C" {

int paged_layout(const int32_t* lengths, const int32_t* new_tokens, int32_t num_seqs, const int32_t* free_pages,
                 int32_t num_free, int32_t* block_table, int64_t table_stride, int32_t table_width,
                 int32_t page_size, int32_t capacity, int32_t* starts, int32_t* slots, int32_t* row_lengths,
                 int32_t* row_seqs, int32_t* pages, hipStream_t stream) {
  REQUIRE(num_seqs >= 0, "num_seqs must be >= 0");
  REQUIRE(num_free >= 0, "num_free must be >= 0");
  REQUIRE(capacity >= 0, "capacity must be >= 0");
  REQUIRE(page_size >= 1, "page_size must be >= 1");
  REQUIRE(table_width >= 1, "table_width must be >= 1");
  REQUIRE(num_seqs <= 1 || table_stride >= table_width, "table_stride must be >= table_width");
  REQUIRE(num_seqs == 0 || (lengths != nullptr && new_tokens != nullptr && block_table != nullptr),
          "null lengths, new_tokens or block_table");
  REQUIRE(num_free == 0 || free_pages != nullptr, "null free_pages");
  REQUIRE(starts != nullptr && pages != nullptr, "null starts or pages");
  REQUIRE(capacity == 0 || (slots != nullptr && row_lengths != nullptr && row_seqs != nullptr),
          "null slots, row_lengths or row_seqs");
  for (const void* p : {(const void*)lengths, (const void*)new_tokens, (const void*)free_pages,
                        (const void*)block_table, (const void*)starts, (const void*)slots, (const void*)row_lengths,
                        (const void*)row_seqs, (const void*)pages})
    REQUIRE(aligned(p, 4), "all arrays must be 4-byte aligned");
  rrt::LayoutParams p{lengths, new_tokens, free_pages, block_table, starts, slots, row_lengths, row_seqs, pages,
                      table_stride, num_seqs, num_free, table_width, page_size, capacity};
  const int64_t grid = std::min<int64_t>(std::max<int64_t>(1, ceil_div(capacity, rrt::kLayoutBlock)), 512);
  return launch(rrt::layout_kernel_ptr(), grid, rrt::kLayoutBlock, &p, stream, "paged_layout");
}

int paged_append(const int32_t* slots, int32_t num_tokens, const paged_part* parts, int32_t num_parts,
                 int32_t page_size, int32_t num_pages, paged_dtype dtype, paged_dtype store, hipStream_t stream) {
  if (int rc = check_types(dtype, store)) return rc;
  REQUIRE(num_tokens >= 0, "num_tokens must be >= 0");
  REQUIRE(num_parts == 1 || num_parts == 2, "num_parts must be 1 or 2");
  REQUIRE(parts != nullptr, "null parts");
  REQUIRE(page_size >= 1 && num_pages >= 0, "page_size must be >= 1 and num_pages >= 0");
  rrt::AppendParams p{};
  const int64_t sz = store == PAGED_E4M3 ? 1 : 2;
  bool wide = true;
  for (int i = 0; i < num_parts; ++i) {
    const paged_part& q = parts[i];
    REQUIRE(q.width >= 1 && q.head_width >= 1 && q.width % q.head_width == 0,
            "a part's head_width must divide its width, both >= 1");
    REQUIRE(q.src_stride >= 0 && q.dst_page_stride >= 0 && q.dst_token_stride >= 0 && q.dst_head_stride >= 0,
            "strides must be >= 0");
    REQUIRE(store == PAGED_E4M3 || q.scales == nullptr, "scales belong to an e4m3 cache");
    REQUIRE(aligned(q.src, 2) && aligned(q.dst, (uintptr_t)sz) && aligned(q.scales, 4),
            "a part's pointers must be aligned to their elements");
    if (num_tokens > 0 && num_pages > 0) REQUIRE(q.src != nullptr && q.dst != nullptr, "null src or dst of a part");
    // 16-byte loads, and stores of as many elements.
    wide = wide && aligned(q.src, 16) && q.src_stride % 8 == 0 && aligned(q.dst, 8 * sz) && q.head_width % 8 == 0 &&
           q.dst_page_stride % 8 == 0 && q.dst_token_stride % 8 == 0 && q.dst_head_stride % 8 == 0;
    p.part[i] = q;
  }
  if (num_tokens == 0 || num_pages == 0) return TOPK_OK;
  REQUIRE(slots != nullptr && aligned(slots, 4), "slots must be 4-byte aligned and not null");
  for (int i = 0; i < num_parts; ++i) p.chunks[i] = wide ? parts[i].width / 8 : parts[i].width;
  REQUIRE((int64_t)p.chunks[0] + p.chunks[1] <= INT32_MAX, "a token's parts are too wide");
  p.slots = slots;
  p.num_tokens = num_tokens;
  p.page_size = page_size;
  p.num_slots = (int64_t)num_pages * page_size;
  const int64_t items = (int64_t)num_tokens * (p.chunks[0] + p.chunks[1]);
  const int64_t grid = std::min<int64_t>(ceil_div(items, rrt::kAppendBlock), 1 << 16);
  return launch(rrt::append_kernel_ptr(dtype, store, wide), grid, rrt::kAppendBlock, &p, stream, "paged_append");
}

int paged_attention_workspace_size(const paged_attention_args* args, hipStream_t stream, size_t* bytes) {
  REQUIRE(bytes != nullptr, "null bytes");
  AttnPlan plan;
  return plan_attention(args, false, stream, &plan, bytes);
}

int paged_attention(const paged_attention_args* args, void* workspace, hipStream_t stream) {
  return run_attention(args, false, workspace, stream);
}

int paged_block_attention_workspace_size(const paged_attention_args* args, int32_t num_blocks, hipStream_t stream,
                                         size_t* bytes) {
  REQUIRE(bytes != nullptr, "null bytes");
  paged_attention_args a;
  const int64_t heads = 0;
  if (int rc = block_args(args, reinterpret_cast<const int32_t*>(16), 0, 0, num_blocks, &a)) return rc;
  AttnPlan plan;
  return plan_attention(&a, false, stream, &plan, bytes, &heads);
}

int paged_block_attention(const paged_attention_args* args, const int32_t* blocks, int64_t blocks_row_stride,
                          int64_t blocks_head_stride, int32_t num_blocks, void* workspace, hipStream_t stream) {
  paged_attention_args a;
  if (int rc = block_args(args, blocks, blocks_row_stride, blocks_head_stride, num_blocks, &a)) return rc;
  return run_attention(&a, false, workspace, stream, &blocks_head_stride);
}

int paged_prefix_attention_workspace_size(const paged_attention_args* args, int32_t num_groups, hipStream_t stream,
                                          size_t* bytes) {
  REQUIRE(bytes != nullptr, "null bytes");
  REQUIRE(num_groups >= 0, "num_groups must be >= 0");
  // A step without groups, which is paged_attention, is served too.
  if (int rc = paged_attention_workspace_size(args, stream, bytes)) return rc;
  if (num_groups == 0) return TOPK_OK;
  const int32_t* any = reinterpret_cast<const int32_t*>(16);
  PrefixPlan plan;
  size_t grouped = 0;
  if (int rc = plan_prefix(args, any, any, num_groups, stream, &plan, &grouped)) return rc;
  *bytes = std::max(*bytes, grouped);
  return TOPK_OK;
}

int paged_prefix_attention(const paged_attention_args* args, const int32_t* group_starts, const int32_t* shared,
                           int32_t num_groups, void* workspace, hipStream_t stream) {
  REQUIRE(num_groups >= 0, "num_groups must be >= 0");
  if (num_groups == 0) return run_attention(args, false, workspace, stream);
  PrefixPlan plan;
  if (int rc = plan_prefix(args, group_starts, shared, num_groups, stream, &plan)) return rc;
  if (args->num_rows == 0) return TOPK_OK;
  if (int rc = check_workspace(workspace, plan.bytes)) return rc;
  rrt::AttnParams& p = plan.p;
  const int64_t outputs = (int64_t)args->num_rows * args->num_heads;
  // The plan first, so that all of it is aligned.
  const int64_t seqs = args->num_rows / args->next_n;
  p.planned = static_cast<rrt::PrefixPlanned*>(workspace);
  p.share = reinterpret_cast<int32_t*>(p.planned + 1);
  p.part_out = reinterpret_cast<float*>(p.share + ceil_div(seqs, 4) * 4);
  p.part_stat = reinterpret_cast<float2*>(p.part_out + outputs * p.pitch * args->head_dim);
  p.items = reinterpret_cast<rrt::PrefixItem*>(p.part_stat + outputs * p.pitch);
  const char* name = "paged_prefix_attention";
  if (int rc = launch(plan.shared_fn, plan.shared_grid, 256, &p, stream, name)) return rc;
  if (int rc = launch(plan.own_fn, plan.own_grid, 256, &p, stream, name)) return rc;
  return launch(rrt::prefix_join_kernel_ptr(args->dtype, args->head_dim), ceil_div(outputs, 4), 256, &p, stream, name);
}

int paged_bounds(const paged_bounds_args* args, hipStream_t stream) {
  if (int rc = check_bounds(args)) return rc;
  if (args->num_seqs == 0 || args->num_tokens == 0) return TOPK_OK;
  rrt::BoundsParams p{};
  p.a = *args;
  p.page = rrt::divisor_of(args->page_size);
  p.units = (int64_t)args->num_tokens / args->page_size + 2 * (int64_t)args->num_seqs;
  return launch(rrt::bounds_kernel_ptr(args->store, args->head_dim),
                ceil_div(p.units * args->num_kv_heads, rrt::kBlocksBlock / 64), rrt::kBlocksBlock, &p, stream,
                "paged_bounds");
}

int paged_block_select_workspace_size(const paged_select_args* args, hipStream_t stream, size_t* bytes) {
  REQUIRE(bytes != nullptr, "null bytes");
  SelectPlan plan;
  return plan_select(args, stream, &plan, bytes);
}

int paged_block_select(const paged_select_args* args, void* workspace, hipStream_t stream) {
  SelectPlan plan;
  if (int rc = plan_select(args, stream, &plan)) return rc;
  if (args->num_rows == 0) return TOPK_OK;
  if (int rc = check_workspace(workspace, plan.bytes)) return rc;
  plan.p.scores = static_cast<float*>(workspace);
  if (int rc = launch(rrt::select_kernel_ptr(args->dtype, args->head_dim, plan.tiles, plan.split), plan.grid,
                      plan.block, &plan.p, stream, "paged_block_select", plan.lds))
    return rc;
  if (!plan.split) return TOPK_OK;
  return launch(rrt::pick_kernel_ptr(), (int64_t)args->num_rows * args->num_kv_heads, rrt::kPickBlock, &plan.p, stream,
                "paged_block_select");
}

int latent_attention_workspace_size(const paged_attention_args* args, hipStream_t stream, size_t* bytes) {
  REQUIRE(bytes != nullptr, "null bytes");
  AttnPlan plan;
  return plan_attention(args, true, stream, &plan, bytes);
}

int latent_attention(const paged_attention_args* args, void* workspace, hipStream_t stream) {
  return run_attention(args, true, workspace, stream);
}

int latent_prefill_workspace_size(const latent_prefill_args* args, hipStream_t stream, size_t* bytes) {
  REQUIRE(bytes != nullptr, "null bytes");
  PrefillPlan plan;
  return plan_prefill(args, stream, &plan, bytes);
}

int latent_prefill(const latent_prefill_args* args, void* workspace, hipStream_t stream) {
  PrefillPlan plan;
  if (int rc = plan_prefill(args, stream, &plan)) return rc;
  if (plan.bytes == 0) return TOPK_OK;
  if (workspace == nullptr) {
    char buf[96];
    std::snprintf(buf, sizeof(buf), "this launch needs a workspace of %zu bytes", plan.bytes);
    return set_error(TOPK_EWORKSPACE, buf);
  }
  REQUIRE(aligned(workspace, 16), "workspace must be 16-byte aligned");
  rrt::PrefillParams& p = plan.p;
  char* ws = static_cast<char*>(workspace);
  p.keys = ws;
  p.lows = ws + plan.low_at;
  p.ropes = ws + plan.rope_at;
  p.values = ws + plan.value_at;
  p.valid = reinterpret_cast<uint64_t*>(ws + plan.valid_at);
  p.flags = reinterpret_cast<uint32_t*>(ws + plan.flag_at);
  p.rope_flags = reinterpret_cast<uint32_t*>(ws + plan.rope_flag_at);
  p.key_exps = reinterpret_cast<int16_t*>(ws + plan.key_exp_at);
  p.rope_exps = reinterpret_cast<int16_t*>(ws + plan.rope_exp_at);
  if (int rc = launch(rrt::expand_kernel_ptr(args->dtype, args->store, args->latent_dim),
                      ceil_div(p.capacity, 2) * args->num_heads, 256, &p, stream, "expansion of latent vectors"))
    return rc;
  p.part_out = reinterpret_cast<float*>(ws + plan.part_at);
  p.part_stat = reinterpret_cast<float2*>(ws + plan.stat_at);
  const int64_t row_tiles = (int64_t)p.row_tiles * args->num_heads;
  if (int rc = launch(rrt::prefill_kernel_ptr(args->dtype), row_tiles * p.parts, 256, &p, stream, "latent_prefill"))
    return rc;
  if (p.parts == 1) return TOPK_OK;
  return launch(rrt::prefill_join_kernel_ptr(args->dtype), row_tiles * (rrt::prefill_rows() / rrt::prefill_join_rows()),
                256, &p, stream, "join of split contexts");
}

int64_t paged_debug_place(const int32_t* table_row, int32_t page_size, int32_t num_pages, int64_t page_stride,
                          int64_t token_stride, int32_t pos) {
  return rrt::locate(table_row, page_size, num_pages, page_stride, token_stride, pos);
}

void paged_debug_split(int32_t n, int32_t most, int32_t least, int32_t unit, int32_t out[2]) {
  const rrt::Split s = rrt::split_of(n, most, least, unit);
  out[0] = s.parts;
  out[1] = s.chunk;
}

}  // extern "C"
