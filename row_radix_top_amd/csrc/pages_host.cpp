// Host side of the operators on pages that sequences share.

#include <algorithm>
#include <cstring>
#include <initializer_list>

#include "paged_host.hpp"

namespace {

constexpr int kBlock = rrt::kPagesBlock;
constexpr int64_t kRowPiece = 4 * kBlock;  // table entries of a workgroup
// Workgroups of a copy (pairs times caches times pieces of a page) up to which each
// pair has its own, and that stride over the pairs of a longer list: a launch takes
// fewer than 2^24, and a list may be half a large pool.  us with one to a pair, and
// striding with 2^13, 2^14 and 2^15:
//   2 caches, 34662 pairs, 13700 of them moves   377  361  357  355
//   2 caches, 2^17 pairs, 10 moves                90   15   15   20
//   8 caches, 2^17 pairs, 60000 moves            623  421  411  404
//   32 caches, 2^18 pairs, 10 moves             2700  199  185  163
// A fork of 512 rows and its copy, 2^14 workgroups: 33.4 with one to a pair, 34.8
// striding, as pairs come by vector loads then.
constexpr int32_t kCopyGroups = 1 << 14;

int check_table(const int32_t* block_table, int64_t table_stride, int32_t table_width, const int32_t* lengths,
                int32_t num_seqs, int32_t page_size) {
  REQUIRE(num_seqs >= 0, "num_seqs must be >= 0");
  REQUIRE(page_size >= 1, "page_size must be >= 1");
  REQUIRE(table_width >= 1, "table_width must be >= 1");
  REQUIRE(num_seqs <= 1 || table_stride >= table_width, "table_stride must be >= table_width");
  REQUIRE(num_seqs == 0 || (block_table != nullptr && lengths != nullptr), "null block_table or lengths");
  REQUIRE(aligned(block_table, 4) && aligned(lengths, 4), "all arrays must be 4-byte aligned");
  return TOPK_OK;
}

// An array of the caller's: rows of `width` entries, `stride` apart.
struct Span {
  const void* data;
  int64_t rows, stride, width;
};
Span list_of(const void* data, int64_t n) { return {data, 1, n, n}; }

// Whether two arrays share an entry.  Views of one buffer that lie between one
// another (two tables side by side) do not.
bool meet(const Span& a, const Span& b) {
  if (a.data == nullptr || b.data == nullptr || a.rows <= 0 || b.rows <= 0 || a.width <= 0 || b.width <= 0) return false;
  const int64_t at = (int64_t)(reinterpret_cast<uintptr_t>(a.data) / 4), to = (int64_t)(reinterpret_cast<uintptr_t>(b.data) / 4);
  if (at >= to + (b.rows - 1) * b.stride + b.width || to >= at + (a.rows - 1) * a.stride + a.width) return false;
  if (a.rows > 1 && b.rows > 1 && a.stride == b.stride) {
    const int64_t off = ((at - to) % b.stride + b.stride) % b.stride;  // of a's rows from the b row before
    if (off >= b.width && off + a.width <= b.stride) return false;
  }
  if (a.rows > b.rows) return meet(b, a);
  for (int64_t i = 0; i < a.rows; ++i) {
    // The first row of b that ends behind this one's beginning.
    const int64_t x = at + i * a.stride, past = x - to - b.width;
    const int64_t j = past < 0 ? 0 : b.rows == 1 ? 1 : past / b.stride + 1;
    if (j < b.rows && to + j * b.stride < x + a.width) return true;
  }
  return false;
}

// Whether an output shares an entry with another one or with an input.
bool overlap(std::initializer_list<Span> outputs, std::initializer_list<Span> inputs) {
  for (const Span* o = outputs.begin(); o != outputs.end(); ++o) {
    for (const Span* p = o + 1; p != outputs.end(); ++p)
      if (meet(*o, *p)) return true;
    for (const Span& in : inputs)
      if (meet(*o, in)) return true;
  }
  return false;
}

// A bitmap of the pool, whole 16 bytes.
int64_t bitmap_words(int32_t num_pages) { return ceil_div(num_pages, 128) * 4; }

rrt::PoolParams pool_params(const int32_t* block_table, int64_t table_stride, int32_t table_width,
                            const int32_t* lengths, int32_t num_seqs, int32_t page_size, int32_t num_pages) {
  rrt::PoolParams p{};
  p.table = block_table;
  p.lengths = lengths;
  p.table_stride = table_stride;
  p.table_width = table_width;
  p.num_seqs = num_seqs;
  p.page_size = page_size;
  p.num_pages = num_pages;
  p.words = (int32_t)bitmap_words(num_pages);
  p.row_pieces = (int32_t)ceil_div(table_width, kRowPiece);
  p.page = rrt::divisor_of(page_size);
  return p;
}

bool small_pool(const rrt::PoolParams& p) {
  return p.num_pages <= rrt::kSmallPages && (int64_t)p.num_seqs * p.table_width <= rrt::kSmallEntries;
}

// Clears the bitmap (and the counts) and sets what the table holds.
int hold(rrt::PoolParams* p, hipStream_t stream, const char* what) {
  const int64_t words = p->refs != nullptr ? p->num_pages : p->words;
  if (int rc = launch(rrt::pool_kernel_ptr(rrt::kPoolClear),
                      std::min<int64_t>(std::max<int64_t>(1, ceil_div(words, kBlock)), 1024), kBlock, p, stream, what))
    return rc;
  if (p->num_seqs == 0) return TOPK_OK;
  return launch(rrt::pool_kernel_ptr(rrt::kPoolHold), (int64_t)p->num_seqs * p->row_pieces, kBlock, p, stream, what);
}

}  // namespace

extern "C" {

int paged_fork(const int32_t* block_table, int64_t table_stride, int32_t table_width, const int32_t* lengths,
               int32_t num_seqs, const int32_t* parents, const int32_t* keep, int32_t num_rows,
               const int32_t* free_pages, int32_t num_free, int32_t page_size, int32_t* out_table,
               int64_t out_stride, int32_t* out_lengths, int32_t* src, int32_t* dst, int32_t* tokens, int32_t* pages,
               hipStream_t stream) {
  if (int rc = check_table(block_table, table_stride, table_width, lengths, num_seqs, page_size)) return rc;
  REQUIRE(num_rows >= 0, "num_rows must be >= 0");
  REQUIRE(num_free >= 0, "num_free must be >= 0");
  REQUIRE(num_rows <= 1 || out_stride >= table_width, "out_stride must be >= table_width");
  REQUIRE(num_free == 0 || free_pages != nullptr, "null free_pages");
  REQUIRE(pages != nullptr, "null pages");
  REQUIRE(num_rows == 0 || (parents != nullptr && out_table != nullptr && out_lengths != nullptr && src != nullptr &&
                            dst != nullptr && tokens != nullptr),
          "null parents, out_table, out_lengths, src, dst or tokens");
  for (const void* p : {(const void*)parents, (const void*)keep, (const void*)free_pages, (const void*)out_table,
                        (const void*)out_lengths, (const void*)src, (const void*)dst, (const void*)tokens,
                        (const void*)pages})
    REQUIRE(aligned(p, 4), "all arrays must be 4-byte aligned");
  REQUIRE(!overlap({{out_table, num_rows, out_stride, table_width}, list_of(out_lengths, num_rows), list_of(src, num_rows),
                    list_of(dst, num_rows), list_of(tokens, num_rows), list_of(pages, 1)},
                   {{block_table, num_seqs, table_stride, table_width}, list_of(lengths, num_seqs), list_of(parents, num_rows),
                    list_of(keep, num_rows), list_of(free_pages, num_free)}),
          "a fork's outputs overlap one another or what it goes on from (table, lengths, parents, keep, free_pages)");
  rrt::ForkParams p{};
  p.table = block_table, p.lengths = lengths, p.parents = parents, p.keep = keep, p.free_pages = free_pages;
  p.out_table = out_table, p.out_lengths = out_lengths, p.src = src, p.dst = dst, p.tokens = tokens, p.pages = pages;
  p.table_stride = table_stride, p.out_stride = out_stride;
  p.table_width = table_width, p.num_seqs = num_seqs, p.num_rows = num_rows, p.num_free = num_free;
  p.page_size = page_size;
  // Each workgroup counts the marks before its rows: 1024 of them at most.
  p.rows_each = (int32_t)std::max<int64_t>(1, ceil_div(num_rows, 1024));
  p.page = rrt::divisor_of(page_size);
  if (num_rows <= rrt::kSmallRows && (int64_t)num_rows * table_width <= rrt::kSmallEntries)
    return launch(rrt::small_kernel_ptr(rrt::kSmallFork), 1, rrt::kSmallBlock, &p, stream, "paged_fork");
  if (num_rows > 0)
    if (int rc = launch(rrt::fork_kernel_ptr(false), ceil_div(num_rows, kBlock / 64), kBlock, &p, stream, "paged_fork"))
      return rc;
  return launch(rrt::fork_kernel_ptr(true), std::max<int64_t>(1, ceil_div(num_rows, p.rows_each)), kBlock, &p, stream,
                "paged_fork");
}

int paged_copy(const int32_t* src, const int32_t* dst, const int32_t* tokens, int32_t num_pairs,
               const paged_pages* caches, int32_t num_caches, int32_t num_pages, hipStream_t stream) {
  REQUIRE(num_pairs >= 0, "num_pairs must be >= 0");
  REQUIRE(num_caches >= 0, "num_caches must be >= 0");
  REQUIRE(num_pages >= 0, "num_pages must be >= 0");
  REQUIRE(num_caches == 0 || caches != nullptr, "null caches");
  for (int i = 0; i < num_caches; ++i) {
    const paged_pages& q = caches[i];
    REQUIRE(q.tokens >= 1 && q.outer >= 1 && q.width >= 1, "a cache's tokens, outer and width must be >= 1");
    REQUIRE((int64_t)q.outer * q.width <= INT32_MAX && (int64_t)q.outer * q.width * q.tokens <= INT32_MAX,
            "a page of a cache must be below 2^31 bytes");
    REQUIRE(q.page_stride >= 0 && q.token_stride >= 0 && q.outer_stride >= 0, "strides must be >= 0");
    REQUIRE(num_pairs == 0 || num_pages == 0 || q.data != nullptr, "null data of a cache");
  }
  if (num_pairs == 0 || num_pages == 0) return TOPK_OK;
  REQUIRE(src != nullptr && dst != nullptr, "null src or dst");
  REQUIRE(aligned(src, 4) && aligned(dst, 4) && aligned(tokens, 4), "all arrays must be 4-byte aligned");
  for (int at = 0; at < num_caches; at += PAGED_COPY_CACHES) {
    rrt::CopyParams p{};
    p.src = src, p.dst = dst, p.tokens = tokens;
    p.num_pairs = num_pairs, p.num_pages = num_pages;
    p.num_caches = std::min(num_caches - at, PAGED_COPY_CACHES);
    int64_t bytes = 0, all = 0;
    for (int i = 0; i < p.num_caches; ++i) {
      const paged_pages& q = p.cache[i] = caches[at + i];
      bytes = std::max(bytes, (int64_t)q.tokens * q.outer * q.width);
      all |= (int64_t)reinterpret_cast<uintptr_t>(q.data) | q.page_stride | (q.tokens > 1 ? q.token_stride : 0) |
             (q.outer > 1 ? q.outer_stride : 0) | q.width;
    }
    const int v = all % 16 == 0 ? 16 : all % 4 == 0 ? 4 : 1;
    for (int i = 0; i < p.num_caches; ++i) {
      p.row[i] = rrt::divisor_of(p.cache[i].width / v);
      p.each[i] = rrt::divisor_of(p.cache[i].width / v * p.cache[i].outer);
    }
    // Four steps of every thread for a whole page.
    p.pieces = (int32_t)std::min<int64_t>(ceil_div(bytes, (int64_t)v * kBlock * 4), 1024);
    const int32_t inner = p.num_caches * p.pieces;
    const bool many = num_pairs > std::max(1, kCopyGroups / inner);
    p.pair_groups = many ? std::max(1, kCopyGroups / inner) : num_pairs;
    if (int rc = launch(rrt::copy_kernel_ptr(v, many), (int64_t)p.pair_groups * inner, kBlock, &p, stream, "paged_copy"))
      return rc;
  }
  return TOPK_OK;
}

int paged_free_workspace_size(int32_t num_pages, size_t* bytes) {
  REQUIRE(bytes != nullptr, "null bytes");
  REQUIRE(num_pages >= 0, "num_pages must be >= 0");
  *bytes = (size_t)bitmap_words(num_pages) * 4;
  return TOPK_OK;
}

int paged_free(const int32_t* block_table, int64_t table_stride, int32_t table_width, const int32_t* lengths,
               int32_t num_seqs, int32_t page_size, int32_t num_pages, int32_t* free_pages, int32_t* refs,
               int32_t* count, void* workspace, hipStream_t stream) {
  if (int rc = check_table(block_table, table_stride, table_width, lengths, num_seqs, page_size)) return rc;
  REQUIRE(num_pages >= 0, "num_pages must be >= 0");
  REQUIRE(count != nullptr && (num_pages == 0 || (free_pages != nullptr && refs != nullptr)),
          "null free_pages, refs or count");
  REQUIRE(aligned(free_pages, 4) && aligned(refs, 4) && aligned(count, 4), "all arrays must be 4-byte aligned");
  if (int rc = check_workspace(workspace, (size_t)bitmap_words(num_pages) * 4)) return rc;
  REQUIRE(!overlap({list_of(free_pages, num_pages), list_of(refs, num_pages), list_of(count, 1),
                    list_of(workspace, bitmap_words(num_pages))},
                   {{block_table, num_seqs, table_stride, table_width}, list_of(lengths, num_seqs)}),
          "free_pages, refs, count and workspace overlap one another or the table or lengths");
  rrt::PoolParams p = pool_params(block_table, table_stride, table_width, lengths, num_seqs, page_size, num_pages);
  p.bits = static_cast<uint32_t*>(workspace);
  p.refs = refs, p.free_pages = free_pages, p.count = count;
  if (small_pool(p))
    return launch(rrt::small_kernel_ptr(rrt::kSmallFree), 1, rrt::kSmallBlock, &p, stream, "paged_free");
  if (int rc = hold(&p, stream, "paged_free")) return rc;
  return launch(rrt::pool_kernel_ptr(rrt::kPoolFree), std::max<int64_t>(1, ceil_div(num_pages, kBlock)), kBlock, &p,
                stream, "paged_free");
}

int paged_compact_workspace_size(int32_t num_pages, size_t* bytes) {
  REQUIRE(bytes != nullptr, "null bytes");
  REQUIRE(num_pages >= 0, "num_pages must be >= 0");
  *bytes = (size_t)bitmap_words(num_pages) * 4 + (size_t)num_pages * 4;
  return TOPK_OK;
}

int paged_compact(const int32_t* block_table, int64_t table_stride, int32_t table_width, const int32_t* lengths,
                  int32_t num_seqs, int32_t page_size, int32_t num_pages, int32_t limit, int32_t* out_table,
                  int64_t out_stride, int32_t* src, int32_t* dst, int32_t* moves, int32_t* live, void* workspace,
                  hipStream_t stream) {
  if (int rc = check_table(block_table, table_stride, table_width, lengths, num_seqs, page_size)) return rc;
  REQUIRE(num_pages >= 0, "num_pages must be >= 0");
  REQUIRE(limit >= -1 && limit <= num_pages, "limit must be in [-1, num_pages]");
  REQUIRE(num_seqs <= 1 || out_stride >= table_width, "out_stride must be >= table_width");
  REQUIRE(num_seqs == 0 || out_table != nullptr, "null out_table");
  REQUIRE(out_table != block_table || num_seqs <= 1 || out_stride == table_stride,
          "a table that is compacted in place keeps its stride");
  REQUIRE(moves != nullptr && live != nullptr && (num_pages < 2 || (src != nullptr && dst != nullptr)),
          "null src, dst, moves or live");
  for (const void* q : {(const void*)out_table, (const void*)src, (const void*)dst, (const void*)moves, (const void*)live})
    REQUIRE(aligned(q, 4), "all arrays must be 4-byte aligned");
  size_t bytes = 0;
  if (int rc = paged_compact_workspace_size(num_pages, &bytes)) return rc;
  if (int rc = check_workspace(workspace, bytes)) return rc;
  const Span table = {block_table, num_seqs, table_stride, table_width}, renamed = {out_table, num_seqs, out_stride, table_width};
  const Span rows = list_of(lengths, num_seqs);
  REQUIRE(!overlap({list_of(src, num_pages / 2), list_of(dst, num_pages / 2), list_of(moves, 1), list_of(live, 1),
                    list_of(workspace, (int64_t)bytes / 4), renamed},
                   {rows}) &&
              (out_table == block_table ||
               !overlap({table}, {list_of(src, num_pages / 2), list_of(dst, num_pages / 2), list_of(moves, 1),
                                  list_of(live, 1), list_of(workspace, (int64_t)bytes / 4), renamed})),
          "src, dst, moves, live, workspace and out_table overlap one another or the table or lengths");
  rrt::PoolParams p = pool_params(block_table, table_stride, table_width, lengths, num_seqs, page_size, num_pages);
  p.bits = static_cast<uint32_t*>(workspace);
  p.rank = reinterpret_cast<int32_t*>(p.bits + p.words);
  p.out_table = out_table, p.out_stride = out_stride;
  p.src = src, p.dst = dst, p.moves = moves, p.live = live;
  p.limit = limit;
  if (small_pool(p))
    return launch(rrt::small_kernel_ptr(rrt::kSmallCompact), 1, rrt::kSmallBlock, &p, stream, "paged_compact");
  if (int rc = hold(&p, stream, "paged_compact")) return rc;
  if (int rc = launch(rrt::pool_kernel_ptr(rrt::kPoolMoves), std::max<int64_t>(1, ceil_div(num_pages, kBlock)), kBlock,
                      &p, stream, "paged_compact"))
    return rc;
  if (num_seqs == 0) return TOPK_OK;
  return launch(rrt::pool_kernel_ptr(rrt::kPoolRename), (int64_t)num_seqs * p.row_pieces, kBlock, &p, stream,
                "paged_compact");
}

}  // extern "C"
