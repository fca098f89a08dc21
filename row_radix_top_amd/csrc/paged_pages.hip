// Pages that sequences share: forks, copies, what is free, and moves that
// bring the held pages together.

#include "paged_device.hpp"

namespace rrt {

constexpr int kBlock = kPagesBlock;

// The sum of x over the workgroup, on all threads; s: a word a wavefront.
__device__ __forceinline__ int32_t block_sum(int32_t x, int32_t* s) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) x += __shfl_xor(x, off);
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = x;
  __syncthreads();
  int32_t sum = 0;
#pragma unroll
  for (int i = 0; i < kBlock / 64; ++i) sum += s[i];
  __syncthreads();
  return sum;
}

__device__ __forceinline__ int32_t pages_of(int32_t n, const Divisor& page) {
  return n == 0 ? 0 : (int32_t)divide((uint32_t)n - 1u, page) + 1;
}

// ---------------------------------------------------------------------------
// Fork.  Row i keeps m tokens of its parent p.  Its last page, if m is no
// multiple of the page size, is the one that the row will write to, so it has
// to be its own: a copy, if another row of the batch holds the page full or a
// row before i holds it in part.  A shared page lies at the same place of every
// row, so the question is one column of the parents' table rows.
//
// Two launches: `mark` answers it, a wavefront a row and the other rows over its
// lanes (src and tokens receive the answer); `write` gives the marked rows their
// free pages, in order (each workgroup counts the marks before its rows by
// itself), and writes the table.  512 rows of 64 pages: 9.4 + 4.0 us, reads that
// wait for one another (parent, length, entry; four rows a lane side by side took
// as long).  Each row looks at every other: a call of 2048 rows takes 27 us, of 8192
// 152, of 32768 3.9 ms.
// ---------------------------------------------------------------------------
__device__ __forceinline__ int32_t kept(const ForkParams& p, int64_t most, int32_t i, int32_t* parent) {
  const int32_t q = p.parents[i];
  *parent = q;
  if ((uint32_t)q >= (uint32_t)p.num_seqs) return 0;
  const int32_t n = clamp_to(p.lengths[q], most);
  return p.keep == nullptr ? n : clamp_to(p.keep[i], n);
}

__global__ void __launch_bounds__(kBlock) fork_mark_kernel(ForkParams p) {
  const int lane = threadIdx.x & 63;
  const int32_t i = (int32_t)(blockIdx.x * (kBlock / 64) + (threadIdx.x >> 6));
  if (i >= p.num_rows) return;
  const int64_t most = table_tokens(p.table_width, p.page_size);
  int32_t parent;
  const int32_t m = kept(p, most, i, &parent);
  const int32_t j = (int32_t)divide((uint32_t)m, p.page), part = m - j * p.page_size;
  const int32_t last = part != 0 ? p.table[(int64_t)parent * p.table_stride + j] : -1;
  bool copy = false;
  if (last >= 0) {
    for (int32_t r0 = 0; r0 < p.num_rows; r0 += 64) {
      const int32_t r = r0 + lane;
      bool other = false;
      if (r < p.num_rows && r != i) {
        int32_t q;
        const int32_t n = kept(p, most, r, &q);
        const int32_t left = n - j * p.page_size;  // tokens that it holds from that page on
        if (left > 0 && (left >= p.page_size || r < i)) other = p.table[(int64_t)q * p.table_stride + j] == last;
      }
      if (__builtin_amdgcn_ballot_w64(other) != 0) {
        copy = true;
        break;
      }
    }
  }
  if (lane == 0) {
    p.out_lengths[i] = m;
    p.src[i] = copy ? last : -1;
    p.tokens[i] = copy ? part : 0;
  }
}

__global__ void __launch_bounds__(kBlock) fork_write_kernel(ForkParams p) {
  __shared__ int32_t sums[kBlock / 64];
  const int tid = threadIdx.x;
  const int32_t first = (int32_t)blockIdx.x * p.rows_each;
  const int32_t stop = p.num_rows - first < p.rows_each ? p.num_rows : first + p.rows_each;
  int32_t before = 0;
  for (int32_t i = tid; i < first; i += kBlock) before += p.src[i] >= 0 ? 1 : 0;
  before = block_sum(before, sums);
  for (int32_t i = first; i < stop; ++i) {
    const int32_t m = p.out_lengths[i], parent = p.parents[i];
    const bool copy = p.src[i] >= 0;
    const int32_t got = copy && before < p.num_free ? p.free_pages[before] : -1;
    if (copy) ++before;
    if (tid == 0) p.dst[i] = got;
    const int32_t need = pages_of(m, p.page);
    const int32_t* from = p.table + (int64_t)(need > 0 ? parent : 0) * p.table_stride;
    int32_t* to = p.out_table + (int64_t)i * p.out_stride;
    for (int32_t j = tid; j < p.table_width; j += kBlock)
      to[j] = j >= need ? -1 : copy && j == need - 1 ? got : from[j];
  }
  if (stop == p.num_rows && tid == 0) p.pages[0] = before;
}

// Few rows (kSmallRows, and kSmallEntries of their tables): both steps by one
// workgroup, a row a wavefront, as launches are what such a call takes: a fork and
// its copy 25.2 us in three of them, 22.3 in two (2.5 us of the device, not 5.6).
__global__ void __launch_bounds__(kSmallBlock) fork_small_kernel(ForkParams p) {
  constexpr int W = kSmallBlock / 64;
  __shared__ int32_t copied[kSmallRows];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  int32_t q = -1, n = 0;  // of row `lane`
  if (lane < p.num_rows) n = kept(p, table_tokens(p.table_width, p.page_size), lane, &q);
  for (int32_t i = w; i < p.num_rows; i += W) {
    const int32_t m = __builtin_amdgcn_readlane(n, i), parent = __builtin_amdgcn_readlane(q, i);
    const int32_t j = (int32_t)divide((uint32_t)m, p.page), part = m - j * p.page_size;
    const int32_t last = part != 0 ? p.table[(int64_t)parent * p.table_stride + j] : -1;
    const int32_t left = n - j * p.page_size;
    bool other = false;
    if (last >= 0 && lane != i && left > 0 && (left >= p.page_size || lane < i))
      other = p.table[(int64_t)q * p.table_stride + j] == last;
    const bool copy = __builtin_amdgcn_ballot_w64(other) != 0;
    if (lane == 0) {
      p.out_lengths[i] = m;
      p.src[i] = copied[i] = copy ? last : -1;
      p.tokens[i] = copy ? part : 0;
    }
  }
  __syncthreads();
  const uint64_t marks = __builtin_amdgcn_ballot_w64(lane < p.num_rows && copied[lane] >= 0);
  for (int32_t i = w; i < p.num_rows; i += W) {
    const int32_t before = __builtin_popcountll(marks & ((1ull << i) - 1ull));
    const bool copy = (marks >> i) & 1u;
    const int32_t got = copy && before < p.num_free ? p.free_pages[before] : -1;
    if (lane == 0) p.dst[i] = got;
    const int32_t need = pages_of(__builtin_amdgcn_readlane(n, i), p.page);
    const int32_t* from = p.table + (int64_t)(need > 0 ? __builtin_amdgcn_readlane(q, i) : 0) * p.table_stride;
    int32_t* to = p.out_table + (int64_t)i * p.out_stride;
    for (int32_t j = lane; j < p.table_width; j += 64) to[j] = j >= need ? -1 : copy && j == need - 1 ? got : from[j];
  }
  if (threadIdx.x == 0) p.pages[0] = __builtin_popcountll(marks);
}

// ---------------------------------------------------------------------------
// Copy.  A workgroup takes a piece of one cache's pages, of one pair or (MANY) of
// every pair_groups-th: it looks at 64 of those at a time, as a compaction's list is
// mostly empty.  V bytes a thread and step, the same for all caches of a launch: what
// their addresses, strides and rows all allow.  Bound by its bytes: 0.88 GB there and
// 0.88 GB back in 343 us, 5.1 TB/s, a large copy's rate; 49 MB each way in 20 us.
// ---------------------------------------------------------------------------
template <int V>
struct Piece;
template <>
struct Piece<16> {
  using type = u32x4;
};
template <>
struct Piece<4> {
  using type = uint32_t;
};
template <>
struct Piece<1> {
  using type = uint8_t;
};

template <int V, bool MANY>
__global__ void __launch_bounds__(kBlock) copy_kernel(CopyParams p) {
  using type = typename Piece<V>::type;
  const uint32_t b = blockIdx.x;
  const uint32_t piece = b % (uint32_t)p.pieces, c = b / (uint32_t)p.pieces % (uint32_t)p.num_caches;
  const uint32_t first = b / (uint32_t)p.pieces / (uint32_t)p.num_caches;
  const paged_pages& q = p.cache[c];
  const Divisor row = p.row[c], each = p.each[c];  // steps of a row, and of a token
  const uint32_t step = (uint32_t)p.pieces * kBlock;
  auto real = [&](int32_t from, int32_t to) {
    return (uint32_t)from < (uint32_t)p.num_pages && (uint32_t)to < (uint32_t)p.num_pages && from != to;
  };
  auto copy = [&](int32_t from, int32_t to, int32_t tokens) __attribute__((always_inline)) {
    const uint32_t items = (uint32_t)tokens * each.by;
    const char* src = (const char*)q.data + (int64_t)from * q.page_stride;
    char* dst = (char*)q.data + (int64_t)to * q.page_stride;
#pragma unroll 4
    for (uint32_t x = piece * kBlock + threadIdx.x; x < items; x += step) {
      const uint32_t t = divide(x, each), y = x - t * each.by, o = divide(y, row);
      const int64_t at = t * q.token_stride + o * q.outer_stride + (int64_t)(y - o * row.by) * V;
      *(type*)(dst + at) = *(const type*)(src + at);
    }
  };
  if constexpr (!MANY) {
    const int32_t from = p.src[first], to = p.dst[first];
    if (!real(from, to)) return;
    copy(from, to, p.tokens == nullptr ? q.tokens : clamp_to(p.tokens[first], q.tokens));
  } else {
    const int lane = threadIdx.x & 63;
    for (int64_t i0 = first; i0 < p.num_pairs; i0 += (int64_t)p.pair_groups * 64) {
      const int64_t i = i0 + (int64_t)lane * p.pair_groups;
      int32_t from = -1, to = -1, tokens = q.tokens;
      if (i < p.num_pairs) {
        from = p.src[i], to = p.dst[i];
        if (p.tokens != nullptr) tokens = clamp_to(p.tokens[i], q.tokens);
      }
      for (uint64_t left = __builtin_amdgcn_ballot_w64(real(from, to)); left != 0; left &= left - 1) {
        const int l = __builtin_ctzll(left);
        copy(__builtin_amdgcn_readlane(from, l), __builtin_amdgcn_readlane(to, l), __builtin_amdgcn_readlane(tokens, l));
      }
    }
  }
}

// ---------------------------------------------------------------------------
// What is held.  `clear` zeroes the counts and a bitmap of the pool, `hold`
// counts the table's entries (adds whose order does not matter) and sets their
// bits, and every workgroup of the last launches counts the bits before its
// pages by itself: 32 pages a word, 32 KB for a pool of 256 K pages, from L2.
// 2048 rows of up to 128 pages of 32 tokens: clear 4.9 us, hold 12 (adds that meet
// in memory), free 4.6, moves 5, rename 5; launches and one trip to memory each.
// Calls for pools of 2^18, 2^20 and 2^22 pages (131 K, 524 K and 2.1 M entries): free
// 20, 62 and 519 us, compact 22, 64 and 534, as every workgroup counts the bitmap.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kBlock) clear_kernel(PoolParams p) {
  const int64_t step = (int64_t)gridDim.x * kBlock, at = (int64_t)blockIdx.x * kBlock + threadIdx.x;
  for (int64_t i = at; i < p.words; i += step) p.bits[i] = 0;
  if (p.refs != nullptr)
    for (int64_t i = at; i < p.num_pages; i += step) p.refs[i] = 0;
}

__device__ __forceinline__ int32_t held_entries(const PoolParams& p, int32_t s) {
  return pages_of(clamp_to(p.lengths[s], table_tokens(p.table_width, p.page_size)), p.page);
}

__global__ void __launch_bounds__(kBlock) hold_kernel(PoolParams p) {
  const int32_t s = (int32_t)(blockIdx.x / (uint32_t)p.row_pieces);
  const int32_t need = held_entries(p, s);
  const int32_t* row = p.table + (int64_t)s * p.table_stride;
  const int32_t j0 = (int32_t)(blockIdx.x % (uint32_t)p.row_pieces) * (kBlock * 4) + (int32_t)threadIdx.x;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int64_t j = (int64_t)j0 + k * kBlock;
    if (j >= need) break;
    const int32_t page = row[j];
    if ((uint32_t)page >= (uint32_t)p.num_pages) continue;
    atomicOr(p.bits + (page >> 5), 1u << (page & 31));
    if (p.refs != nullptr) atomicAdd(p.refs + page, 1);
  }
}

// Held pages among [0, 32 * words), all threads.
__device__ __forceinline__ int32_t bits_before(const PoolParams& p, int32_t words, int32_t* s) {
  int32_t n = 0;
  const int32_t whole = words & ~3;
  for (int32_t i = (int32_t)threadIdx.x * 4; i < whole; i += kBlock * 4) {
    const u32x4 x = *(const u32x4*)(p.bits + i);
    n += __builtin_popcount(x[0]) + __builtin_popcount(x[1]) + __builtin_popcount(x[2]) + __builtin_popcount(x[3]);
  }
  if ((int32_t)threadIdx.x < words - whole) n += __builtin_popcount(p.bits[whole + threadIdx.x]);
  return block_sum(n, s);
}

// A workgroup looks after kPoolPages pages: eight words, two wavefronts' worth
// of bits each.  rank: held pages before the thread's page.
__device__ __forceinline__ int32_t rank_of(const PoolParams& p, int32_t page, int32_t* s) {
  const int32_t word0 = (int32_t)blockIdx.x * (kBlock / 32);
  int32_t n = bits_before(p, word0, s);
  for (int32_t i = word0; i < (page >> 5) && i < p.words; ++i) n += __builtin_popcount(p.bits[i]);
  if ((page >> 5) < p.words) n += __builtin_popcount(p.bits[page >> 5] & ((1u << (page & 31)) - 1u));
  return n;
}

__global__ void __launch_bounds__(kBlock) free_kernel(PoolParams p) {
  __shared__ int32_t sums[kBlock / 64];
  const int32_t page = (int32_t)(blockIdx.x * kBlock + threadIdx.x);
  const int32_t before = rank_of(p, page, sums);
  const int32_t live = bits_before(p, p.words, sums);
  if (page == 0) p.count[0] = p.num_pages - live;
  if (page >= p.num_pages) return;
  const bool held = (p.bits[page >> 5] >> (page & 31)) & 1u;
  if (!held) p.free_pages[page - before] = page;
  // The places behind the last one, as many as there are held pages.
  if (held) p.free_pages[p.num_pages - live + before] = -1;
}

// The k-th held page from the limit on and the k-th free one below it.
__global__ void __launch_bounds__(kBlock) moves_kernel(PoolParams p) {
  __shared__ int32_t sums[kBlock / 64];
  const int32_t page = (int32_t)(blockIdx.x * kBlock + threadIdx.x);
  const int32_t before = rank_of(p, page, sums);
  const int32_t live = bits_before(p, p.words, sums);
  const int32_t limit = p.limit < 0 ? live : p.limit;
  // Held pages below the limit.
  int32_t low = bits_before(p, limit >> 5, sums);
  if (limit & 31) low += __builtin_popcount(p.bits[limit >> 5] & ((1u << (limit & 31)) - 1u));
  const int32_t holes = limit - low, movers = live - low, moves = holes < movers ? holes : movers;
  if (page == 0) p.moves[0] = moves, p.live[0] = live;
  if (page < p.num_pages / 2 && page >= moves) p.src[page] = -1, p.dst[page] = -1;
  if (page >= p.num_pages) return;
  const bool held = (p.bits[page >> 5] >> (page & 31)) & 1u;
  if (page < limit) {
    const int32_t k = page - before;
    if (!held && k < moves) p.dst[k] = page;
  } else {
    const int32_t k = before - low;
    if (held && k < moves) p.src[k] = page;
    p.rank[page] = held && k < moves ? k : -1;
  }
}

__global__ void __launch_bounds__(kBlock) rename_kernel(PoolParams p) {
  const int32_t s = (int32_t)(blockIdx.x / (uint32_t)p.row_pieces);
  const int32_t need = held_entries(p, s), limit = p.limit < 0 ? p.live[0] : p.limit;
  const int32_t* row = p.table + (int64_t)s * p.table_stride;
  int32_t* to = p.out_table + (int64_t)s * p.out_stride;
  const int32_t j0 = (int32_t)(blockIdx.x % (uint32_t)p.row_pieces) * (kBlock * 4) + (int32_t)threadIdx.x;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int64_t j = (int64_t)j0 + k * kBlock;
    if (j >= p.table_width) break;
    int32_t page = row[j];
    if (j < need && page >= limit && page < p.num_pages) {
      const int32_t at = p.rank[page];
      if (at >= 0) page = p.dst[at];
    }
    to[j] = page;
  }
}

// A small pool (kSmallPages) and a small table (kSmallEntries): everything by one
// workgroup, with the counts in LDS, as launches are what such a call takes (a pool
// of some thousand pages: free, compact and copy 50 us in eight of them, 34 in
// three; 3.3 and 5.2 us of the device for the first two).
template <bool COMPACT>
__global__ void __launch_bounds__(kSmallBlock) small_pool_kernel(PoolParams p) {
  constexpr int EACH = kSmallPages / kSmallBlock, W = kSmallBlock / 64;
  __shared__ int32_t refs[kSmallPages];  // then, compact: the move of a page from the limit on, or -1
  __shared__ int32_t to_page[COMPACT ? kSmallPages / 2 : 1];
  __shared__ int32_t sums[W], lows[W];
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  for (int32_t i = tid; i < kSmallPages; i += kSmallBlock) refs[i] = 0;
  __syncthreads();
  for (int32_t s = w; s < p.num_seqs; s += W) {
    const int32_t need = held_entries(p, s);
    const int32_t* row = p.table + (int64_t)s * p.table_stride;
    for (int32_t j = lane; j < need; j += 64) {
      const int32_t page = row[j];
      if ((uint32_t)page < (uint32_t)p.num_pages) atomicAdd(&refs[page], 1);
    }
  }
  __syncthreads();
  // A thread looks after EACH pages.  before: held ones before them.
  const int32_t first = tid * EACH;
  uint32_t held = 0;
#pragma unroll
  for (int e = 0; e < EACH; ++e) held |= (refs[first + e] != 0 ? 1u : 0u) << e;
  int32_t upto = __builtin_popcount(held);
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int32_t x = __shfl_up(upto, off);
    if (lane >= off) upto += x;
  }
  if (lane == 63) sums[w] = upto;
  __syncthreads();
  int32_t before = upto - __builtin_popcount(held), live = 0;
#pragma unroll
  for (int k = 0; k < W; ++k) {
    if (k < w) before += sums[k];
    live += sums[k];
  }
  if constexpr (!COMPACT) {
    if (tid == 0) p.count[0] = p.num_pages - live;
#pragma unroll
    for (int e = 0; e < EACH; ++e) {
      const int32_t page = first + e;
      if (page >= p.num_pages) break;
      p.refs[page] = refs[page];
      if ((held >> e) & 1u) p.free_pages[p.num_pages - live + before++] = -1;
      else p.free_pages[page - before] = page;
    }
  } else {
    const int32_t limit = p.limit < 0 ? live : p.limit;
    const int32_t mine = limit - first;  // of the thread's pages, below the limit
    int32_t low = __builtin_popcount(mine >= EACH ? held : mine <= 0 ? 0u : held & ((1u << mine) - 1u));
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) low += __shfl_xor(low, off);
    if (lane == 0) lows[w] = low;
    __syncthreads();
    low = 0;
#pragma unroll
    for (int k = 0; k < W; ++k) low += lows[k];
    const int32_t holes = limit - low, movers = live - low, moves = holes < movers ? holes : movers;
    if (tid == 0) p.moves[0] = moves, p.live[0] = live;
    for (int32_t k = moves + tid; k < p.num_pages / 2; k += kSmallBlock) p.src[k] = -1, p.dst[k] = -1;
#pragma unroll
    for (int e = 0; e < EACH; ++e) {
      const int32_t page = first + e;
      if (page >= p.num_pages) break;
      const bool is = (held >> e) & 1u;
      if (page < limit) {
        const int32_t k = page - before;
        if (!is && k < moves) p.dst[k] = to_page[k] = page;
      } else {
        const int32_t k = before - low;
        if (is && k < moves) p.src[k] = page;
        refs[page] = is && k < moves ? k : -1;
      }
      before += is ? 1 : 0;
    }
    __syncthreads();
    for (int32_t s = w; s < p.num_seqs; s += W) {
      const int32_t need = held_entries(p, s);
      const int32_t* row = p.table + (int64_t)s * p.table_stride;
      int32_t* to = p.out_table + (int64_t)s * p.out_stride;
      for (int32_t j = lane; j < p.table_width; j += 64) {
        int32_t page = row[j];
        if (j < need && page >= limit && page < p.num_pages) {
          const int32_t k = refs[page];
          if (k >= 0) page = to_page[k];
        }
        to[j] = page;
      }
    }
  }
}

const void* small_kernel_ptr(int what) {
  return what == kSmallFork ? (const void*)&fork_small_kernel : what == kSmallFree ? (const void*)&small_pool_kernel<false>
                                                              : (const void*)&small_pool_kernel<true>;
}
const void* fork_kernel_ptr(bool write) {
  return write ? (const void*)&fork_write_kernel : (const void*)&fork_mark_kernel;
}
template <bool MANY>
const void* copy_bytes(int bytes) {
  return bytes == 16 ? (const void*)&copy_kernel<16, MANY> : bytes == 4 ? (const void*)&copy_kernel<4, MANY>
                                                                       : (const void*)&copy_kernel<1, MANY>;
}
const void* copy_kernel_ptr(int bytes, bool many) { return many ? copy_bytes<true>(bytes) : copy_bytes<false>(bytes); }
const void* pool_kernel_ptr(int step) {
  switch (step) {
    case kPoolClear: return (const void*)&clear_kernel;
    case kPoolHold: return (const void*)&hold_kernel;
    case kPoolFree: return (const void*)&free_kernel;
    case kPoolMoves: return (const void*)&moves_kernel;
    default: return (const void*)&rename_kernel;
  }
}

}  // namespace rrt
