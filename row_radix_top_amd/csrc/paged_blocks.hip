// Bounds of a cache's pages in 8 bits, and the choice of pages by them.

#include <cfloat>

#include "paged_device.hpp"

namespace rrt {

// A scale is the largest magnitude times this rounded number, here and wherever
// the same bounds are formed.
constexpr float kOver127 = 1.0f / 127.0f;

using i32x4 = int __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float as_e4m3(uint32_t w, int i) {
  return i == 0 ? __builtin_amdgcn_cvt_f32_fp8((int)w, 0) : i == 1 ? __builtin_amdgcn_cvt_f32_fp8((int)w, 1)
       : i == 2 ? __builtin_amdgcn_cvt_f32_fp8((int)w, 2) : __builtin_amdgcn_cvt_f32_fp8((int)w, 3);
}

// ---------------------------------------------------------------------------
// Bounds.  A wavefront takes a page and a key-value head: LPR lanes hold a
// token's row, 64 / LPR tokens a step, and the largest and smallest value of
// each dim meet over the lanes at the end.  Bound by reading the keys; one new
// token of each of 64 sequences, 8 heads, pages of 32: 6 us, a chain of dependent
// reads (starts, lengths, table, keys).
//
// Which page: sequence s gets floor(starts[s] / P) + 2 s as its first unit, and so
// at least floor(new / P) + 2 of them, as many as `new` tokens at any offset may
// touch; the search for the unit's sequence probes 64 at a time.  Of a step that is
// longer than num_tokens the tokens past it were never written: a sequence ends for
// its bounds before the first of them.
// ---------------------------------------------------------------------------
template <typename T, bool F8, int D>
__global__ void __launch_bounds__(kBlocksBlock) bounds_kernel(BoundsParams p) {
  constexpr int SZ = F8 ? 1 : 2, E = 16 / SZ, LPR = D / E, TPI = 64 / LPR;
  const paged_bounds_args& a = p.a;
  const int lane = threadIdx.x & 63;
  const int64_t wave = (int64_t)blockIdx.x * (kBlocksBlock / 64) + __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int64_t u = wave / a.num_kv_heads;
  const int32_t head = (int32_t)(wave - u * a.num_kv_heads);
  if (u >= p.units) return;
  auto first_unit = [&](int32_t s) {
    return (int64_t)divide((uint32_t)clamp_to(a.starts[s], a.num_tokens), p.page) + 2 * (int64_t)s;
  };
  int32_t s = 0;
  for (int32_t n = a.num_seqs; n > 1;) {
    const int32_t step = (n + 63) / 64, at = lane * step;
    const uint64_t below = __builtin_amdgcn_ballot_w64(at < n && first_unit(s + at) <= u);
    const int32_t c = below == 0 ? 0 : __builtin_popcountll(below) - 1;
    s += c * step;
    n = n - c * step < step ? n - c * step : step;
  }
  const int64_t most = table_tokens(a.table_width, a.page_size);
  const int32_t len = clamp_to(a.lengths[s], most);
  const int64_t fresh = (int64_t)a.starts[s + 1] - a.starts[s];
  const int32_t room = a.num_tokens - clamp_to(a.starts[s], a.num_tokens);  // for the sequence's new tokens
  if (fresh <= 0 || len == 0 || room == 0) return;
  const int32_t held = fresh < len ? len - (int32_t)fresh : 0;
  const int32_t end = len - held < room ? len : held + room;
  const int64_t j = (int64_t)divide((uint32_t)held, p.page) + (u - first_unit(s));
  if (j < 0 || j * a.page_size >= end) return;
  const int32_t page = a.block_table[(int64_t)s * a.table_stride + j];
  if ((uint32_t)page >= (uint32_t)a.num_pages) return;
  const int32_t left = end - (int32_t)j * a.page_size, count = left < a.page_size ? left : a.page_size;

  float hi[E], lo[E];
#pragma unroll
  for (int e = 0; e < E; ++e) hi[e] = -INFINITY, lo[e] = INFINITY;
  const char* k = (const char*)a.k + ((int64_t)page * a.page_stride + (int64_t)head * a.head_stride) * SZ + (lane % LPR) * 16;
#pragma unroll 4
  for (int32_t t = lane / LPR; t < count; t += TPI) {
    const u32x4 x = *(const u32x4*)(k + (int64_t)t * a.token_stride * SZ);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      float y;
      if constexpr (F8) y = as_e4m3(x[e >> 2], e & 3);
      else y = (e & 1) ? T::hi(x[e >> 1]) : T::lo(x[e >> 1]);
      hi[e] = fmaxf(hi[e], y);  // either of them passes over NaN
      lo[e] = fminf(lo[e], y);
    }
  }
  constexpr float kMost = F8 ? 448.0f : T::kLargest;
  float top = 0.0f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
#pragma unroll
    for (int off = LPR; off < 64; off <<= 1) {
      hi[e] = fmaxf(hi[e], __shfl_xor(hi[e], off));
      lo[e] = fminf(lo[e], __shfl_xor(lo[e], off));
    }
    if (hi[e] < lo[e]) hi[e] = lo[e] = 0.0f;  // NaN alone
    hi[e] = fminf(fmaxf(hi[e], -kMost), kMost);
    lo[e] = fminf(fmaxf(lo[e], -kMost), kMost);
    top = fmaxf(top, fmaxf(fabsf(hi[e]), fabsf(lo[e])));
  }
#pragma unroll
  for (int off = 1; off < LPR; off <<= 1) top = fmaxf(top, __shfl_xor(top, off));
  const float scale = top * kOver127, by = scale == 0.0f ? 1.0f : scale;
  uint32_t up[E / 4], down[E / 4];
#pragma unroll
  for (int i = 0; i < E / 4; ++i) {
    up[i] = down[i] = 0;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int x = (int)fminf(fmaxf(ceilf(hi[i * 4 + c] / by), -127.0f), 127.0f);
      const int y = (int)fminf(fmaxf(floorf(lo[i * 4 + c] / by), -127.0f), 127.0f);
      up[i] |= (uint32_t)(x & 0xff) << (8 * c);
      down[i] |= (uint32_t)(y & 0xff) << (8 * c);
    }
  }
  if (lane >= LPR) return;
  char* to = (char*)a.bounds + (int64_t)page * a.bounds_page_stride + (int64_t)head * a.bounds_head_stride + lane * E;
  if constexpr (E == 8) {
    *(u32x2*)to = u32x2{up[0], up[1]};
    *(u32x2*)(to + D) = u32x2{down[0], down[1]};
  } else {
    *(u32x4*)to = u32x4{up[0], up[1], up[2], up[3]};
    *(u32x4*)(to + D) = u32x4{down[0], down[1], down[2], down[3]};
  }
  if (lane == 0) a.scales[(int64_t)page * a.scales_stride + head] = scale;
}

// ---------------------------------------------------------------------------
// Choice.  With Q+ = max(Q, 0) and Q- = min(Q, 0),
//   sum_d max(Q_d B_d, Q_d b_d) = [Q+ Q-] . [B b],
// one product of 8-bit numbers of length 2 D: S[head][block] = queries x bounds,
// 16 heads x 16 blocks a matrix instruction, 64 of the 2 D at a time.  The
// order of those 64 is the same for both operands, so each lane loads 16
// consecutive bytes of a page's bounds as they lie.  Sums are whole numbers
// below 2^21, exact in fp32.
//
// The 16 are the heads of 16 / hp2 rows of a sequence, hp2 the power of two from
// heads a key-value head up (more than 16 heads: one row, several sixteens; places
// without a head repeat the first).  A lane holds four of them for one block, so
// the largest head is a maximum in the lane and over at most four lanes, and a
// block's scale, page and place are the lane's own.  Infinities mark the blocks that
// are always taken and those without a page, so a score that passes fp32's range (an
// infinite query or key) is kept as the largest number there is.  (Blocks along the other side:
// a block's four numbers each need shuffles and four maxima across lanes, 148 us
// for 1024 rows of 1250 to 3125 blocks.)
//
// Fused: a workgroup scores all blocks of its rows into LDS, then each wavefront
// picks for its rows.  Split: many workgroups score into the workspace and a
// second launch picks.
//
// The pick: keys in registers (fp32 bits in order) and, between the lowest and the
// highest finite one, the largest threshold that at least K reach, found by halving
// (it ends where exactly K do: ten steps or so of the 32 that bits would take),
// counted by ballots on the scalar unit; ranks by ballots again.
//
// 64 rows of up to 1024 blocks, 64 heads on 8, bf16: 26 us for 71 MB of bounds (11
// at a large read's rate): the chain of lengths, table, bounds, then the longest
// rows.  1024 rows of 1400 to 3125 blocks in four sequences, 32 heads on 4, fp16: 96 us,
// of which the pick is 23; eight rows' scores fill most of a CU's LDS, so its eight
// wavefronts score, then pick, with nothing beside them (four rows to a workgroup and
// two workgroups a CU: 106).
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t b = __float_as_uint(x);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
constexpr uint32_t kInfKey = 0xff800000u;  // infinity's

// n scores (n > k) to the k best's indices, ascending.  TEAM wavefronts (the
// workgroup's, or one alone) hold 64 KEYS scores each.
template <int TEAM, int KEYS>
__device__ __forceinline__ void pick(const float* scores, int32_t n, int32_t k, int32_t* out, int w, int lane, int32_t* s) {
  uint32_t key[KEYS];
  const int32_t base = w * KEYS * 64 + lane;
  uint32_t low = kInfKey, high = 1;  // of this lane's finite scores
#pragma unroll
  for (int i = 0; i < KEYS; ++i) {
    const bool in = base + i * 64 < n;
    const uint32_t x = in ? order_of(scores[base + i * 64]) : 1u;
    const uint32_t y = x < 1u ? 1u : x > kInfKey ? kInfKey : x;  // NaN among the ends
    key[i] = in ? y : 0u;
    low = in && y < low ? y : low;
    high = y < kInfKey && y > high ? y : high;
  }
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const uint32_t x = (uint32_t)__shfl_xor((int)low, off), y = (uint32_t)__shfl_xor((int)high, off);
    low = x < low ? x : low;
    high = y > high ? y : high;
  }
  if constexpr (TEAM > 1) {
    if (lane == 0) s[w] = (int32_t)low, s[TEAM + w] = (int32_t)high;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < TEAM; ++i) {
      const uint32_t x = (uint32_t)s[i], y = (uint32_t)s[TEAM + i];
      low = x < low ? x : low;
      high = y > high ? y : high;
    }
    __syncthreads();
  }
  auto reach = [&](uint32_t t) -> int32_t {  // how many of the team's do
    int32_t c = 0;
#pragma unroll
    for (int i = 0; i < KEYS; ++i) {
      c += __builtin_popcountll(__builtin_amdgcn_ballot_w64(key[i] >= t));
      if (i % 8 == 7) __builtin_amdgcn_sched_barrier(0);  // few ballots at a time: scalar registers
    }
    if constexpr (TEAM == 1) return c;
    if (lane == 0) s[w] = c;
    __syncthreads();
    c = 0;
#pragma unroll
    for (int i = 0; i < TEAM; ++i) c += s[i];
    __syncthreads();
    return c;
  };
  // k reach t, and fewer reach `end`.
  uint32_t t = (uint32_t)__builtin_amdgcn_readfirstlane((int)low), end = (uint32_t)__builtin_amdgcn_readfirstlane((int)high) + 1u;
  int32_t c = reach(kInfKey);
  if (c >= k) t = kInfKey, end = kInfKey + 1u;
  while (end - t > 1u && c != k) {
    const uint32_t want = t + (end - t) / 2;
    c = reach(want);
    if (c >= k) t = want;
    else end = want;
  }
  if (TEAM == 1 && c == k) {  // no ties to part
    int32_t rank = 0;
#pragma unroll
    for (int i = 0; i < KEYS; ++i) {
      const bool in = key[i] >= t;
      const uint64_t all = __builtin_amdgcn_ballot_w64(in);
      if (in) out[rank + __builtin_amdgcn_mbcnt_hi((uint32_t)(all >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)all, 0))] = base + i * 64;
      rank += __builtin_popcountll(all);
    }
    return;
  }
  int32_t above = 0, level = 0;
#pragma unroll
  for (int i = 0; i < KEYS; ++i) {
    above += __builtin_popcountll(__builtin_amdgcn_ballot_w64(key[i] > t));
    level += __builtin_popcountll(__builtin_amdgcn_ballot_w64(key[i] == t));
  }
  asm volatile("" : "+v"(t));  // ballots are taken again below: all of them would fill the scalar registers
  int32_t ties = k, rank = 0;  // entries at the threshold still wanted; the next entry's place
  if constexpr (TEAM == 1) {
    ties -= above;
  } else {
    if (lane == 0) s[w] = above, s[TEAM + w] = level;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < TEAM; ++i) ties -= s[i];
    for (int i = 0; i < w; ++i) {
      const int32_t took = s[TEAM + i] < ties ? s[TEAM + i] : ties;
      rank += s[i] + took;
      ties -= took;
    }
  }
#pragma unroll
  for (int i = 0; i < KEYS; ++i) {
    const uint64_t equal = __builtin_amdgcn_ballot_w64(key[i] == t);
    const int32_t before = __builtin_amdgcn_mbcnt_hi((uint32_t)(equal >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)equal, 0));
    const bool in = key[i] > t || (key[i] == t && before < ties);
    const uint64_t all = __builtin_amdgcn_ballot_w64(in);
    if (in) out[rank + __builtin_amdgcn_mbcnt_hi((uint32_t)(all >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)all, 0))] = base + i * 64;
    rank += __builtin_popcountll(all);
    const int32_t n_equal = __builtin_popcountll(equal);
    ties -= n_equal < ties ? n_equal : ties;
  }
}

__device__ __forceinline__ int32_t blocks_of(const SelectParams& p, int32_t row) {
  const int32_t n = clamp_to(p.a.lengths[row], table_tokens(p.a.table_width, p.a.page_size));
  return n == 0 ? 0 : (int32_t)divide((uint32_t)n - 1u, p.page) + 1;
}

// One row's choice from its scores, by one wavefront.  Its registers hold what its
// row has and not the most there may be, as every step goes over all of them; us of a
// choice from n blocks, 256 rows x 8 heads of 64 dims, with these forms, and where rows
// took the next larger one or the largest:
//   n                    200   1024   2048   3000
//   these              25.9   57.5    101    141
//   the next larger    29.3   66.5    109    193
//   the largest        71.5    119    176    209
__device__ __forceinline__ void pick_row(const SelectParams& p, const float* scores, int32_t n, int32_t* out, int lane) {
  const int32_t k = p.a.num_blocks;
  if (n <= k) {
    for (int32_t i = lane; i < k; i += 64) out[i] = i < n ? i : -1;
  } else if (n <= 4 * 64) {
    pick<1, 4>(scores, n, k, out, 0, lane, nullptr);
  } else if (n <= 16 * 64) {
    pick<1, 16>(scores, n, k, out, 0, lane, nullptr);
  } else if (n <= 32 * 64) {
    pick<1, 32>(scores, n, k, out, 0, lane, nullptr);
  } else if (n <= 48 * 64) {
    pick<1, 48>(scores, n, k, out, 0, lane, nullptr);
  } else {
    pick<1, 64>(scores, n, k, out, 0, lane, nullptr);
  }
}

template <typename T, int D, int NT, bool SPLIT>
__global__ void __launch_bounds__(kSelectBlock, 2) select_kernel(SelectParams p) {
  constexpr int QS = D / 64, KS = 2 * QS;  // steps over the dims, and over both bounds
  extern __shared__ __align__(16) float scores[];
  __shared__ u32x4 sq[NT][KS][64];  // a lane's queries
  __shared__ __align__(16) float sby[NT][16];
  const paged_select_args& a = p.a;
  const int lane = threadIdx.x & 63, c16 = lane & 15, g = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  uint32_t unit = blockIdx.x;
  const int32_t kvh = (int32_t)(unit % (uint32_t)a.num_kv_heads);
  unit /= (uint32_t)a.num_kv_heads;
  int32_t part = 0;
  if constexpr (SPLIT) {
    part = (int32_t)(unit % (uint32_t)p.parts);
    unit /= (uint32_t)p.parts;
  }
  const int32_t seq = (int32_t)(unit / (uint32_t)p.seq_units);
  const int32_t j0 = (int32_t)(unit - (uint32_t)seq * (uint32_t)p.seq_units) * p.unit_rows;
  const int32_t rows = a.next_n - j0 < p.unit_rows ? a.next_n - j0 : p.unit_rows;
  const int32_t r0 = seq * a.next_n + j0;
  const int32_t per = a.num_heads / a.num_kv_heads;
  const int32_t passes = per <= 16 ? 1 : (per + 16 * NT - 1) / (16 * NT);
  const int32_t hp2 = p.hp2, hp2_log = __builtin_ctz((uint32_t)hp2);

  // Of the first turns' blocks, looked up before the lengths are there to say which
  // count: nothing reads the scores of others.
  const int32_t* table = a.block_table + (int64_t)seq * a.table_stride;
  const int32_t W = (int32_t)blockDim.x >> 6, first_tile = SPLIT ? part * p.part_tiles : 0;
  auto pages_at = [&](int32_t four) -> int32_t {
    const int32_t b = (first_tile + four * 4) * 16 + lane;
    return b < a.table_width ? table[b] : -1;
  };
  const int32_t page0 = pages_at(w), page1 = pages_at(w + W);
  const int32_t mine = lane < rows ? blocks_of(p, r0 + lane) : 0;  // blocks of the lane's row
  int32_t have = mine, least = lane < rows ? mine : INT32_MAX;     // and of the longest and the shortest
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int32_t x = __shfl_xor(have, off), y = __shfl_xor(least, off);
    have = x > have ? x : have;
    least = y < least ? y : least;
  }
  have = __builtin_amdgcn_readfirstlane(have);
  least = __builtin_amdgcn_readfirstlane(least);
  int32_t t0 = 0, t1 = (have + 15) / 16;
  if constexpr (SPLIT) {
    t0 = first_tile;
    t1 = t1 - t0 < p.part_tiles ? t1 : t0 + p.part_tiles;
    if (t0 >= t1) return;
  }
  const char* bounds = (const char*)a.bounds + (int64_t)kvh * a.bounds_head_stride;
  auto score_at = [&](int32_t j) -> float* {
    if constexpr (SPLIT) return p.scores + ((int64_t)(r0 + j) * a.num_kv_heads + kvh) * p.pitch;
    else return scores + (int64_t)j * p.pitch;
  };

  for (int32_t pass = 0; pass < passes; ++pass) {
    // A wavefront takes four tiles at a time.  Their bounds are read four tiles
    // ahead, and where they lie is looked up, a block a lane, four more before that.
    const int32_t fours = (t1 - t0 + 3) / 4;
    u32x4 ring[4][KS];
    float scales[4];
    int32_t pages[4];
    auto fetch = [&](int d, int32_t page) __attribute__((always_inline)) {
      pages[d] = __shfl(page, d * 16 + c16);
      const int64_t at = (uint32_t)pages[d] < (uint32_t)a.num_pages ? pages[d] : 0;
      const char* from = bounds + at * a.bounds_page_stride + g * 16;
#pragma unroll
      for (int i = 0; i < KS; ++i) ring[d][i] = *(const u32x4*)(from + i * 64);
      scales[d] = a.scales[at * a.scales_stride + kvh];
    };
    int32_t page = page0, page_next = page1;
    if (w < fours) {
#pragma unroll
      for (int d = 0; d < 4; ++d) fetch(d, page);
    }

    // The queries, a sixteen a wavefront.
    if (w < NT) {
      const int32_t j = per <= 16 ? (w * 16 + c16) >> hp2_log : 0;
      const int32_t head = per <= 16 ? (c16 & (hp2 - 1)) : (pass * NT + w) * 16 + c16;
      const char* from = (const char*)a.q + 2 * ((int64_t)(r0 + (j < rows ? j : 0)) * a.q_row_stride +
                                                 (int64_t)(kvh * per + (head < per ? head : 0)) * a.q_head_stride);
      float x[QS][16], top = 0.0f;
#pragma unroll
      for (int i = 0; i < QS; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const u32x4 y = *(const u32x4*)(from + i * 128 + g * 32 + h * 16);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float v = (e & 1) ? T::hi(y[e >> 1]) : T::lo(y[e >> 1]);
            v = v != v ? 0.0f : fminf(fmaxf(v, -T::kLargest), T::kLargest);
            x[i][h * 8 + e] = v;
            top = fmaxf(top, fabsf(v));
          }
        }
      top = max_xor32(max_xor16(top));
      top *= kOver127;
      if (g == 0) sby[w][c16] = top;
      const float div = top == 0.0f ? 1.0f : top;
#pragma unroll
      for (int i = 0; i < QS; ++i) {
        u32x4 ups, downs;
#pragma unroll
        for (int e4 = 0; e4 < 4; ++e4) {
          uint32_t up = 0, down = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            int v = (int)fminf(fmaxf(rintf(x[i][e4 * 4 + e] / div), -127.0f), 127.0f);
            up |= (uint32_t)(v > 0 ? v : 0) << (8 * e);
            down |= (uint32_t)((v < 0 ? v : 0) & 0xff) << (8 * e);
          }
          ups[e4] = up;
          downs[e4] = down;
        }
        sq[w][i][lane] = ups;
        sq[w][QS + i][lane] = downs;
      }
    }
    __syncthreads();
    u32x4 q[NT][KS];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < KS; ++i) q[t][i] = sq[t][i][lane];
    for (int32_t four = w; four < fours; four += W) {
      page = page_next;
      page_next = pages_at(four + 2 * W);
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const int32_t tile = t0 + four * 4 + d, at = tile * 16 + c16;
        i32x4 sum[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          sum[t] = i32x4{0, 0, 0, 0};
#pragma unroll
          for (int i = 0; i < KS; ++i)
            sum[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, q[t][i]), __builtin_bit_cast(i32x4, ring[d][i]),
                                                           sum[t], 0, 0, 0);
        }
        const float scale = scales[d];
        const bool valid = (uint32_t)pages[d] < (uint32_t)a.num_pages;
        if (four + W < fours) fetch(d, page);
        if (tile >= t1) continue;
        const bool ends = tile * 16 < a.first || tile * 16 + 16 > least - a.last;  // blocks that some row always takes
        float best[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const f32x4 by = *(const f32x4*)&sby[t][g * 4];
          float y[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            y[i] = (float)sum[t][i] * by[i];
            if (per > 16) y[i] = best[i] = fmaxf(best[i], y[i]);
          }
          if (per > 16 && t + 1 < NT) continue;
          if (hp2 >= 2) y[0] = fmaxf(y[0], y[1]), y[1] = fmaxf(y[2], y[3]);
          if (hp2 >= 4) y[0] = fmaxf(y[0], y[1]);
          if (hp2 >= 8) y[0] = max_xor16(y[0]);
          if (hp2 >= 16) y[0] = max_xor32(y[0]);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            if (r > 0 && r * hp2 >= 4) break;
            const int32_t j = per > 16 ? 0 : ((t * 16 + g * 4) >> hp2_log) + r;
            float z = __builtin_amdgcn_fmed3f(y[r] * scale, -FLT_MAX, FLT_MAX);  // NaN: the smallest
            if (ends) {
              const int32_t n = __shfl(mine, j & 63);
              z = at < a.first || at >= n - a.last ? INFINITY : z;
            }
            z = valid ? z : -INFINITY;
            if (j >= rows || ((g * 4) & (hp2 - 1)) != 0) continue;
            float* to = score_at(j) + at;
            if (pass > 0) z = fmaxf(z, *to);
            *to = z;
          }
        }
      }
    }
    __syncthreads();  // the queries and their scales are read, the scores there
  }
  if constexpr (SPLIT) return;
  for (int32_t j = w; j < rows; j += (int32_t)blockDim.x >> 6)
    pick_row(p, score_at(j), blocks_of(p, r0 + j), a.blocks + ((int64_t)(r0 + j) * a.num_kv_heads + kvh) * a.num_blocks, lane);
}

// The choice of one row and key-value head from scores in the workspace.  Up to 4096
// blocks in four registers a lane: one row of 4096 x 8 heads 18 us, 34 with 32.
__global__ void __launch_bounds__(kPickBlock) pick_kernel(SelectParams p) {
  constexpr int TEAM = kPickBlock / 64;
  __shared__ int32_t s[2 * TEAM];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int32_t row = (int32_t)(blockIdx.x / (uint32_t)p.a.num_kv_heads), k = p.a.num_blocks;
  const int32_t n = blocks_of(p, row);
  const float* scores = p.scores + (int64_t)blockIdx.x * p.pitch;
  int32_t* out = p.a.blocks + (int64_t)blockIdx.x * k;
  if (n <= k) {
    for (int32_t i = threadIdx.x; i < k; i += kPickBlock) out[i] = i < n ? i : -1;
  } else if (n <= TEAM * 64 * 4) {
    pick<TEAM, 4>(scores, n, k, out, w, lane, s);
  } else {
    pick<TEAM, 32>(scores, n, k, out, w, lane, s);
  }
}

namespace {
template <typename T, bool F8>
const void* bounds_dims(int dim) {
  return dim == 64 ? (const void*)&bounds_kernel<T, F8, 64> : dim == 128 ? (const void*)&bounds_kernel<T, F8, 128> : nullptr;
}
template <typename T, int D, bool SPLIT>
const void* select_tiles(int tiles) {
  return tiles == 4 ? (const void*)&select_kernel<T, D, 4, SPLIT> : tiles == 2 ? (const void*)&select_kernel<T, D, 2, SPLIT>
                                                                  : (const void*)&select_kernel<T, D, 1, SPLIT>;
}
template <typename T>
const void* select_dims(int dim, int tiles, bool split) {
  if (dim == 64) return split ? select_tiles<T, 64, true>(tiles) : select_tiles<T, 64, false>(tiles);
  if (dim == 128) return split ? select_tiles<T, 128, true>(tiles) : select_tiles<T, 128, false>(tiles);
  return nullptr;
}
}  // namespace

const void* bounds_kernel_ptr(int store, int head_dim) {
  return store == PAGED_E4M3 ? bounds_dims<Bf16, true>(head_dim)
       : store == PAGED_BF16 ? bounds_dims<Bf16, false>(head_dim) : bounds_dims<Fp16, false>(head_dim);
}
const void* select_kernel_ptr(int dtype, int head_dim, int tiles, bool split) {
  return dtype == PAGED_BF16 ? select_dims<Bf16>(head_dim, tiles, split) : select_dims<Fp16>(head_dim, tiles, split);
}
const void* pick_kernel_ptr() { return (const void*)&pick_kernel; }

}  // namespace rrt
