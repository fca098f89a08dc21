// Attention over positions that many rows share: their keys and values are read
// once for all of them.

#include <type_traits>

#include "lds_device.hpp"

namespace rrt {

// ---------------------------------------------------------------------------
// The columns are the heads (that share a key-value head) of all rows of a
// group, so that this is a product with as many columns as a prompt has rows and
// no mask: a row either sees the whole shared part or takes no part here.
//
// A workgroup takes 32 CW columns of a group, a key-value head and a part of the
// shared positions; CW of its four wavefronts lie along the columns, the others
// along the tokens of a tile, and join at the end.  S^T = K Q^T and O^T = V^T P
// in matrix instructions of 32 x 32, a column and its maximum, sum, weights and
// output in one lane (and the lane 32 further).
//
// A tile's keys and values go straight to LDS as they lie, row by row; 16-byte
// chunk c of token t's row is kept at c ^ turn(t), so that neither the key
// operand (16 tokens, one chunk) nor the transposed reads of the values (4 tokens
// x 4 chunks) meet a bank twice.  Keys have three buffers (two where tiles are
// of 128 tokens or pages of other than 16), values two.  (e4m3: raw bytes wait in
// LDS and are widened from there into the tiles, by writes that do meet: 8 % of the
// cycles that a CU is at work.)
//
// The weights are relative to a reference that follows the running maximum
// lazily: only a score that passes it by 2^8 moves it (they then stay below 2^8,
// or 2^15 as fp16 keeps them).  They are rounded to the 16-bit type for the
// second product (half a step relative to each); references, sums, outputs and
// parts stay fp32.
//
// Bound by the two products where 32 rows and more share: 64 rows of 64 heads on 8
// behind 32768 tokens, bf16: 90 to 101 us with the clock (82 at best) for 69 GFLOP (43 at the rate of a large product),
// of which 65 are the loop, matrix units busy two thirds of it; the rest is the
// start (3 us for the shares, 8 until the first tiles are there: every workgroup
// asks at once) and 34 MB of parts (6).  Two wavefronts a SIMD: eight to a
// workgroup, alone on its CU with four buffers of each, took as long (98).
// Twelve groups of 1 to 32 rows, 40 heads on 8, e4m3: 70 to 79 us (66 at best).  Eight rows
// behind 2000 tokens: 13 us, the chain of dependent reads.
// ---------------------------------------------------------------------------
constexpr float kLazyStep = 8.0f;
// Past this a reference's own rounding shows in the difference of a score to it.
constexpr float kFar = 1048576.0f;
constexpr int kAhead = 3;  // operands in flight from LDS, and one in use
constexpr int32_t kSharedLeast = 256;  // positions of a part

__device__ __forceinline__ int32_t prefix_scan(int32_t x, int lane) {
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int32_t y = __shfl_up(x, off);
    if (lane >= off) x = __builtin_elementwise_add_sat(x, y);
  }
  return x;
}

template <int D>
__device__ __forceinline__ uint32_t turn(uint32_t t) {
  return D == 128 ? ((t & 3) << 2) | ((t >> 2) & 3) : (((t >> 1) & 1) << 2) | ((t >> 2) & 3);
}

// ---------------------------------------------------------------------------
// Who does what.  A group has ceil(columns / wide) tiles of columns and `n` shared
// positions; a part of those is a `workgroups`-th of all that there is to read,
// positions times tiles times heads, so that groups of any sizes make workgroups
// alike, and few more of them than that.  Every workgroup finds its own by sums
// over the groups, 64 at a time.
// ---------------------------------------------------------------------------
struct GroupWork {
  int32_t first, count;  // sequences
  int32_t tiles, n;      // of columns; shared positions
};
__device__ __forceinline__ GroupWork work_of_group(const AttnParams& p, int32_t g, int32_t per_seq, int32_t wide, int64_t most) {
  GroupWork w = {0, 0, 0, 0};
  if (g >= p.num_groups) return w;
  group_of(p, g, &w.first, &w.count);
  w.tiles = (int32_t)(((int64_t)w.count * per_seq + wide - 1) / wide);
  w.n = clamp_to(p.shared[g], most);
  return w;
}
__device__ __forceinline__ int32_t shared_part(const AttnParams& p, int32_t per_seq, int32_t wide, int64_t most, int lane) {
  int64_t all = 0;
  GroupWork mine;
  for (int32_t g0 = 0; g0 < p.num_groups; g0 += 64) {
    mine = work_of_group(p, g0 + lane, per_seq, wide, most);
    all += (int64_t)mine.tiles * mine.n;
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) all += shfl64(all, lane ^ off);
  const int32_t part = part_size(readlane64(all, 0) * p.a.num_kv_heads, p.shared_workgroups, kSharedLeast, p.shared_unit);
  if (p.num_groups > 64 || p.num_groups == 1) return part;
  // Each group's last part is a short one, so that there are some more of them than
  // workgroups that run at once, and the last few would start when the others end
  // (twelve groups: 16 of 528, 95 us for 64).  Lane l tries l units more: the first that
  // makes no more than run at once.
  const float by = 1.0f / (float)(part + lane * p.shared_unit);
  float all_of = 0.0f;
  for (int32_t g = 0; g < p.num_groups; ++g) {
    const float parts = __builtin_ceilf((float)__builtin_amdgcn_readlane(mine.n, g) * by);
    all_of += fminf(parts, (float)p.shared_most) * (float)__builtin_amdgcn_readlane(mine.tiles, g);
  }
  const uint64_t fit = __builtin_amdgcn_ballot_w64(all_of * (float)p.a.num_kv_heads <= (float)p.shared_workgroups);
  return fit == 0 ? part : part + __builtin_ctzll(fit) * p.shared_unit;
}

// One workgroup, beside the others: what each sequence shares, and the list of
// own parts for the launch behind this one (a sequence whose rows end with the
// shared positions has none).
__device__ __forceinline__ void plan_own(const AttnParams& p, int32_t per_seq, int32_t wide, int tid, int lane, char* lds) {
  const paged_attention_args& a = p.a;
  const int32_t seqs = a.num_rows / a.next_n, w = tid >> 6;
  const int64_t most = table_tokens(a.table_width, a.page_size);
  int64_t* sums = (int64_t*)lds;  // a wavefront each
  int32_t* counts = (int32_t*)(lds + 64);
  auto own_of = [&](int32_t s) {
    int32_t n = 0;
    for (int32_t j = 0; j < a.next_n; ++j) {
      const int32_t x = clamp_to(a.lengths[(int64_t)s * a.next_n + j], most);
      n = x > n ? x : n;
    }
    return n;
  };
  int64_t all = 0;
  for (int32_t s = tid; s < seqs; s += 256) {
    // The last group that starts at or before it.
    int32_t at = -1, end = p.num_groups;
    while (end - at > 1) {
      const int32_t mid = at + (end - at) / 2;
      if (p.group_starts[mid] <= s) at = mid;
      else end = mid;
    }
    int32_t shared = 0;
    if (at >= 0) {
      int32_t first, count;
      group_of(p, at, &first, &count);
      const int32_t n = clamp_to(p.shared[at], most);
      if (s >= first && s - first < count && takes_part(a, s, n, most)) shared = n;
    }
    p.share[s] = shared;
    all += own_of(s) - shared;
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) all += shfl64(all, lane ^ off);
  if (lane == 0) sums[w] = all;
  __syncthreads();
  all = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) all += sums[k];
  const int32_t part = part_size(all * (a.num_kv_heads * p.col_tiles), p.workgroups, p.least, p.unit);
  int32_t base = 0;
  for (int32_t s0 = 0; s0 < seqs; s0 += 256) {
    const int32_t s = s0 + tid;
    const int32_t parts = s < seqs ? split_by(own_of(s) - p.share[s], part, p.most, p.unit).parts : 0;
    const int32_t upto = prefix_scan(parts, lane);
    if (lane == 63) counts[w] = upto;
    __syncthreads();
    int32_t at = base + upto - parts;
    for (int k = 0; k < 4; ++k) {
      if (k < w) at += counts[k];
      base += counts[k];
    }
    for (int32_t k = 0; k < parts; ++k) p.items[at + k] = PrefixItem{s, k};
    __syncthreads();
  }
  const int32_t shared = shared_part(p, per_seq, wide, most, lane);
  if (tid == 0) *p.planned = PrefixPlanned{base, part, shared, 0};
}

template <typename T, bool F8, int D, int CW, bool P16>
__global__ void __launch_bounds__(256, 2) prefix_kernel(AttnParams p) {
  constexpr int NW = 4;                 // wavefronts
  constexpr int TB = CW == 4 ? 2 : 1;   // blocks of 32 tokens of a wavefront in a tile
  constexpr int TW = NW / CW;           // wavefronts along the tokens
  constexpr int TT = 32 * TB * TW;      // tokens of a tile
  constexpr int QT = TT / NW;           // and of a wavefront's loads
  constexpr int NP = TT / 64;                  // words of a tile's mask; tokens that a lane looks up
  constexpr int KS = D / 16, DB = D / 32;      // steps over the key dims; blocks of value dims
  constexpr uint32_t ROW = D * 2, TILE = TT * ROW;
  constexpr int SZ = F8 ? 1 : 2;
  constexpr int LPR = D * SZ / 16, RPL = 64 / LPR;  // lanes of a row's load; rows of a load
  constexpr int NL = QT / RPL < 1 ? 1 : QT / RPL;   // loads of a wavefront's share of a tile
  constexpr int NG = QT < 16 ? NL : 16 / RPL;       // and of 16 tokens of it
  static_assert(QT % RPL == 0, "whole loads");
  // Tiles of keys and of values in LDS, and of raw e4m3 bytes: what 80 KB hold, so
  // that two workgroups fit a CU, or (eight wavefronts, which have it to themselves)
  // as far ahead as memory takes.
  constexpr int KB = F8 || CW == 1 || !P16 ? 2 : 3, VB = 2;
  constexpr int RB = F8 ? 1 : 0;
  __shared__ __align__(1024) char sk[KB][TILE];
  __shared__ __align__(1024) char sv[VB][TILE];
  __shared__ __align__(1024) char sraw[F8 ? RB : 1][2][F8 ? TT * D : 16];
  const paged_attention_args& a = p.a;
  const int tid = threadIdx.x, lane = tid & 63, col = lane & 31, half = lane >> 5;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6), cw = w % CW, tw = w / CW;

  const int32_t per = a.num_heads / a.num_kv_heads, per_seq = per * a.next_n;
  if (blockIdx.x == 0) {
    plan_own(p, per_seq, 32 * CW, tid, lane, &sk[0][0]);
    return;
  }
  // The parts of a group, times the heads, go round the XCDs, and tiles of columns
  // that read the same positions follow one another on one of them.
  const int64_t most = table_tokens(a.table_width, a.page_size);
  const uint32_t block = blockIdx.x - 1, xcd = block & 7;
  const int32_t want = (int32_t)(block >> 3), part_of = shared_part(p, per_seq, 32 * CW, most, lane);
  GroupWork mine;
  Split sp;
  int32_t base = 0, before = 0;  // tiles before the group's on this XCD
  bool found = false;
  for (int32_t g0 = 0; g0 < p.num_groups && !found; g0 += 64) {
    mine = work_of_group(p, g0 + lane, per_seq, 32 * CW, most);
    sp = split_by(mine.n, part_of, p.shared_most, TT);
    const int32_t tiles = (int32_t)(((int64_t)sp.parts * a.num_kv_heads + 7) / 8) * mine.tiles;
    const int32_t upto = __builtin_elementwise_add_sat(base, prefix_scan(tiles, lane));
    const uint64_t past = __builtin_amdgcn_ballot_w64(upto > want);
    found = past != 0;
    if (found) {
      const int l = __builtin_ctzll(past);
      before = l == 0 ? base : __builtin_amdgcn_readlane(upto, l - 1);
      mine.first = __builtin_amdgcn_readlane(mine.first, l);
      mine.count = __builtin_amdgcn_readlane(mine.count, l);
      mine.tiles = __builtin_amdgcn_readlane(mine.tiles, l);
      mine.n = __builtin_amdgcn_readlane(mine.n, l);
    }
    base = __builtin_amdgcn_readlane(upto, 63);
  }
  if (!found) return;
  mine = {__builtin_amdgcn_readfirstlane(mine.first), __builtin_amdgcn_readfirstlane(mine.count),
          __builtin_amdgcn_readfirstlane(mine.tiles), __builtin_amdgcn_readfirstlane(mine.n)};
  before = __builtin_amdgcn_readfirstlane(before);
  const int32_t n = mine.n;
  sp = split_by(n, part_of, p.shared_most, TT);
  const int32_t turn_of = (want - before) / mine.tiles, col_tile = want - before - turn_of * mine.tiles;
  const uint32_t outer = (uint32_t)turn_of * 8 + ((xcd + (uint32_t)turn_of) & 7);
  const int32_t part = (int32_t)(outer / (uint32_t)a.num_kv_heads), kvh = (int32_t)(outer - (uint32_t)part * (uint32_t)a.num_kv_heads);
  if (part >= sp.parts) return;
  const int32_t begin = part * sp.chunk, end = n - begin < sp.chunk ? n : begin + sp.chunk;
  const int32_t tiles = (end - begin + TT - 1) / TT;

  // The table row of the first sequence that takes part.
  int32_t reader = -1;
  for (int32_t s0 = 0; s0 < mine.count && reader < 0; s0 += 64) {
    const uint64_t in = __builtin_amdgcn_ballot_w64(s0 + lane < mine.count && takes_part(a, mine.first + s0 + lane, n, most));
    if (in != 0) reader = mine.first + s0 + (int32_t)__builtin_ctzll(in);
  }
  if (reader < 0) return;
  const int32_t* table = a.block_table + (int64_t)reader * a.table_stride;

  // The lane's column.
  const int32_t c = (col_tile * CW + cw) * 32 + col;
  const int32_t j = c / per, seq = mine.first + j / a.next_n;
  const bool real = c < mine.count * per_seq && takes_part(a, seq, n, most);
  const int64_t row = (int64_t)mine.first * a.next_n + (c < mine.count * per_seq ? j : 0);
  const int32_t head = kvh * per + (c < mine.count * per_seq ? c - j * per : 0);
  // The scale's sign goes into the queries, so that the largest product has the
  // largest score (and products are 0 where the scale is).
  const float total = p.scale_log2 * (F8 && a.k_scales != nullptr ? a.k_scales[kvh] : 1.0f);
  const float sign = total < 0.0f ? -1.0f : total == 0.0f ? 0.0f : 1.0f;
  const float scale = total == 0.0f ? 1.0f : fabsf(total);
  u32x4 q[KS];
  {
    const char* qp = (const char*)a.q + 2 * (row * a.q_row_stride + (int64_t)head * a.q_head_stride);
#pragma unroll
    for (int s = 0; s < KS; ++s) q[s] = *(const u32x4*)(qp + s * 32 + half * 16);
    if (sign != 1.0f) {
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int e = 0; e < 4; ++e) q[s][e] = T::pack(T::lo(q[s][e]) * sign, T::hi(q[s][e]) * sign);
    }
  }

  // --- places -----------------------------------------------------------------
  // Where the rows of a wavefront's loads lie, and which tokens of a tile count.
  // Pages of a multiple of 16 tokens (P16): sixteen tokens have one page, and a
  // lane's place inside them is fixed.  Lane l looks up the l-th sixteen of BT
  // tiles at once, a batch ahead, and a tile takes its own by a lane's number: no
  // wait for vector memory among the tiles' loads but one in BT tiles, and few
  // scalar instructions (looked up tile by tile through the scalar cache, they
  // were as many as the vector ones and half of a wavefront's time).  Others: lane
  // l looks up tokens l (and 64 + l) of a tile, and a load's lanes get them there.
  const char* kbase = (const char*)a.k + (int64_t)kvh * a.head_stride * SZ;
  const char* vbase = (const char*)a.v + (int64_t)kvh * a.head_stride * SZ;
  const uint32_t sub = (uint32_t)lane / LPR, pos = (uint32_t)lane % LPR;
  const uint32_t row0 = (uint32_t)w * QT;
  constexpr int GT = TT / 16, BT = 64 / GT;
  struct Place {
    int64_t at[P16 ? (QT + 15) / 16 : NL];  // bytes: of sixteen tokens, or of the lane's row in each load
    uint64_t mask[NP];
    __device__ __forceinline__ bool whole() const {
      return mask[0] == ~0ull && mask[NP - 1] == ~0ull;
    }
  };
  int32_t page[P16 ? 1 : NP];  // of what is placed next
  uint32_t in[NP];             // and the tokens' offsets in them
  int64_t group_at = 0;        // P16: the lane's sixteen
  int32_t group_count = 0;
  uint64_t group_whole = 0;
  auto look_up = [&](int32_t i) {
    if constexpr (P16) {
      const int32_t x = begin + i * TT + lane * 16;
      page[0] = x < end ? table[divide((uint32_t)x, p.page)] : -1;
    } else {
#pragma unroll
      for (int k = 0; k < NP; ++k) {
        const int32_t x = begin + i * TT + k * 64 + lane;
        const uint32_t y = x < end ? (uint32_t)x : 0u, at = divide(y, p.page);
        in[k] = x < end ? y - at * p.page.by : ~0u;
        page[k] = table[at];
      }
    }
  };
  // Tile i's places; starts the look-up of the next one's, or batch's.
  auto place = [&](int32_t i) __attribute__((always_inline)) -> Place {
    Place out;
    if constexpr (P16) {
      if (i % BT == 0) {
        const int32_t x = begin + i * TT + lane * 16, left = end - x;
        const bool ok = left > 0 && (uint32_t)page[0] < (uint32_t)a.num_pages;
        const uint32_t y = ok ? (uint32_t)x : 0u, inner = y - divide(y, p.page) * p.page.by;
        group_at = ok ? ((int64_t)page[0] * a.page_stride + (int64_t)inner * a.token_stride) * SZ : 0;
        group_count = !ok ? 0 : left < 16 ? left : 16;
        group_whole = __builtin_amdgcn_ballot_w64(group_count == 16);
        if (i + BT < tiles) look_up(i + BT);
      }
      const int g0 = i % BT * GT;
#pragma unroll
      for (int g = 0; g < (QT + 15) / 16; ++g) out.at[g] = readlane64(group_at, g0 + (int)row0 / 16 + g);
#pragma unroll
      for (int k = 0; k < NP; ++k) out.mask[k] = ~0ull;
      if ((~(group_whole >> g0) & ((1u << GT) - 1u)) != 0) {
#pragma unroll
        for (int k = 0; k < NP; ++k) {
          out.mask[k] = 0;
#pragma nounroll
          for (int g = 0; g < 4; ++g)
            out.mask[k] |= (uint64_t)((1u << __builtin_amdgcn_readlane(group_count, g0 + k * 4 + g)) - 1u) << (g * 16);
        }
      }
    } else {
      int64_t at[NP];
#pragma unroll
      for (int k = 0; k < NP; ++k) {
        const bool ok = in[k] != ~0u && (uint32_t)page[k] < (uint32_t)a.num_pages;
        out.mask[k] = __builtin_amdgcn_ballot_w64(ok);
        at[k] = ok ? ((int64_t)page[k] * a.page_stride + (int64_t)in[k] * a.token_stride) * SZ : 0;
      }
#pragma unroll
      for (int k = 0; k < NL; ++k) {
        const int t = (int)row0 + k * RPL;  // of the tile, before the lane's row
        const int64_t mine = NP == 1 || t < 64 ? at[0] : at[NP - 1];
        out.at[k] = shfl64(mine, (t & 63) + (int)sub);
      }
      if (i + 1 < tiles) look_up(i + 1);
    }
    return out;
  };
  uint32_t inside[NG];  // bytes from the first of sixteen tokens to the lane's chunk
#pragma unroll
  for (int k = 0; k < NG; ++k) {
    const uint32_t t = row0 % 16 + k * RPL + sub, chunk = F8 ? pos : pos ^ turn<D>(t);
    inside[k] = t * (uint32_t)a.token_stride * SZ + chunk * 16;
  }
  // A tile's mask from token t on.
  auto mask_from = [&](const Place& m, uint32_t t) __attribute__((always_inline)) -> uint64_t {
    uint64_t x = m.mask[0];
    if constexpr (NP > 1) {
      const uint64_t y = m.mask[1];
      x = t < 64 ? x : y;
    }
    return x >> (t & 63);
  };

  // --- tiles to LDS -------------------------------------------------------------
  // Straight to LDS: 16-bit rows at their turned places, raw e4m3 bytes as they are.
  auto issue = [&](const char* base, const Place& at, char* to) __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < NL; ++k) {
      const uint32_t where = lds_at(to) + (row0 + k * RPL) * (D * SZ);
      if constexpr (P16) load_to_lds(base + readlane64(at.at[k / NG], 0), inside[k % NG], where);
      else load_to_lds(base + at.at[k] + (F8 ? pos : pos ^ turn<D>(row0 + k * RPL + sub)) * 16, where);
    }
  };
  // e4m3: the wavefront's raw bytes, widened, into a tile.
  auto put = [&](const char* raw, char* to, const Place& m) __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < NL; ++k) {
      const uint32_t t = row0 + k * RPL + sub;
      const u32x4 x = lds_read16(lds_at(raw) + t * D + pos * 16);
      // Tokens that do not count become zeros: their places may hold NaN.
      const bool ok = (mask_from(m, t) & 1u) != 0;
      const u32x4 lo = widen<T>(u32x2{x[0], x[1]}), hi = widen<T>(u32x2{x[2], x[3]});
      const uint32_t at = lds_at(to) + t * ROW + (((pos * 2) ^ turn<D>(t)) << 4);
      *(lds_u32x4*)at = ok ? lo : u32x4{0, 0, 0, 0};
      *(lds_u32x4*)(at ^ 16) = ok ? hi : u32x4{0, 0, 0, 0};
    }
  };
  // Waits until all but the last n tiles' loads (of keys, or of values) have arrived.
  auto wait_tiles = [&](int n) __attribute__((always_inline)) {
    switch (n) {
      case 0: return wait_loads<0>();
      case 1: return wait_loads<NL>();
      case 2: return wait_loads<2 * NL>();
      case 3: return wait_loads<3 * NL>();
      default: return wait_loads<4 * NL>();
    }
  };
  // The wavefront's rows of a values' tile that do not count (16 bits).
  auto clear = [&](char* to, const Place& m) {
    constexpr uint32_t kAll = QT == 32 ? ~0u : (1u << QT) - 1u;
    const uint32_t mine = (uint32_t)mask_from(m, row0) & kAll;
    if (mine == kAll) return;
#pragma nounroll
    for (int t = 0; t < QT; ++t)
      if (((mine >> t) & 1u) == 0 && lane < D / 8) *(lds_u32x4*)(lds_at(to) + (row0 + t) * ROW + lane * 16) = u32x4{0, 0, 0, 0};
  };

  // --- one tile -------------------------------------------------------------------
  // The matrix unit works behind a wavefront's back, so every product is issued
  // among vector instructions that do not need it: the scores of tile i + 1 among
  // the weights of tile i, the values of tile i among the maximum of tile i + 1.
  // (A tile's steps one after the other: 4600 cycles for a wavefront alone of which
  // 1024 on the matrix unit, and two wavefronts on a SIMD did not fill it.)
  // The barriers keep the order as it is written.
  constexpr int E = TB * 16;         // scores of a lane
  constexpr int M = TB * KS;         // products of a tile's scores,
  constexpr int N = 2 * TB * DB;     // and of its values
  float ref = -INFINITY, sum = 0.0f;  // base-2 logarithm; of this lane's tokens
  float by = scale, r = 0.0f, sum_a = 0.0f, sum_b = 0.0f;
  f32x16 o[DB];
#pragma unroll
  for (int d = 0; d < DB; ++d) o[d] = f32x16{};
  u32x4 pw[2 * TB];
  const uint32_t key_at = (uint32_t)(tw * TB * 32 + col) * ROW + (((uint32_t)half ^ turn<D>((uint32_t)col)) << 4);
  // Weights of scores e and e + 1.
  using Scores = f32x16[TB];
  auto weigh = [&](const Scores& s, int e) __attribute__((always_inline)) {
    const float x = exp2_fast(fmaf(s[e >> 4][e & 15], by, r)), y = exp2_fast(fmaf(s[(e + 1) >> 4][(e + 1) & 15], by, r));
    sum_a += x;
    sum_b += y;
    uint32_t both = T::pack(x, y);
    asm volatile("" : "+v"(both), "+v"(sum_a), "+v"(sum_b));  // formed here, not where they are used first
    pw[e >> 3][(e & 7) >> 1] = both;
  };
  // Scores of the keys at `base` into s, the weights of `from` among them.
  auto scores = [&](uint32_t base, Scores& s, const Scores& from, auto among) __attribute__((always_inline)) {
    const uint32_t at = base + key_at;
    auto key = [&](int m) { return lds_read16((at ^ (uint32_t)((m % KS) << 5)) + (uint32_t)(m / KS) * (32 * ROW)); };
    u32x4 ring[kAhead];
#pragma unroll
    for (int m = 0; m < kAhead - 1; ++m) ring[m] = key(m);
#pragma unroll
    for (int tb = 0; tb < TB; ++tb) s[tb] = f32x16{};
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int m = 0; m < M; ++m) {
      if (m + kAhead - 1 < M) ring[(m + kAhead - 1) % kAhead] = key(m + kAhead - 1);
      s[m / KS] = T::mfma32(ring[m % kAhead], q[m % KS], s[m / KS]);
      if constexpr (decltype(among)::value) {
#pragma unroll
        for (int e = m * (E / M); e < (m + 1) * (E / M); e += 2) weigh(from, e);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  auto leave_out = [&](Scores& s, const Place& m) __attribute__((always_inline)) {
#pragma unroll
    for (int tb = 0; tb < TB; ++tb) {
      const uint32_t bits = (uint32_t)mask_from(m, (uint32_t)(tw * (TB * 32) + tb * 32)) >> (half * 4);
#pragma unroll
      for (int e = 0; e < 16; ++e) s[tb][e] = (bits >> ((e >> 2) * 8 + (e & 3))) & 1u ? s[tb][e] : -INFINITY;
    }
  };
  // The reference for scores s whose largest product is `top`.
  auto refer = [&](Scores& s, float top) __attribute__((always_inline)) {
    top = max_xor32(top) * scale;
    if (__builtin_amdgcn_ballot_w64(top > ref + kLazyStep) != 0) {
      const float m = fmaxf(ref, top);
      const float less = m == ref ? 1.0f : exp2_fast(ref - m);
      ref = m;
      sum *= less;
#pragma unroll
      for (int d = 0; d < DB; ++d) o[d] *= less;
    }
    // A difference to the reference comes unrounded out of one fma, but the
    // reference is a rounded product: far out products are rounded first, so
    // that the largest is the reference.
    by = scale;
    if (__builtin_amdgcn_ballot_w64(fabsf(ref) > kFar && ref != -INFINITY) != 0) {
#pragma unroll
      for (int tb = 0; tb < TB; ++tb) s[tb] *= scale;
      by = 1.0f;
    }
    r = ref == -INFINITY ? 0.0f : lift<T>(kLazyStep) - ref;
    sum_a = sum_b = 0.0f;
  };
  // Lane i of each 16 gives the address of 4 dims of token i / 4.
  const uint32_t i16 = (uint32_t)lane & 15, vt = (uint32_t)half * 4 + (i16 >> 2);
  const uint32_t vchunk = (((uint32_t)lane >> 4) & 1) * 2 + ((i16 & 3) >> 1);
  const uint32_t value_at = ((uint32_t)(tw * TB * 32) + vt) * ROW + ((vchunk ^ turn<D>(vt)) << 4) + (i16 & 1) * 8;
  // The values at `base` by the weights, the largest of s among them.
  auto values = [&](uint32_t base, const Scores& s, auto among) __attribute__((always_inline)) -> float {
    const uint32_t at = base + value_at;
    // Tokens vt .. and, eight rows further, vt + 8 ..: turn() differs by one bit.
    auto value = [&](int m) {
      const uint32_t x = (at ^ (uint32_t)((m % DB) << 6)) + (uint32_t)(m / DB) * (16 * ROW);
      const u32x2 lo = lds_read_tr(x), hi = lds_read_tr((x ^ 32) + 8 * ROW);
      return u32x4{lo[0], lo[1], hi[0], hi[1]};
    };
    u32x4 ring[kAhead];
#pragma unroll
    for (int m = 0; m < kAhead - 1; ++m) ring[m] = value(m);
    float top = -INFINITY;
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int m = 0; m < N; ++m) {
      if (m + kAhead - 1 < N) ring[(m + kAhead - 1) % kAhead] = value(m + kAhead - 1);
      o[m % DB] = T::mfma32(ring[m % kAhead], pw[m / DB], o[m % DB]);
      if constexpr (decltype(among)::value) {
#pragma unroll
        for (int e = m * (E / N); e < (m + 1) * (E / N); e += 2)
          top = fmaxf(fmaxf(top, s[e >> 4][e & 15]), s[(e + 1) >> 4][(e + 1) & 15]);
        asm volatile("" : "+v"(top));
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    return top;
  };
  auto highest = [&](const Scores& s) __attribute__((always_inline)) -> float {
    float top = -INFINITY;
#pragma unroll
    for (int e = 0; e < E; e += 2) top = fmaxf(fmaxf(top, s[e >> 4][e & 15]), s[(e + 1) >> 4][(e + 1) & 15]);
    return top;
  };
  auto close = [&] __attribute__((always_inline)) { sum += sum_a + sum_b; };

  // Step i: the weights of tile i and the scores of tile i + 1; then, once the
  // values of tile i and the keys of tile i + 2 have arrived for every wavefront,
  // the values.  That one barrier also says that the keys of tile i + 1 and the
  // values of tile i - 1 are read: the next loads into them start behind it.
  constexpr int AHEAD = F8 ? RB + 2 : KB;  // tiles that keys are placed ahead
  Place at_tile[AHEAD + 1], whole;         // of tiles i, i + 1, ...; of one that is not masked
#pragma unroll
  for (int k = 0; k < NP; ++k) whole.mask[k] = ~0ull;
  const auto keys_of = [&](int32_t i) -> char* { return &sk[0][0] + (uint32_t)(i % KB) * TILE; };
  const auto values_of = [&](int32_t i) -> char* { return &sv[0][0] + (uint32_t)(i % VB) * TILE; };
  const auto raw_of = [&](int32_t i, int which) -> char* { return &sraw[F8 ? i % (RB > 0 ? RB : 1) : 0][which][0]; };
  Scores s0, s1;
  constexpr std::bool_constant<true> kAmong;
  constexpr std::bool_constant<false> kAlone;
  look_up(0);
#pragma unroll
  for (int d = 0; d < AHEAD; ++d) {
    if (d == 0 || d < tiles) at_tile[d] = place(d);
    else at_tile[d] = at_tile[d - 1];
  }
  at_tile[AHEAD] = at_tile[AHEAD - 1];
  if constexpr (!F8) {
#pragma unroll
    for (int d = 0; d < KB; ++d)
      if (d < tiles) issue(kbase, at_tile[d], keys_of(d));
#pragma unroll
    for (int d = 0; d < VB - 1; ++d)
      if (d < tiles) issue(vbase, at_tile[d], values_of(d));
    wait_loads<0>();
  } else {
    // The first two tiles of keys and the first of values, and RB behind each.
#pragma unroll
    for (int d = 0; d < 2; ++d) {
      if (d >= tiles) break;
      issue(kbase, at_tile[d], raw_of(d, 0));
      if (d == 0) issue(vbase, at_tile[0], raw_of(0, 1));
      wait_loads<0>();
      put(raw_of(d, 0), keys_of(d), whole);
      if (d == 0) put(raw_of(0, 1), values_of(0), at_tile[0]);
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the raw bytes are read
    }
#pragma unroll
    for (int d = 0; d < RB; ++d) {
      if (d + 2 < tiles) issue(kbase, at_tile[d + 2], raw_of(d + 2, 0));
      if (d + 1 < tiles) issue(vbase, at_tile[d + 1], raw_of(d + 1, 1));
    }
  }
  if constexpr (!F8)
    if (!at_tile[0].whole()) clear(values_of(0), at_tile[0]);
  __syncthreads();
  scores(lds_at(keys_of(0)), s0, s1, kAlone);
  if (!at_tile[0].whole()) leave_out(s0, at_tile[0]);
  float top = highest(s0);
  __syncthreads();  // the first tile's keys are read
  auto step = [&](int32_t i, Scores& s, Scores& t) __attribute__((always_inline)) {
    // Behind the last barrier: the keys of tile i and the values of tile i - 1.
    const bool more = i + AHEAD < tiles;
    if (more) at_tile[AHEAD] = place(i + AHEAD);
    if constexpr (!F8) {
      if (more) issue(kbase, at_tile[AHEAD], keys_of(i + KB));
    } else if (i + 2 < tiles) {
      // Behind these: RB - 1 more of keys and RB of values, while there are any.
      if (more) wait_loads<(2 * RB - 1) * NL>();
      else wait_loads<0>();
      put(raw_of(i + 2, 0), keys_of(i + 2), whole);
      if (more) {
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        issue(kbase, at_tile[AHEAD], raw_of(i + AHEAD, 0));
      }
    }
    refer(s, top);
    scores(lds_at(keys_of(i + 1)), t, s, kAmong);
    close();
    if constexpr (!F8) {
      // Behind the values of tile i and the keys of tile i + 2: values up to tile
      // i + VB - 2, keys up to tile i + KB.
      const int32_t keys = (i + KB < tiles ? i + KB : tiles - 1) - (i + 2), some = (i + VB - 2 < tiles ? i + VB - 2 : tiles - 1) - i;
      wait_tiles((keys > 0 ? keys : 0) + some);
      if (!at_tile[0].whole()) clear(values_of(i), at_tile[0]);
    }
    __syncthreads();
    if constexpr (!F8) {
      if (i + VB - 1 < tiles) issue(vbase, at_tile[VB - 1], values_of(i + VB - 1));
    } else {
      if (more) wait_loads<(2 * RB - 1) * NL>();
      else wait_loads<0>();
      put(raw_of(i + 1, 1), values_of(i + 1), at_tile[1]);
      if (i + 1 + RB < tiles) {
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        issue(vbase, at_tile[1 + RB], raw_of(i + 1 + RB, 1));
      }
    }
    if (!at_tile[1].whole()) leave_out(t, at_tile[1]);
    top = values(lds_at(values_of(i)), t, kAmong);
#pragma unroll
    for (int d = 0; d < AHEAD; ++d) at_tile[d] = at_tile[d + 1];
  };
  {
    int32_t i = 0;
    for (; i + 2 < tiles; i += 2) {
      step(i, s0, s1);
      step(i + 1, s1, s0);
    }
    if (i + 1 < tiles) {
      step(i, s0, s1);
#pragma unroll
      for (int tb = 0; tb < TB; ++tb) s0[tb] = s1[tb];
    }
  }
  // The last tile's weights and values.
  refer(s0, top);
#pragma unroll
  for (int e = 0; e < E; e += 2) weigh(s0, e);
  close();
  if constexpr (!F8) {
    wait_loads<0>();
    if (tiles > 1 && !at_tile[0].whole()) clear(values_of(tiles - 1), at_tile[0]);
  }
  __syncthreads();
  values(lds_at(values_of(tiles - 1)), s0, kAlone);

  sum += __shfl_xor(sum, 32);
  if constexpr (TW > 1) {
    // The wavefronts along the tokens meet where the tiles were.
    __syncthreads();
    f32x4* so = (f32x4*)&sv[0][0];          // [TW - 1][CW][DB * 4][64]
    float2(*stat)[32] = (float2(*)[32])&sk[0][0];
    if (half == 0) stat[w][col] = float2{ref, sum};
    __syncthreads();
    float top = ref;
#pragma unroll
    for (int k = 0; k < TW; ++k) top = fmaxf(top, stat[k * CW + cw][col].x);
    const float by = ref == top ? 1.0f : exp2_fast(ref - top);
#pragma unroll
    for (int d = 0; d < DB; ++d) o[d] *= by;
    if (tw > 0) {
#pragma unroll
      for (int x = 0; x < DB * 4; ++x)
        so[(((tw - 1) * CW + cw) * (DB * 4) + x) * 64 + lane] =
            f32x4{o[x >> 2][(x & 3) * 4], o[x >> 2][(x & 3) * 4 + 1], o[x >> 2][(x & 3) * 4 + 2], o[x >> 2][(x & 3) * 4 + 3]};
    }
    __syncthreads();
    if (tw > 0) return;
    sum = 0.0f;
#pragma unroll
    for (int k = 0; k < TW; ++k) {
      const float2 m = stat[k * CW + cw][col];
      sum += m.y * (m.x == top ? 1.0f : exp2_fast(m.x - top));
      if (k == 0) continue;
#pragma unroll
      for (int x = 0; x < DB * 4; ++x) {
        const f32x4 y = so[(((k - 1) * CW + cw) * (DB * 4) + x) * 64 + lane];
#pragma unroll
        for (int e = 0; e < 4; ++e) o[x >> 2][(x & 3) * 4 + e] += y[e];
      }
    }
    ref = top;
  }
  if (!real) return;
  const float v_scale = F8 && a.v_scales != nullptr ? a.v_scales[kvh] : 1.0f;
  const int64_t pi = (row * a.num_heads + head) * p.pitch + part;
#pragma unroll
  for (int d = 0; d < DB; ++d)
#pragma unroll
    for (int k = 0; k < 4; ++k)
      *(f32x4*)(p.part_out + pi * D + d * 32 + k * 8 + half * 4) =
          f32x4{o[d][k * 4] * v_scale, o[d][k * 4 + 1] * v_scale, o[d][k * 4 + 2] * v_scale, o[d][k * 4 + 3] * v_scale};
  if (half == 0) p.part_stat[pi] = float2{ref - lift<T>(kLazyStep), sum};
}

// ---------------------------------------------------------------------------
// Join of a row's shared and own parts: a wavefront for each (row, head).  Its
// lanes take the statistics of at most 64 parts; D / 4 of them cover the dims, and
// as many parts are read side by side as fit, eight deep.  Rows whose one own part
// is all they have were finished with it.
// ---------------------------------------------------------------------------
template <typename T, int D>
__global__ void __launch_bounds__(256) prefix_join_kernel(AttnParams p) {
  constexpr int LD = D / 4, SIDE = 64 / LD, DEEP = 8;
  const paged_attention_args& a = p.a;
  const int lane = threadIdx.x & 63;
  const int64_t at = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  if (at >= (int64_t)a.num_rows * a.num_heads) return;
  const int32_t seq = (int32_t)(at / a.num_heads) / a.next_n;
  const int64_t most = table_tokens(a.table_width, a.page_size);
  const int32_t shared = p.share[seq];
  int32_t n = 0;
  for (int32_t j = 0; j < a.next_n; ++j) {
    const int32_t x = clamp_to(a.lengths[(int64_t)seq * a.next_n + j], most);
    n = x > n ? x : n;
  }
  const PrefixPlanned planned = *p.planned;
  const int32_t own = split_by(n - shared, planned.own_part, p.most, p.unit).parts;
  const int32_t first = split_by(shared, planned.shared_part, p.shared_most, p.shared_unit).parts;
  if (first == 0 && own == 1) return;
  const int32_t parts = first + own, side = lane / LD, dim = lane % LD * 4;
  auto place = [&](int32_t i) { return i < first ? i : p.shared_most + (i - first); };  // of the i-th part
  const float2* stat = p.part_stat + at * p.pitch;
  const float2 m = lane < parts ? stat[place(lane)] : float2{-INFINITY, 0.0f};
  const float* po = p.part_out + at * p.pitch * D + dim;
  f32x4 x[DEEP];
  auto read = [&](int32_t i0) {
#pragma unroll
    for (int k = 0; k < DEEP; ++k) {
      const int32_t i = i0 + k * SIDE + side;
      x[k] = i < parts ? *(const f32x4*)(po + (int64_t)place(i) * D) : f32x4{0, 0, 0, 0};
    }
  };
  read(0);  // beside the statistics
  float top = m.x;
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor(top, off));
  const float by = m.x == top ? 1.0f : exp2_fast(m.x - top);
  float sum = m.y * by;
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off);
  f32x4 o = {0, 0, 0, 0};
  for (int32_t i0 = 0;;) {
#pragma unroll
    for (int k = 0; k < DEEP; ++k) {
      const float weight = __shfl(by, (i0 + k * SIDE + side) & 63);
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] += weight * x[k][e];
    }
    i0 += DEEP * SIDE;
    if (i0 >= parts) break;
    read(i0);
  }
#pragma unroll
  for (int off = LD; off < 64; off <<= 1)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] += __shfl_xor(o[e], off);
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  if (side == 0)
    *(u32x2*)((uint16_t*)a.out + at * D + dim) = u32x2{T::pack(o[0] * inv, o[1] * inv), T::pack(o[2] * inv, o[3] * inv)};
  if (lane == 0 && a.lse != nullptr) a.lse[at] = sum == 0.0f ? -INFINITY : (top + __log2f(sum)) * kLn2;
}

namespace {
template <typename T, bool F8, int D, bool P16>
const void* prefix_waves(int waves) {
  return waves == 4 ? (const void*)&prefix_kernel<T, F8, D, 4, P16> : waves == 2 ? (const void*)&prefix_kernel<T, F8, D, 2, P16>
                                                                  : (const void*)&prefix_kernel<T, F8, D, 1, P16>;
}
template <typename T, bool F8>
const void* prefix_dims(int dim, int waves, bool p16) {
  if (dim == 64) return p16 ? prefix_waves<T, F8, 64, true>(waves) : prefix_waves<T, F8, 64, false>(waves);
  if (dim == 128) return p16 ? prefix_waves<T, F8, 128, true>(waves) : prefix_waves<T, F8, 128, false>(waves);
  return nullptr;
}
}  // namespace

const void* prefix_kernel_ptr(int dtype, int store, int head_dim, int waves, bool p16) {
  if (dtype == PAGED_BF16)
    return store == PAGED_E4M3 ? prefix_dims<Bf16, true>(head_dim, waves, p16) : prefix_dims<Bf16, false>(head_dim, waves, p16);
  return store == PAGED_E4M3 ? prefix_dims<Fp16, true>(head_dim, waves, p16) : prefix_dims<Fp16, false>(head_dim, waves, p16);
}
const void* prefix_join_kernel_ptr(int dtype, int head_dim) {
  if (dtype == PAGED_BF16)
    return head_dim == 64 ? (const void*)&prefix_join_kernel<Bf16, 64> : (const void*)&prefix_join_kernel<Bf16, 128>;
  return head_dim == 64 ? (const void*)&prefix_join_kernel<Fp16, 64> : (const void*)&prefix_join_kernel<Fp16, 128>;
}
int prefix_unit(int waves) { return waves == 1 ? 128 : 64; }

}  // namespace rrt
