// Attention over positions that many rows share: their keys and values are read
// once for all of them.

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
// x 4 chunks) meet a bank twice.  Keys have one buffer, values two: the next
// tile's values load under this one's scores, its keys under the rest.  (e4m3:
// raw bytes wait in registers, and are widened on the way to LDS.)
//
// The weights are relative to a reference that follows the running maximum
// lazily: only a score that passes it by 2^8 moves it (they then stay below 2^8,
// or 2^15 as fp16 keeps them).
// ---------------------------------------------------------------------------
constexpr float kLazyStep = 8.0f;
// Past this a reference's own rounding shows in the difference of a score to it.
constexpr float kFar = 1048576.0f;
constexpr int kAhead = 4;  // operands in flight from LDS, and one in use
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
  for (int32_t g0 = 0; g0 < p.num_groups; g0 += 64) {
    const GroupWork w = work_of_group(p, g0 + lane, per_seq, wide, most);
    all += (int64_t)w.tiles * w.n;
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) all += shfl64(all, lane ^ off);
  return part_size(readlane64(all, 0) * p.a.num_kv_heads, p.workgroups, kSharedLeast, p.shared_unit);
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
  all = (sums[0] + sums[1]) + (sums[2] + sums[3]);
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
  constexpr int TB = CW == 4 ? 2 : 1;          // blocks of 32 tokens of a wavefront in a tile
  constexpr int TW = 4 / CW;                   // wavefronts along the tokens
  constexpr int TT = 32 * TB * TW;             // tokens of a tile
  constexpr int QT = TT / 4;                   // and of a wavefront's loads
  constexpr int NP = TT / 64;                  // words of a tile's mask; tokens that a lane looks up
  constexpr int KS = D / 16, DB = D / 32;      // steps over the key dims; blocks of value dims
  constexpr uint32_t ROW = D * 2, TILE = TT * ROW;
  constexpr int SZ = F8 ? 1 : 2;
  constexpr int LPR = D * SZ / 16, RPL = 64 / LPR;  // lanes of a row's load; rows of a load
  constexpr int NL = QT / RPL, NG = 16 / RPL;       // loads of a wavefront's quarter of a tile, of 16 tokens
  constexpr int KB = F8 || CW == 1 ? 2 : 3;         // keys' tiles in LDS
  __shared__ __align__(1024) char sk[KB][TILE];
  __shared__ __align__(1024) char sv[2][TILE];
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
    int64_t at[P16 ? QT / 16 : NL];  // bytes: of sixteen tokens, or of the lane's row in each load
    uint64_t mask[NP];
    bool whole;                      // every token counts
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
  auto place = [&](int32_t i, Place* out) {
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
      for (int g = 0; g < QT / 16; ++g) out->at[g] = readlane64(group_at, g0 + w * (QT / 16) + g);
      out->whole = (~(group_whole >> g0) & ((1u << GT) - 1u)) == 0;
#pragma unroll
      for (int k = 0; k < NP; ++k) out->mask[k] = ~0ull;
      if (!out->whole) {
#pragma unroll
        for (int k = 0; k < NP; ++k) {
          out->mask[k] = 0;
#pragma nounroll
          for (int g = 0; g < 4; ++g)
            out->mask[k] |= (uint64_t)((1u << __builtin_amdgcn_readlane(group_count, g0 + k * 4 + g)) - 1u) << (g * 16);
        }
      }
    } else {
      int64_t at[NP];
      out->whole = true;
#pragma unroll
      for (int k = 0; k < NP; ++k) {
        const bool ok = in[k] != ~0u && (uint32_t)page[k] < (uint32_t)a.num_pages;
        out->mask[k] = __builtin_amdgcn_ballot_w64(ok);
        out->whole = out->whole && out->mask[k] == ~0ull;
        at[k] = ok ? ((int64_t)page[k] * a.page_stride + (int64_t)in[k] * a.token_stride) * SZ : 0;
      }
#pragma unroll
      for (int k = 0; k < NL; ++k) {
        const int t = (int)row0 + k * RPL;  // of the tile, before the lane's row
        const int64_t mine = NP == 1 || t < 64 ? at[0] : at[NP - 1];
        out->at[k] = shfl64(mine, (t & 63) + (int)sub);
      }
      if (i + 1 < tiles) look_up(i + 1);
    }
  };
  uint32_t inside[NG];  // bytes from the first of sixteen tokens to the lane's chunk
#pragma unroll
  for (int k = 0; k < NG; ++k) {
    const uint32_t t = k * RPL + sub, chunk = F8 ? pos : pos ^ turn<D>(t);
    inside[k] = t * (uint32_t)a.token_stride * SZ + chunk * 16;
  }
  // The tokens of a tile that count, 32 for this wavefront's block tb.
  auto counts = [&](const uint64_t* m, int tb) -> uint32_t {
    const int t = tw * (TB * 32) + tb * 32;
    return (uint32_t)((NP == 1 || t < 64 ? m[0] : m[NP - 1]) >> (t & 63));
  };

  // --- tiles to LDS -------------------------------------------------------------
  u32x4 rk[F8 ? NL : 1], rv[F8 ? NL : 1];
  auto issue = [&](const char* base, const Place& at, char* to) {  // 16 bits: straight to LDS
#pragma unroll
    for (int k = 0; k < NL; ++k) {
      const uint32_t where = lds_at(to) + (row0 + k * RPL) * ROW;
      if constexpr (P16) load_to_lds(base + at.at[k / NG], inside[k % NG], where);
      else load_to_lds(base + at.at[k] + (pos ^ turn<D>(row0 + k * RPL + sub)) * 16, where);
    }
  };
  auto fetch = [&](const char* base, const Place& at, u32x4* r) {  // e4m3: to registers
#pragma unroll
    for (int k = 0; k < NL; ++k) {
      if constexpr (P16) r[k] = *(const u32x4*)(base + at.at[k / NG] + inside[k % NG]);
      else r[k] = *(const u32x4*)(base + at.at[k] + pos * 16);
    }
  };
  auto put = [&](const u32x4* r, char* to, const Place* m) {
#pragma unroll
    for (int k = 0; k < NL; ++k) {
      const uint32_t t = row0 + k * RPL + sub;
      // Tokens that do not count become zeros: their places may hold NaN.
      const bool ok = m == nullptr || m->whole || (((NP == 1 || t < 64 ? m->mask[0] : m->mask[NP - 1]) >> (t & 63)) & 1u) != 0;
      const u32x4 lo = widen<T>(u32x2{r[k][0], r[k][1]}), hi = widen<T>(u32x2{r[k][2], r[k][3]});
      const uint32_t at = lds_at(to) + t * ROW + (((pos * 2) ^ turn<D>(t)) << 4);
      *(lds_u32x4*)at = ok ? lo : u32x4{0, 0, 0, 0};
      *(lds_u32x4*)(at ^ 16) = ok ? hi : u32x4{0, 0, 0, 0};
    }
  };
  // The wavefront's rows of a values' tile that do not count (16 bits).
  auto clear = [&](char* to, const uint64_t* m) {
    constexpr uint32_t kAll = QT == 32 ? ~0u : (1u << QT) - 1u;
    const uint32_t mine = (uint32_t)((NP == 1 || row0 < 64 ? m[0] : m[NP - 1]) >> (row0 & 63)) & kAll;
    if (mine == kAll) return;
#pragma nounroll
    for (int t = 0; t < QT; ++t)
      if (((mine >> t) & 1u) == 0 && lane < D / 8) *(lds_u32x4*)(lds_at(to) + (row0 + t) * ROW + lane * 16) = u32x4{0, 0, 0, 0};
  };

  // --- one tile -------------------------------------------------------------------
  float ref = -INFINITY, sum = 0.0f;  // base-2 logarithm; of this lane's tokens
  f32x16 o[DB], s[TB];
#pragma unroll
  for (int d = 0; d < DB; ++d) o[d] = f32x16{};
  u32x4 pw[2 * TB];
  const uint32_t key_at = (uint32_t)(tw * TB * 32 + col) * ROW + (((uint32_t)half ^ turn<D>((uint32_t)col)) << 4);
  auto scores = [&](uint32_t base) {
    const uint32_t at = base + key_at;
    auto key = [&](int m) { return lds_read16((at ^ (uint32_t)((m % KS) << 5)) + (uint32_t)(m / KS) * (32 * ROW)); };
    u32x4 ring[kAhead];
#pragma unroll
    for (int m = 0; m < kAhead - 1; ++m) ring[m] = key(m);
#pragma unroll
    for (int tb = 0; tb < TB; ++tb) s[tb] = f32x16{};
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int m = 0; m < TB * KS; ++m) {
      if (m + kAhead - 1 < TB * KS) ring[(m + kAhead - 1) % kAhead] = key(m + kAhead - 1);
      s[m / KS] = T::mfma32(ring[m % kAhead], q[m % KS], s[m / KS]);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  auto leave_out = [&](const uint64_t* m) {
#pragma unroll
    for (int tb = 0; tb < TB; ++tb) {
      const uint32_t bits = counts(m, tb);
      if (bits == 0xffffffffu) continue;
#pragma unroll
      for (int e = 0; e < 16; ++e) s[tb][e] = (bits >> ((e >> 2) * 8 + half * 4 + (e & 3))) & 1u ? s[tb][e] : -INFINITY;
    }
  };
  auto weights = [&] {
    float top = s[0][0];
#pragma unroll
    for (int e = 1; e < TB * 16; ++e) top = fmaxf(top, s[e >> 4][e & 15]);
    top = max_xor32(top) * scale;
    if (__builtin_amdgcn_ballot_w64(top > ref + kLazyStep) != 0) {
      const float m = fmaxf(ref, top);
      const float by = m == ref ? 1.0f : exp2_fast(ref - m);
      ref = m;
      sum *= by;
#pragma unroll
      for (int d = 0; d < DB; ++d) o[d] *= by;
    }
    // A difference to the reference comes unrounded out of one fma, but the
    // reference is a rounded product: far out products are rounded first, so
    // that the largest is the reference.
    float by = scale;
    if (__builtin_amdgcn_ballot_w64(fabsf(ref) > kFar && ref != -INFINITY) != 0) {
#pragma unroll
      for (int tb = 0; tb < TB; ++tb) s[tb] *= scale;
      by = 1.0f;
    }
    const float r = ref == -INFINITY ? 0.0f : lift<T>(kLazyStep) - ref;
    float part4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < 2 * TB; ++k) {
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] = exp2_fast(fmaf(s[k >> 1][(k & 1) * 8 + e], by, r));
        part4[e & 3] += x[e];
      }
      pw[k] = u32x4{T::pack(x[0], x[1]), T::pack(x[2], x[3]), T::pack(x[4], x[5]), T::pack(x[6], x[7])};
    }
    sum += (part4[0] + part4[1]) + (part4[2] + part4[3]);
  };
  // Lane i of each 16 gives the address of 4 dims of token i / 4.
  const uint32_t i16 = (uint32_t)lane & 15, vt = (uint32_t)half * 4 + (i16 >> 2);
  const uint32_t vchunk = (((uint32_t)lane >> 4) & 1) * 2 + ((i16 & 3) >> 1);
  const uint32_t value_at = ((uint32_t)(tw * TB * 32) + vt) * ROW + ((vchunk ^ turn<D>(vt)) << 4) + (i16 & 1) * 8;
  auto values = [&](uint32_t base) {
    const uint32_t at = base + value_at;
    // Tokens vt .. and, eight rows further, vt + 8 ..: turn() differs by one bit.
    auto value = [&](int m) {
      const uint32_t x = (at ^ (uint32_t)((m % DB) << 6)) + (uint32_t)(m / DB) * (16 * ROW);
      const u32x2 lo = lds_read_tr(x), hi = lds_read_tr((x ^ 32) + 8 * ROW);
      return u32x4{lo[0], lo[1], hi[0], hi[1]};
    };
    constexpr int N = 2 * TB * DB;
    u32x4 ring[kAhead];
#pragma unroll
    for (int m = 0; m < kAhead - 1; ++m) ring[m] = value(m);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int m = 0; m < N; ++m) {
      if (m + kAhead - 1 < N) ring[(m + kAhead - 1) % kAhead] = value(m + kAhead - 1);
      o[m % DB] = T::mfma32(ring[m % kAhead], pw[m / DB], o[m % DB]);
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  // Tile i: its scores and weights; then, once its values (and the next tile's
  // keys) have arrived for every wavefront, its values.  That one barrier also
  // says that the keys of tile i and the values of tile i - 1 are read: the next
  // loads into them start behind it, values one tile ahead and keys two.
  Place now, next, after;
  look_up(0);
  place(0, &now);
  if constexpr (!F8) {
    constexpr int AHEAD = KB - 1;  // tiles that keys are ahead
    issue(kbase, now, &sk[0][0]);
    issue(vbase, now, &sv[0][0]);
    next = now;
    if (tiles > 1) {
      place(1, &next);
      if constexpr (AHEAD == 2) issue(kbase, next, &sk[1][0]);
    }
    after = next;
    if (AHEAD == 2 && tiles > 1) wait_loads<2 * NL>();
    else wait_loads<NL>();
    __syncthreads();  // the first tile's keys
    int ring = 0;     // of tile i in sk
    for (int32_t i = 0; i < tiles; ++i) {
      const bool more = i + AHEAD < tiles;
      const int to = ring == 0 ? KB - 1 : ring - 1;
      if (more) {
        if constexpr (AHEAD == 2) place(i + 2, &after);
        issue(kbase, AHEAD == 2 ? after : next, &sk[to][0]);
      }
      scores(lds_at(&sk[0][0]) + (uint32_t)ring * TILE);
      if (!now.whole) leave_out(now.mask);
      weights();
      // All but the keys issued above: with keys one tile ahead those too.
      if (AHEAD == 2 && more) wait_loads<NL>();
      else wait_loads<0>();
      if (!now.whole) clear(&sv[i & 1][0], now.mask);
      __syncthreads();
      if (i + 1 < tiles) issue(vbase, next, &sv[(i + 1) & 1][0]);
      now = next;
      if constexpr (AHEAD == 2) next = after;
      else if (i + 2 < tiles) place(i + 2, &next);
      ring = ring + 1 == KB ? 0 : ring + 1;
      values(lds_at(&sv[i & 1][0]));
    }
  } else {
    // Raw bytes of tile i + 2 load while tile i is used.
    fetch(kbase, now, rk);
    fetch(vbase, now, rv);
    put(rk, &sk[0][0], nullptr);
    put(rv, &sv[0][0], &now);
    next = now;
    if (tiles > 1) {
      place(1, &next);
      fetch(kbase, next, rk);
      fetch(vbase, next, rv);
    }
    after = next;
    __syncthreads();
    for (int32_t i = 0; i < tiles; ++i) {
      if (i + 1 < tiles) put(rk, &sk[(i + 1) & 1][0], nullptr);
      if (i + 2 < tiles) {
        place(i + 2, &after);
        fetch(kbase, after, rk);
      }
      scores(lds_at(&sk[i & 1][0]));
      if (!now.whole) leave_out(now.mask);
      weights();
      __syncthreads();
      if (i + 1 < tiles) put(rv, &sv[(i + 1) & 1][0], &next);
      if (i + 2 < tiles) fetch(vbase, after, rv);
      now = next;
      next = after;
      values(lds_at(&sv[i & 1][0]));
    }
  }

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
