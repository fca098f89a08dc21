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

// The group of a tile of columns, the tile's place in it, and the sequences.
struct ColTile {
  int32_t group, local, first, count;
};
__device__ __forceinline__ bool col_tile_of(const AttnParams& p, int32_t want, int32_t per_seq, int32_t wide, int lane, ColTile* t) {
  int32_t base = 0;
  for (int32_t g0 = 0; g0 < p.num_groups; g0 += 64) {
    const int32_t g = g0 + lane;
    int32_t from = 0, n = 0;
    if (g < p.num_groups) group_of(p, g, &from, &n);
    const int32_t mine = (int32_t)(((int64_t)n * per_seq + wide - 1) / wide);
    const int32_t upto = __builtin_elementwise_add_sat(base, prefix_scan(mine, lane));
    const uint64_t past = __builtin_amdgcn_ballot_w64(upto > want);
    if (past != 0) {
      const int l = __builtin_ctzll(past);
      t->group = g0 + l;
      t->local = want - (l == 0 ? base : __builtin_amdgcn_readlane(upto, l - 1));
      t->first = __builtin_amdgcn_readlane(from, l);
      t->count = __builtin_amdgcn_readlane(n, l);
      return true;
    }
    base = __builtin_amdgcn_readlane(upto, 63);
  }
  return false;
}

template <typename T, bool F8, int D, int CW>
__global__ void __launch_bounds__(256, 2) prefix_kernel(AttnParams p) {
  constexpr int TB = CW == 4 ? 2 : 1;          // blocks of 32 tokens of a wavefront in a tile
  constexpr int TW = 4 / CW;                   // wavefronts along the tokens
  constexpr int TT = 32 * TB * TW;             // tokens of a tile
  constexpr int NP = TT / 64;                  // tokens of a tile that a lane looks up
  constexpr int KS = D / 16, DB = D / 32;      // steps over the key dims; blocks of value dims
  constexpr uint32_t ROW = D * 2, TILE = TT * ROW;
  constexpr int SZ = F8 ? 1 : 2;
  constexpr int LPR = D * SZ / 16, RPL = 64 / LPR;  // lanes of a row's load; rows of a load
  constexpr int NL = TT / 4 / RPL;                  // loads of a wavefront's quarter of a tile
  __shared__ __align__(1024) char sk[TILE];
  __shared__ __align__(1024) char sv[2][TILE];
  __shared__ float2 stat[4][32];
  const paged_attention_args& a = p.a;
  const int tid = threadIdx.x, lane = tid & 63, col = lane & 31, half = lane >> 5;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6), cw = w % CW, tw = w / CW;

  // Tiles of columns that read the same tokens follow one another on one XCD; a
  // part's heads go round the XCDs (see work_of).
  const uint32_t idx = blockIdx.x >> 3, eight = idx / (uint32_t)p.shared_tiles;
  const uint32_t outer = eight * 8 + (((blockIdx.x & 7) + eight) & 7);
  const int32_t part = (int32_t)(outer / (uint32_t)a.num_kv_heads), kvh = (int32_t)(outer - (uint32_t)part * (uint32_t)a.num_kv_heads);
  if (part >= p.shared_most) return;
  const int32_t per = a.num_heads / a.num_kv_heads, per_seq = per * a.next_n;
  ColTile ct;
  if (!col_tile_of(p, (int32_t)(idx - eight * (uint32_t)p.shared_tiles), per_seq, 32 * CW, lane, &ct)) return;
  const int64_t most = table_tokens(a.table_width, a.page_size);
  const int32_t n = clamp_to(p.shared[ct.group], most);
  const Split sp = split_of(n, p.shared_most, p.shared_least, TT);
  if (n == 0 || part >= sp.parts) return;
  const int32_t begin = part * sp.chunk, end = n - begin < sp.chunk ? n : begin + sp.chunk;
  const int32_t tiles = (end - begin + TT - 1) / TT;

  // The table row of the first sequence that takes part.
  int32_t reader = -1;
  for (int32_t s0 = 0; s0 < ct.count && reader < 0; s0 += 64) {
    const uint64_t in = __builtin_amdgcn_ballot_w64(s0 + lane < ct.count && takes_part(a, ct.first + s0 + lane, n, most));
    if (in != 0) reader = ct.first + s0 + (int32_t)__builtin_ctzll(in);
  }
  if (reader < 0) return;
  const int32_t* table = a.block_table + (int64_t)reader * a.table_stride;

  // The lane's column.
  const int32_t c = (ct.local * CW + cw) * 32 + col;
  const int32_t j = c / per, seq = ct.first + j / a.next_n;
  const bool real = c < ct.count * per_seq && takes_part(a, seq, n, most);
  const int64_t row = (int64_t)ct.first * a.next_n + (c < ct.count * per_seq ? j : 0);
  const int32_t head = kvh * per + (c < ct.count * per_seq ? c - j * per : 0);
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
  // Lane l looks up tokens l (and 64 + l) of a tile; every wavefront does so for
  // the whole tile, which gives it the tile's mask.  A page is read a tile
  // before it is used.
  const char* kbase = (const char*)a.k + (int64_t)kvh * a.head_stride * SZ;
  const char* vbase = (const char*)a.v + (int64_t)kvh * a.head_stride * SZ;
  int32_t page[NP];
  uint32_t in[NP];
  auto look_up = [&](int32_t i) {
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      const int32_t pos = begin + i * TT + k * 64 + lane;
      const bool ok = pos < end;
      const uint32_t x = ok ? (uint32_t)pos : 0u, at = divide(x, p.page);
      in[k] = ok ? x - at * p.page.by : ~0u;
      page[k] = table[at];
    }
  };
  int64_t off[NL];  // of the lane's rows in the next tile to load, in bytes
  uint64_t mask[NP];
  auto place = [&] {
    int64_t at[NP];
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      const bool ok = in[k] != ~0u && (uint32_t)page[k] < (uint32_t)a.num_pages;
      mask[k] = __builtin_amdgcn_ballot_w64(ok);
      at[k] = ok ? ((int64_t)page[k] * a.page_stride + (int64_t)in[k] * a.token_stride) * SZ : 0;
    }
#pragma unroll
    for (int k = 0; k < NL; ++k) {
      const int t = w * (TT / 4) + k * RPL;  // of the tile, before the lane's row
      const int64_t mine = NP == 1 || t < 64 ? at[0] : at[NP - 1];
      off[k] = shfl64(mine, (t & 63) + lane / LPR);
    }
  };
  // The tokens of a tile that count, 32 for this wavefront's block tb.
  auto counts = [&](const uint64_t* m, int tb) -> uint32_t {
    const int t = tw * (TB * 32) + tb * 32;
    return (uint32_t)(m[t >> 6] >> (t & 63));
  };

  // --- tiles to LDS -------------------------------------------------------------
  const uint32_t sub = (uint32_t)lane / LPR, pos = (uint32_t)lane % LPR;
  const uint32_t row0 = (uint32_t)w * (TT / 4);
  u32x4 rk[F8 ? NL : 1], rv[F8 ? NL : 1];
  auto issue = [&](const char* base, const char* to) {  // 16 bits: straight to LDS
#pragma unroll
    for (int k = 0; k < NL; ++k) {
      const uint32_t chunk = pos ^ turn<D>(row0 + k * RPL + sub);
      load_to_lds(base + off[k] + chunk * 16, lds_at(to) + (row0 + k * RPL) * ROW);
    }
  };
  auto fetch = [&](const char* base, u32x4* r) {  // e4m3: to registers
#pragma unroll
    for (int k = 0; k < NL; ++k) r[k] = *(const u32x4*)(base + off[k] + pos * 16);
  };
  auto put = [&](const u32x4* r, char* to, const uint64_t* m) {
#pragma unroll
    for (int k = 0; k < NL; ++k) {
      const uint32_t t = row0 + k * RPL + sub;
      // Tokens that do not count become zeros: their places may hold NaN.
      const bool ok = m == nullptr || ((m[NP == 1 ? 0 : t >> 6] >> (t & 63)) & 1u) != 0;
      const u32x4 lo = widen<T>(u32x2{r[k][0], r[k][1]}), hi = widen<T>(u32x2{r[k][2], r[k][3]});
      const uint32_t at = lds_at(to) + t * ROW + (((pos * 2) ^ turn<D>(t)) << 4);
      *(lds_u32x4*)at = ok ? lo : u32x4{0, 0, 0, 0};
      *(lds_u32x4*)(at ^ 16) = ok ? hi : u32x4{0, 0, 0, 0};
    }
  };
  // The wavefront's rows of a values' tile that do not count (16 bits).
  auto clear = [&](char* to, const uint64_t* m) {
    constexpr uint32_t kAll = TT / 4 == 32 ? ~0u : (1u << (TT / 4)) - 1u;
    const uint32_t mine = (uint32_t)(m[NP == 1 ? 0 : row0 >> 6] >> (row0 & 63)) & kAll;
    if (mine == kAll) return;
#pragma nounroll
    for (int t = 0; t < TT / 4; ++t)
      if (((mine >> t) & 1u) == 0 && lane < D / 8) *(lds_u32x4*)(lds_at(to) + (row0 + t) * ROW + lane * 16) = u32x4{0, 0, 0, 0};
  };

  // --- one tile -------------------------------------------------------------------
  float ref = -INFINITY, sum = 0.0f;  // base-2 logarithm; of this lane's tokens
  f32x16 o[DB], s[TB];
#pragma unroll
  for (int d = 0; d < DB; ++d) o[d] = f32x16{};
  u32x4 pw[2 * TB];
  const uint32_t key_at = lds_at(&sk[0]) + (uint32_t)(tw * TB * 32 + col) * ROW + (((uint32_t)half ^ turn<D>((uint32_t)col)) << 4);
  auto scores = [&] {
    auto key = [&](int m) { return lds_read16((key_at ^ (uint32_t)((m % KS) << 5)) + (uint32_t)(m / KS) * (32 * ROW)); };
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

  uint64_t now[NP];
  if constexpr (!F8) {
    look_up(0);
    place();
    issue(kbase, &sk[0]);
    issue(vbase, &sv[0][0]);
    if (tiles > 1) look_up(1);
    for (int32_t i = 0; i < tiles; ++i) {
      const bool more = i + 1 < tiles;
#pragma unroll
      for (int k = 0; k < NP; ++k) now[k] = mask[k];
      wait_loads<0>();
      clear(&sv[i & 1][0], now);
      __syncthreads();
      if (more) {
        place();
        issue(vbase, &sv[(i + 1) & 1][0]);
      }
      scores();
      __syncthreads();  // the keys are read
      if (more) issue(kbase, &sk[0]);
      if (i + 2 < tiles) look_up(i + 2);
      leave_out(now);
      weights();
      values(lds_at(&sv[i & 1][0]));
    }
  } else {
    uint64_t next[NP];
    look_up(0);
    place();
    fetch(kbase, rk);
    fetch(vbase, rv);
    if (tiles > 1) look_up(1);
#pragma unroll
    for (int k = 0; k < NP; ++k) now[k] = mask[k];
    put(rk, &sk[0], nullptr);
    put(rv, &sv[0][0], now);
    if (tiles > 1) {
      place();
      fetch(kbase, rk);
      fetch(vbase, rv);
      if (tiles > 2) look_up(2);
    }
    for (int32_t i = 0; i < tiles; ++i) {
#pragma unroll
      for (int k = 0; k < NP; ++k) next[k] = mask[k];
      __syncthreads();
      scores();
      __syncthreads();  // the keys are read
      if (i + 1 < tiles) {
        put(rk, &sk[0], nullptr);
        put(rv, &sv[(i + 1) & 1][0], next);
      }
      if (i + 2 < tiles) {
        place();
        fetch(kbase, rk);
        fetch(vbase, rv);
        if (i + 3 < tiles) look_up(i + 3);
      }
      leave_out(now);
      weights();
      values(lds_at(&sv[i & 1][0]));
#pragma unroll
      for (int k = 0; k < NP; ++k) now[k] = next[k];
    }
  }

  sum += __shfl_xor(sum, 32);
  if constexpr (TW > 1) {
    // The wavefronts along the tokens meet in the values' buffers.
    __syncthreads();
    f32x4* so = (f32x4*)&sv[0][0];  // [TW - 1][CW][DB * 4][64]
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
// Join of a row's shared and own parts: a wavefront for each (row, head), its
// lanes the statistics of at most 64 parts and then the dims.  Rows whose one
// own part is all they have were finished with it.
// ---------------------------------------------------------------------------
template <typename T, int D>
__global__ void __launch_bounds__(256) prefix_join_kernel(AttnParams p) {
  constexpr int E = D / 64;
  const paged_attention_args& a = p.a;
  const int lane = threadIdx.x & 63;
  const int64_t at = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  if (at >= (int64_t)a.num_rows * a.num_heads) return;
  const int32_t seq = (int32_t)(at / a.num_heads) / a.next_n;
  const int64_t most = table_tokens(a.table_width, a.page_size);
  const int32_t shared = shared_of(p, seq, most, lane);
  int32_t n = 0;
  for (int32_t j = 0; j < a.next_n; ++j) {
    const int32_t x = clamp_to(a.lengths[(int64_t)seq * a.next_n + j], most);
    n = x > n ? x : n;
  }
  const int32_t own = split_of(n - shared, p.most, p.least, p.unit).parts;
  const int32_t first = shared == 0 ? 0 : split_of(shared, p.shared_most, p.shared_least, p.shared_unit).parts;
  if (first == 0 && own == 1) return;
  const float2* stat = p.part_stat + at * p.pitch;
  const bool here = lane < first || (lane >= p.shared_most && lane < p.shared_most + own);
  const float2 m = here ? stat[lane] : float2{-INFINITY, 0.0f};
  float top = m.x;
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor(top, off));
  const float by = m.x == top ? 1.0f : exp2_fast(m.x - top);
  float sum = m.y * by;
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off);
  const float* po = p.part_out + at * p.pitch * D + lane * E;
  float o[E] = {};
#pragma unroll 4
  for (int32_t i = 0; i < first + own; ++i) {
    const int32_t x = i < first ? i : p.shared_most + (i - first);
    const float weight = __shfl(by, x);
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] += weight * po[(int64_t)x * D + e];
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  uint16_t* out = (uint16_t*)a.out + at * D + lane * E;
  if constexpr (E == 1) *out = (uint16_t)T::pack(o[0] * inv, 0.0f);
  else *(uint32_t*)out = T::pack(o[0] * inv, o[1] * inv);
  if (lane == 0 && a.lse != nullptr) a.lse[at] = sum == 0.0f ? -INFINITY : (top + __log2f(sum)) * kLn2;
}

namespace {
template <typename T, bool F8, int D>
const void* prefix_waves(int waves) {
  return waves == 4 ? (const void*)&prefix_kernel<T, F8, D, 4> : waves == 2 ? (const void*)&prefix_kernel<T, F8, D, 2>
                                                             : (const void*)&prefix_kernel<T, F8, D, 1>;
}
template <typename T, bool F8>
const void* prefix_dims(int dim, int waves) {
  return dim == 64 ? prefix_waves<T, F8, 64>(waves) : dim == 128 ? prefix_waves<T, F8, 128>(waves) : nullptr;
}
}  // namespace

const void* prefix_kernel_ptr(int dtype, int store, int head_dim, int waves) {
  if (dtype == PAGED_BF16)
    return store == PAGED_E4M3 ? prefix_dims<Bf16, true>(head_dim, waves) : prefix_dims<Bf16, false>(head_dim, waves);
  return store == PAGED_E4M3 ? prefix_dims<Fp16, true>(head_dim, waves) : prefix_dims<Fp16, false>(head_dim, waves);
}
const void* prefix_join_kernel_ptr(int dtype, int head_dim) {
  if (dtype == PAGED_BF16)
    return head_dim == 64 ? (const void*)&prefix_join_kernel<Bf16, 64> : (const void*)&prefix_join_kernel<Bf16, 128>;
  return head_dim == 64 ? (const void*)&prefix_join_kernel<Fp16, 64> : (const void*)&prefix_join_kernel<Fp16, 128>;
}
int prefix_unit(int waves) { return waves == 1 ? 128 : 64; }

}  // namespace rrt
