// Attention of single tokens over a paged cache of keys and values, and the
// join of rows that were split over several workgroups.

#include "paged_device.hpp"

namespace rrt {

// ---------------------------------------------------------------------------
// o = softmax(s q K^T) V in one pass over K and V, with the running maximum m
// (of base-2 logarithms) and sum l of each query column.
//
// A workgroup takes one part of one key-value head's positions; its four
// wavefronts take tiles of 32 tokens in turn, each with its own m, l and
// output, and join them in LDS at the end.  The columns of a tile are the
// query heads that share the key-value head, for every row of the sequence
// (multi-token rows read the cache once).
//
// Nothing passes through LDS on the way in.  With S^T = K Q^T the K operand's
// lane layout (row l % 16, 8 consecutive dims) is what a 16-byte load of a
// cache row gives, and S^T's layout (column l % 16, rows l / 16 * 4 + i) is
// the layout of the P operand of O^T = V^T P if lane group g = l / 16 counts
// tokens g*4 .. g*4+3 and 16+g*4 .. 16+g*4+3 as its eight: the order of the
// summed-over tokens is free as long as V follows it.  So each lane loads V
// rows of those eight tokens (a load of a wavefront covers four whole rows)
// and transposes its own 8 x 8 block with byte permutes.  m, l, P and O^T then
// all live in the lane of their column: no exchange but the maximum's.
//
// P is rounded to the 16-bit type for the matrix instruction (half a step
// relative to each weight, which is lifted into the type's range); m, l, S and O
// stay fp32.
//
// Bound by reading the cache.  64 rows of 1 to 32768 positions, 64 heads on 8,
// bf16: 744 us, 5.6 TB/s where a plain read reaches 6.4 (e4m3: 397, 5.2); 4 rows
// of 8192: 24.6 us, 5.5 TB/s; 64 rows of 2048 chosen positions, 40 heads on 4:
// 47.7 us, 5.7 TB/s of scattered rows, e4m3 34, 4.0 TB/s; 32 x 2 rows of 16384
// positions, 64 heads on 4: 215 us, 5.0 TB/s, e4m3 114, 4.7.
// ---------------------------------------------------------------------------
constexpr int kAttnBlock = 256;
constexpr int kTok = 32;  // tokens of a wavefront's tile

__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) x = fmaxf(x, __shfl_xor(x, off));
  return x;
}

// The longest row of a group, all lanes.
__device__ __forceinline__ int32_t group_length(const AttnParams& p, int32_t r0, int64_t most, int lane) {
  int32_t n = 0;
  for (int32_t j = lane; j < p.group_rows; j += 64) {
    const int32_t x = clamp_to(p.a.lengths[r0 + j], most);
    n = x > n ? x : n;
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) {
    const int32_t x = __shfl_xor(n, off);
    n = x > n ? x : n;
  }
  return __builtin_amdgcn_readfirstlane(n);
}

template <bool F8, int D>
struct KvTile {
  static constexpr int KL = F8 ? D / 64 : D / 32;                // 16-byte key loads per token of a lane group
  static constexpr int VW = F8 ? D / 64 : D / 32;                // words of a lane's value dims
  u32x4 k[2][KL];
  uint32_t v[8][VW];
};

// off: place of the tile's token `lane % 32`, in elements (-1: none; the load
// then takes the pool's first token, and the tile's mask leaves it out).
template <bool F8, int D>
__device__ __forceinline__ void load_keys(KvTile<F8, D>& b, const char* k, int64_t off, int lane) {
  constexpr int SZ = F8 ? 1 : 2;
  const int64_t at = off < 0 ? 0 : off * SZ;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const char* kp = k + shfl64(at, u * 16 + (lane & 15)) + (lane >> 4) * 16;
#pragma unroll
    for (int i = 0; i < KvTile<F8, D>::KL; ++i) b.k[u][i] = *(const u32x4*)(kp + i * 64);
  }
}
template <bool F8, int D>
__device__ __forceinline__ void load_values(KvTile<F8, D>& b, const char* v, int64_t off, int lane) {
  using Tile = KvTile<F8, D>;
  constexpr int SZ = F8 ? 1 : 2;
  const int64_t at = off < 0 ? 0 : off * SZ;
#pragma unroll
  for (int t = 0; t < 8; ++t) {
    const char* vp = v + shfl64(at, (t >> 2) * 16 + (lane >> 4) * 4 + (t & 3)) + (lane & 15) * (Tile::VW * 4);
    if constexpr (Tile::VW == 4) {
      const u32x4 x = *(const u32x4*)vp;
#pragma unroll
      for (int i = 0; i < 4; ++i) b.v[t][i] = x[i];
    } else if constexpr (Tile::VW == 2) {
      const u32x2 x = *(const u32x2*)vp;
      b.v[t][0] = x[0], b.v[t][1] = x[1];
    } else {
      b.v[t][0] = *(const uint32_t*)vp;
    }
  }
}

// What a row reads: all its positions (kOne: a sequence has one row; kRows:
// several, which share the reads but may end at different places), or chosen
// ones.
enum { kOne, kRows, kChosen };

template <bool B>
struct Flag {
  static constexpr bool value = B;
};

template <typename T, bool F8, int D, int MODE, int NT>
__global__ void __launch_bounds__(kAttnBlock, NT == 1 && MODE != kRows ? 3 : 2) attn_kernel(AttnParams p) {
  constexpr bool CHOSEN = MODE == kChosen;
  constexpr int KS = D / 32;  // matrix steps over the key dims
  constexpr int VD = D / 16;  // value dims of a lane
  constexpr int SZ = F8 ? 1 : 2;
  constexpr int LD = D + 4;   // row pitch of the joined outputs in LDS
  __shared__ float so[4][16][LD];
  __shared__ float sm[4][16], sl[4][16];
  const paged_attention_args& a = p.a;
  const int lane = threadIdx.x & 63, col16 = lane & 15, g = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);

  Work work;
  if (!work_of<CHOSEN>(blockIdx.x, (uint32_t)(a.num_kv_heads * p.col_tiles), (uint32_t)p.groups, (uint32_t)p.most, &work)) return;
  const int64_t most = table_tokens(a.table_width, a.page_size);
  const int32_t part = work.part;
  const int32_t group = CHOSEN ? work.group : by_length(a, work.group, p.groups, p.group_rows, most, lane);
  const int32_t kvh = work.unit % a.num_kv_heads, tile = work.unit / a.num_kv_heads;
  const int32_t r0 = group * p.group_rows;
  const int32_t heads_per = a.num_heads / a.num_kv_heads;

  const int32_t n = CHOSEN ? a.num_chosen : group_length(p, r0, most, lane);
  const Split sp = split_of(n, p.most, p.least, p.unit);
  if (part >= sp.parts) return;
  const int32_t begin = part * sp.chunk;
  const int32_t end = n - begin < sp.chunk ? n : begin + sp.chunk;

  // Columns: (row of the group, head of the key-value head).
  int32_t collen[NT], colrow[NT];
  u32x4 q[NT][KS];
  int32_t shortest = INT32_MAX, jlo = INT32_MAX, jhi = -1;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int32_t c = (tile * NT + t) * 16 + col16;
    const bool real = c < p.group_rows * heads_per;
    const int32_t j = real ? c / heads_per : 0;
    collen[t] = real ? clamp_to(a.lengths[r0 + j], most) : 0;
    colrow[t] = real ? j : -1;
    if (real) {
      shortest = collen[t] < shortest ? collen[t] : shortest;
      jlo = j < jlo ? j : jlo;
      jhi = j > jhi ? j : jhi;
    }
    // Columns past the last one compute with the first head and see nothing.
    const int32_t head = kvh * heads_per + (real ? c - j * heads_per : 0);
    const char* qp = (const char*)a.q + 2 * ((int64_t)(r0 + j) * a.q_row_stride + (int64_t)head * a.q_head_stride);
#pragma unroll
    for (int i = 0; i < KS; ++i) {
      // The dims that the lane's key words hold at matrix step i.
      const int dim = F8 ? (i >> 1) * 64 + g * 16 + (i & 1) * 8 : i * 32 + g * 8;
      q[t][i] = *(const u32x4*)(qp + 2 * dim);
    }
  }
#pragma unroll
  for (int off = 8; off > 0; off >>= 1) {
    const int32_t x = __shfl_xor(shortest, off), y = __shfl_xor(jlo, off), z = __shfl_xor(jhi, off);
    shortest = x < shortest ? x : shortest;
    jlo = y < jlo ? y : jlo;
    jhi = z > jhi ? z : jhi;
  }
  shortest = __builtin_amdgcn_readfirstlane(shortest);
  jlo = __builtin_amdgcn_readfirstlane(jlo);
  jhi = __builtin_amdgcn_readfirstlane(jhi);

  const float scale = p.scale_log2 * (F8 && a.k_scales != nullptr ? a.k_scales[kvh] : 1.0f);
  const char* kbase = (const char*)a.k + (int64_t)kvh * a.head_stride * SZ;
  const char* vbase = (const char*)a.v + (int64_t)kvh * a.head_stride * SZ;
  const int32_t* table = a.block_table + (int64_t)(r0 / a.next_n) * a.table_stride;
  const int32_t* chosen = CHOSEN ? a.chosen + (int64_t)r0 * a.chosen_stride : nullptr;
  const int32_t seen = CHOSEN ? clamp_to(a.lengths[r0], most) : 0;

  // Places of the lane's tokens (both halves of the wavefront hold the same
  // 32); a part is never empty unless its row is.
  constexpr int kStep = 4 * kTok;
  Places<CHOSEN> places{table, chosen, a.page_stride, a.token_stride, p.page, a.num_pages, seen, end, kStep};

  float m[NT], l[NT];
  f32x4 o[NT][VD];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    m[t] = -INFINITY, l[t] = 0.0f;
#pragma unroll
    for (int d = 0; d < VD; ++d) o[t][d] = f32x4{0, 0, 0, 0};
  }

  // One tile: `next` is called when its keys are no longer needed.  ragged:
  // some column ends inside the tile, or before it.
  KvTile<F8, D> b;
  auto compute = [&](uint32_t valid, int32_t t0, auto is_ragged, auto&& next) {
    constexpr bool ragged = decltype(is_ragged)::value;
    const bool whole = valid == 0xffffffffu;  // bit i: token i is in the cache and inside the part
    f32x4 s[NT][2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      u32x4 kk[KS];
      if constexpr (F8) {
#pragma unroll
        for (int i = 0; i < KS; ++i) kk[i] = widen<T>(u32x2{b.k[u][i >> 1][(i & 1) * 2], b.k[u][i >> 1][(i & 1) * 2 + 1]});
      } else {
#pragma unroll
        for (int i = 0; i < KS; ++i) kk[i] = b.k[u][i];
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        s[t][u] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < KS; ++i) s[t][u] = T::mfma16(kk[i], q[t][i], s[t][u]);
      }
    }
    // The barriers keep the scheduler from starting the next loads into further
    // registers before these are free.
    __builtin_amdgcn_sched_barrier(0);
    next();
    __builtin_amdgcn_sched_barrier(0);
    u32x4 pk[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = s[t][e >> 2][e & 3] * scale;
      if (!whole || ragged) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int i = (e >> 2) * 16 + g * 4 + (e & 3);
          const bool in = ((valid >> i) & 1u) != 0 && (!ragged || t0 + i < collen[t]);
          x[e] = in ? x[e] : -INFINITY;
        }
      }
      float mt = x[0];
#pragma unroll
      for (int e = 1; e < 8; ++e) mt = fmaxf(mt, x[e]);
      mt = max_xor32(max_xor16(mt));
      if (__builtin_amdgcn_ballot_w64(mt > m[t]) != 0) {
        const float mn = fmaxf(m[t], mt);
        const float by = mn == m[t] ? 1.0f : exp2_fast(m[t] - mn);
        m[t] = mn;
        l[t] *= by;
#pragma unroll
        for (int d = 0; d < VD; ++d) o[t][d] *= by;
      }
      const float ref = m[t] == -INFINITY ? 0.0f : m[t] - T::kLift;
      float sum = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] = exp2_fast(x[e] - ref);
        sum += x[e];
      }
      l[t] += sum;
      pk[t] = u32x4{T::pack(x[0], x[1]), T::pack(x[2], x[3]), T::pack(x[4], x[5]), T::pack(x[6], x[7])};
    }
    // Values as 16-bit pairs of dims.  Tokens that do not count become zeros
    // below: their places may hold NaN, which a weight of zero would not stop.
    uint32_t v[8][VD / 2];
#pragma unroll
    for (int e = 0; e < 8; ++e)
#pragma unroll
      for (int i = 0; i < VD / 2; ++i) {
        if constexpr (F8)
          v[e][i] = (i & 1) ? T::template from_e4m3<true>(b.v[e][i >> 1]) : T::template from_e4m3<false>(b.v[e][i >> 1]);
        else
          v[e][i] = b.v[e][i];
      }
    // One matrix step for value dim d of each lane's block; the words of
    // `keep` are all ones where the pair's tokens count.
    auto accumulate = [&](int d, u32x4 keep, int t) {
      const uint32_t sel = (d & 1) ? 0x07060302u : 0x05040100u;
      const int i = d >> 1;
      u32x4 vt = {__builtin_amdgcn_perm(v[1][i], v[0][i], sel), __builtin_amdgcn_perm(v[3][i], v[2][i], sel),
                  __builtin_amdgcn_perm(v[5][i], v[4][i], sel), __builtin_amdgcn_perm(v[7][i], v[6][i], sel)};
      return T::mfma16(vt & keep, pk[t], o[t][d]);
    };
    auto keep_words = [&](uint32_t bits) {  // bits: the tile's tokens that count
      u32x4 k;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = (e >> 1) * 16 + g * 4 + (e & 1) * 2;
        k[e] = ((bits >> i) & 1u ? 0x0000ffffu : 0u) | ((bits >> i) & 2u ? 0xffff0000u : 0u);
      }
      return k;
    };
    if constexpr (!ragged) {
      u32x4 keep = {~0u, ~0u, ~0u, ~0u};
      if (!whole) keep = keep_words(valid);
#pragma unroll
      for (int d = 0; d < VD; ++d)
#pragma unroll
        for (int t = 0; t < NT; ++t) o[t][d] = accumulate(d, keep, t);
      return;
    }
    // Rows of the sequence end at different places in this tile: one row's
    // columns at a time, with the tokens that the row does not see as zeros.
    for (int32_t j = jlo; j <= jhi; ++j) {
      const int32_t left = clamp_to(a.lengths[r0 + j], most) - t0;
      if (left <= 0) continue;  // its weights in this tile are zeros
      const u32x4 keep = keep_words(left >= 32 ? valid : valid & ((1u << left) - 1u));
#pragma unroll
      for (int d = 0; d < VD; ++d)
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const f32x4 x = accumulate(d, keep, t);
#pragma unroll
          for (int i = 0; i < 4; ++i) o[t][d][i] = colrow[t] == j ? x[i] : o[t][d][i];
        }
    }
  };

  // The next tile's keys are loaded once this one's scores are formed, its
  // values once this one's are summed: the registers of one tile, and loads in
  // flight all the time.  (Two whole tiles in registers left room for two
  // wavefronts on a SIMD instead of three.)
  int32_t t = begin + w * kTok;
  if (t < end) {
    places.start(t + (lane & 31));
    int64_t off = places.take();
    load_keys<F8, D>(b, kbase, off, lane);
    load_values<F8, D>(b, vbase, off, lane);
    bool more = true;
    auto step = [&](auto is_ragged) {
      const uint32_t valid = (uint32_t)__builtin_amdgcn_ballot_w64(off >= 0);
      more = t + kStep < end;
      compute(valid, t, is_ragged, [&] {
        if (more) {
          off = places.take();
          load_keys<F8, D>(b, kbase, off, lane);
        }
      });
      if (!more) return;
      __builtin_amdgcn_sched_barrier(0);
      load_values<F8, D>(b, vbase, off, lane);
      t += kStep;
    };
    // Ragged tiles come last and in a loop of their own: the copies of the
    // sums that they need cost the others registers and spills (32 x 2 rows of
    // 16384 positions, 64 heads on 4, a call: 329 us against 229, e4m3 240 against 129).
    if constexpr (MODE == kRows) {
      while (more && t + kTok <= shortest) step(Flag<false>{});
      while (more) step(Flag<true>{});
    } else {
      while (more) step(Flag<false>{});
    }
  }

  const float v_scale = F8 && a.v_scales != nullptr ? a.v_scales[kvh] : 1.0f;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    l[t] += __shfl_xor(l[t], 16);
    l[t] += __shfl_xor(l[t], 32);
    if (t > 0) __syncthreads();
    if (lane < 16) sm[w][lane] = m[t], sl[w][lane] = l[t];
    __syncthreads();
    const float top = fmaxf(fmaxf(sm[0][col16], sm[1][col16]), fmaxf(sm[2][col16], sm[3][col16]));
    const float by = (m[t] == top ? 1.0f : exp2_fast(m[t] - top)) * v_scale;
#pragma unroll
    for (int d = 0; d < VD; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i) so[w][col16][(g * 4 + i) * VD + d] = o[t][d][i] * by;
    __syncthreads();
    for (int32_t i = threadIdx.x; i < 16 * (D / 2); i += kAttnBlock) {
      const int32_t c16 = i / (D / 2), dim = (i - c16 * (D / 2)) * 2;
      const int32_t c = (tile * NT + t) * 16 + c16;
      if (c >= p.group_rows * heads_per) continue;
      const int32_t j = c / heads_per;
      const int64_t at = (int64_t)(r0 + j) * a.num_heads + kvh * heads_per + (c - j * heads_per);
      const float cm = fmaxf(fmaxf(sm[0][c16], sm[1][c16]), fmaxf(sm[2][c16], sm[3][c16]));
      float sum = 0.0f, x = 0.0f, y = 0.0f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        sum += sl[k][c16] * (sm[k][c16] == cm ? 1.0f : exp2_fast(sm[k][c16] - cm));
        x += so[k][c16][dim];
        y += so[k][c16][dim + 1];
      }
      if (sp.parts == 1) {
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        *(uint32_t*)((uint16_t*)a.out + at * D + dim) = T::pack(x * inv, y * inv);
        if (dim == 0 && a.lse != nullptr) a.lse[at] = sum == 0.0f ? -INFINITY : (cm - T::kLift + __log2f(sum)) * kLn2;
      } else {
        const int64_t pi = at * p.most + part;
        *(float2*)(p.part_out + pi * D + dim) = float2{x, y};
        if (dim == 0) p.part_stat[pi] = float2{cm - T::kLift, sum};
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Join: out = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i over a row's
// parts, M the largest m_i; rows of one part were finished by the attention
// kernel.
//
// Many parts (MANY): a workgroup for each (row, head); D / 4 threads cover the
// dims, the groups of threads beside each other take every G-th part and meet
// in LDS, so a row of many parts is not a chain of as many reads (20 heads of
// 512 dims in 64 parts: 5.8 us, 13.7 us with one wavefront each).  Up to four
// parts: one wavefront for each (row, head) and no LDS (8192 of them, two
// parts: 9.1 us, 13.7 us with a workgroup each).
// ---------------------------------------------------------------------------
template <typename T, int D, bool MANY>
__global__ void __launch_bounds__(kAttnBlock) join_kernel(AttnParams p) {
  constexpr int TD = MANY ? D / 4 : 64;     // threads of a (row, head) along the dims
  constexpr int E = D / TD;                 // dims of a thread
  constexpr int G = MANY ? kAttnBlock / TD : 1;
  __shared__ float acc[MANY ? G : 1][MANY ? D : 1];
  __shared__ float weight[MANY ? 128 : 1];
  const paged_attention_args& a = p.a;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t at = MANY ? blockIdx.x : (int64_t)blockIdx.x * (kAttnBlock / 64) + w;
  if (at >= (int64_t)a.num_rows * a.num_heads) return;
  const int32_t row = (int32_t)(at / a.num_heads);
  const int64_t most = table_tokens(a.table_width, a.page_size);
  const int32_t n = a.chosen != nullptr ? a.num_chosen : group_length(p, row / p.group_rows * p.group_rows, most, lane);
  const Split sp = split_of(n, p.most, p.least, p.unit);
  if (sp.parts == 1) return;
  // Every wavefront forms the weights: at most 128, two a lane.
  const float2* stat = p.part_stat + at * p.most;
  const float2 s0 = lane < sp.parts ? stat[lane] : float2{-INFINITY, 0.0f};
  const float2 s1 = MANY && lane + 64 < sp.parts ? stat[lane + 64] : float2{-INFINITY, 0.0f};
  const float top = wave_max(fmaxf(s0.x, s1.x));
  const float w0 = s0.x == top ? 1.0f : exp2_fast(s0.x - top), w1 = s1.x == top ? 1.0f : exp2_fast(s1.x - top);
  float sum = s0.y * w0 + s1.y * w1;
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off);
  const int g = MANY ? (int)threadIdx.x / TD : 0, d = MANY ? (int)threadIdx.x % TD : lane;
  const float* po = p.part_out + at * p.most * D + d * E;
  float o[E] = {};
  if constexpr (MANY) {
    if (w == 0) weight[lane] = w0, weight[lane + 64] = w1;
    __syncthreads();
#pragma unroll 8
    for (int32_t i = g; i < sp.parts; i += G) {
      const f32x4 x = *(const f32x4*)(po + (int64_t)i * D);
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] += weight[i] * x[e];
    }
  } else {
#pragma unroll 4
    for (int32_t i = 0; i < sp.parts; ++i) {
      const float by = __shfl(w0, i);
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] += by * po[(int64_t)i * D + e];
    }
  }
  if constexpr (MANY) {
#pragma unroll
    for (int e = 0; e < E; ++e) acc[g][d * E + e] = o[e];
    __syncthreads();
    if (threadIdx.x >= TD) return;
#pragma unroll
    for (int k = 1; k < G; ++k)
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] += acc[k][d * E + e];
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  uint16_t* out = (uint16_t*)a.out + at * D + d * E;
  if constexpr (E == 1) {
    *out = (uint16_t)T::pack(o[0] * inv, 0.0f);
  } else {
#pragma unroll
    for (int e = 0; e < E; e += 2) *(uint32_t*)(out + e) = T::pack(o[e] * inv, o[e + 1] * inv);
  }
  if (d == 0 && a.lse != nullptr) a.lse[at] = sum == 0.0f ? -INFINITY : (top + __log2f(sum)) * kLn2;
}

namespace {

template <typename T, bool F8, int D, int MODE>
const void* attn_tiles(int tiles) {
  return tiles == 2 ? (const void*)&attn_kernel<T, F8, D, MODE, 2> : (const void*)&attn_kernel<T, F8, D, MODE, 1>;
}
template <typename T, bool F8, int D>
const void* attn_modes(int mode, int tiles) {
  return mode == kOne ? attn_tiles<T, F8, D, kOne>(tiles)
       : mode == kRows ? attn_tiles<T, F8, D, kRows>(tiles) : attn_tiles<T, F8, D, kChosen>(tiles);
}
template <typename T, bool F8>
const void* attn_dims(int head_dim, int mode, int tiles) {
  if (head_dim == 64) return attn_modes<T, F8, 64>(mode, tiles);
  if (head_dim == 128) return attn_modes<T, F8, 128>(mode, tiles);
  return nullptr;
}
template <typename T>
const void* join_dims(int head_dim, bool many) {
  switch (head_dim) {
    case 64: return many ? (const void*)&join_kernel<T, 64, true> : (const void*)&join_kernel<T, 64, false>;
    case 128: return many ? (const void*)&join_kernel<T, 128, true> : (const void*)&join_kernel<T, 128, false>;
    case 256: return many ? (const void*)&join_kernel<T, 256, true> : (const void*)&join_kernel<T, 256, false>;
    case 512: return many ? (const void*)&join_kernel<T, 512, true> : (const void*)&join_kernel<T, 512, false>;
    default: return nullptr;
  }
}

}  // namespace

const void* attn_kernel_ptr(int dtype, int store, int head_dim, bool chosen, int rows, int tiles) {
  const int mode = chosen ? kChosen : rows > 1 ? kRows : kOne;
  if (dtype == PAGED_BF16)
    return store == PAGED_E4M3 ? attn_dims<Bf16, true>(head_dim, mode, tiles)
                               : attn_dims<Bf16, false>(head_dim, mode, tiles);
  return store == PAGED_E4M3 ? attn_dims<Fp16, true>(head_dim, mode, tiles)
                             : attn_dims<Fp16, false>(head_dim, mode, tiles);
}

const void* join_kernel_ptr(int dtype, int head_dim, bool many) {
  return dtype == PAGED_BF16 ? join_dims<Bf16>(head_dim, many) : join_dims<Fp16>(head_dim, many);
}

}  // namespace rrt
