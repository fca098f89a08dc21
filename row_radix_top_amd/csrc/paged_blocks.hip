// Bounds of a cache's pages in 8 bits, and the choice of pages by them.

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
// each dim meet over the lanes at the end.  Bound by reading the keys.
//
// Which page: sequence s gets floor(starts[s] / P) + 2 s as its first unit, and so
// at least floor(new / P) + 2 of them, as many as `new` tokens at any offset may
// touch; the search for the unit's sequence probes 64 at a time.
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
  if (fresh <= 0 || len == 0) return;
  const int32_t held = fresh < len ? len - (int32_t)fresh : 0;
  const int64_t j = (int64_t)divide((uint32_t)held, p.page) + (u - first_unit(s));
  if (j < 0 || j * a.page_size >= len) return;
  const int32_t page = a.block_table[(int64_t)s * a.table_stride + j];
  if ((uint32_t)page >= (uint32_t)a.num_pages) return;
  const int32_t left = len - (int32_t)j * a.page_size, count = left < a.page_size ? left : a.page_size;

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
// one product of 8-bit numbers of length 2 D: S[block][head] = bounds x queries,
// 16 blocks x 16 columns a matrix instruction, 64 of the 2 D at a time.  The
// order of those 64 is the same for both operands, so each lane loads 16
// consecutive bytes of a page's bounds as they lie.  Sums are whole numbers
// below 2^21, exact in fp32.
//
// The columns of a 16 are the heads of 16 / hp2 rows of a sequence, hp2 the power
// of two from heads a key-value head up (more than 16 heads: one row, several
// sixteens), so a row's largest head is a maximum over neighbouring lanes.
//
// Fused: a workgroup scores all blocks of its rows into LDS, then each wavefront
// picks for its rows.  Split: many workgroups score into the workspace and a
// second launch picks.
//
// The pick: keys in registers (fp32 bits in order), bit by bit the largest
// threshold that at least K reach, counted by ballots on the scalar unit, and
// ranks by ballots again.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t b = __float_as_uint(x);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}

// n scores (n > k) to the k best's indices, ascending.  TEAM wavefronts (the
// workgroup's, or one alone) hold 64 KEYS scores each.
template <int TEAM, int KEYS>
__device__ __forceinline__ void pick(const float* scores, int32_t n, int32_t k, int32_t* out, int w, int lane, int32_t* s) {
  uint32_t key[KEYS];
  const int32_t base = w * KEYS * 64 + lane;
#pragma unroll
  for (int i = 0; i < KEYS; ++i) key[i] = base + i * 64 < n ? order_of(scores[base + i * 64]) : 0u;
  auto total = [&](int32_t x) -> int32_t {  // over the team
    if constexpr (TEAM == 1) return x;
    if (lane == 0) s[w] = x;
    __syncthreads();
    int32_t sum = 0;
#pragma unroll
    for (int i = 0; i < TEAM; ++i) sum += s[i];
    __syncthreads();
    return sum;
  };
  uint32_t t = 0;
  for (int bit = 31; bit >= 0; --bit) {
    const uint32_t want = t | 1u << bit;
    int32_t c = 0;
#pragma unroll
    for (int i = 0; i < KEYS; ++i) c += __builtin_popcountll(__builtin_amdgcn_ballot_w64(key[i] >= want));
    c = total(c);
    if (c >= k) t = want;
    if (c == k) break;
  }
  int32_t above = 0, level = 0;
#pragma unroll
  for (int i = 0; i < KEYS; ++i) {
    above += __builtin_popcountll(__builtin_amdgcn_ballot_w64(key[i] > t));
    level += __builtin_popcountll(__builtin_amdgcn_ballot_w64(key[i] == t));
  }
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

// One row's choice from its scores, by one wavefront.
__device__ __forceinline__ void pick_row(const SelectParams& p, const float* scores, int32_t n, int32_t* out, int lane) {
  const int32_t k = p.a.num_blocks;
  if (n <= k) {
    for (int32_t i = lane; i < k; i += 64) out[i] = i < n ? i : -1;
  } else if (n <= 256) {
    pick<1, 4>(scores, n, k, out, 0, lane, nullptr);
  } else if (n <= 1024) {
    pick<1, 16>(scores, n, k, out, 0, lane, nullptr);
  } else {
    pick<1, 64>(scores, n, k, out, 0, lane, nullptr);
  }
}

template <int CTRL>
__device__ __forceinline__ float max_dpp(float x) {
  return fmaxf(x, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xf, 0xf, true)));
}
// The largest over aligned groups of `wide` (1, 2, 4, 8, 16) lanes.
__device__ __forceinline__ float group_max(float x, int wide) {
  if (wide > 1) x = max_dpp<0xb1>(x);    // lanes 1 0 3 2
  if (wide > 2) x = max_dpp<0x4e>(x);    // 2 3 0 1
  if (wide > 4) x = max_dpp<0x141>(x);   // mirrored within 8
  if (wide > 8) x = max_dpp<0x140>(x);   // within 16
  return x;
}

template <typename T, int D, int NT, bool SPLIT>
__global__ void __launch_bounds__(kBlocksBlock) select_kernel(SelectParams p) {
  constexpr int QS = D / 64, KS = 2 * QS;  // steps over the dims, and over both bounds
  extern __shared__ __align__(16) float scores[];
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
  const int32_t row_cols = per <= 16 ? p.hp2 : 16;

  int32_t have = 0;  // of the unit's longest row
  for (int32_t j = 0; j < rows; ++j) {
    const int32_t n = blocks_of(p, r0 + j);
    have = n > have ? n : have;
  }
  int32_t t0 = 0, t1 = (have + 15) / 16;
  if constexpr (SPLIT) {
    t0 = part * p.part_tiles;
    t1 = t1 - t0 < p.part_tiles ? t1 : t0 + p.part_tiles;
    if (t0 >= t1) return;
  }
  const int32_t* table = a.block_table + (int64_t)seq * a.table_stride;
  const char* bounds = (const char*)a.bounds + (int64_t)kvh * a.bounds_head_stride;
  auto score_at = [&](int32_t j) -> float* {
    if constexpr (SPLIT) return p.scores + ((int64_t)(r0 + j) * a.num_kv_heads + kvh) * p.pitch;
    else return scores + (int64_t)j * p.pitch;
  };

  for (int32_t pass = 0; pass < passes; ++pass) {
    u32x4 q[NT][KS];
    float by[NT];
    int32_t col_row[NT], col_have[NT];
    bool head_real[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int32_t j = per <= 16 ? (t * 16 + c16) / row_cols : 0;
      const int32_t head = per <= 16 ? c16 % row_cols : (pass * NT + t) * 16 + c16;
      col_row[t] = j < rows ? j : -1;
      head_real[t] = head < per && j < rows;
      col_have[t] = j < rows ? blocks_of(p, r0 + j) : 0;
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
      by[t] = top * kOver127;
      const float div = by[t] == 0.0f ? 1.0f : by[t];
#pragma unroll
      for (int i = 0; i < QS; ++i)
#pragma unroll
        for (int e4 = 0; e4 < 4; ++e4) {
          uint32_t up = 0, down = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            int v = (int)fminf(fmaxf(rintf(x[i][e4 * 4 + e] / div), -127.0f), 127.0f);
            up |= (uint32_t)(v > 0 ? v : 0) << (8 * e);
            down |= (uint32_t)((v < 0 ? v : 0) & 0xff) << (8 * e);
          }
          q[t][i][e4] = up;
          q[t][QS + i][e4] = down;
        }
    }

    // A tile's pages are looked up two tiles ahead of it, its bounds one.
    auto page_at = [&](int32_t tile) -> int32_t {
      const int32_t b = tile * 16 + c16;
      return b < have ? table[b] : -1;
    };
    u32x4 next[KS];
    float next_scale = 0.0f;
    auto fetch = [&](int32_t page) {
      const int64_t at = (uint32_t)page < (uint32_t)a.num_pages ? page : 0;
      const char* from = bounds + at * a.bounds_page_stride + g * 16;
#pragma unroll
      for (int i = 0; i < KS; ++i) next[i] = *(const u32x4*)(from + i * 64);
      next_scale = a.scales[at * a.scales_stride + kvh];
    };
    constexpr int W = kBlocksBlock / 64;
    int32_t tile = t0 + w;
    int32_t page = tile < t1 ? page_at(tile) : -1;
    int32_t page_next = tile + W < t1 ? page_at(tile + W) : -1;
    if (tile < t1) fetch(page);
    for (; tile < t1; tile += W) {
      u32x4 b[KS];
#pragma unroll
      for (int i = 0; i < KS; ++i) b[i] = next[i];
      const float scale = next_scale;
      const uint32_t valid = (uint32_t)__builtin_amdgcn_ballot_w64((uint32_t)page < (uint32_t)a.num_pages);
      page = page_next;
      page_next = tile + 2 * W < t1 ? page_at(tile + 2 * W) : -1;
      if (tile + W < t1) fetch(page);
      float best[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        i32x4 sum = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < KS; ++i)
          sum = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, b[i]), __builtin_bit_cast(i32x4, q[t][i]),
                                                      sum, 0, 0, 0);
        float y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          y[i] = group_max(head_real[t] ? (float)sum[i] * by[t] : -INFINITY, row_cols);
          if (per > 16) best[i] = fmaxf(best[i], y[i]);
        }
        if (per > 16 && t + 1 < NT) continue;
        f32x4 z;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int blk = g * 4 + i;
          const float v = (per > 16 ? best[i] : y[i]) * __shfl(scale, blk);
          const int32_t at = tile * 16 + blk;
          const bool always = at < a.first || at >= col_have[per > 16 ? 0 : t] - a.last;
          z[i] = ((valid >> blk) & 1u) == 0 ? -INFINITY : always ? INFINITY : v;
        }
        const int32_t j = per > 16 ? 0 : col_row[t];
        if (j < 0 || c16 % row_cols != 0) continue;
        f32x4* to = (f32x4*)(score_at(j) + tile * 16 + g * 4);
        if (pass > 0) {
          const f32x4 old = *to;
#pragma unroll
          for (int i = 0; i < 4; ++i) z[i] = fmaxf(z[i], old[i]);
        }
        *to = z;
      }
    }
  }
  if constexpr (SPLIT) return;
  __syncthreads();
  for (int32_t j = w; j < rows; j += kBlocksBlock / 64)
    pick_row(p, score_at(j), blocks_of(p, r0 + j), a.blocks + ((int64_t)(r0 + j) * a.num_kv_heads + kvh) * a.num_blocks, lane);
}

// The choice of one row and key-value head from scores in the workspace.
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
