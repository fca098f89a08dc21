// The expanded form of latent attention: keys and values of every head formed
// from the latent vectors of the context, then causal attention over them.

#include <type_traits>

#include "paged_device.hpp"

namespace rrt {

// ---------------------------------------------------------------------------
// Two kernels (and a join where few rows share out their contexts).  `expand`
// forms k_h = W_k,h c and v_h = W_v,h c for every context token and head (2 DC
// 256 flop each) and leaves them in the workspace in fragment order: 1 KB blocks
// that are, lane by lane, the operands that the attention's matrix instructions
// take.  `prefill` streams them through LDS with plain linear copies, and no
// operand needs a shuffle, a transpose or a swizzle there.
//
// A context tile is 64 tokens.  With tb = token / 32, half = lane / 32:
//   key block (tb, s):   lane holds token tb*32 + lane % 32, dims s*16 + half*8 .. +8
//   value block (tb, ks, db): lane holds dim db*32 + lane % 32, tokens
//     tb*32 + ks*16 + half*4 + {0..3, 8..11}: the tokens whose weights the lane
//     holds after S^T = K Q^T, so the weights go from one product into the
//     next without leaving the lane.
// Expanded values are rounded to the 16-bit type, as a program that keeps them
// would (one past fp16's range is an infinity).  Keys, which a score of 20 takes
// twenty times as they are off, are rounded to fp16 for bf16 too, at the same
// rate and eight times closer, and with them rope parts and queries.  The range
// is that of fp32 all the same: a token's key, its rope part and a row's queries
// are kept times powers of two wherever their size asks for it (keep_exp), which
// costs tiles of ordinary sizes nothing (8192 tokens x 32 heads, a call: 807 us;
// 899 with one small token in its midst, 1082 with small keys everywhere).
// A key's rounding moves a score by at most u sum |q k| over the 128 formed dims,
// u = 2^-11.  A row of many tokens with scores alike averages that away, as
// 1 / sqrt(n), so the keys of a sequence's first kExactTiles tiles come with what
// their rounding left, as a second fp16 number, and score with both (for rows of
// few tokens all that they see).  A key behind them that outweighs a row's
// others is averaged with nothing: the log-sum-exp is then off by up to 1.2e-3
// at a score of 20, against 6e-6 among the first.  The weights of the first
// kExactWeights tiles are taken in two parts too: an output of few tokens is off
// by 1.35 times its own rounding so, 1.55 times without.
// 8192 tokens x 32 heads, bf16, attention side by side: 703 us with bf16 keys, 721
// with fp16 (what fp16's products draw of the power limit).  With bf16
// keys it was 634 us without second parts, 680 with those of 16 tiles' keys,
// 729 with 32 tiles', 872 with all.
//
// A scale of the cache multiplies the scores, not the keys.
// ---------------------------------------------------------------------------
constexpr int kExpandBlock = 256;
constexpr int kHead = PAGED_HEAD_DIM;
constexpr int kRopeDim = PAGED_ROPE_DIM;
constexpr int kBlock16 = 1024;                              // bytes of a block
constexpr int kExactWeights = 4;                            // tiles whose weights come in two parts
constexpr int kKeyTile = 16 * kBlock16, kRopeTile = 8 * kBlock16, kValueTile = 16 * kBlock16;

using lds_u32x4 = __attribute__((address_space(3))) u32x4;

__device__ __forceinline__ uint32_t lds_at(const void* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const char*)p;
}
__device__ __forceinline__ u32x4 lds_read16(uint32_t at) { return *(lds_u32x4*)at; }
// 16 bytes from each lane's address to LDS at `to` (wave uniform) + 16 x lane.
// No register is written: wait_loads() alone waits for it.
__device__ __forceinline__ void load_to_lds(const char* from, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(__builtin_amdgcn_readfirstlane(to)), "v"(from) : "memory", "m0");
}
__device__ __forceinline__ void load_to_lds(const char* from, uint32_t offset, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(__builtin_amdgcn_readfirstlane(to)), "v"(offset), "s"(from) : "memory", "m0");
}
__device__ __forceinline__ void wait_loads() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// keep_exp: a token's key (or rope part) is kept in fp16 times 2^-this, given its
// largest magnitude: 0 for the ordinary, 2^-8 to 2^15 (and for what is not finite),
// else what makes the largest as large as fp16 takes.  A dim below 2^-30 of its token's
// largest loses bits, and is lost in a score's fp32 sum unless the queries are as
// uneven the other way.
constexpr int kKeepLeast = -112, kKeepMost = 113;
__device__ __forceinline__ int keep_exp(float most) {
  if (!(most > 0.0f && most < INFINITY) || (most >= 0.00390625f && most <= 32768.0f)) return 0;
  const int e = __builtin_amdgcn_frexp_expf(most) - 15;
  return e < kKeepLeast ? kKeepLeast : e > kKeepMost ? kKeepMost : e;
}

__device__ __forceinline__ int32_t context_of(const PrefillParams& p, int32_t s) {
  return clamp_to(p.a.lengths[s], table_tokens(p.a.table_width, p.a.page_size));
}
__device__ __forceinline__ int32_t tiles_of(int32_t n, int32_t per) { return (int32_t)(((int64_t)n + per - 1) / per); }

// Inclusive sums over the wavefront; they stop at 2^31 - 1, so that lengths
// that do not fit the workspace by far still lie past it.
__device__ __forceinline__ int32_t scan_up(int32_t x, int lane) {
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int32_t y = __shfl_up(x, off);
    if (lane >= off) x = __builtin_elementwise_add_sat(x, y);
  }
  return x;
}

// The sequence that context tile `tile` belongs to and the tiles before that
// sequence; -1 if the tile lies past the last sequence.  All lanes take part.
__device__ __forceinline__ int32_t sequence_of_tile(const PrefillParams& p, int32_t tile, int lane, int32_t* before) {
  int32_t base = 0;
  for (int32_t s0 = 0; s0 < p.a.num_seqs; s0 += 64) {
    const int32_t mine = s0 + lane < p.a.num_seqs ? tiles_of(context_of(p, s0 + lane), kCtxTile) : 0;
    const int32_t upto = __builtin_elementwise_add_sat(base, scan_up(mine, lane));
    const uint64_t past = __builtin_amdgcn_ballot_w64(upto > tile);
    if (past != 0) {
      const int l = __builtin_ctzll(past);
      *before = l == 0 ? base : __builtin_amdgcn_readlane(upto, l - 1);
      return s0 + l;
    }
    base = __builtin_amdgcn_readlane(upto, 63);
  }
  return -1;
}

// ---------------------------------------------------------------------------
// Expansion: one head's 128 keys and 128 values for two context tiles a
// workgroup, a product of [128 tokens x DC] and [DC x 256].  Each wavefront
// forms 64 x 128 of it: 0 and 1 half of the key dims for all tokens, 2 and 3
// all value dims for a tile, so that keys come out with consecutive dims in a
// lane and values with consecutive tokens, as their fragments want them.
// Latent vectors and weights pass through LDS in slices of 32 of the summed
// dims, two slices deep (48 KB: two workgroups a CU hide each other's waits;
// 8192 tokens x 32 heads take 95 to 110 us, 0.7 PFLOP/s, and a third slice or
// several heads a workgroup no less),
// 16-byte chunks at c ^ (row / 4 % 4): a read's 16 rows then meet every bank
// once.
// ---------------------------------------------------------------------------
template <typename T, bool F8, int DC>
__global__ void __launch_bounds__(kExpandBlock, 2) expand_kernel(PrefillParams p) {
  constexpr int SL = 32;             // dims of a slice
  constexpr int NS = DC / SL;
  constexpr int TOK = 2 * kCtxTile;  // tokens of a workgroup
  constexpr int ROWS = TOK + 2 * kHead;
  constexpr int PITCH = SL * 2;      // bytes of a slice's row
  __shared__ __align__(1024) char sm[2][ROWS * PITCH];  // tokens, key weights, value weights
  __shared__ int64_t splace[TOK];
  __shared__ float smost[2][TOK];  // each token's largest magnitude in the key dims of a wavefront
  __shared__ int32_t slow[2];  // where the tiles' second parts go, -1 where they have none
  const latent_prefill_args& a = p.a;
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int32_t head = (int32_t)(blockIdx.x % (uint32_t)a.num_heads);
  const int32_t tile0 = (int32_t)(blockIdx.x / (uint32_t)a.num_heads) * 2;

  // Places of the tokens: wavefronts 0 and 1 find a tile's each.
  if (w < 2) {
    int64_t off = -1;
    int32_t before = 0;
    const int32_t tile = tile0 + w;
    const int32_t s = tile < p.capacity ? sequence_of_tile(p, tile, lane, &before) : -1;
    if (s >= 0) {
      const int32_t pos = (tile - before) * kCtxTile + lane;
      if (pos < context_of(p, s))
        off = locate(a.block_table + (int64_t)s * a.table_stride, a.page_size, a.num_pages, a.page_stride,
                     a.token_stride, pos);
      const uint64_t bits = __builtin_amdgcn_ballot_w64(off >= 0);
      if (head == 0 && lane == 0) p.valid[tile] = bits;
    }
    splace[w * 64 + lane] = s < 0 ? -2 : off;
    if (lane == 0) slow[w] = s >= 0 && tile - before < kExactTiles ? low_tile(p, s, tile - before, tile) : -1;
  }
  __syncthreads();
  const bool real[2] = {splace[0] != -2, splace[64] != -2};
  if (!real[0] && !real[1]) return;

  // A wavefront loads 64 rows of weights and 32 of tokens of each slice, 16
  // rows (of four lanes) at a time.
  constexpr int SZ = F8 ? 1 : 2;
  const int r16 = lane >> 2, c4 = lane & 3;
  const int swap = c4 ^ ((r16 >> 2) & 3);  // the chunk that lands at the lane's place
  const char* cache = (const char*)a.cache;
  const char* wrow = (w < 2 ? (const char*)a.w_k : (const char*)a.w_v) +
                     ((int64_t)head * kHead + (w & 1) * 64 + r16) * (DC * 2) + swap * 16;
  const char* xrow[2];
  bool gone[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t off = splace[w * 32 + i * 16 + r16];
    gone[i] = off < 0;
    xrow[i] = cache + (off < 0 ? 0 : off) * SZ + (F8 ? c4 * 8 : swap * 16);
  }
  const bool any_gone = __builtin_amdgcn_ballot_w64(gone[0] || gone[1]) != 0;
  u32x2 stage[2];
  auto issue = [&](int k, int b) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      load_to_lds(wrow + i * (16 * DC * 2) + k * PITCH, lds_at(&sm[b][(TOK + w * 64 + i * 16) * PITCH]));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if constexpr (F8)
        stage[i] = *(const u32x2*)(xrow[i] + k * SL);
      else
        load_to_lds(xrow[i] + k * PITCH, lds_at(&sm[b][(w * 32 + i * 16) * PITCH]));
    }
  };
  auto mine = [&](int b, int i) { return (u32x4*)&sm[b][(w * 32 + i * 16 + r16) * PITCH]; };
  auto store = [&](int b) {
    if constexpr (F8) {
#pragma unroll
      for (int i = 0; i < 2; ++i) mine(b, i)[swap] = widen<T>(stage[i]);
    }
  };

  f32x16 acc[2][4];  // [block of 32 rows][block of 32 columns]
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x16{};
  // Keys: rows are dims, columns tokens.  Values: rows are tokens, columns dims.
  const bool keys = w < 2;
  const int arow = keys ? TOK + w * 64 : (w & 1) * 64, brow = keys ? 0 : TOK + kHead;
  const uint32_t lrow = (uint32_t)(lane & 31) * PITCH, lswap = (uint32_t)(lane >> 2) & 3;
  issue(0, 0);
  store(0);
  for (int k = 0; k < NS; ++k) {
    const int b = k & 1;
    wait_loads();
    if (any_gone) {  // tokens that are not there count as zeros
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (gone[i]) mine(b, i)[c4] = u32x4{0, 0, 0, 0};
    }
    __syncthreads();
    if (k + 1 < NS) issue(k + 1, b ^ 1);
    const uint32_t abase = lds_at(&sm[b][0]) + (uint32_t)arow * PITCH + lrow;
    const uint32_t bbase = lds_at(&sm[b][0]) + (uint32_t)brow * PITCH + lrow;
#pragma unroll
    for (int s = 0; s < SL / 16; ++s) {
      const uint32_t c = (((uint32_t)(s * 2 + half)) ^ lswap) * 16;
      u32x4 x[2], y[4];
#pragma unroll
      for (int i = 0; i < 2; ++i) x[i] = lds_read16(abase + i * (32 * PITCH) + c);
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] = lds_read16(bbase + j * (32 * PITCH) + c);
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = T::mfma32(x[i], y[j], acc[i][j]);
    }
    if (k + 1 < NS) store(b ^ 1);
  }

  if (keys) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float most = 0.0f;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) most = fmaxf(most, fabsf(acc[i][j][e]));
      most = max_xor32(most);
      if (half == 0) smost[w][j * 32 + lane] = most;
    }
  }
  __syncthreads();
  if (keys) {
    bool uneven = false;
#pragma unroll
    for (int j = 0; j < 4; ++j) {  // 32 tokens
      if (!real[j >> 1]) continue;
      const int64_t at = ((int64_t)head * p.capacity + tile0 + (j >> 1)) * kKeyTile;
      const int32_t low = slow[j >> 1];
      const int e2 = keep_exp(fmaxf(smost[0][j * 32 + (lane & 31)], smost[1][j * 32 + (lane & 31)]));
      const float key_by = ldexpf(1.0f, -e2);
      if (w == 0) {
        const int64_t tile_at = (int64_t)head * p.capacity + tile0 + (j >> 1);
        const bool any = __builtin_amdgcn_ballot_w64(e2 != 0) != 0;
        if (j & 1) uneven = uneven || any;
        else uneven = any;
        if (half == 0) p.key_exps[tile_at * kCtxTile + (j & 1) * 32 + lane] = (int16_t)e2;
        if ((j & 1) && lane == 0) ((uint16_t*)(p.flags + tile_at))[1] = uneven ? 1 : 0;
      }
      const int64_t low_at = ((int64_t)head * p.low_tiles + low) * kKeyTile;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {  // dims w*64 + i*32 + e*8 + half*4 .. +4 of the lane's token
          float x[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) x[c] = acc[i][j][e * 4 + c] * key_by;
          const u32x2 high = {Fp16::pack(x[0], x[1]), Fp16::pack(x[2], x[3])};
          const int to = ((j & 1) * 8 + w * 4 + i * 2 + (e >> 1)) * kBlock16 + (e & 1) * 512 + (lane & 31) * 16 + half * 8;
          *(u32x2*)(p.keys + at + to) = high;
          if (low < 0) continue;
#pragma unroll
          for (int c = 0; c < 4; ++c) {  // what the rounding left; nothing of what is not finite
            const float h = c & 1 ? Fp16::hi(high[c >> 1]) : Fp16::lo(high[c >> 1]);
            x[c] = fabsf(h) <= Fp16::kLargest ? x[c] - h : 0.0f;
          }
          *(u32x2*)(p.lows + low_at + to) = u32x2{Fp16::pack(x[0], x[1]), Fp16::pack(x[2], x[3])};
        }
    }
  } else if (real[w & 1]) {
    const float by = F8 && a.scale != nullptr ? a.scale[0] : 1.0f;
    const int32_t tile = tile0 + (w & 1);
    char* to = p.values + ((int64_t)head * p.capacity + tile) * kValueTile + lane * 16;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          float x[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            x[e] = acc[i][j][ks * 8 + e] * by;
            bad = bad || !(fabsf(x[e]) <= T::kLargest);
          }
          *(u32x4*)(to + ((i * 2 + ks) * 4 + j) * kBlock16) =
              u32x4{T::pack(x[0], x[1]), T::pack(x[2], x[3]), T::pack(x[4], x[5]), T::pack(x[6], x[7])};
        }
    const uint64_t any = __builtin_amdgcn_ballot_w64(bad);
    if (lane == 0) ((uint16_t*)(p.flags + (int64_t)head * p.capacity + tile))[0] = any != 0 ? 1 : 0;
  }
  // Rope parts, copied once for all heads: wavefront w takes 32 tokens.
  if (head == 0 && real[w >> 1]) {
    const int64_t rtile = tile0 + (w >> 1);
    const int64_t off = splace[w * 32 + (lane & 31)];
    const char* from = cache + (off < 0 ? 0 : off) * SZ + DC * SZ;
    u32x4 x[4];
    float most = 0.0f;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      if constexpr (F8)
        x[s] = widen<T>(*(const u32x2*)(from + s * 16 + half * 8));
      else
        x[s] = *(const u32x4*)(from + s * 32 + half * 16);
      if (off < 0) x[s] = u32x4{0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < 4; ++i) most = fmaxf(most, fmaxf(fabsf(T::lo(x[s][i])), fabsf(T::hi(x[s][i]))));
    }
    const int e2 = keep_exp(max_xor32(most));
    const float rope_by = ldexpf(1.0f, -e2);
    const uint64_t uneven = __builtin_amdgcn_ballot_w64(e2 != 0);
    if (lane == 0) ((uint16_t*)(p.rope_flags + rtile))[w & 1] = uneven != 0 ? 1 : 0;
    if (half == 0) p.rope_exps[rtile * kCtxTile + (w & 1) * 32 + lane] = (int16_t)e2;
    char* to = p.ropes + rtile * kRopeTile + (w & 1) * (4 * kBlock16) + lane * 16;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[s][i] = Fp16::pack(T::lo(x[s][i]) * rope_by, T::hi(x[s][i]) * rope_by);
      *(u32x4*)(to + s * kBlock16) = x[s];
    }
  }
}

// ---------------------------------------------------------------------------
// Attention of 128 query rows of one head a workgroup, 32 a wavefront, over
// the context's tiles in order.  Values lie in LDS twice, being loaded and in
// use; keys once (72 KB with their second parts, so that two workgroups fit a
// CU): the next tile's come under the softmax and the product with the values,
// which measures as two buffers do.  S^T and O^T keep a query row in a lane (and the lane 32 further), so
// the maximum takes one exchange and everything else none.  The reference of
// the weights moves only when a score passes it by 2^8 (see the absorbed
// form).
//
// The tiles that all rows see come first, in a loop of their own: what the
// last few need (keys past a row's end masked, values that are not finite kept
// from rows that do not see them) costs registers, and the copies and spills
// that came with it cost the loop a wait for memory on every tile (790 us
// against 690 for 8192 tokens x 32 heads, both without second parts).  The dozen
// registers that spill still lie around that last path, none in this loop.
//
// 8192 tokens x 32 heads take 709 us (766 on a hot card), 0.97 PFLOP/s, at the
// 1.65 to 1.8 GHz that the power limit leaves under this load.  While a CU is at
// work its matrix units are busy 63 % of the time and its LDS 32 %; a wavefront
// waits for its turn to issue 45 % of the time and for loads or barriers 18 %.
// So it is the two wavefronts of a SIMD taking turns, not one full unit: longer
// rings of reads, both token blocks' chains in turn and wave priorities changed
// nothing.
// ---------------------------------------------------------------------------
constexpr int kRows = 128;
constexpr int kLeastTiles = 4;  // of a part of a split context
constexpr float kLazyStep = 8.0f;
constexpr float kFar = 1048576.0f;
constexpr int kAheadBlocks = 4;

// A tile of query rows: its sequence, its place within the sequence's chunk
// (the last one first: it has the most work), the context tiles before the
// sequence's, the chunk's first row and rows.  False past the last one.
struct RowTile {
  int32_t seq, local, tile0, start, count;
};
__device__ __forceinline__ bool row_tile_of(const PrefillParams& p, int32_t want, int lane, RowTile* t) {
  const latent_prefill_args& a = p.a;
  int32_t rows_base = 0, ctx_base = 0;
  for (int32_t s0 = 0; s0 < a.num_seqs; s0 += 64) {
    const int32_t s = s0 + lane;
    int32_t from = 0, n = 0, ctx = 0;
    if (s < a.num_seqs) {
      from = clamp_to(a.starts[s], a.num_tokens);
      n = clamp_to(a.starts[s + 1], a.num_tokens) - from;
      n = n < 0 ? 0 : n;
      ctx = tiles_of(context_of(p, s), kCtxTile);
    }
    const int32_t mine = tiles_of(n, kRows);
    const int32_t upto = __builtin_elementwise_add_sat(rows_base, scan_up(mine, lane));
    const int32_t cupto = __builtin_elementwise_add_sat(ctx_base, scan_up(ctx, lane));
    const uint64_t past = __builtin_amdgcn_ballot_w64(upto > want);
    if (past != 0) {
      const int l = __builtin_ctzll(past);
      t->seq = s0 + l;
      t->local = __builtin_amdgcn_readlane(mine, l) - 1 -
                 (want - (l == 0 ? rows_base : __builtin_amdgcn_readlane(upto, l - 1)));
      t->tile0 = l == 0 ? ctx_base : __builtin_amdgcn_readlane(cupto, l - 1);
      t->start = __builtin_amdgcn_readlane(from, l);
      t->count = __builtin_amdgcn_readlane(n, l);
      return true;
    }
    rows_base = __builtin_amdgcn_readlane(upto, 63);
    ctx_base = __builtin_amdgcn_readlane(cupto, 63);
  }
  return false;
}
// Parts that a row tile's context tiles are shared out to.
__device__ __forceinline__ int32_t parts_of(int32_t tiles, int32_t most) {
  const int32_t n = tiles / kLeastTiles;
  return n < 1 ? 1 : n < most ? n : most;
}

template <typename T>
__global__ void __launch_bounds__(256, 2) prefill_kernel(PrefillParams p) {
  // Keys, rope parts and what the keys' rounding left: one tile; values: two.
  __shared__ __align__(1024) char sk[kKeyTile + kRopeTile + kKeyTile];
  __shared__ __align__(1024) char sv[2][kValueTile];
  const latent_prefill_args& a = p.a;
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int32_t head = (int32_t)(blockIdx.x % (uint32_t)a.num_heads);
  const int32_t slot = (int32_t)(blockIdx.x / (uint32_t)a.num_heads), part = slot % p.parts;

  RowTile at_tile;
  if (!row_tile_of(p, slot / p.parts, lane, &at_tile)) return;
  const int32_t seq = at_tile.seq, local = at_tile.local, tile0 = at_tile.tile0, start = at_tile.start, count = at_tile.count;
  const int32_t ctx = context_of(p, seq);
  const int32_t row0 = local * kRows;  // first row of the tile, within the chunk
  const bool fits = (int64_t)tile0 + tiles_of(ctx, kCtxTile) <= p.capacity;

  // Row of this lane; how many positions it sees (0 for rows past the chunk).
  const int32_t j = row0 + w * 32 + (lane & 31);
  const bool real = j < count;
  const int32_t sees = real ? (ctx - count + j + 1 < 0 ? 0 : ctx - count + j + 1) : 0;
  const int32_t last = row0 + kRows < count ? row0 + kRows : count;  // rows of the tile end here
  const int32_t longest = ctx - count + last;                        // positions its last row sees
  const int32_t tiles = longest > 0 && fits ? tiles_of(longest, kCtxTile) : 0;
  const int32_t parts = parts_of(tiles, p.parts);
  if (part >= parts) return;
  const int32_t chunk = (tiles + parts - 1) / parts;
  const int32_t begin = part * chunk < tiles ? part * chunk : tiles, stop = tiles - begin < chunk ? tiles : begin + chunk;
  // Positions that any row of the wavefront sees.
  const int32_t wfirst = row0 + w * 32, wlast = wfirst + 31 < count - 1 ? wfirst + 31 : count - 1;
  const int32_t any_see = wfirst < count ? ctx - count + wlast + 1 : 0;

  u32x4 q[12];
  {
    const char* qp = (const char*)a.q + 2 * ((int64_t)(start + (real ? j : row0)) * a.q_row_stride + (int64_t)head * a.q_head_stride);
#pragma unroll
    for (int s = 0; s < 12; ++s) q[s] = *(const u32x4*)(qp + s * 32 + half * 16);
  }
  // The scale's sign goes into the queries, so that the largest product has the
  // largest score (and products are 0 where the scale is).  A bf16 row goes to
  // fp16 times 2^-qe, which makes it as large as fp16 takes: exact for what lies
  // within 2^-31 of its largest.  Its rope part has a power of its own where that
  // would cost it bits or the others: 2^-(qe + qgap).
  const float total = p.scale_log2 * (a.scale == nullptr ? 1.0f : a.scale[0]);
  const float sign = total < 0.0f ? -1.0f : total == 0.0f ? 0.0f : 1.0f;
  const float scale = total == 0.0f ? 1.0f : fabsf(total);
  int qe = 0, qgap = 0;
  if constexpr (!std::is_same_v<T, Fp16>) {
    float most[2] = {0.0f, 0.0f};
#pragma unroll
    for (int s = 0; s < 12; ++s)
#pragma unroll
      for (int e = 0; e < 4; ++e) most[s >> 3] = fmaxf(most[s >> 3], fmaxf(fabsf(T::lo(q[s][e])), fabsf(T::hi(q[s][e]))));
    most[0] = max_xor32(most[0]), most[1] = max_xor32(most[1]);
    const bool ordinary = total != 0.0f && most[0] < INFINITY && most[1] < INFINITY;
    if (ordinary && fmaxf(most[0], most[1]) > 0.0f) {
      const int en = __builtin_amdgcn_frexp_expf(most[0]) - 15, er = __builtin_amdgcn_frexp_expf(most[1]) - 15;
      const bool one = most[0] == 0.0f || most[1] == 0.0f || (en - er <= 12 && er - en <= 12);
      qe = one ? __builtin_amdgcn_frexp_expf(fmaxf(most[0], most[1])) - 15 : en;
      qgap = one ? 0 : er - en;
    }
  }
#pragma unroll
  for (int s = 0; s < 12; ++s)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int by = s < 8 ? -qe : -(qe + qgap);
      q[s][e] = Fp16::pack(ldexpf(T::lo(q[s][e]) * sign, by), ldexpf(T::hi(q[s][e]) * sign, by));
    }

  // 16 blocks of keys, 8 of rope parts, 16 of values, and 16 of what the keys'
  // rounding left, a quarter of each a wavefront, as they lie.
  const char* kp = p.keys + ((int64_t)head * p.capacity + tile0) * kKeyTile + w * kBlock16;
  const char* lp = p.lows + ((int64_t)head * p.low_tiles + low_tile(p, seq, 0, tile0)) * kKeyTile + w * kBlock16;
  const char* rp = p.ropes + (int64_t)tile0 * kRopeTile + w * kBlock16;
  const char* vp = p.values + ((int64_t)head * p.capacity + tile0) * kValueTile + w * kBlock16;
  const uint32_t lane16 = (uint32_t)lane * 16;
  auto issue_keys = [&](int32_t i) {
    const uint32_t to = lds_at(&sk[0]) + (uint32_t)w * kBlock16;
#pragma unroll
    for (int k = 0; k < 4; ++k) load_to_lds(kp + (int64_t)i * kKeyTile + k * 4096, lane16, to + k * 4096);
#pragma unroll
    for (int k = 0; k < 2; ++k) load_to_lds(rp + (int64_t)i * kRopeTile + k * 4096, lane16, to + kKeyTile + k * 4096);
    if (i < kExactTiles)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        load_to_lds(lp + (int64_t)i * kKeyTile + k * 4096, lane16, to + kKeyTile + kRopeTile + k * 4096);
  };
  auto issue_values = [&](int32_t i) {
    const uint32_t to = lds_at(&sv[i & 1][0]) + (uint32_t)w * kBlock16;
#pragma unroll
    for (int k = 0; k < 4; ++k) load_to_lds(vp + (int64_t)i * kValueTile + k * 4096, lane16, to + k * 4096);
  };
  // Which of a tile's tokens are in the cache; read through the scalar cache
  // and a tile ahead, so that no wait for vector memory is among the loads.
  using scalar_u64 = const __attribute__((address_space(4))) uint64_t;
  scalar_u64* valid_of = (scalar_u64*)(p.valid + tile0);
  using scalar_u32 = const __attribute__((address_space(4))) uint32_t;
  scalar_u32* flag_of = (scalar_u32*)(p.flags + (int64_t)head * p.capacity + tile0);
  scalar_u32* rope_flag_of = (scalar_u32*)(p.rope_flags + tile0);

  float ref = -INFINITY, sum = 0.0f;  // base-2 logarithm; of this lane's tokens
  f32x16 o[4];
#pragma unroll
  for (int d = 0; d < 4; ++d) o[d] = f32x16{};
  f32x16 s[2];
  u32x4 pw[4];

  // Powers of two that the keys (rope parts) of the lane's tokens e*8 + half*4 .. +4
  // of a block of 32 are kept smaller by.
  auto powers = [&](const int16_t* of_tile, int tb, int e, int* x) __attribute__((always_inline)) {
    const u32x2 two = *(const u32x2*)(of_tile + tb * 32 + e * 8 + half * 4);
#pragma unroll
    for (int c = 0; c < 4; ++c) x[c] = c & 1 ? (int)two[c >> 1] >> 16 : (int)(int16_t)(two[c >> 1] & 0xffffu);
  };
  // uneven: some token of tile i or some row has a power of its own.  Rope parts
  // come first and are then brought level with the keys; scores then take the
  // scale alone, without 2^qe.
  auto scores = [&](bool exact, int32_t i, bool uneven) __attribute__((always_inline)) {
    const int16_t* ke = p.key_exps + ((int64_t)head * p.capacity + tile0 + i) * kCtxTile;
    const int16_t* re = p.rope_exps + ((int64_t)tile0 + i) * kCtxTile;
    const uint32_t base = lds_at(&sk[0]) + lane16;
    auto key = [&](int n) {  // n: token block * 12 + step
      const int tb = n / 12, k = n % 12;
      return lds_read16(base + (k < 4 ? kKeyTile + (tb * 4 + k) * kBlock16 : (tb * 8 + k - 4) * kBlock16));
    };
    u32x4 ring[kAheadBlocks];
#pragma unroll
    for (int n = 0; n < kAheadBlocks - 1; ++n) ring[n] = key(n);
    s[0] = f32x16{}, s[1] = f32x16{};
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int n = 0; n < 24; ++n) {
      if (n + kAheadBlocks - 1 < 24) ring[(n + kAheadBlocks - 1) % kAheadBlocks] = key(n + kAheadBlocks - 1);
      if (uneven && n % 12 == 4) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          int kx[4], rx[4];
          powers(ke, n / 12, e, kx), powers(re, n / 12, e, rx);
#pragma unroll
          for (int c = 0; c < 4; ++c) s[n / 12][e * 4 + c] = ldexpf(s[n / 12][e * 4 + c], rx[c] - kx[c] + qgap);
        }
      }
      s[n / 12] = Fp16::mfma32(ring[n % kAheadBlocks], q[(n + 8) % 12], s[n / 12]);
      __builtin_amdgcn_sched_barrier(0);
    }
    auto finish = [&] {
      if (!uneven) return;
#pragma unroll
      for (int tb = 0; tb < 2; ++tb)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          int kx[4];
          powers(ke, tb, e, kx);
#pragma unroll
          for (int c = 0; c < 4; ++c) s[tb][e * 4 + c] = ldexpf(s[tb][e * 4 + c], kx[c] + qe);
        }
    };
    if (!exact) return finish();
    auto low = [&](int n) { return lds_read16(base + kKeyTile + kRopeTile + n * kBlock16); };
#pragma unroll
    for (int n = 0; n < kAheadBlocks - 1; ++n) ring[n] = low(n);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int n = 0; n < 16; ++n) {
      if (n + kAheadBlocks - 1 < 16) ring[(n + kAheadBlocks - 1) % kAheadBlocks] = low(n + kAheadBlocks - 1);
      s[n / 8] = Fp16::mfma32(ring[n % kAheadBlocks], q[n % 8], s[n / 8]);
      __builtin_amdgcn_sched_barrier(0);
    }
    finish();
  };
  // Leaves out tokens that are not in the cache or past `left` (of the tile).
  auto mask = [&](uint64_t valid, int32_t left) {
#pragma unroll
    for (int tb = 0; tb < 2; ++tb) {
      const uint32_t bits = (uint32_t)(valid >> (tb * 32)) >> (half * 4);
      const int32_t rest = left - tb * 32 - half * 4;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int t = (e >> 2) * 8 + (e & 3);
        s[tb][e] = t < rest && ((bits >> t) & 1u) != 0 ? s[tb][e] : -INFINITY;
      }
    }
  };
  auto weights = [&](float by_tile) {
    float top = s[0][0];
#pragma unroll
    for (int e = 1; e < 32; ++e) top = fmaxf(top, s[e >> 4][e & 15]);
    top = max_xor32(top) * by_tile;
    if (__builtin_amdgcn_ballot_w64(top > ref + kLazyStep) != 0) {
      const float m = fmaxf(ref, top);
      const float by = m == ref ? 1.0f : exp2_fast(ref - m);
      ref = m;
      sum *= by;
#pragma unroll
      for (int d = 0; d < 4; ++d) o[d] *= by;
    }
    // Differences to the reference come unrounded out of one fma, but the reference
    // is a rounded product: far out, where half a step of it is a factor, products
    // are rounded first, so that the largest is the reference.
    float by = by_tile;
    if (__builtin_amdgcn_ballot_w64(fabsf(ref) > kFar && ref != -INFINITY) != 0) {
      s[0] *= by_tile, s[1] *= by_tile;
      by = 1.0f;
    }
    const float r = ref == -INFINITY ? 0.0f : lift<T>(kLazyStep) - ref;
    float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] = exp2_fast(fmaf(s[k >> 1][(k & 1) * 8 + e], by, r));
        s[k >> 1][(k & 1) * 8 + e] = x[e];
        part[e & 3] += x[e];
      }
      pw[k] = u32x4{T::pack(x[0], x[1]), T::pack(x[2], x[3]), T::pack(x[4], x[5]), T::pack(x[6], x[7])};
    }
    sum += (part[0] + part[1]) + (part[2] + part[3]);
  };
  auto values = [&](uint32_t vbase, bool exact) {
    auto value = [&](int n) { return lds_read16(vbase + n * kBlock16); };
    u32x4 ring[kAheadBlocks];
#pragma unroll
    for (int n = 0; n < kAheadBlocks - 1; ++n) ring[n] = value(n);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int n = 0; n < 16; ++n) {
      if (n + kAheadBlocks - 1 < 16) ring[(n + kAheadBlocks - 1) % kAheadBlocks] = value(n + kAheadBlocks - 1);
      o[n & 3] = T::mfma32(ring[n % kAheadBlocks], pw[n >> 2], o[n & 3]);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (!exact) return;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      u32x4 left;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int e = (k & 1) * 8 + c * 2;
        left[c] = T::pack(s[k >> 1][e] - T::lo(pw[k][c]), s[k >> 1][e + 1] - T::hi(pw[k][c]));
      }
#pragma unroll
      for (int d = 0; d < 4; ++d) o[d] = T::mfma32(value(k * 4 + d), left, o[d]);
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  // Tiles that every row of the workgroup sees whole, up to the first that is not
  // of ordinary size; none where a row of the wavefront is not.  (Both loops have
  // the same two barriers a tile, so wavefronts may part here.)
  const int32_t first_sees = ctx - count + row0 + 1;
  const int32_t all_whole = first_sees > 0 && fits ? first_sees / kCtxTile : 0;
  int32_t whole = all_whole < begin ? begin : all_whole < stop ? all_whole : stop;
  uint64_t valid = 0;
  if (begin < stop) {
    issue_keys(begin);
    issue_values(begin);
    valid = valid_of[begin];
  }
  const bool uneven_rows = __builtin_amdgcn_ballot_w64(qgap != 0) != 0;
  for (int32_t i = begin; i < whole; i += 64) {
    const int32_t at = i + lane < whole ? i + lane : whole - 1;
    const uint64_t uneven = __builtin_amdgcn_ballot_w64(
        (p.flags[(int64_t)head * p.capacity + tile0 + at] >> 16) != 0 || p.rope_flags[tile0 + at] != 0);
    if (uneven != 0) {
      const int32_t first = i + (int32_t)__builtin_ctzll(uneven);
      whole = first < whole ? first : whole;
      break;
    }
  }
  if (uneven_rows) whole = begin;
  const float row_scale = fmaxf(ldexpf(scale, qe), 1.17549435e-38f);  // masked scores times 0 are no numbers
  for (int32_t i = begin; i < whole; ++i) {
    wait_loads();
    __syncthreads();
    if (i + 1 < stop) issue_values(i + 1);
    const uint64_t now = valid;
    if (i + 1 < stop) valid = valid_of[i + 1];
    scores(i < kExactTiles, i, false);
    __syncthreads();  // the keys are read
    if (i + 1 < stop) issue_keys(i + 1);
    if (now != ~0ull) mask(now, kCtxTile);
    weights(row_scale);
    // The second parts of weights meet finite values only.
    values(lds_at(&sv[i & 1][0]) + lane16, i < kExactWeights && (flag_of[i] & 0xffffu) == 0);
  }
  // Tiles that some row sees in part or not at all, and others from the first on
  // that is out of the ordinary.
  for (int32_t i = whole; i < stop; ++i) {
    wait_loads();
    __syncthreads();
    if (i + 1 < stop) issue_values(i + 1);
    const uint64_t now = valid;
    if (i + 1 < stop) valid = valid_of[i + 1];
    const uint32_t flags = flag_of[i];
    const bool odd = (flags & 0xffffu) != 0;  // some value is not finite
    const bool uneven = uneven_rows || (flags >> 16) != 0 || rope_flag_of[i] != 0;
    const int32_t t0 = i * kCtxTile;
    const bool any = t0 < any_see;  // else nothing here for this wavefront
    if (any) scores(i < kExactTiles, i, uneven);
    __syncthreads();
    if (i + 1 < stop) issue_keys(i + 1);
    if (!any) continue;
    const uint32_t vbase = lds_at(&sv[i & 1][0]) + lane16;
    mask(now, sees - t0);
    weights(uneven ? scale : row_scale);
    if (!odd) {
      values(vbase, i < kExactWeights);
      continue;
    }
    // Values that are not finite: one token at a time, into the rows that see
    // it.
    for (int32_t t = 0; t < kCtxTile; ++t) {
      const int k = t >> 4, in = t & 15;  // block of 16 tokens; the token's half and element there
      const bool mine = half == ((in >> 2) & 1);
      const int e = (in >> 3) * 4 + (in & 3);
      u32x4 keep = {0, 0, 0, 0};
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (mine && (e >> 1) == c) keep[c] = (e & 1) ? 0xffff0000u : 0x0000ffffu;
      u32x4 weight = {0, 0, 0, 0};
#pragma unroll
      for (int c = 0; c < 4; ++c) weight = k == c ? pw[c] : weight;
      weight &= keep;
      const bool here = t0 + t < sees && ((now >> t) & 1u) != 0;
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const f32x16 x = T::mfma32(lds_read16(vbase + (k * 4 + d) * kBlock16) & keep, weight, o[d]);
#pragma unroll
        for (int c = 0; c < 16; ++c) o[d][c] = here ? x[c] : o[d][c];
      }
    }
  }

  sum += __shfl_xor(sum, 32);
  if (!real) return;
  ref -= lift<T>(kLazyStep);  // of the weights as they are kept
  const int64_t at = (int64_t)(start + j) * a.num_heads + head;
  if (parts > 1) {
    const int64_t pi = at * p.parts + part;
#pragma unroll
    for (int d = 0; d < 4; ++d)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        *(f32x4*)(p.part_out + pi * kHead + d * 32 + k * 8 + half * 4) =
            f32x4{o[d][k * 4], o[d][k * 4 + 1], o[d][k * 4 + 2], o[d][k * 4 + 3]};
    if (half == 0) p.part_stat[pi] = float2{ref, sum};
    return;
  }
  const float by = !fits ? NAN : sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
  for (int d = 0; d < 4; ++d)
#pragma unroll
    for (int k = 0; k < 4; ++k)
      *(u32x2*)((uint16_t*)a.out + at * kHead + d * 32 + k * 8 + half * 4) =
          u32x2{T::pack(o[d][k * 4] * by, o[d][k * 4 + 1] * by), T::pack(o[d][k * 4 + 2] * by, o[d][k * 4 + 3] * by)};
  if (half == 0 && a.lse != nullptr)
    a.lse[at] = !fits ? NAN : sum == 0.0f ? -INFINITY : (ref + __log2f(sum)) * kLn2;
}

// Joins the parts of split contexts: eight rows of a row tile and head a
// workgroup, 32 threads of four dims each.
constexpr int kJoinRows = 8;
template <typename T>
__global__ void __launch_bounds__(256) prefill_join_kernel(PrefillParams p) {
  const latent_prefill_args& a = p.a;
  const int tid = threadIdx.x, lane = tid & 63;
  const int32_t head = (int32_t)(blockIdx.x % (uint32_t)a.num_heads);
  const int32_t slot = (int32_t)(blockIdx.x / (uint32_t)a.num_heads);
  RowTile t;
  if (!row_tile_of(p, slot / (kRows / kJoinRows), lane, &t)) return;
  const int32_t row0 = t.local * kRows, ctx = context_of(p, t.seq);
  const int32_t longest = ctx - t.count + (row0 + kRows < t.count ? row0 + kRows : t.count);
  const bool fits = (int64_t)t.tile0 + tiles_of(ctx, kCtxTile) <= p.capacity;
  const int32_t parts = parts_of(longest > 0 && fits ? tiles_of(longest, kCtxTile) : 0, p.parts);
  const int32_t j = row0 + slot % (kRows / kJoinRows) * kJoinRows + (tid >> 5);
  if (parts == 1 || j >= t.count) return;
  const int64_t at = (int64_t)(t.start + j) * a.num_heads + head;
  const float2* stat = p.part_stat + at * p.parts;
  const float* from = p.part_out + at * p.parts * kHead + (tid & 31) * 4;
  float top = -INFINITY;
  for (int32_t i = 0; i < parts; ++i) top = fmaxf(top, stat[i].x);
  float sum = 0.0f;
  f32x4 o = {0, 0, 0, 0};
#pragma unroll 4
  for (int32_t i = 0; i < parts; ++i) {
    const float2 m = stat[i];
    const float by = m.x == top ? 1.0f : exp2_fast(m.x - top);
    sum += m.y * by;
    o += *(const f32x4*)(from + i * kHead) * by;
  }
  const float by = sum == 0.0f ? 0.0f : 1.0f / sum;
  *(u32x2*)((uint16_t*)a.out + at * kHead + (tid & 31) * 4) = u32x2{T::pack(o[0] * by, o[1] * by), T::pack(o[2] * by, o[3] * by)};
  if ((tid & 31) == 0 && a.lse != nullptr) a.lse[at] = sum == 0.0f ? -INFINITY : (top + __log2f(sum)) * kLn2;
}

namespace {
template <typename T>
const void* expand_dims(int store, int dim) {
  if (dim == 256) return store == PAGED_E4M3 ? (const void*)&expand_kernel<T, true, 256> : (const void*)&expand_kernel<T, false, 256>;
  if (dim == 512) return store == PAGED_E4M3 ? (const void*)&expand_kernel<T, true, 512> : (const void*)&expand_kernel<T, false, 512>;
  return nullptr;
}
}  // namespace

const void* expand_kernel_ptr(int dtype, int store, int latent_dim) {
  return dtype == PAGED_BF16 ? expand_dims<Bf16>(store, latent_dim) : expand_dims<Fp16>(store, latent_dim);
}
const void* prefill_kernel_ptr(int dtype) {
  return dtype == PAGED_BF16 ? (const void*)&prefill_kernel<Bf16> : (const void*)&prefill_kernel<Fp16>;
}
const void* prefill_join_kernel_ptr(int dtype) {
  return dtype == PAGED_BF16 ? (const void*)&prefill_join_kernel<Bf16> : (const void*)&prefill_join_kernel<Fp16>;
}
int prefill_rows() { return kRows; }
int prefill_join_rows() { return kJoinRows; }

}  // namespace rrt
