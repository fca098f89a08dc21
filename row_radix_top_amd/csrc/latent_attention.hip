// The absorbed form of latent attention: all heads of a row read one shared
// vector a token, as keys whole and as values without its rope part.

#include <type_traits>

#include "paged_device.hpp"

namespace rrt {

// ---------------------------------------------------------------------------
// o_h = softmax(s q_h c^T) c[:DC], for HT heads of one row and one part of its
// positions a workgroup.
//
// 2 (2 DC + 64) flop a head and token against 2 (DC + 64) bytes a token: with
// 128 heads near the card's balance of matrix rate and memory rate, with few
// heads bound by memory.  Every token's vector is used by all
// heads and twice (scores, values), so a tile of 64 tokens is staged in LDS
// once, in 16 bits, two buffers deep: the next tile's loads go straight to LDS
// while this one is used.  (An e4m3 cache: the raw bytes go to one buffer of
// half the size, and each wavefront widens its own tokens into one tile.  Their
// part of the buffer is its own too, so it starts the next tile's loads into it
// once it has read this one's, with no barrier between.)
//
//   S^T[token][head] = C Q^T: 2 x 4 wavefronts split heads and tokens; each
//     keeps the queries of its heads in registers for the whole part.
//   O^T[dim][head] += C^T P^T: each wavefront owns an eighth of the value dims
//     for all heads, so the values are read from LDS once in all; their
//     transpose is the LDS read instruction's.  P passes through LDS.
//
// Eight wavefronts, two on a SIMD, with 256 registers each: queries 128 (two
// 16-head columns a wavefront, so a key operand serves two products; their rope
// parts lie in LDS) and outputs 64 at 512 dims and 64 heads.  One wavefront a SIMD with all 512 was
// slower however its products were overlapped: loads, addresses, weights and
// LDS latencies then add up, with no second wavefront to run meanwhile
// (5300 cycles for 32 tokens of which 1090 on the matrix unit).
//
// The weights are relative to a reference that follows the running maximum
// lazily: only when a score passes it by 2^8 does the workgroup agree on a new
// one, form the weights again and rescale (P then stays below 2^8, or below 2^15
// as fp16 keeps it, sums below that times n: far inside fp32).
//
// No unit is full: 64 rows of 2048 chosen positions, 128 heads, bf16, take 70 us
// (0.48 PFLOP/s) with the matrix units busy 30 % of a CU's time at work and LDS
// 26 %; 1024 rows of 1024, 64 heads, e4m3, 259 us with 25 % and 37 %.  A
// wavefront waits for loads or barriers 37 % of its time and for its turn to
// issue 28 %: all eight go through scores, weights and values of a tile together,
// two barriers a tile (e4m3: three) and one workgroup on a CU.
//
// LDS rows are a multiple of all banks wide; 16-byte chunk c of token t's row
// is kept at c ^ swizzle(t), which spreads both the 16 tokens of a key operand
// and the 4 tokens x 2 chunks of a transposed read over the banks.
// ---------------------------------------------------------------------------
constexpr int kRope = PAGED_ROPE_DIM;
constexpr float kLazy = 8.0f;
constexpr int kAhead = 4;  // key operands in flight from LDS, and one in use

using i16x4 = short __attribute__((ext_vector_type(4)));
using lds_i16x4 = __attribute__((address_space(3))) i16x4;
using lds_u32x4 = __attribute__((address_space(3))) u32x4;
using lds_i32 = __attribute__((address_space(3))) int32_t;
using lds_u32x2 = __attribute__((address_space(3))) u32x2;

__device__ __forceinline__ uint32_t lds_at(const void* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const char*)p;
}
__device__ __forceinline__ u32x4 lds_read16(uint32_t at) { return *(lds_u32x4*)at; }
// Four 16-bit values of one column from four rows: lane i of a group of 16
// gives the address of 4 columns of row i / 4 and gets column i.
__device__ __forceinline__ u32x2 lds_read_tr(uint32_t at) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)at));
}
// The value again, opaque to the compiler: addresses derived from it inside a
// loop are formed there instead of being kept in registers across it.
__device__ __forceinline__ uint32_t fresh(uint32_t x) {
  asm volatile("" : "+v"(x));
  return x;
}

constexpr int kLatentBlock = 512;

template <int DC, int HT>
struct LatentShape {
  static constexpr int NW = 8;                  // wavefronts
  static constexpr int TT = 64;                 // tokens of a tile
  static constexpr int WT = 4;                  // wavefronts along the tokens of the scores, 16 each
  static constexpr int WH = 2;                  // and along the heads
  static constexpr int NH = HT / 16 / WH;       // 16-head columns of a wavefront's scores
  static constexpr int KS = (DC + kRope) / 32;  // matrix steps over the key dims
  static constexpr int ND = DC / 16 / NW;       // 16-dim rows of a wavefront's output
  static constexpr int NC = HT / 16;            // 16-head columns of the output
  static constexpr int PT = TT + 16;            // pitch of the weights (rows 40 banks apart)
};

// Sixteen-byte reads are served in groups of lanes {0-3, 12-15, 20-27} and so
// on: tokens 0-3 and 12-15 of one lane group with 4-11 of the next, whose
// chunk is the neighbour.  swz is a permutation of 0..15 that maps {4..11} to
// whole pairs (2i, 2i+1), so such a group meets every bank once; and its upper
// three bits differ over tokens {0-3, 8-11} and over {4-7, 12-15}, which are
// the rows that a transposed read touches together.  (A rotation of t, without
// the second lane group in mind, spent 42% of the LDS cycles in conflicts.)
__device__ __forceinline__ int swz(int t) {
  return ((t & 3) << 1) | ((t >> 2) & 1) | ((((t >> 2) ^ (t >> 3)) & 1) << 3);
}
__device__ __forceinline__ int swz_rope(int t) { return (t >> 1) & 7; }

// Loads straight to LDS: 16 (4) bytes from each active lane's address to `to`
// (wave uniform) + 16 (4) x lane.  No register is written, so nothing but
// wait_loads() below waits for them; as instructions that the compiler knows
// to write LDS, they made it wait for all of them before every transposed read.
__device__ __forceinline__ void load_to_lds(const char* from, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(__builtin_amdgcn_readfirstlane(to)), "v"(from) : "memory", "m0");
}
__device__ __forceinline__ void load_to_lds(const char* from, uint32_t offset, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(__builtin_amdgcn_readfirstlane(to)), "v"(offset), "s"(from) : "memory", "m0");
}
__device__ __forceinline__ void load4_to_lds(const int32_t* from, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(__builtin_amdgcn_readfirstlane(to)), "v"(from) : "memory", "m0");
}
// Waits until all but the last N loads have arrived.
template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

template <typename T, bool F8, int DC, bool CHOSEN, int HT>
__global__ void __launch_bounds__(kLatentBlock, 2) latent_kernel(AttnParams p) {
  using S = LatentShape<DC, HT>;
  constexpr int NW = S::NW, TT = S::TT, NH = S::NH, KS = S::KS, ND = S::ND, NC = S::NC, PT = S::PT, WT = S::WT;
  constexpr int TW = TT / NW;                 // tokens that a wavefront loads
  constexpr int SZ = F8 ? 1 : 2;
  constexpr int ROW = (DC + kRope) * SZ;      // bytes of a raw token
  constexpr uint32_t kTileBytes = TT * DC * 2, kRawBytes = TT * ROW;
  constexpr int NB = F8 ? 1 : 2;              // tiles in 16 bits
  __shared__ __align__(1024) uint16_t sc[NB][TT * DC];
  __shared__ __align__(1024) uint16_t sr[TT * kRope];
  __shared__ __align__(1024) char sraw[F8 ? kRawBytes : 16];
  __shared__ __align__(1024) u32x4 sq[S::WH * NH * (kRope / 32)][64];
  __shared__ __align__(16) uint16_t sp_[HT * PT];
  __shared__ float smax[WT][HT], ssum[WT][HT], salpha[HT];
  __shared__ int32_t spos[2][TT], spage[2][TT];
  __shared__ __align__(8) uint8_t svalid[2][NW];
  __shared__ int32_t sflag[2];  // the tile (plus one) whose scores pass the reference
  const paged_attention_args& a = p.a;
  const int tid = threadIdx.x, lane = tid & 63, col = lane & 15, g = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wh = w % S::WH, wt = w / S::WH;

  Work work;
  if (!work_of<CHOSEN>(blockIdx.x, (uint32_t)p.col_tiles, (uint32_t)p.groups, (uint32_t)p.most, &work)) return;
  const int64_t most = table_tokens(a.table_width, a.page_size);
  const int32_t part = work.part, head0 = work.unit * HT;
  const int32_t row = CHOSEN ? work.group : by_length(a, work.group, p.groups, 1, most, lane);
  const int32_t seen = clamp_to(a.lengths[row], most);
  const int32_t n = CHOSEN ? a.num_chosen : seen;
  const Split sp = split_of(n, p.most, p.least, p.unit);
  if (part >= sp.parts) return;
  const int32_t begin = part * sp.chunk;
  const int32_t end = n - begin < sp.chunk ? n : begin + sp.chunk;
  const int32_t tiles = (end - begin + TT - 1) / TT;

  const int32_t* table = a.block_table + (int64_t)(row / a.next_n) * a.table_stride;
  const int32_t* chosen = CHOSEN ? a.chosen + (int64_t)row * a.chosen_stride : nullptr;
  const char* cache = (const char*)a.k;

  // --- places of a tile's tokens -------------------------------------------
  // Lane l looks after the wavefront's token l % TW.  The chosen position of a
  // token of tile t + 2, the page of one of tile t + 1 and tile t's data are
  // on their way at the same time, all of them straight to LDS, so that the
  // one wait of a tile covers each and nothing waits for a place alone.
  const int32_t first = begin + w * TW;
  constexpr uint32_t kSlot = TT * 4;
  const uint32_t pos_at = lds_at(&spos[0][0]) + (uint32_t)w * (TW * 4), page_at = lds_at(&spage[0][0]) + (uint32_t)w * (TW * 4);
  auto fetch_chosen = [&](int32_t t) {
    if constexpr (CHOSEN) {
      const uint32_t ln = fresh((uint32_t)lane);
      const int32_t i = first + t * TT + (int32_t)(ln & (TW - 1));
      if (ln < TW) load4_to_lds(chosen + (i < end ? i : end - 1), pos_at + ((uint32_t)t & 1) * kSlot);
    }
  };
  // Starts the page's load; returns the token's offset inside it (all ones: no
  // such token).
  auto fetch_page = [&](int32_t t) -> uint32_t {
    const uint32_t slot = ((uint32_t)t & 1) * kSlot;
    const uint32_t ln = fresh((uint32_t)lane), l8 = ln & (TW - 1);
    const int32_t i = first + t * TT + (int32_t)l8;
    int32_t pos = i;
    if constexpr (CHOSEN) pos = *(lds_i32*)(pos_at + slot + l8 * 4);
    const bool ok = i < end && (!CHOSEN || (uint32_t)pos < (uint32_t)seen);
    const uint32_t x = ok ? (uint32_t)pos : 0u, j = divide(x, p.page);
    if (ln < TW) load4_to_lds(table + j, page_at + slot);
    return ok ? x - j * p.page.by : ~0u;
  };
  auto place = [&](int32_t t, uint32_t in) -> int64_t {
    const int32_t page = *(lds_i32*)(page_at + ((uint32_t)t & 1) * kSlot + (fresh((uint32_t)lane) & (TW - 1)) * 4);
    return in == ~0u || (uint32_t)page >= (uint32_t)a.num_pages
               ? -1
               : (int64_t)page * a.page_stride + (int64_t)in * a.token_stride;
  };

  // --- loads of a tile -----------------------------------------------------
  // LT lanes of 16 bytes hold a token's latent part, RT its rope part.  swz is
  // linear over the bits of its argument, so a lane's chunk offset is its own
  // part, fixed, and a wave-uniform part for each load.  Raw e4m3 rows lie as
  // they are.
  constexpr int LT = DC * SZ / 16, PER = 64 / LT, NL = TW / PER;
  constexpr int RT = kRope * SZ / 16;
  uint32_t recent = 0;  // which of the wavefront's tokens count, a byte a tile, the last one lowest
  // Rope parts have one buffer: theirs start when the scores before them are
  // formed (e4m3: with the rest; the raw bytes are the wavefront's own).
  const char* rope_from = nullptr;
  auto issue = [&](int32_t t, uint32_t in) {
    const uint32_t b = (uint32_t)t & 1;
    const int64_t off = place(t, in);
    const uint32_t valid = (uint32_t)__builtin_amdgcn_ballot_w64(off >= 0) & ((1u << TW) - 1u);
    recent = recent << 8 | valid;
    const int64_t at = (off < 0 ? 0 : off) * SZ;
    const uint32_t ln = fresh((uint32_t)lane);
    if (ln == 0) svalid[b][w] = (uint8_t)valid;
    const uint32_t sub = PER == 1 ? 0u : ln / LT, chunk = ln % LT;
    const uint32_t lane_chunk = F8 ? chunk * 16 : (chunk ^ (uint32_t)swz((int)sub)) << 4;
    const uint32_t wave_swz = F8 ? 0u : (uint32_t)swz(w * TW) << 4;
    const uint32_t to = F8 ? lds_at(&sraw[0]) + (uint32_t)(w * TW) * DC
                           : lds_at(&sc[0][0]) + b * kTileBytes + (uint32_t)(w * TW) * (DC * 2);
#pragma unroll
    for (int k = 0; k < NL; ++k) {
      const uint32_t offset = F8 ? lane_chunk : lane_chunk ^ (wave_swz ^ ((uint32_t)swz(k * PER) << 4));
      if constexpr (PER == 1) {
        load_to_lds(cache + readlane64(at, k), offset, to + (uint32_t)k * 1024);
      } else {
        int64_t where = readlane64(at, k * PER);
#pragma unroll
        for (int j = 1; j < PER; ++j) where = sub >= (uint32_t)j ? readlane64(at, k * PER + j) : where;
        load_to_lds(cache + where + offset, to + (uint32_t)k * 1024);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    const uint32_t tok = (ln / RT) & (TW - 1), rchunk = ln % RT;
    const char* rope = cache + shfl64(at, (int)tok) + DC * SZ;
    if constexpr (F8) {
      if (ln < TW * RT)
        load_to_lds(rope + rchunk * 16, lds_at(&sraw[0]) + TT * DC + (uint32_t)(w * TW) * kRope);
    } else {
      rope_from = rope + ((rchunk ^ (uint32_t)swz_rope(w * TW + (int)tok)) << 4);
    }
  };
  auto issue_rope = [&] {
    if constexpr (!F8) load_to_lds(rope_from, lds_at(&sr[0]) + (uint32_t)(w * TW) * (kRope * 2));
  };
  // e4m3: the wavefront's raw tokens of tile t, widened, into the tile.
  auto widen_tile = [&] {
    if constexpr (F8) {
      const uint32_t ln = fresh((uint32_t)lane);
      const uint32_t raw = lds_at(&sraw[0]) + (uint32_t)(w * TW) * DC + ln * 16;
      const uint32_t sub = ln / LT;
      const uint32_t base = lds_at(&sc[0][0]) + ((uint32_t)(w * TW) + sub) * (DC * 2) +
                            ((((ln % LT) * 2) ^ (uint32_t)swz((int)sub) ^ (uint32_t)swz(w * TW)) << 4);
#pragma unroll
      for (int k = 0; k < NL; ++k) {
        const u32x4 x = lds_read16(raw + (uint32_t)k * 1024);
        const uint32_t to = (base ^ ((uint32_t)swz(k * PER) << 4)) + (uint32_t)(k * PER) * (DC * 2);
        *(lds_u32x4*)to = widen<T>(u32x2{x[0], x[1]});
        *(lds_u32x4*)(to ^ 16) = widen<T>(u32x2{x[2], x[3]});
      }
      if (ln < TW * RT) {
        const uint32_t tt = (uint32_t)(w * TW) + ln / RT;
        const u32x4 x = lds_read16(lds_at(&sraw[0]) + TT * DC + (uint32_t)(w * TW) * kRope + ln * 16);
        const uint32_t to = lds_at(&sr[0]) + tt * (kRope * 2) + ((((ln % RT) * 2) ^ (uint32_t)swz_rope((int)tt)) << 4);
        *(lds_u32x4*)to = widen<T>(u32x2{x[0], x[1]});
        *(lds_u32x4*)(to ^ 16) = widen<T>(u32x2{x[2], x[3]});
      }
    }
  };
  // Tokens of the wavefront that do not count become zeros: their places may
  // hold NaN.  Before the barrier that shows the tile.
  auto clear = [&](uint32_t b, uint32_t valid) {
    if (valid == (1u << TW) - 1u) return;
#pragma nounroll
    for (int t = 0; t < TW; ++t) {
      if ((valid >> t) & 1u) continue;
      const uint32_t tt = (uint32_t)(w * TW + t);
      if (lane < DC / 8) *(lds_u32x4*)(lds_at(&sc[0][0]) + b * kTileBytes + tt * (DC * 2) + (uint32_t)lane * 16) = u32x4{0, 0, 0, 0};
      if (lane < kRope / 8) *(lds_u32x4*)(lds_at(&sr[0]) + tt * (kRope * 2) + (uint32_t)lane * 16) = u32x4{0, 0, 0, 0};
    }
  };

  // Queries of the wavefront's heads, as the scores' second operand.  The
  // latent part stays in the half of the register file that only matrix
  // instructions read, and fills it; the rope part lies in LDS.
  constexpr int KL = DC / 32, KR = kRope / 32;
  u32x4 q[NH][KL];
  // They come through LDS, where the tile that is not yet in use takes all
  // heads' rows once (each wavefront reading its own from memory, in 64-byte
  // pieces and four times over, took 9 us).
  auto issue_queries = [&] {
    constexpr int QL = DC / 8, QPER = 64 / QL, HW = HT / NW;
    static_assert(S::WH * NH * KR <= NW, "a rope fragment a wavefront");
    const uint32_t ln = (uint32_t)lane;
    auto row_of_head = [&](int32_t head) {  // columns past the last head compute a copy of head 0 that is not written
      return (const char*)a.q + 2 * ((int64_t)row * a.q_row_stride +
                                     (int64_t)(head < a.num_heads ? head : 0) * a.q_head_stride);
    };
#pragma unroll
    for (int k = 0; k < HW / QPER; ++k) {
      const int h = w * HW + k * QPER + (int)(ln / QL);
      load_to_lds(row_of_head(head0 + h) + (((ln % QL) ^ (uint32_t)swz(h)) << 4),
                  lds_at(&sc[NB - 1][0]) + (uint32_t)(w * HW + k * QPER) * (DC * 2));
    }
    if (w < S::WH * NH * KR)
      load_to_lds(row_of_head(head0 + (w / KR) * 16 + col) + (DC + (w % KR) * 32 + g * 8) * 2, lds_at(&sq[w][0]));
  };
  auto rope_query = [&](int h, int i) { return lds_at(&sq[(wh * NH + h) * KR + i][0]) + fresh((uint32_t)lane) * 16; };
  // The first tile's chain of reads (positions, pages, data) and the queries
  // are on their way together: one trip to memory after the other is most of a
  // short part's time.
  uint32_t in = ~0u;  // of the tile that is issued next
  uint32_t in0 = ~0u;
  for (int32_t t = 0; t < 2 && t < tiles; ++t) fetch_chosen(t);
  issue_queries();
  wait_loads<HT * DC / 8 / 64 / NW>();  // all but the queries
  if (tiles > 0) in0 = fetch_page(0);
  if (tiles > 1) in = fetch_page(1);
  if (tiles > 2) fetch_chosen(2);  // into the first tile's slot, read by then
  wait_loads<0>();
  if (tiles > 0) {
    issue(0, in0);
    issue_rope();
  }
  __syncthreads();
#pragma unroll
  for (int h = 0; h < NH; ++h) {
    const int t = (wh * NH + h) * 16 + col;
    const uint32_t at = lds_at(&sc[NB - 1][0]) + (uint32_t)t * (DC * 2) + (((uint32_t)g ^ (uint32_t)swz(t)) << 4);
#pragma unroll
    for (int i = 0; i < KL; ++i) q[h][i] = lds_read16((at ^ ((i & 3) << 6)) + (i >> 2) * 256);
#pragma unroll
    for (int i = 0; i < KL; ++i) asm volatile("" : "+a"(q[h][i]));
  }
  const float by_cache = F8 && a.k_scales != nullptr ? a.k_scales[0] : 1.0f;
  const float scale = p.scale_log2 * by_cache;

  float ref[NH], sum[NH];
#pragma unroll
  for (int h = 0; h < NH; ++h) ref[h] = -INFINITY, sum[h] = 0.0f;
  f32x4 o[NC][ND];
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int d = 0; d < ND; ++d) o[c][d] = f32x4{0, 0, 0, 0};
  if (tid < 2) sflag[tid] = 0;

  for (int32_t i = 0; i < tiles; ++i) {
    const uint32_t b = F8 ? 0u : (uint32_t)i & 1;
    wait_loads<0>();  // the tile, the next one's pages and the positions after that
    if constexpr (F8) {
      __syncthreads();  // the tile before is no longer read
      widen_tile();
    }
    clear(b, recent & ((1u << TW) - 1u));
    __syncthreads();
    // Scores.  Address bits 4..7 of a row's chunk are (4 (k % 4) + g) ^ swz, so
    // step k is one exclusive-or away from step 0.  A ring keeps the reads some
    // steps ahead; the scheduling barriers keep the compiler from reading all
    // operands at once into registers that it does not have.
    const uint32_t ln = fresh((uint32_t)lane), lcol = ln & 15, lg = ln >> 4;
    const uint32_t ktok = (uint32_t)wt * 16 + lcol;
    const uint32_t krow = lds_at(&sc[0][0]) + b * kTileBytes + ktok * (DC * 2) + ((lg ^ (uint32_t)swz((int)ktok)) << 4);
    const uint32_t rrow = lds_at(&sr[0]) + ktok * (kRope * 2) + ((lg ^ (uint32_t)swz_rope((int)ktok)) << 4);
    auto key = [&](int k) {
      return k < KL ? lds_read16((krow ^ ((k & 3) << 6)) + (k >> 2) * 256) : lds_read16(rrow ^ ((k - KL) << 6));
    };
    // The next tile's loads.  Half the wavefronts, one of the two on each
    // SIMD, start them before their scores and half behind, so that one's
    // addresses are formed under the other's matrix products.
    auto ahead = [&] {
      if (i + 3 < tiles) fetch_chosen(i + 3);
      const uint32_t next = i + 2 < tiles ? fetch_page(i + 2) : ~0u;
      if (i + 1 < tiles) issue(i + 1, in);
      in = next;
      __builtin_amdgcn_sched_barrier(0);
    };
    if (w < NW / 2) ahead();
    const uint32_t shown = *(const uint16_t*)&svalid[i & 1][wt * 2];
    u32x4 ring[kAhead];
#pragma unroll
    for (int n = 0; n < kAhead - 1; ++n) ring[n] = key(n);
    f32x4 s[NH];
#pragma unroll
    for (int h = 0; h < NH; ++h) s[h] = f32x4{0, 0, 0, 0};
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int n = 0; n < KS; ++n) {
      if (n + kAhead - 1 < KS) ring[(n + kAhead - 1) % kAhead] = key(n + kAhead - 1);
#pragma unroll
      for (int h = 0; h < NH; ++h)
        s[h] = T::mfma16(ring[n % kAhead], n < KL ? q[h][n < KL ? n : 0] : lds_read16(rope_query(h, n < KL ? 0 : n - KL)), s[h]);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (w >= NW / 2) ahead();
    // Scaled and masked, and each head's maximum over the wavefront's tokens.
    const uint32_t bits = __builtin_amdgcn_readfirstlane(shown);
    float top[NH], kept[NH];
    bool past = false;
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      s[h] *= scale;
      if (bits != 0xffffu) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s[h][e] = (bits >> (lg * 4 + e)) & 1u ? s[h][e] : -INFINITY;
      }
      top[h] = max_xor32(max_xor16(fmaxf(fmaxf(s[h][0], s[h][1]), fmaxf(s[h][2], s[h][3]))));
      past = past || top[h] > ref[h] + kLazy;
      kept[h] = sum[h];
    }
    if (__builtin_amdgcn_ballot_w64(past) != 0 && ln == 0) sflag[i & 1] = i + 1;
    // Weights under the present reference.
    auto weights = [&] {
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        const float r = ref[h] == -INFINITY ? 0.0f : ref[h] - lift<T>(kLazy);
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = exp2_fast(s[h][e] - r);
        sum[h] = kept[h] + ((x[0] + x[1]) + (x[2] + x[3]));
        *(lds_u32x2*)(lds_at(sp_) + ((((wh * NH + h) * 16 + lcol) * PT + wt * 16 + lg * 4) * 2)) =
            u32x2{T::pack(x[0], x[1]), T::pack(x[2], x[3])};
      }
    };
    weights();
    __syncthreads();
    if (i + 1 < tiles) issue_rope();
    const int32_t flag = sflag[i & 1];
    // Values.  The wavefront's dims are 16 of every 128, so that they are a
    // fixed distance apart whatever the swizzle.
    const uint32_t prow = lds_at(sp_) + lcol * (PT * 2) + lg * 16;
    const uint32_t dims = (uint32_t)w * 2 + ((lcol & 3) >> 1);
    u32x4 v[ND];
    auto values = [&](int k) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const uint32_t tt = k * 32 + lg * 8 + half * 4 + (lcol >> 2);
        const uint32_t at = lds_at(&sc[0][0]) + b * kTileBytes + tt * (DC * 2) + ((dims ^ (uint32_t)swz((int)tt)) << 4) + (lcol & 1) * 8;
#pragma unroll
        for (int d = 0; d < ND; ++d) {
          const u32x2 x = lds_read_tr(at + d * 256);
          v[d][half * 2] = x[0], v[d][half * 2 + 1] = x[1];
        }
      }
    };
    values(0);
    __builtin_amdgcn_sched_barrier(0);
    if (__builtin_amdgcn_readfirstlane(flag) == i + 1) {
      // A new reference for every head, the maximum so far.
      if (ln < 16) {
#pragma unroll
        for (int h = 0; h < NH; ++h) smax[wt][(wh * NH + h) * 16 + ln] = top[h];
      }
      __syncthreads();
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        const int at = (wh * NH + h) * 16 + (int)lcol;
        float m = ref[h];
#pragma unroll
        for (int k = 0; k < WT; ++k) m = fmaxf(m, smax[k][at]);
        const float by = m == ref[h] ? 1.0f : exp2_fast(ref[h] - m);
        ref[h] = m;
        kept[h] *= by;
        if (wt == 0 && ln < 16) salpha[at] = by;
      }
      weights();
      __syncthreads();
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const float by = salpha[c * 16 + lcol];
#pragma unroll
        for (int d = 0; d < ND; ++d) o[c][d] *= by;
      }
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int k = 0; k < TT / 32; ++k) {
      u32x4 pw[2];
      pw[0] = lds_read16(prow + k * 64);
      if (k > 0) values(k);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        if (c + 1 < NC) pw[(c + 1) & 1] = lds_read16(prow + (c + 1) * (16 * PT * 2) + k * 64);
#pragma unroll
        for (int d = 0; d < ND; ++d) o[c][d] = T::mfma16(v[d], pw[c & 1], o[c][d]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }

  // Sums over the lanes and wavefronts that share a head.
#pragma unroll
  for (int h = 0; h < NH; ++h) {
    sum[h] += __shfl_xor(sum[h], 16);
    sum[h] += __shfl_xor(sum[h], 32);
    if (lane < 16) {
      ssum[wt][(wh * NH + h) * 16 + lane] = sum[h];
      if (wt == 0) smax[0][(wh * NH + h) * 16 + lane] = ref[h];
    }
  }
  __syncthreads();
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int32_t head = head0 + c * 16 + col;
    if (head >= a.num_heads) continue;
    float total = 0.0f;
#pragma unroll
    for (int k = 0; k < WT; ++k) total += ssum[k][c * 16 + col];
    const float m = smax[0][c * 16 + col] - lift<T>(kLazy);
    const int64_t at = (int64_t)row * a.num_heads + head;
    if (sp.parts == 1) {
      const float by = total == 0.0f ? 0.0f : by_cache / total;
#pragma unroll
      for (int d = 0; d < ND; ++d)
        *(u32x2*)((uint16_t*)a.out + at * DC + d * 128 + w * 16 + g * 4) =
            u32x2{T::pack(o[c][d][0] * by, o[c][d][1] * by), T::pack(o[c][d][2] * by, o[c][d][3] * by)};
      if (w == 0 && lane < 16 && a.lse != nullptr) a.lse[at] = total == 0.0f ? -INFINITY : (m + __log2f(total)) * kLn2;
    } else {
      const int64_t pi = at * p.most + part;
#pragma unroll
      for (int d = 0; d < ND; ++d)
        *(f32x4*)(p.part_out + pi * DC + d * 128 + w * 16 + g * 4) = o[c][d] * by_cache;
      if (w == 0 && lane < 16) p.part_stat[pi] = float2{m, total};
    }
  }
}

namespace {

template <typename T, bool F8, int DC, bool CHOSEN>
const void* latent_heads(int heads) {
  switch (heads) {
    case 32: return (const void*)&latent_kernel<T, F8, DC, CHOSEN, 32>;
    case 64: return (const void*)&latent_kernel<T, F8, DC, CHOSEN, 64>;
    default: return nullptr;
  }
}
template <typename T, bool F8>
const void* latent_dims(int head_dim, bool chosen, int heads) {
  if (head_dim == 256)
    return chosen ? latent_heads<T, F8, 256, true>(heads) : latent_heads<T, F8, 256, false>(heads);
  if (head_dim == 512)
    return chosen ? latent_heads<T, F8, 512, true>(heads) : latent_heads<T, F8, 512, false>(heads);
  return nullptr;
}

}  // namespace

const void* latent_kernel_ptr(int dtype, int store, int head_dim, bool chosen, int heads) {
  if (dtype == PAGED_BF16)
    return store == PAGED_E4M3 ? latent_dims<Bf16, true>(head_dim, chosen, heads)
                               : latent_dims<Bf16, false>(head_dim, chosen, heads);
  return store == PAGED_E4M3 ? latent_dims<Fp16, true>(head_dim, chosen, heads)
                             : latent_dims<Fp16, false>(head_dim, chosen, heads);
}

}  // namespace rrt
