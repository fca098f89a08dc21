// The absorbed form of latent attention: all heads of a row read one shared
// vector a token, as keys whole and as values without its rope part.

#include "paged_device.hpp"

namespace rrt {

// ---------------------------------------------------------------------------
// o_h = softmax(s q_h c^T) c[:DC], for HT heads of one row and one part of its
// positions a workgroup.
//
// 2 (2 DC + 64) flop a head and token against 2 (DC + 64) bytes a token: with
// 128 heads near the card's balance of matrix rate and memory rate, with few
// heads bound by memory.  Every token's vector is used by all heads and twice
// (scores, values), so a tile of TT tokens is staged in LDS once, in 16 bits,
// two buffers deep: the next tile's loads go straight to LDS while this one is
// used (an e4m3 cache goes through registers, where it is widened).
//
//   S^T[token][head] = C Q^T: WH x WT wavefronts split heads and tokens; each
//     keeps the queries of its heads in registers for the whole part.
//   O^T[dim][head] += C^T P^T: each wavefront owns a quarter of the value dims
//     for all heads, so the values are read from LDS once in all; their
//     transpose is the LDS read instruction's.  P passes through LDS.
//
// The weights are relative to a reference that follows the running maximum
// lazily: only when a score passes it by 2^8 does the workgroup agree on a new
// one and rescale (P then stays below 2^8, sums below 2^8 n: far inside
// fp32; relative precision does not depend on the reference).  So most tiles
// take two barriers and no rescaling.
//
// LDS rows are a multiple of all banks wide; 16-byte chunk c of token t's row
// is kept at c ^ swizzle(t), which spreads both the 16 tokens of a key operand
// and the 4 tokens x 2 chunks of a transposed read over the banks.
// ---------------------------------------------------------------------------
constexpr int kRope = PAGED_ROPE_DIM;
constexpr float kLazy = 8.0f;
constexpr int kAhead = 4;  // operands in flight from LDS

using i16x4 = short __attribute__((ext_vector_type(4)));
using lds_i16x4 = __attribute__((address_space(3))) i16x4;
using lds_u32x4 = __attribute__((address_space(3))) u32x4;
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

constexpr int latent_waves(int heads) { return heads == 32 ? 8 : 4; }

template <int DC, int HT>
struct LatentShape {
  static constexpr int NW = latent_waves(HT);        // wavefronts
  static constexpr int TT = 64;                     // tokens of a tile
  static constexpr int WT = HT == 64 ? 2 : 4;                   // wavefronts along the tokens of the scores
  static constexpr int WH = NW / WT;                // and along the heads
  static constexpr int NH = HT / 16 / WH;           // 16-head columns of a wavefront's scores
  static constexpr int NU = TT / 16 / WT;           // 16-token rows of a wavefront's scores
  static constexpr int KS = (DC + kRope) / 32;      // matrix steps over the key dims
  static constexpr int ND = DC / 16 / NW;           // 16-dim rows of a wavefront's output
  static constexpr int NC = HT / 16;                // 16-head columns of the output
  static constexpr int PT = TT + 16;                // pitch of the weights (rows 40 banks apart)
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

// 64 lanes x 16 bytes from the lanes' addresses to 1 KB of LDS at `to` (wave
// uniform); counted by vmcnt, no registers are written.
__device__ __forceinline__ void load_to_lds(const char* from, uint32_t to) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) uint32_t*)from,
                                   (__attribute__((address_space(3))) uint32_t*)(uintptr_t)to, 16, 0, 0);
}
__device__ __forceinline__ void wait_loads() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

template <typename T, bool F8, int DC, bool CHOSEN, int HT>
__global__ void __launch_bounds__(latent_waves(HT) * 64, latent_waves(HT) / 4) latent_kernel(AttnParams p) {
  using S = LatentShape<DC, HT>;
  constexpr int TT = S::TT, NH = S::NH, NU = S::NU, KS = S::KS, ND = S::ND, NC = S::NC, PT = S::PT, WT = S::WT, NW = S::NW;
  constexpr int TW = TT / NW;  // tokens that a wavefront loads
  constexpr int SZ = F8 ? 1 : 2;
  __shared__ __align__(1024) uint16_t sc[2][TT * DC];
  __shared__ __align__(1024) uint16_t sr[2][TT * kRope];
  __shared__ __align__(16) uint16_t sp_[HT * PT];
  __shared__ float smax[WT][HT], ssum[WT][HT], salpha[HT];
  __shared__ uint32_t svalid[2][NW];
  __shared__ uint32_t sflag[2];
  const paged_attention_args& a = p.a;
  const int tid = threadIdx.x, lane = tid & 63, col = lane & 15, g = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wh = w % S::WH, wt = w / S::WH;

  Work work;
  if (!work_of(blockIdx.x, (uint32_t)p.col_tiles, (uint32_t)p.groups, (uint32_t)p.most, &work)) return;
  const int32_t part = work.part, row = work.group, head0 = work.unit * HT;
  const int64_t most = table_tokens(a.table_width, a.page_size);
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

  // Places of the wavefront's token `lane % TW` of each tile.
  Places<CHOSEN> places{table, chosen, a.page_stride, a.token_stride, p.page, a.num_pages, seen, end, TT};

  // --- loads of a tile -----------------------------------------------------
  constexpr int LT = F8 ? DC / 16 : DC / 8;      // lanes (16 bytes each) of a token's latent part
  constexpr int PER = 64 / LT;                   // tokens of one load
  constexpr int NL = TW / PER;                   // loads
  constexpr int RT = F8 ? 4 : 8;                 // lanes of a token's rope part
  constexpr int NR = (TW * RT + 63) / 64;        // loads of the rope parts
  u32x4 stage[F8 ? NL : 1], stage_r[F8 ? NR : 1];

  auto issue = [&](int64_t off, int b) {
    const uint32_t valid = (uint32_t)__builtin_amdgcn_ballot_w64(off >= 0) & (TW == 32 ? ~0u : (1u << TW) - 1u);
    if (lane == 0) svalid[b][w] = valid;
    const int64_t at = (off < 0 ? 0 : off) * SZ;
    const int lane = (int)fresh((uint32_t)threadIdx.x & 63u);
    int64_t rope_at[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) rope_at[i] = shfl64(at, (i * (64 / RT) + lane / RT) & (TW - 1));
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int t = i * PER + lane / LT;  // of the wavefront's tokens
      const int c = lane % LT;
      int64_t place = readlane64(at, i * PER);
#pragma unroll
      for (int k = 1; k < PER; ++k) place = lane / LT >= k ? readlane64(at, i * PER + k) : place;
      const char* from = cache + place;
      if constexpr (F8) {
        stage[i] = *(const u32x4*)(from + c * 16);
      } else {
        const int tt = w * TW + t;
        load_to_lds(from + (uint32_t)((c ^ swz(tt)) * 16), lds_at(&sc[b][(w * TW + i * PER) * DC]));
      }
    }
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const int t = i * (64 / RT) + lane / RT;
      const int c = lane % RT;
      const char* from = cache + rope_at[i] + DC * SZ;
      if constexpr (F8) {
        stage_r[i] = *(const u32x4*)(from + c * 16);
      } else {
        const int tt = w * TW + t;
        load_to_lds(from + ((c ^ swz_rope(tt)) * 16), lds_at(&sr[b][(w * TW + i * (64 / RT)) * kRope]));
      }
    }
  };
  // e4m3: the staged tile, widened, into its buffer.
  auto store = [&](int b) {
    if constexpr (F8) {
      const int lane = (int)fresh((uint32_t)threadIdx.x & 63u);
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        const int tt = w * TW + i * PER + lane / LT, c = (lane % LT) * 2;
        u32x4* rowp = (u32x4*)&sc[b][tt * DC];
        rowp[c ^ swz(tt)] = widen<T>(u32x2{stage[i][0], stage[i][1]});
        rowp[(c + 1) ^ swz(tt)] = widen<T>(u32x2{stage[i][2], stage[i][3]});
      }
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        const int t = i * (64 / RT) + lane / RT, c = (lane % RT) * 2;
        if (t >= TW) continue;
        const int tt = w * TW + t;
        u32x4* rowp = (u32x4*)&sr[b][tt * kRope];
        rowp[c ^ swz_rope(tt)] = widen<T>(u32x2{stage_r[i][0], stage_r[i][1]});
        rowp[(c + 1) ^ swz_rope(tt)] = widen<T>(u32x2{stage_r[i][2], stage_r[i][3]});
      }
    }
  };

  if (tiles > 0) {
    places.start(begin + w * TW + (lane & (TW - 1)));
    issue(places.take(), 0);
  }

  // Queries of the wavefront's heads, as the scores' second operand.
  u32x4 q[NH][KS];
#pragma unroll
  for (int h = 0; h < NH; ++h) {
    const int32_t head = head0 + (wh * NH + h) * 16 + col;
    // Columns past the last head compute a copy of head 0 that is not written.
    const char* qp = (const char*)a.q + 2 * ((int64_t)row * a.q_row_stride +
                                             (int64_t)(head < a.num_heads ? head : 0) * a.q_head_stride);
#pragma unroll
    for (int i = 0; i < KS; ++i) q[h][i] = *(const u32x4*)(qp + 2 * (i * 32 + g * 8));
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
  if (tiles > 0) store(0);

  for (int32_t i = 0; i < tiles; ++i) {
    const int b = i & 1;
    if constexpr (!F8) wait_loads();
    // Tokens that do not count become zeros: their places may hold NaN.
    {
      const uint32_t mine = __builtin_amdgcn_readfirstlane(svalid[b][w]);
      constexpr uint32_t all = TW == 32 ? ~0u : (1u << TW) - 1u;
      if (mine != all) {
        for (int t = 0; t < TW; ++t) {
          if ((mine >> t) & 1u) continue;
          const int tt = w * TW + t;
          for (int c = lane; c < DC / 8; c += 64) ((u32x4*)&sc[b][tt * DC])[c] = u32x4{0, 0, 0, 0};
          if (lane < 8) ((u32x4*)&sr[b][tt * kRope])[lane] = u32x4{0, 0, 0, 0};
        }
      }
    }
    __syncthreads();
    if (tid == 0) sflag[b ^ 1] = 0;
    if (i + 1 < tiles) issue(places.take(), b ^ 1);

    // Scores.  Address bits 4..7 of a row's chunk are (4 (k % 4) + g) ^ swz, so
    // step k is one exclusive-or away from step 0.
    const uint32_t ln = fresh((uint32_t)lane), lcol = ln & 15, lg = ln >> 4;
    const uint32_t buf = lds_at(&sc[0][0]) + (uint32_t)b * (TT * DC * 2), bufr = lds_at(&sr[0][0]) + (uint32_t)b * (TT * kRope * 2);
    uint32_t krow[NU], rrow[NU];
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const uint32_t tt = (uint32_t)(wt * NU + u) * 16 + lcol;
      krow[u] = buf + tt * (DC * 2) + ((lg ^ (uint32_t)swz((int)tt)) << 4);
      rrow[u] = bufr + tt * (kRope * 2) + ((lg ^ (uint32_t)swz_rope((int)tt)) << 4);
    }
    f32x4 s[NH][NU];
#pragma unroll
    for (int h = 0; h < NH; ++h)
#pragma unroll
      for (int u = 0; u < NU; ++u) s[h][u] = f32x4{0, 0, 0, 0};
    // A ring of key operands, so that reads are some steps ahead; the barriers
    // keep the scheduler from reading all of them at once into registers that
    // the accumulators need.
    auto key = [&](int k, int u) {
      return k < DC / 32 ? lds_read16((krow[u] ^ ((k & 3) << 6)) + (k >> 2) * 256)
                         : lds_read16(rrow[u] ^ ((k - DC / 32) << 6));
    };
    u32x4 kk[kAhead][NU];
#pragma unroll
    for (int k = 0; k < kAhead - 1; ++k)
#pragma unroll
      for (int u = 0; u < NU; ++u) kk[k][u] = key(k, u);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      if (k + kAhead - 1 < KS) {
#pragma unroll
        for (int u = 0; u < NU; ++u) kk[(k + kAhead - 1) % kAhead][u] = key(k + kAhead - 1, u);
      }
#pragma unroll
      for (int u = 0; u < NU; ++u)
#pragma unroll
        for (int h = 0; h < NH; ++h) s[h][u] = T::mfma16(kk[k % kAhead][u], q[h][k], s[h][u]);
      __builtin_amdgcn_sched_barrier(0);
    }
    float top[NH];
    uint64_t valid = 0;
#pragma unroll
    for (int k = NW - 1; k >= 0; --k) valid = (valid << TW) | __builtin_amdgcn_readfirstlane(svalid[b][k]);
    constexpr uint64_t every = TT == 64 ? ~0ull : (1ull << (TT & 63)) - 1ull;
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      top[h] = -INFINITY;
#pragma unroll
      for (int u = 0; u < NU; ++u) {
        s[h][u] *= scale;
        if (valid != every) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            s[h][u][e] = (valid >> ((wt * NU + u) * 16 + g * 4 + e)) & 1u ? s[h][u][e] : -INFINITY;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) top[h] = fmaxf(top[h], s[h][u][e]);
      }
      top[h] = fmaxf(top[h], __shfl_xor(top[h], 16));
      top[h] = fmaxf(top[h], __shfl_xor(top[h], 32));
    }
    auto weights = [&]() {
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        const float r = ref[h] == -INFINITY ? 0.0f : ref[h];
#pragma unroll
        for (int u = 0; u < NU; ++u) {
          float x[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = exp2_fast(s[h][u][e] - r);
          sum[h] += (x[0] + x[1]) + (x[2] + x[3]);
          *(u32x2*)&sp_[((wh * NH + h) * 16 + col) * PT + (wt * NU + u) * 16 + g * 4] =
              u32x2{T::pack(x[0], x[1]), T::pack(x[2], x[3])};
        }
      }
    };
    bool past = false;
#pragma unroll
    for (int h = 0; h < NH; ++h) past = past || top[h] > ref[h] + kLazy;
    if (__builtin_amdgcn_ballot_w64(past) != 0) {
      if (lane == 0) sflag[b] = 1;
    }
    float kept[NH];
#pragma unroll
    for (int h = 0; h < NH; ++h) kept[h] = sum[h];
    weights();
    __syncthreads();
    if (__builtin_amdgcn_readfirstlane(sflag[b]) != 0) {
      // A new reference for every head, the maximum so far.
      if (lane < 16) {
#pragma unroll
        for (int h = 0; h < NH; ++h) smax[wt][(wh * NH + h) * 16 + lane] = top[h];
      }
      __syncthreads();
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        const int at = (wh * NH + h) * 16 + col;
        float m = ref[h];
#pragma unroll
        for (int k = 0; k < WT; ++k) m = fmaxf(m, smax[k][at]);
        const float by = m == ref[h] ? 1.0f : exp2_fast(ref[h] - m);
        ref[h] = m;
        sum[h] = kept[h] * by;
        if (wt == 0 && lane < 16) salpha[at] = by;
      }
      weights();
      __syncthreads();
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const float by = salpha[c * 16 + col];
#pragma unroll
        for (int d = 0; d < ND; ++d) o[c][d] *= by;
      }
    }

    // Values.  Dims d of the wavefront's quarter: again an exclusive-or away.
    const uint32_t prow = lds_at(sp_) + lcol * (PT * 2) + lg * 16;
#pragma unroll
    for (int k = 0; k < TT / 32; ++k) {
      u32x4 pw[NC];
#pragma unroll
      for (int c = 0; c < NC; ++c) pw[c] = lds_read16(prow + c * (16 * PT * 2) + k * 64);
      uint32_t vrow[2];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const uint32_t tt = k * 32 + lg * 8 + half * 4 + (lcol >> 2);
        const uint32_t chunk = (uint32_t)w * (DC / 8 / NW) + ((lcol & 3) >> 1);
        vrow[half] = buf + tt * (DC * 2) + ((chunk ^ (uint32_t)swz((int)tt)) << 4) + (lcol & 1) * 8;
      }
      auto value = [&](int d) {
        const u32x2 x = lds_read_tr(vrow[0] ^ (d << 5)), y = lds_read_tr(vrow[1] ^ (d << 5));
        return u32x4{x[0], x[1], y[0], y[1]};
      };
      u32x4 v[kAhead];
#pragma unroll
      for (int d = 0; d < kAhead - 1 && d < ND; ++d) v[d] = value(d);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int d = 0; d < ND; ++d) {
        if (d + kAhead - 1 < ND) v[(d + kAhead - 1) % kAhead] = value(d + kAhead - 1);
#pragma unroll
        for (int c = 0; c < NC; ++c) o[c][d] = T::mfma16(v[d % kAhead], pw[c], o[c][d]);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if (i + 1 < tiles) store(b ^ 1);
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
    const float m = smax[0][c * 16 + col];
    const int64_t at = (int64_t)row * a.num_heads + head;
    if (sp.parts == 1) {
      const float by = total == 0.0f ? 0.0f : by_cache / total;
#pragma unroll
      for (int d = 0; d < ND; ++d)
        *(u32x2*)((uint16_t*)a.out + at * DC + w * (DC / NW) + d * 16 + g * 4) =
            u32x2{T::pack(o[c][d][0] * by, o[c][d][1] * by), T::pack(o[c][d][2] * by, o[c][d][3] * by)};
      if (w == 0 && lane < 16 && a.lse != nullptr) a.lse[at] = total == 0.0f ? -INFINITY : (m + __log2f(total)) * kLn2;
    } else {
      const int64_t pi = at * p.most + part;
#pragma unroll
      for (int d = 0; d < ND; ++d)
        *(f32x4*)(p.part_out + pi * DC + w * (DC / NW) + d * 16 + g * 4) = o[c][d] * by_cache;
      if (w == 0 && lane < 16) p.part_stat[pi] = float2{m, total};
    }
  }
}

namespace {

template <typename T, bool F8, int DC, bool CHOSEN>
const void* latent_heads(int heads) {
  switch (heads) {
    case 16: return (const void*)&latent_kernel<T, F8, DC, CHOSEN, 16>;
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

int latent_threads(int heads) { return latent_waves(heads) * 64; }

const void* latent_kernel_ptr(int dtype, int store, int head_dim, bool chosen, int heads) {
  if (dtype == PAGED_BF16)
    return store == PAGED_E4M3 ? latent_dims<Bf16, true>(head_dim, chosen, heads)
                               : latent_dims<Bf16, false>(head_dim, chosen, heads);
  return store == PAGED_E4M3 ? latent_dims<Fp16, true>(head_dim, chosen, heads)
                             : latent_dims<Fp16, false>(head_dim, chosen, heads);
}

}  // namespace rrt
