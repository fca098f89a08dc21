// Device helpers of the paged-cache kernels: 16-bit types and their matrix
// instructions, e4m3 conversions, lane exchanges.
#pragma once

#include <hip/hip_runtime.h>

#include "paged_internal.h"

namespace rrt {

using f32x16 = float __attribute__((ext_vector_type(16)));
using f32x4 = float __attribute__((ext_vector_type(4)));
using u32x2 = uint32_t __attribute__((ext_vector_type(2)));
using u32x4 = uint32_t __attribute__((ext_vector_type(4)));
using bf16x2 = __bf16 __attribute__((ext_vector_type(2)));
using bf16x8 = __bf16 __attribute__((ext_vector_type(8)));
using f16x2 = _Float16 __attribute__((ext_vector_type(2)));
using f16x8 = _Float16 __attribute__((ext_vector_type(8)));

// The two 16-bit types.  pack: two fp32 values to a pair, each rounded to
// nearest even; from_e4m3: two of the four 8-bit values of a word, exactly;
// mfma16: D[16][16] += A[16][32] B[32][16], lane l holding A's row l % 16 and
// B's column l % 16 for the 8 values k = l / 16 * 8 .. + 8, and D's column
// l % 16 for the rows l / 16 * 4 .. + 4; mfma32: D[32][32] += A[32][16]
// B[16][32], A's row and B's column l % 32 for k = l / 32 * 8 .. + 8, D's column
// l % 32 for the rows 8 j + l / 32 * 4 + i as value 4 j + i.
// kLift: a softmax weight of at most 1 is kept times 2^kLift.  fp16 holds nothing
// below 2^-24 and full precision only from 2^-14 up, and the many small weights
// of a long row with one large one matter together: 65,535 weights of e^-18 are
// 1e-3 of the output, and were zeros beside a weight of 1.  2^15 is the most
// that fp16 takes; bf16 has the exponents of fp32 and needs none.  Sums are of
// lifted weights too, so an output does not change and a log-sum-exp by kLift.
struct Bf16 {
  using elem = __bf16;
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    bf16x2 v = {(__bf16)lo, (__bf16)hi};
    return __builtin_bit_cast(uint32_t, v);
  }
  static __device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
  static __device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
  template <bool HI>
  static __device__ __forceinline__ uint32_t from_e4m3(uint32_t w) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HI));
  }
  static __device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
  }
  static __device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
  }
  static constexpr float kLargest = 3.3895313892515355e38f;
  static constexpr float kLift = 0.0f;
};

struct Fp16 {
  using elem = _Float16;
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    f16x2 v = {(_Float16)lo, (_Float16)hi};
    return __builtin_bit_cast(uint32_t, v);
  }
  static __device__ __forceinline__ float lo(uint32_t w) { return (float)__builtin_bit_cast(f16x2, w)[0]; }
  static __device__ __forceinline__ float hi(uint32_t w) { return (float)__builtin_bit_cast(f16x2, w)[1]; }
  template <bool HI>
  static __device__ __forceinline__ uint32_t from_e4m3(uint32_t w) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, HI));
  }
  static __device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0,
                                                  0);
  }
  static __device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0,
                                                  0);
  }
  static constexpr float kLargest = 65504.0f;
  static constexpr float kLift = 15.0f;
};

// Eight e4m3 values (two words) to eight 16-bit ones (four words).
template <typename T>
__device__ __forceinline__ u32x4 widen(u32x2 w) {
  return u32x4{T::template from_e4m3<false>(w[0]), T::template from_e4m3<true>(w[0]),
               T::template from_e4m3<false>(w[1]), T::template from_e4m3<true>(w[1])};
}

__device__ __forceinline__ int64_t shfl64(int64_t v, int lane) {
  const int lo = __shfl((int)(uint32_t)v, lane), hi = __shfl((int)(v >> 32), lane);
  return (int64_t)(((uint64_t)(uint32_t)hi << 32) | (uint32_t)lo);
}

__device__ __forceinline__ int64_t readlane64(int64_t v, int lane) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, lane);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(v >> 32), lane);
  return (int64_t)(((uint64_t)hi << 32) | lo);
}

// Places of a lane's tokens, one a tile, `step` positions of the row apart.
// A place takes up to two dependent reads (the chosen position, its page);
// memory reads return in order, so each is issued one tile before it is
// needed and ahead of that tile's data, and nothing waits for it alone:
//   start(i); loop { off = take(); ... issue the data loads at off ... }
// take() returns the place of the next tile (in elements, -1: nothing there)
// and issues the reads for the two after it.
template <bool CHOSEN>
struct Places {
  const int32_t* table;
  const int32_t* chosen;
  int64_t page_stride, token_stride;
  Divisor by;          // page size
  int32_t num_pages, seen, end, step;
  int32_t at;          // row index of the entry in `ahead`
  int32_t ahead;       // the chosen position there
  int32_t page;        // the next tile's page
  uint32_t in;         // and the offset inside it, all ones where there is no position

  __device__ __forceinline__ int32_t read(int32_t i) const {
    if constexpr (CHOSEN) return chosen[i < end ? i : end - 1];
    return i;
  }
  __device__ __forceinline__ void look_up() {
    const bool ok = at < end && (!CHOSEN || (uint32_t)ahead < (uint32_t)seen);
    const uint32_t pos = ok ? (uint32_t)ahead : 0u, j = divide(pos, by);
    in = ok ? pos - j * by.by : ~0u;
    page = table[j];
    at += step;
    ahead = read(at);
  }
  __device__ __forceinline__ void start(int32_t i) {
    at = i;
    ahead = read(i);
    look_up();
  }
  __device__ __forceinline__ int64_t take() {
    const int64_t off = in == ~0u || (uint32_t)page >= (uint32_t)num_pages
                            ? -1
                            : (int64_t)page * page_stride + (int64_t)in * token_stride;
    look_up();
    return off;
  }
};

// The larger of a lane's value and that of the lane 16 (32) further or before:
// a register swap between rows of lanes, no trip through LDS.
__device__ __forceinline__ float max_xor16(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float max_xor32(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// The exponent's offset that lifts weights which are at most 2^lazy, relative to
// their reference.
template <typename T>
constexpr float lift(float lazy) {
  return T::kLift > lazy ? T::kLift - lazy : 0.0f;
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Which (group of rows, part) and which of its `inner` units (heads, column
// tiles) a workgroup takes.  Workgroups go to the eight XCDs in turn; all units
// of a (group, part) are given to one XCD, one after the other.  They read
// neighbouring bytes of the same tokens: with head h of every token on XCD
// h % 8 each XCD's L2 would see one 256-byte column of the cache, a fraction
// of its channels.
// Rows of chosen positions are alike: a group's parts go to one XCD, whose L2
// then holds its table once (64 rows of 2048 of up to 32768 positions: 70 us against
// 72).  Others: side by side, as a sequence on one XCD alone would leave the
// XCDs with unequal shares, and every other eight in the reverse order, so that
// none gets the longer of each two.  False past the last one.
struct Work {
  int32_t group, part, unit;
};
template <bool CHOSEN>
__device__ __forceinline__ bool work_of(uint32_t block, uint32_t inner, uint32_t groups, uint32_t most, Work* w) {
  const uint32_t idx = block >> 3, eight = idx / inner;
  w->unit = (int32_t)(idx % inner);
  if constexpr (CHOSEN) {
    const uint32_t outer = eight * 8 + (block & 7);
    w->part = (int32_t)(outer / groups);
    w->group = (int32_t)(outer - (uint32_t)w->part * groups);
    return w->part < (int32_t)most;
  }
  const uint32_t outer = eight * 8 + ((block & 7) ^ (eight & 1 ? 7u : 0u));
  w->group = (int32_t)(outer / most);
  w->part = (int32_t)(outer - (uint32_t)w->group * most);
  return w->group < (int32_t)groups;
}
// Groups longest first, within each 64 of them: the group that stands at place
// `at`.  What starts last ends the launch and is better short: 64 rows of 1 to
// 32768 positions x 8 heads took 880 us in their own order with a sequence's
// parts on one XCD, 755 so.  Wave uniform; every wavefront finds the same.
__device__ __forceinline__ int32_t by_length(const paged_attention_args& a, int32_t at, int32_t groups, int32_t group_rows,
                                             int64_t most, int lane) {
  const int32_t base = at & ~63, count = groups - base < 64 ? groups - base : 64;
  const bool here = lane < count;
  const int32_t len = here ? clamp_to(a.lengths[(int64_t)(base + lane) * group_rows + group_rows - 1], most) : -1;
  if (__builtin_amdgcn_ballot_w64(here && len != __builtin_amdgcn_readfirstlane(len)) == 0) return at;
  int32_t before = 0;
  for (int32_t j = 0; j < count; ++j) {
    const int32_t other = __builtin_amdgcn_readlane(len, j);
    before += other > len || (other == len && j < lane) ? 1 : 0;
  }
  return base + (int32_t)__builtin_ctzll(__builtin_amdgcn_ballot_w64(here && before == at - base));
}

constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kLog2e = 1.44269504088896340736f;

}  // namespace rrt
