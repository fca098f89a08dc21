// Block tables and slot maps of a serving step, and the write of its new
// tokens into the paged cache.

#include "paged_device.hpp"

namespace rrt {

// ---------------------------------------------------------------------------
// Layout.  With held = ceil((len - new) / P) and need = ceil(len / P), sequence
// s takes need - held pages from the free list, after those of the sequences
// before it, and its new token i sits at position len - new + i.  Everything a
// token or a new table entry needs is two prefix sums over the sequences.
//
// One launch and no workspace: every workgroup forms both prefix sums by
// itself (2048 segments of consecutive sequences, two a thread; the sequences'
// 8 bytes each come from L2), then takes its share of the tokens and of the
// new table entries, each found by a search over the segments in LDS and a
// walk inside one segment (no walk for up to 2048 sequences).  A launch of two
// kernels with the sums in memory would read less and wait for a second
// launch, which costs more than the sums for any batch that is served.
//
// Bound by the chain of waits (lengths, sums, search, table), not by bytes, so
// a segment's first position lies in LDS too and a workgroup is 1024 threads,
// a token each: 2048 sequences with 66,400 new tokens took 12.1 us with 256
// threads, 256 segments and walks through memory, 6.7 us so.
//
// Sums stop at 2^31 - 1: lengths whose sum passes that leave a table of the
// first tokens, as any other sum past the capacity does.
// ---------------------------------------------------------------------------
constexpr int kSegments = 2 * kLayoutBlock;

struct SeqInfo {
  int32_t len, fresh, held, take;  // tokens, new tokens, pages held before and taken now
};

__device__ __forceinline__ SeqInfo seq_info(const LayoutParams& p, int64_t most, int32_t s) {
  SeqInfo q;
  q.len = clamp_to(p.lengths[s], most);
  q.fresh = clamp_to(p.new_tokens[s], q.len);
  const uint32_t P = (uint32_t)p.page_size;
  q.held = (int32_t)(((uint32_t)(q.len - q.fresh) + P - 1) / P);
  q.take = (int32_t)(((uint32_t)q.len + P - 1) / P) - q.held;
  return q;
}

__device__ __forceinline__ int32_t plus(int32_t a, int32_t b) { return __builtin_elementwise_add_sat(a, b); }

// The last segment whose prefix is <= x (x is below the total, so the segment
// found holds it); `top`: the largest power of two below the segments in use.
__device__ __forceinline__ int find_segment(const int32_t* prefix, int top, int32_t x) {
  int lo = 0;
  for (int step = top; step > 0; step >>= 1)
    if (prefix[lo + step] <= x) lo += step;
  return lo;
}

__global__ void __launch_bounds__(kLayoutBlock) layout_kernel(LayoutParams p) {
  constexpr int W = kLayoutBlock / 64;
  __shared__ int32_t tok[kSegments + 1], page[kSegments + 1];
  __shared__ SeqInfo info[kSegments];  // of a segment's first sequence
  __shared__ __align__(16) int32_t wave_tok[W], wave_page[W];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int64_t most = table_tokens(p.table_width, p.page_size);
  const int32_t per = (int32_t)(((int64_t)p.num_seqs + kSegments - 1) / kSegments);
  const int32_t used = per == 0 ? 0 : (p.num_seqs - 1) / per + 1;
  const int top = used > 1 ? 1 << (31 - __builtin_clz((uint32_t)(used - 1))) : 0;
  int32_t nt[2] = {0, 0}, np[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int64_t first = (int64_t)(tid * 2 + j) * per;
    if (first >= p.num_seqs) continue;
    const SeqInfo q = seq_info(p, most, (int32_t)first);
    info[tid * 2 + j] = q;
    nt[j] = q.fresh;
    np[j] = q.take;
  }
  for (int32_t i = 1; i < per; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int64_t s = (int64_t)(tid * 2 + j) * per + i;
      if (s >= p.num_seqs) continue;
      const SeqInfo q = seq_info(p, most, (int32_t)s);
      nt[j] = plus(nt[j], q.fresh);
      np[j] = plus(np[j], q.take);
    }
  int32_t it = plus(nt[0], nt[1]), ip = plus(np[0], np[1]);  // sums up to here: the wavefront's, the workgroup's
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int32_t a = __shfl_up(it, off), b = __shfl_up(ip, off);
    if (lane >= off) it = plus(it, a), ip = plus(ip, b);
  }
  const int32_t bt = __shfl_up(it, 1), bp = __shfl_up(ip, 1);
  if (lane == 63) wave_tok[w] = it, wave_page[w] = ip;
  __syncthreads();
  int32_t at_tok = lane == 0 ? 0 : bt, at_page = lane == 0 ? 0 : bp, tokens = 0, taken = 0;
#pragma unroll
  for (int i = 0; i < W; ++i) {
    if (i < w) at_tok = plus(at_tok, wave_tok[i]), at_page = plus(at_page, wave_page[i]);
    tokens = plus(tokens, wave_tok[i]);
    taken = plus(taken, wave_page[i]);
  }
  tok[tid * 2] = at_tok;
  page[tid * 2] = at_page;
  tok[tid * 2 + 1] = plus(at_tok, nt[0]);
  page[tid * 2 + 1] = plus(at_page, np[0]);
  if (tid == 0) tok[kSegments] = tokens, page[kSegments] = taken;
  __syncthreads();
  const uint32_t P = (uint32_t)p.page_size;

  if (blockIdx.x == 0) {
    for (int seg = tid; seg < used; seg += kLayoutBlock) {
      int32_t at = tok[seg];
      for (int32_t i = 0; i < per && (int64_t)seg * per + i < p.num_seqs; ++i) {
        const int32_t s = seg * per + i;
        p.starts[s] = at;
        if (i + 1 < per) at = plus(at, (i == 0 ? info[seg] : seq_info(p, most, s)).fresh);
      }
    }
    if (tid == 0) p.starts[p.num_seqs] = tokens, p.pages[0] = taken;
  }

  const int64_t gid = (int64_t)blockIdx.x * kLayoutBlock + tid, step = (int64_t)gridDim.x * kLayoutBlock;
  for (int64_t t = gid; t < p.capacity; t += step) {
    int32_t slot = -1, length = 0, seq = -1;
    if (t < tokens) {
      const int seg = find_segment(tok, top, (int32_t)t);
      int32_t at = tok[seg], pg = page[seg];
      seq = seg * per;
      SeqInfo q = info[seg];
      while (plus(at, q.fresh) <= t) {
        at += q.fresh;
        pg = plus(pg, q.take);
        q = seq_info(p, most, ++seq);
      }
      const int32_t pos = q.len - q.fresh + ((int32_t)t - at);
      const int32_t j = (int32_t)((uint32_t)pos / P);
      int32_t id;
      if (j < q.held) {
        id = p.table[(int64_t)seq * p.table_stride + j];
      } else {  // a page of this step: its table entry may not be written yet
        const int32_t i = plus(pg, j - q.held);
        id = i < p.num_free ? p.free_pages[i] : -1;
      }
      const int64_t place = (int64_t)id * p.page_size + (int32_t)((uint32_t)pos % P);
      slot = id < 0 || place > INT32_MAX ? -1 : (int32_t)place;
      length = pos + 1;
    }
    p.slots[t] = slot;
    p.row_lengths[t] = length;
    p.row_seqs[t] = seq;
  }
  for (int64_t i = gid; i < taken; i += step) {
    const int seg = find_segment(page, top, (int32_t)i);
    int32_t pg = page[seg], seq = seg * per;
    SeqInfo q = info[seg];
    while (plus(pg, q.take) <= i) {
      pg += q.take;
      q = seq_info(p, most, ++seq);
    }
    p.table[(int64_t)seq * p.table_stride + q.held + ((int32_t)i - pg)] = i < p.num_free ? p.free_pages[i] : -1;
  }
}

// ---------------------------------------------------------------------------
// Append.  One work item is 8 consecutive elements of a part's row (wide: all
// strides and pointers allow 16-byte loads and 16- or 8-byte stores) or one
// element.  A copy: bound by its bytes, or by the launch for a decode step
// (3 us).  16,000 latent tokens of 576 values rounded to 8 bits, 27.6 MB, take
// 11.5 us; four items a thread in flight took 12.5, and a quotient from
// the scale's inverse instead of the division saved nothing that showed.
// ---------------------------------------------------------------------------

// x / scale to e4m3, to nearest even; magnitudes past 448 become 448, NaN
// stays NaN (the comparisons are false for it).
__device__ __forceinline__ float saturate(float x, float scale) {
  float y = x / scale;
  y = y > 448.0f ? 448.0f : y;
  return y < -448.0f ? -448.0f : y;
}

template <typename T, bool F8>
__device__ __forceinline__ void append_item(const AppendParams& p, const paged_part& q, int64_t slot,
                                            int32_t c, bool wide, u32x4 x) {
  const uint32_t P = (uint32_t)p.page_size;
  const int64_t pg = (int64_t)((uint64_t)slot / P);
  const int64_t base = pg * q.dst_page_stride + (slot - pg * P) * q.dst_token_stride;
  const int32_t col = wide ? c * 8 : c;
  const int32_t head = col / q.head_width;
  const int64_t to = base + head * q.dst_head_stride + (col - head * q.head_width);
  const float scale = F8 && q.scales != nullptr ? q.scales[head] : 1.0f;
  if (wide) {
    if constexpr (F8) {
      u32x2 y;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        int w = 0;
        w = __builtin_amdgcn_cvt_pk_fp8_f32(saturate(T::lo(x[2 * i]), scale), saturate(T::hi(x[2 * i]), scale), w,
                                            false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(saturate(T::lo(x[2 * i + 1]), scale),
                                            saturate(T::hi(x[2 * i + 1]), scale), w, true);
        y[i] = (uint32_t)w;
      }
      *(u32x2*)((uint8_t*)q.dst + to) = y;
    } else {
      *(u32x4*)((uint16_t*)q.dst + to) = x;
    }
  } else if constexpr (F8) {
    const float y = saturate(T::lo(x[0]), scale);
    ((uint8_t*)q.dst)[to] = (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(y, y, 0, false);
  } else {
    ((uint16_t*)q.dst)[to] = (uint16_t)x[0];
  }
}

template <typename T, bool F8, bool WIDE>
__global__ void __launch_bounds__(kAppendBlock) append_kernel(AppendParams p) {
  const uint32_t each = (uint32_t)(p.chunks[0] + p.chunks[1]);
  const int64_t items = (int64_t)p.num_tokens * each;
  const int64_t step = (int64_t)gridDim.x * kAppendBlock;
  for (int64_t i = (int64_t)blockIdx.x * kAppendBlock + threadIdx.x; i < items; i += step) {
    const int64_t t = (uint64_t)i >> 32 ? i / each : (int64_t)((uint32_t)i / each);
    int32_t c = (int32_t)(i - t * each);
    const int64_t slot = p.slots[t];
    const bool second = c >= p.chunks[0];
    if (second) c -= p.chunks[0];
    const paged_part& q = p.part[second ? 1 : 0];
    const uint16_t* src = (const uint16_t*)q.src + t * q.src_stride + (WIDE ? c * 8 : c);
    u32x4 x = {};  // read beside the slot, not after it
    if constexpr (WIDE) x = *(const u32x4*)src;
    else x[0] = *src;
    if (slot < 0 || slot >= p.num_slots) continue;
    append_item<T, F8>(p, q, slot, c, WIDE, x);
  }
}

const void* layout_kernel_ptr() { return (const void*)&layout_kernel; }

const void* append_kernel_ptr(int dtype, int store, bool wide) {
  const bool bf = dtype == PAGED_BF16;
  if (store == PAGED_E4M3) {
    if (bf) return wide ? (const void*)&append_kernel<Bf16, true, true> : (const void*)&append_kernel<Bf16, true, false>;
    return wide ? (const void*)&append_kernel<Fp16, true, true> : (const void*)&append_kernel<Fp16, true, false>;
  }
  return wide ? (const void*)&append_kernel<Bf16, false, true> : (const void*)&append_kernel<Bf16, false, false>;
}

}  // namespace rrt
