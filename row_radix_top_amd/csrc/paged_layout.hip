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
// itself (256 segments of consecutive sequences, one a thread; the sequences'
// 8 bytes each come from L2), then takes its share of the tokens and of the
// new table entries, each found by a search over the segments in LDS and a
// walk inside one segment (no walk for up to 256 sequences).  A launch of two
// kernels with the sums in memory would read less and wait for a second
// launch, which costs more than the sums for any batch that is served.
// ---------------------------------------------------------------------------
constexpr int kLayoutBlock = 256;

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

// The last segment whose prefix is <= x (x is below the total, so the segment
// found holds it).
__device__ __forceinline__ int find_segment(const int32_t* prefix, int32_t x) {
  int lo = 0;
#pragma unroll
  for (int step = kLayoutBlock / 2; step > 0; step >>= 1)
    if (prefix[lo + step] <= x) lo += step;
  return lo;
}

__global__ void __launch_bounds__(kLayoutBlock) layout_kernel(LayoutParams p) {
  __shared__ int32_t tok[kLayoutBlock + 1], page[kLayoutBlock + 1];
  __shared__ int32_t wave_tok[4], wave_page[4];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int64_t most = table_tokens(p.table_width, p.page_size);
  const int32_t per = (p.num_seqs + kLayoutBlock - 1) / kLayoutBlock;
  const int64_t first = (int64_t)tid * per;
  int32_t nt = 0, np = 0;
  for (int32_t i = 0; i < per && first + i < p.num_seqs; ++i) {
    const SeqInfo q = seq_info(p, most, (int32_t)(first + i));
    nt += q.fresh;
    np += q.take;
  }
  int32_t it = nt, ip = np;  // inclusive sums over the wavefront, then the workgroup
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int32_t a = __shfl_up(it, off), b = __shfl_up(ip, off);
    if (lane >= off) it += a, ip += b;
  }
  if (lane == 63) wave_tok[w] = it, wave_page[w] = ip;
  __syncthreads();
  for (int i = 0; i < w; ++i) it += wave_tok[i], ip += wave_page[i];
  tok[tid] = it - nt;
  page[tid] = ip - np;
  if (tid == kLayoutBlock - 1) tok[kLayoutBlock] = it, page[kLayoutBlock] = ip;
  __syncthreads();
  const int32_t tokens = tok[kLayoutBlock], taken = page[kLayoutBlock];
  const uint32_t P = (uint32_t)p.page_size;

  if (blockIdx.x == 0) {
    int32_t at = tok[tid];
    for (int32_t i = 0; i < per && first + i < p.num_seqs; ++i) {
      p.starts[first + i] = at;
      at += seq_info(p, most, (int32_t)(first + i)).fresh;
    }
    if (tid == 0) p.starts[p.num_seqs] = tokens, p.pages[0] = taken;
  }

  const int64_t gid = (int64_t)blockIdx.x * kLayoutBlock + tid, step = (int64_t)gridDim.x * kLayoutBlock;
  for (int64_t t = gid; t < p.capacity; t += step) {
    int32_t slot = -1, length = 0, seq = -1;
    if (t < tokens) {
      const int seg = find_segment(tok, (int32_t)t);
      int32_t at = tok[seg], pg = page[seg];
      seq = seg * per;
      SeqInfo q = seq_info(p, most, seq);
      while (at + q.fresh <= t) {
        at += q.fresh;
        pg += q.take;
        q = seq_info(p, most, ++seq);
      }
      const int32_t pos = q.len - q.fresh + ((int32_t)t - at);
      const int32_t j = (int32_t)((uint32_t)pos / P);
      int32_t id;
      if (j < q.held) {
        id = p.table[(int64_t)seq * p.table_stride + j];
      } else {  // a page of this step: its table entry may not be written yet
        const int32_t i = pg + (j - q.held);
        id = i < p.num_free ? p.free_pages[i] : -1;
      }
      slot = id < 0 ? -1 : id * p.page_size + (int32_t)((uint32_t)pos % P);
      length = pos + 1;
    }
    p.slots[t] = slot;
    p.row_lengths[t] = length;
    p.row_seqs[t] = seq;
  }
  for (int64_t i = gid; i < taken; i += step) {
    const int seg = find_segment(page, (int32_t)i);
    int32_t pg = page[seg], seq = seg * per;
    SeqInfo q = seq_info(p, most, seq);
    while (pg + q.take <= i) {
      pg += q.take;
      q = seq_info(p, most, ++seq);
    }
    p.table[(int64_t)seq * p.table_stride + q.held + ((int32_t)i - pg)] = i < p.num_free ? p.free_pages[i] : -1;
  }
}

// ---------------------------------------------------------------------------
// Append.  One work item is 8 consecutive elements of a part's row (wide: all
// strides and pointers allow 16-byte loads and 16- or 8-byte stores) or one
// element.  A copy: bound by its bytes, or by the launch for a decode step.
// ---------------------------------------------------------------------------
constexpr int kAppendBlock = 256;

// x / scale to e4m3, to nearest even; magnitudes past 448 become 448, NaN
// stays NaN (the comparisons are false for it).
__device__ __forceinline__ float saturate(float x, float scale) {
  float y = x / scale;
  y = y > 448.0f ? 448.0f : y;
  return y < -448.0f ? -448.0f : y;
}

template <typename T, bool F8>
__device__ __forceinline__ void append_item(const AppendParams& p, const paged_part& q, int64_t t, int64_t slot,
                                            int32_t c, bool wide) {
  const uint32_t P = (uint32_t)p.page_size;
  const int64_t pg = (int64_t)((uint64_t)slot / P);
  const int64_t base = pg * q.dst_page_stride + (slot - pg * P) * q.dst_token_stride;
  const int32_t col = wide ? c * 8 : c;
  const int32_t head = col / q.head_width;
  const int64_t to = base + head * q.dst_head_stride + (col - head * q.head_width);
  const uint16_t* src = (const uint16_t*)q.src + t * q.src_stride + col;
  const float scale = F8 && q.scales != nullptr ? q.scales[head] : 1.0f;
  if (wide) {
    const u32x4 x = *(const u32x4*)src;
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
    const float y = saturate(T::lo(*src), scale);
    ((uint8_t*)q.dst)[to] = (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(y, y, 0, false);
  } else {
    ((uint16_t*)q.dst)[to] = *src;
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
    if (slot < 0 || slot >= p.num_slots) continue;
    const bool second = c >= p.chunks[0];
    if (second) c -= p.chunks[0];
    append_item<T, F8>(p, p.part[second ? 1 : 0], t, slot, c, WIDE);
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
