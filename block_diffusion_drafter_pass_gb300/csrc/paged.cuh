// paged.cuh - what the operators over caller-owned page pools share: the
// device view of a batch, the token types, and the token -> (sequence,
// position) map.
//
// Page layout (one page = 64 tokens, as the contexts' own pools): keys
// [n_kv][64][d], then values transposed [n_kv][d][64], 16-bit elements; a
// pool is n_pages of them. Sequence i owns the new tokens q_start[i] ..
// q_start[i+1]-1 of the token buffers, and its cache holds kv_len[i] tokens,
// those new ones last: new token j sits at position kv_len - q_len + j, slot
// position % 64 of page page_table[i][position / 64].
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "dflash.h"
#include "internal.h"
#include "ptx.cuh"

namespace dfl {

constexpr int kPagedMaxSeqs = 1024;      // sequences of one call (their bounds are held in shared memory)
constexpr int kPagedMaxTable = 1 << 20;  // pages of one sequence: positions stay below 2^26, a batch's steps of keys below 2^30

// The batch as the kernels read it. All arrays are on the device.
struct PagedView {
  int n_heads, n_kv, group;   // query heads, kv heads, query heads per kv head
  int n_seq, n_tokens, n_pages;
  int table_pages;            // entries of one page-table row
  long long table_stride;
  const int32_t* page_table;
  const int32_t* q_start;     // [n_seq + 1]
  const int32_t* kv_len;      // [n_seq]
  uint16_t* pool;
  int32_t* status;
};

// Checks what the host can see of a batch; the message of the first fault, or null.
const char* paged_check(const dflash_paged_batch* b);
PagedView paged_view(const dflash_paged_batch& b);
inline bool misaligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) & 15; }
// A row stride, in elements, that rows of `width` elements with 16-byte loads allow.
inline bool bad_stride(long long s, long long width) { return s < width || s % 8 || s > (1ll << 36); }

// Whether two buffers of n rows of 16-bit elements share bytes. Columns of one
// wider matrix (equal strides) interleave without sharing any; other interleaved
// layouts count as shared.
inline bool rows_overlap(const void* x, long long x_stride, long long x_width, const void* y, long long y_stride,
                         long long y_width, long long n) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(x), b = reinterpret_cast<uintptr_t>(y);
  if (a > b) return rows_overlap(y, y_stride, y_width, x, x_stride, x_width, n);
  if (n < 1 || static_cast<uintptr_t>(((n - 1) * x_stride + x_width) * 2) <= b - a) return false;
  if (x_stride != y_stride || n == 1) return true;
  const long long off = static_cast<long long>((b - a) / 2 % x_stride);
  return off < x_width || off + y_width > x_stride;
}

// Whether a token buffer reaches into the batch's pool.
inline bool in_pool(const dflash_paged_batch& b, const void* x, long long stride, long long width) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(x), pool = reinterpret_cast<uintptr_t>(b.pool);
  const uintptr_t end = at + static_cast<uintptr_t>(((b.n_tokens - 1) * stride + width) * 2);
  const uintptr_t page = static_cast<uintptr_t>(2) * b.n_kv_heads * kPage * b.head_dim * 2;
  return at < pool + b.n_pages * page && pool < end;
}

template <bool F16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (F16) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  } else {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  }
}

template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if constexpr (F16) asm volatile("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm volatile("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// The bounds of the sequences' new tokens, read into shared memory as
// non-decreasing numbers within [0, n_tokens]: what a caller's broken array
// says otherwise is bent to that (and latched), so no index derived from it
// leaves a buffer. All threads of the block call it; ends with a barrier.
__device__ __forceinline__ void load_q_start(const PagedView& b, int* s_q) {
  bool bent = false;
  for (int i = threadIdx.x; i <= b.n_seq; i += blockDim.x) {
    const int raw = b.q_start[i], v = min(max(raw, 0), b.n_tokens);
    s_q[i] = v;
    bent |= v != raw;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < b.n_seq; i += blockDim.x) bent |= s_q[i + 1] < s_q[i];
  if (__syncthreads_or(bent)) {
    if (threadIdx.x == 0) {
      latch_status(b.status, kDevBounds);
      for (int i = 0; i < b.n_seq; ++i) s_q[i + 1] = max(s_q[i + 1], s_q[i]);
    }
    __syncthreads();
  }
}

// The sequence whose new tokens hold token t: the last i in [0, n_seq) with
// s_q[i] <= t (sequences without new tokens share their start with the next
// one and are passed over). t in [s_q[0], s_q[n_seq]).
__device__ __forceinline__ int seq_of_token(const int* s_q, int n_seq, int t) {
  int lo = 0, hi = n_seq - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s_q[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Cached tokens (`raw`, as kv_len says), bent to what a page-table row can hold.
__device__ __forceinline__ int cached_tokens(const PagedView& b, int raw) {
  const int v = min(max(raw, 0), b.table_pages * kPage);
  if (v != raw) latch_status(b.status, kDevBounds);
  return v;
}

}  // namespace dfl
