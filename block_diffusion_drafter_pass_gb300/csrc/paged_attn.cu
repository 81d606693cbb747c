// paged_attn.cu - attention of ragged query blocks over a caller's page pool:
// over each sequence's own cache, with a sliding window and first tokens that
// stay visible, or over one prefix that all sequences share and then their own
// cache.
//
// Row (token t, head h) of sequence i at position p = kv_len - q_len + j:
//     o = sum_k w_k v_k / sum_k w_k,  w_k = exp(scale q.k),  k over what it sees:
// causal keys k <= p; with a window those with k > p - window or k < sinks.
// Behind a prefix of P tokens the sequence's own positions start at P, and the
// prefix is seen whole (up to P + p when a cache holds fewer tokens than the
// block has). A row that sees nothing is zero.
//
// One warp per (token, head), page by page with the running maximum and sum of
// the softmax.
#include <cmath>
#include <cstring>

#include "paged.cuh"
#include "paged_row.cuh"

namespace dfl {
namespace {

constexpr int kWarps = 4;

struct PagedAttnArgs {
  PagedView b;
  const int32_t* prefix_table;
  int prefix_len;
  const uint16_t* q;
  long long q_stride;
  uint16_t* out;
  long long out_stride;
  int window, sinks, causal;
  float scale_log2;
};

template <int D, bool F16>
__global__ void __launch_bounds__(kWarps * 32) paged_rows_kernel(const __grid_constant__ PagedAttnArgs a) {
  __shared__ int s_q[kPagedMaxSeqs + 1];
  __shared__ int s_part[kWarps];
  grid_dep_wait();
  grid_dep_launch();
  load_q_start(a.b, s_q, s_part);
  const int lane = threadIdx.x & 31, h = blockIdx.x * kWarps + (threadIdx.x >> 5), t = blockIdx.y;
  if (h >= a.b.n_heads || t < s_q[0] || t >= s_q[a.b.n_seq]) return;
  const int i = seq_of_token(s_q, a.b.n_seq, t);
  const int len = cached_tokens(a.b, i);
  const int pos = len - (s_q[i + 1] - s_q[i]) + (t - s_q[i]);
  const int kvh = h / a.b.group;
  const uint16_t* q = a.q + t * a.q_stride + h * D;
  const size_t page_elems = static_cast<size_t>(2) * a.b.n_kv * kPage * D;
  RowState<D> r;
  r.clear();
  auto walk = [&](const int32_t* table, const RowSpan& span, int end) {
    const int pages = (min(end, span.hi == INT32_MAX ? end : span.hi + 1) + kPage - 1) / kPage;
    for (int g = 0; g < pages; ++g) {
      const unsigned long long vis = row_sees(span, g * kPage, end);
      if (vis == 0) continue;
      const int page = table[g];
      if (page < 0 || page >= a.b.n_pages) {
        if (lane == 0) latch_status(a.b.status, kDevBounds);
        continue;
      }
      const uint16_t* kp = a.b.pool + page * page_elems + static_cast<size_t>(kvh) * kPage * D;
      row_page<D, F16>(r, q, kp, kp + static_cast<size_t>(a.b.n_kv) * kPage * D, a.scale_log2, vis, lane);
    }
  };
  if (a.prefix_len > 0)
    walk(a.prefix_table, RowSpan{0, a.causal ? a.prefix_len + pos : INT32_MAX, 0}, a.prefix_len);
  walk(a.b.page_table + i * a.b.table_stride,
       RowSpan{a.window > 0 ? max(0, pos - a.window + 1) : 0, a.causal ? pos : INT32_MAX, a.sinks}, len);
  const float inv = r.l > 0.f || r.l != r.l ? 1.f / r.l : 0.f;
  uint16_t* o = a.out + t * a.out_stride + h * D + lane * (D / 32);
#pragma unroll
  for (int e = 0; e < D / 32; e += 2)
    *reinterpret_cast<uint32_t*>(o + e) = pack2<F16>(r.acc[e] * inv, r.acc[e + 1] * inv);
}

const char* attn_check(const dflash_paged_batch* b, const void* q, long long q_stride, const void* out,
                       long long out_stride, float scale) {
  if (const char* why = paged_check(b)) return why;
  if (!(scale > 0.f) || !std::isfinite(scale)) return "scale must be positive and finite";
  if (b->n_seq == 0 || b->n_tokens == 0) return nullptr;
  const long long width = static_cast<long long>(b->n_heads) * b->head_dim;
  if (!q || !out) return "null pointer";
  if (bad_stride(q_stride, width) || bad_stride(out_stride, width))
    return "token strides must be multiples of 8 elements and at least a token's row";
  if (misaligned16(q) || misaligned16(out)) return "q and out must be 16-byte aligned";
  return nullptr;
}

dflash_status run(const dflash_paged_batch& b, PagedAttnArgs& a, void* workspace, size_t workspace_bytes, void* stream) {
  (void)workspace;
  (void)workspace_bytes;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const dim3 grid((b.n_heads + kWarps - 1) / kWarps, b.n_tokens);
  cudaError_t e;
  if (b.head_dim == 128) {
    e = b.dtype == DFLASH_FP16 ? launch_pdl(paged_rows_kernel<128, true>, grid, dim3(kWarps * 32), 0, s, a)
                               : launch_pdl(paged_rows_kernel<128, false>, grid, dim3(kWarps * 32), 0, s, a);
  } else {
    e = b.dtype == DFLASH_FP16 ? launch_pdl(paged_rows_kernel<64, true>, grid, dim3(kWarps * 32), 0, s, a)
                               : launch_pdl(paged_rows_kernel<64, false>, grid, dim3(kWarps * 32), 0, s, a);
  }
  if (e != cudaSuccess) {
    set_unattached_error("paged attention: kernel launch failed");
    return DFLASH_ECUDA;
  }
  return DFLASH_OK;
}

PagedAttnArgs attn_args(const dflash_paged_batch& b, const void* q, long long q_stride, void* out, long long out_stride,
                        int causal, float scale) {
  PagedAttnArgs a;
  std::memset(&a, 0, sizeof(a));
  a.b = paged_view(b);
  a.q = static_cast<const uint16_t*>(q);
  a.q_stride = q_stride;
  a.out = static_cast<uint16_t*>(out);
  a.out_stride = out_stride;
  a.causal = causal ? 1 : 0;
  a.scale_log2 = scale * 1.4426950408889634f;
  return a;
}

dflash_status refuse(const char* why) {
  set_unattached_error(why);
  return DFLASH_EINVAL;
}

}  // namespace
}  // namespace dfl

using namespace dfl;

extern "C" dflash_status dflash_paged_attn_workspace(const dflash_paged_batch* b, size_t* bytes) {
  if (!bytes) return refuse("null pointer");
  *bytes = 0;
  if (const char* why = paged_check(b)) return refuse(why);
  return DFLASH_OK;
}

extern "C" dflash_status dflash_paged_attn(const dflash_paged_batch* b, const void* q, long long q_stride, void* out,
                                           long long out_stride, int window, int sinks, int causal, float scale,
                                           void* workspace, size_t workspace_bytes, void* stream) {
  if (const char* why = attn_check(b, q, q_stride, out, out_stride, scale)) return refuse(why);
  if (window < 0 || sinks < 0) return refuse("window and sinks must not be negative");
  if (b->n_seq == 0 || b->n_tokens == 0) return DFLASH_OK;
  PagedAttnArgs a = attn_args(*b, q, q_stride, out, out_stride, causal, scale);
  a.window = window;
  a.sinks = window > 0 ? sinks : 0;
  return run(*b, a, workspace, workspace_bytes, stream);
}

extern "C" dflash_status dflash_shared_prefix_attn(const dflash_paged_batch* b, const int32_t* prefix_table,
                                                   int prefix_len, const void* q, long long q_stride, void* out,
                                                   long long out_stride, int causal, float scale, void* workspace,
                                                   size_t workspace_bytes, void* stream) {
  if (const char* why = attn_check(b, q, q_stride, out, out_stride, scale)) return refuse(why);
  if (prefix_len < 0 || prefix_len > (1 << 30)) return refuse("prefix_len must be 0..2^30");
  if (b->n_seq == 0 || b->n_tokens == 0) return DFLASH_OK;
  if (prefix_len > 0 && !prefix_table) return refuse("null pointer");
  PagedAttnArgs a = attn_args(*b, q, q_stride, out, out_stride, causal, scale);
  a.prefix_table = prefix_table;
  a.prefix_len = prefix_len;
  return run(*b, a, workspace, workspace_bytes, stream);
}
