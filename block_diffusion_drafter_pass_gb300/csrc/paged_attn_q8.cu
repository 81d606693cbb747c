// paged_attn_q8.cu - the attention of paged_attn.cu over 8-bit pages: the same
// rows, masks and prefixes, with keys and values that stand for code * scale.
//
// One warp takes one row (token, head): lanes take keys for the scores and head
// dims for the product with the values, page by page with a running maximum and
// sum, everything in fp32.
#include "paged_walk.cuh"

namespace dfl {
namespace {

constexpr int kRowWarps = 8;

template <int D, bool F16>
__global__ void __launch_bounds__(kRowWarps * 32) paged_rows_q8_kernel(const __grid_constant__ PagedAttnArgs a) {
  __shared__ int s_q[kPagedMaxSeqs + 1];
  grid_dep_wait();
  grid_dep_launch();
  load_q_start(a.b, s_q);
  const int lane = threadIdx.x & 31, n_q = a.b.n_heads;
  const long long row = static_cast<long long>(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
  const int t = static_cast<int>(row / n_q), head = static_cast<int>(row % n_q), kvh = head / a.b.group;
  if (t < s_q[0] || t >= s_q[a.b.n_seq]) return;
  const int i = seq_of_token(s_q, a.b.n_seq, t);
  const int len = cached_tokens(a.b, a.b.kv_len[i]);
  const int pos = len - s_q[i + 1] + t;
  const uint16_t* q = a.q + t * a.q_stride + static_cast<long long>(head) * D;
  float m = -INFINITY, l = 0.f, acc[D / 32] = {};
  for (int run = 0; run < 2; ++run) {
    if (run == 0 && a.prefix_len == 0) continue;
    const int32_t* table = run == 0 ? a.prefix_table : a.b.page_table + i * a.b.table_stride;
    const int end = run == 0 ? a.prefix_len : len;
    RowSpan sp{0, a.causal ? pos : kNoEnd, 0};
    if (run == 0) sp.hi = a.causal ? pos + a.prefix_len : kNoEnd;
    else if (a.window > 0) sp.lo = max(0, pos - a.window + 1), sp.sinks = a.sinks;
    for (int key0 = 0; key0 < end; key0 += kPage) {
      const unsigned long long vis = sp.hi >= 0 ? row_sees(sp, key0, end) : 0ull;
      if (vis == 0) continue;
      const int page = table[key0 / kPage];
      if (page < 0 || page >= a.b.n_pages) {
        if (lane == 0) latch_status(a.b.status, kDevBounds);
        continue;
      }
      const uint8_t* block = reinterpret_cast<const uint8_t*>(a.b.pool) + (static_cast<long long>(page) * a.b.n_kv + kvh) * q8_block_bytes(D);
      const float* ks = reinterpret_cast<const float*>(block + q8_key_scales_at(D));
      const float* vs = reinterpret_cast<const float*>(block + q8_value_scales_at(D));
      float s[2] = {-INFINITY, -INFINITY};
      for (int u = 0; u < 2; ++u) {
        const int c = lane + 32 * u;
        if (!(vis >> c & 1)) continue;
        float x = 0.f;
        for (int e = 0; e < D; e += 2) {
          const float2 f = unpack2<F16>(*reinterpret_cast<const uint32_t*>(q + e));
          x = fmaf(f.x, static_cast<int>(block[c * D + e]) - 128, x);
          x = fmaf(f.y, static_cast<int>(block[c * D + e + 1]) - 128, x);
        }
        s[u] = x * ks[c] * a.scale_log2;
      }
      float mx = fmaxf(s[0], s[1]);
      for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const float nm = fmaxf(m, mx), ref = nm == -INFINITY ? 0.f : nm, alpha = exp2f(m - ref);
      float p[2], w[2], sum = 0.f;
      for (int u = 0; u < 2; ++u) {
        const int c = lane + 32 * u;
        const bool sees = vis >> c & 1;
        p[u] = sees ? exp2f(s[u] - ref) : 0.f;
        w[u] = sees ? p[u] * vs[c] : 0.f;
        sum += p[u];
      }
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      l = l * alpha + sum;
      m = nm;
      for (int e = 0; e < D / 32; ++e) acc[e] *= alpha;
      for (int c = 0; c < kPage; ++c) {
        const float wc = __shfl_sync(0xffffffffu, c < 32 ? w[0] : w[1], c & 31);
        if (!(vis >> c & 1)) continue;
        for (int e = 0; e < D / 32; ++e)
          acc[e] = fmaf(wc, static_cast<int>(block[q8_values_at(D) + c * D + lane * (D / 32) + e]) - 128, acc[e]);
      }
    }
  }
  const float f = l > 0.f || l != l ? 1.f / l : 0.f;
  uint16_t* o = out_row(a, t, kvh, head % a.b.group, D) + lane * (D / 32);
  for (int e = 0; e < D / 32; e += 2) *reinterpret_cast<uint32_t*>(o + e) = pack2<F16>(acc[e] * f, acc[e + 1] * f);
}

__global__ void no_pieces_kernel(const __grid_constant__ PagedAttnArgs a) {
  grid_dep_wait();
  a.split[blockIdx.x] = make_int4(0, 0, 0, 0);
  a.piece[blockIdx.x] = 0;
}

}  // namespace

cudaError_t launch_paged_attn_q8(const PagedAttnArgs& a, int head_dim, bool f16, int, int ctas, cudaStream_t s) {
  const long long blocks = (static_cast<long long>(a.b.n_tokens) * a.b.n_heads + kRowWarps - 1) / kRowWarps;
  cudaError_t e = launch_pdl(no_pieces_kernel, dim3(ctas), dim3(1), 0, s, a);
  if (e != cudaSuccess) return e;
  auto go = [&](auto kernel) { return launch_pdl(kernel, dim3(static_cast<unsigned>(blocks)), dim3(kRowWarps * 32), 0, s, a); };
  if (head_dim == 128) return f16 ? go(paged_rows_q8_kernel<128, true>) : go(paged_rows_q8_kernel<128, false>);
  return f16 ? go(paged_rows_q8_kernel<64, true>) : go(paged_rows_q8_kernel<64, false>);
}

}  // namespace dfl
