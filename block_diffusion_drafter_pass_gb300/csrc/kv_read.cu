// kv_read.cu - cached keys and values out of a caller's page pool, as rows of
// the token buffers: the way back of dflash_kv_append (its rotation stays).
//
// 16-bit pages are copied, 8-bit ones give code * scale, an exact product of
// fp32 rounded once to the tokens' type.
//
// Bound: memory, the pages read once, the rows written once. A block takes 64
// tokens of one kv head, whose rows lie together in a page: of 8-bit pages and
// of 16-bit keys a thread has 16 bytes of a row at a time, 16-bit values, which
// the pages hold transposed, are turned over in shared memory. Of 8-bit pages
// 150 thousand tokens (8 heads of 128) take 149 us, 92% of the copy bandwidth for
// codes and scales read and rows written; 300 tokens of 4 heads 2.7 us.
#include <cstring>

#include "paged.cuh"

namespace dfl {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 64;   // tokens of a block

struct ReadArgs {
  PagedView b;
  uint16_t *k, *v;
  long long k_stride, v_stride;   // elements between tokens
};

template <int D, bool F16>
__device__ __forceinline__ uint4 decode8(uint2 w, float scale) {
  uint4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t two = (i < 2 ? w.x : w.y) >> (16 * (i & 1));
    (&r.x)[i] = pack2<F16>((static_cast<int>(two & 255u) - 128) * scale, (static_cast<int>(two >> 8 & 255u) - 128) * scale);
  }
  return r;
}

template <int D, bool F16, bool Q8>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const __grid_constant__ ReadArgs a) {
  __shared__ int s_q[kPagedMaxSeqs + 1], s_len[kPagedMaxSeqs];
  __shared__ long long s_page[kTokens];   // the token's page in the pool, -1: none
  __shared__ int s_slot[kTokens];
  __shared__ uint32_t s_v[Q8 ? 1 : kTokens][D / 2 + 1];
  grid_dep_wait();
  grid_dep_launch();
  const int tid = threadIdx.x, n_kv = a.b.n_kv;
  const int t0 = blockIdx.x / n_kv * kTokens, h = blockIdx.x % n_kv;
  for (int i = tid; i < a.b.n_seq; i += kThreads) s_len[i] = a.b.kv_len[i];
  load_q_start(a.b, s_q);
  if (tid < kTokens) {
    const Place p = place_of(a.b, s_q, s_len, t0 + tid, n_kv * (Q8 ? q8_block_bytes(D) : 4ll * kPage * D));
    s_page[tid] = p.page;
    s_slot[tid] = p.slot;
  }
  __syncthreads();
  const uint8_t* pool = reinterpret_cast<const uint8_t*>(a.b.pool);
  if constexpr (Q8) {
    constexpr int kOf = D / 16;   // threads of a row
#pragma unroll
    for (int e = tid; e < kTokens * kOf; e += kThreads) {
      const int r = e / kOf, c = e % kOf;
      if (s_page[r] < 0) continue;
      const uint8_t* block = pool + s_page[r] + static_cast<long long>(h) * q8_block_bytes(D);
      const int at = s_slot[r] * D + c * 16;
      const uint4 kw = __ldg(reinterpret_cast<const uint4*>(block + at));
      const uint4 vw = __ldg(reinterpret_cast<const uint4*>(block + q8_values_at(D) + at));
      const float ks = __ldg(reinterpret_cast<const float*>(block + q8_key_scales_at(D)) + s_slot[r]);
      const float vs = __ldg(reinterpret_cast<const float*>(block + q8_value_scales_at(D)) + s_slot[r]);
      uint4* k = reinterpret_cast<uint4*>(a.k + (t0 + r) * a.k_stride + h * D + c * 16);
      uint4* v = reinterpret_cast<uint4*>(a.v + (t0 + r) * a.v_stride + h * D + c * 16);
      k[0] = decode8<D, F16>(make_uint2(kw.x, kw.y), ks);
      k[1] = decode8<D, F16>(make_uint2(kw.z, kw.w), ks);
      v[0] = decode8<D, F16>(make_uint2(vw.x, vw.y), vs);
      v[1] = decode8<D, F16>(make_uint2(vw.z, vw.w), vs);
    }
  } else {
    constexpr int kOf = D / 8;
    for (int e = tid; e < kTokens * kOf; e += kThreads) {
      const int r = e / kOf, c = e % kOf;
      if (s_page[r] < 0) continue;
      const uint16_t* row = reinterpret_cast<const uint16_t*>(pool + s_page[r]) + (h * kPage + s_slot[r]) * D;
      *reinterpret_cast<uint4*>(a.k + (t0 + r) * a.k_stride + h * D + c * 8) = __ldg(reinterpret_cast<const uint4*>(row) + c);
    }
    const int lane = tid & 31, warp = tid >> 5;
    for (int r = lane; r < kTokens; r += 32) {
      if (s_page[r] < 0) continue;
      const uint16_t* col = reinterpret_cast<const uint16_t*>(pool + s_page[r]) + ((n_kv + h) * D) * kPage + s_slot[r];
      for (int c = warp; c < D / 2; c += kThreads / 32)
        s_v[r][c] = __ldg(col + 2 * c * kPage) | static_cast<uint32_t>(__ldg(col + (2 * c + 1) * kPage)) << 16;
    }
    __syncthreads();
    for (int e = tid; e < kTokens * kOf; e += kThreads) {
      const int r = e / kOf, c = e % kOf;
      if (s_page[r] < 0) continue;
      *reinterpret_cast<uint4*>(a.v + (t0 + r) * a.v_stride + h * D + c * 8) =
          make_uint4(s_v[r][4 * c], s_v[r][4 * c + 1], s_v[r][4 * c + 2], s_v[r][4 * c + 3]);
    }
  }
}

}  // namespace
}  // namespace dfl

using namespace dfl;

extern "C" dflash_status dflash_kv_read(const dflash_paged_batch* b, void* k_out, long long k_stride, void* v_out,
                                        long long v_stride, void* stream) {
  auto refuse = [](const char* why) {
    set_unattached_error(why);
    return DFLASH_EINVAL;
  };
  if (const char* why = paged_check(b)) return refuse(why);
  if (b->n_seq == 0 || b->n_tokens == 0) return DFLASH_OK;
  if (!k_out || !v_out) return refuse("null pointer");
  const long long w = static_cast<long long>(b->n_kv_heads) * b->head_dim;
  if (bad_stride(k_stride, w) || bad_stride(v_stride, w))
    return refuse("token strides must be multiples of 8 elements and at least a token's row");
  if (misaligned16(k_out) || misaligned16(v_out)) return refuse("k_out and v_out must be 16-byte aligned");
  if (rows_overlap(k_out, k_stride, w, v_out, v_stride, w, b->n_tokens)) return refuse("k_out and v_out must not overlap");
  if (in_pool(*b, k_out, k_stride, w) || in_pool(*b, v_out, v_stride, w)) return refuse("k_out and v_out must not lie in the pool");
  ReadArgs a;
  std::memset(&a, 0, sizeof(a));
  a.b = paged_view(*b);
  a.k = static_cast<uint16_t*>(k_out);
  a.v = static_cast<uint16_t*>(v_out);
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  const long long blocks = (b->n_tokens + kTokens - 1ll) / kTokens * b->n_kv_heads;   // at most 2^25
  auto go = [&](auto kernel) {
    return launch_pdl(kernel, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, static_cast<cudaStream_t>(stream), a);
  };
  const bool f16 = b->dtype & DFLASH_FP16, wide = b->head_dim == 128;
  cudaError_t e;
  if (!(b->dtype & DFLASH_POOL_Q8)) e = wide ? go(kv_read_kernel<128, false, false>) : go(kv_read_kernel<64, false, false>);
  else if (wide) e = f16 ? go(kv_read_kernel<128, true, true>) : go(kv_read_kernel<128, false, true>);
  else e = f16 ? go(kv_read_kernel<64, true, true>) : go(kv_read_kernel<64, false, true>);
  if (e != cudaSuccess) {
    set_unattached_error("dflash_kv_read: kernel launch failed");
    return DFLASH_ECUDA;
  }
  return DFLASH_OK;
}
