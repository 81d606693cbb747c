// kv_append.cu - new keys and values into a caller's page pool, with the
// position rotation applied on the way, and the queries rotated beside them.
//
// Rotation of pair (x_i, x_{i+d/2}) of a head row at position p: by the angle
// p * base^(-2i/d). The angle's fraction of a turn is what cos and sin need,
// and at far positions a float (or float product) has lost it, so the host
// gives base^(-2i/d) / (2 pi) as a 64-bit fraction of a turn and the kernel
// multiplies by p in integers: whole turns fall off the top, exactly. The
// fraction comes from doubles: two powers (1 ulp each), 2 pi, a quotient and a
// product, together less than 2^-50 of it, so the angle is off by at most
// |p| * 2^-50 rad: 2^-24 at the farthest cache position (2^26), 2^-19 at the
// farthest int32 (found over 400 bases: 2^-20.8). sincospif takes it from there.
//
// Bound: memory, q, k and v read once, q and the pages written once.
// Queries and keys: one thread per (token, 8 pairs), which computes its 8
// rotations once and walks up to 8 heads with them: 16-byte loads and stores,
// 128 bytes of a head row in a row of lanes. Values: one block per (64
// tokens, kv head) turns the rows over in shared memory, since the pages hold
// them transposed. Few tokens are cut finer (fewer heads a thread, ranges of
// the values' dims), until the blocks fill the device: one token of 32
// sequences (32 + 8 + 8 heads of 128) takes 3.4 us, with whole blocks 6.4;
// 10.6 thousand tokens take 46 us, 83% of the copy bandwidth for q, k and v
// read and written once.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "paged.cuh"

namespace dfl {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxHeads = 8;   // heads one thread rotates with the same angles, at most
constexpr int kAtOnce = 2;     // of them under way together (4 took registers, and 4% at 260 MB)
constexpr int kVTokens = 64;   // tokens of a value block
constexpr int kQ8Threads = 128, kQ8Ahead = 2;   // 8-bit pages

struct AppendArgs {
  PagedView b;
  const uint16_t *k, *v, *q;
  long long k_stride, v_stride, q_stride, out_stride;   // elements between tokens
  uint16_t* q_out;
  const int32_t* positions;        // [n_tokens] rotation positions, or null: the cache positions
  int rotate;
  int heads;                       // heads of a rotation block
  int qk_tiles, qk_groups;         // blocks of the rotation part: token tiles x head groups
  int v_split;                     // value blocks that share a (tokens, head): ranges of dims
  unsigned long long turn[64];     // base^(-2i/d) / (2 pi) in units of 2^-64 turns
};

// The rotations of 8 pairs at position `at`.
__device__ __forceinline__ void rotation(const AppendArgs& a, long long at, int oct, float (&cs)[8], float (&sn)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const unsigned long long turns = static_cast<unsigned long long>(at) * a.turn[oct * 8 + e];
    // the signed upper half is the fraction of a turn in units of 2^-32
    const float half_turns = static_cast<float>(static_cast<int32_t>(turns >> 32)) * 0x1p-31f;
    sincospif(half_turns, &sn[e], &cs[e]);
  }
}

template <int D, bool F16>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int kOct = D / 16;                 // threads of a token: 8 pairs each
  constexpr int kTokens = kThreads / kOct;
  __shared__ int s_q[kPagedMaxSeqs + 1], s_len[kPagedMaxSeqs];
  __shared__ long long s_dst[kVTokens];        // values: element offset of the token's column, -1: none
  __shared__ uint32_t s_v[kVTokens][D / 2 + 1];
  grid_dep_wait();
  grid_dep_launch();
  const int tid = threadIdx.x;
  const int n_kv = a.b.n_kv;
  for (int i = tid; i < a.b.n_seq; i += kThreads) s_len[i] = a.b.kv_len[i];
  // The rows are read as soon as their addresses are known, before what says
  // where they go (a short call is the chain of these reads).
  if (static_cast<int>(blockIdx.x) < a.qk_tiles * a.qk_groups) {
    const int tile = blockIdx.x / a.qk_groups, grp = blockIdx.x % a.qk_groups;
    const int t = tile * kTokens + tid / kOct, oct = tid % kOct;
    const int n_q = a.q ? a.b.n_heads : 0;
    const int h0 = grp * a.heads, h1 = t < a.b.n_tokens ? min(n_q + n_kv, h0 + a.heads) : h0;
    uint4 lo[kAtOnce], hi[kAtOnce];
    auto read = [&](int h) {
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        if (h + u >= h1) continue;
        const uint16_t* src = h + u < n_q ? a.q + t * a.q_stride + (h + u) * D : a.k + t * a.k_stride + (h + u - n_q) * D;
        lo[u] = __ldg(reinterpret_cast<const uint4*>(src + oct * 8));
        hi[u] = __ldg(reinterpret_cast<const uint4*>(src + D / 2 + oct * 8));
      }
    };
    read(h0);
    load_q_start(a.b, s_q);
    const Place p = place_of(a.b, s_q, s_len, t, 2ll * n_kv * kPage * D);
    if (p.pos < 0) return;
    float cs[8], sn[8];
    if (a.rotate) rotation(a, a.positions ? a.positions[t] : p.pos, oct, cs, sn);
#pragma unroll 1
    for (int h = h0; h < h1; h += kAtOnce) {
      if (h > h0) read(h);
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        const bool is_q = h + u < n_q;
        if (h + u >= h1 || (!is_q && p.page < 0)) continue;
        uint16_t* dst = is_q ? a.q_out + t * a.out_stride + (h + u) * D
                             : a.b.pool + p.page + (static_cast<long long>(h + u - n_q) * kPage + p.slot) * D;
        uint4 ro = lo[u], rh = hi[u];
        if (a.rotate) {
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const float2 x = unpack2<F16>((&lo[u].x)[w]), y = unpack2<F16>((&hi[u].x)[w]);
            (&ro.x)[w] = pack2<F16>(x.x * cs[2 * w] - y.x * sn[2 * w], x.y * cs[2 * w + 1] - y.y * sn[2 * w + 1]);
            (&rh.x)[w] = pack2<F16>(y.x * cs[2 * w] + x.x * sn[2 * w], y.y * cs[2 * w + 1] + x.y * sn[2 * w + 1]);
          }
        }
        *reinterpret_cast<uint4*>(dst + oct * 8) = ro;
        *reinterpret_cast<uint4*>(dst + D / 2 + oct * 8) = rh;
      }
    }
    return;
  }
  const int vb = (blockIdx.x - a.qk_tiles * a.qk_groups) / a.v_split;
  const int t0 = vb / n_kv * kVTokens, h = vb % n_kv;
  // this block's dims, in pieces of 8
  const int of = D / 8 / a.v_split, c0 = (blockIdx.x - a.qk_tiles * a.qk_groups) % a.v_split * of, c1 = c0 + of;
  constexpr int kPieces = kVTokens * (D / 8) / kThreads;
  uint4 rows[kPieces];
#pragma unroll
  for (int u = 0; u < kPieces; ++u) {
    const int e = tid + u * kThreads, r = e / (D / 8), c = e % (D / 8);
    rows[u] = make_uint4(0, 0, 0, 0);
    if (t0 + r < a.b.n_tokens && c >= c0 && c < c1) rows[u] = __ldg(reinterpret_cast<const uint4*>(a.v + (t0 + r) * a.v_stride + h * D + c * 8));
  }
  load_q_start(a.b, s_q);
  if (tid < kVTokens) {
    const Place p = place_of(a.b, s_q, s_len, t0 + tid, 2ll * n_kv * kPage * D);
    s_dst[tid] = p.page < 0 ? -1 : p.page + (static_cast<long long>(n_kv) * kPage + h * kPage) * D + p.slot;
  }
#pragma unroll
  for (int u = 0; u < kPieces; ++u) {
    const int e = tid + u * kThreads, r = e / (D / 8), c = e % (D / 8);
#pragma unroll
    for (int w = 0; w < 4; ++w) s_v[r][c * 4 + w] = (&rows[u].x)[w];
  }
  __syncthreads();
  const int lane = tid & 31, warp = tid >> 5;
#pragma unroll
  for (int half = 0; half < kVTokens / 32; ++half) {
    const int r = half * 32 + lane;
    const long long at = s_dst[r];
    if (at < 0) continue;
    for (int c = c0 * 4 + warp; c < c1 * 4; c += kThreads / 32) {
      const uint32_t w = s_v[r][c];
      a.b.pool[at + (2 * c) * kPage] = static_cast<uint16_t>(w);
      a.b.pool[at + (2 * c + 1) * kPage] = static_cast<uint16_t>(w >> 16);
    }
  }
}

// Rows for 8-bit pages, in blocks of kOct lanes: each holds 8 pairs (or, of
// values, the same 16 places) of a head row. The row's largest magnitude is a
// maximum of bit patterns, under which NaN and infinity come out on top; such a
// row is held as the scale NaN, so that all of it reads back as NaN.
template <int D>
__device__ __forceinline__ void write_q8(const float (&x)[16], uint8_t* codes, float* scale, int oct, unsigned group) {
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < 16; ++e) top = max(top, __float_as_uint(x[e]) & 0x7FFFFFFFu);
#pragma unroll
  for (int o = D / 32; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(group, top, o));
  const float most = __uint_as_float(top);
  const bool finite = top < 0x7F800000u, held = finite && most >= kQ8Least;
  const float inv = held ? __fdiv_rn(kQ8Codes, most) : 0.f;
  // the nearest code (halves to the even one) and 128, in the low byte of a float's bits
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    uint32_t b[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) b[c] = __float_as_uint(__fadd_rn(__fmul_rn(x[4 * e + c], inv), 12582912.f + 128.f));
    w[e] = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
    if (!held) w[e] = 0x80808080u;
  }
  *reinterpret_cast<uint2*>(codes + oct * 8) = make_uint2(w[0], w[1]);
  *reinterpret_cast<uint2*>(codes + D / 2 + oct * 8) = make_uint2(w[2], w[3]);
  if (oct == 0) *scale = held ? __fdiv_rn(most, kQ8Codes) : finite ? 0.f : __uint_as_float(0x7FC00000u);
}

// The same work for 8-bit pages. Keys and values alike lie in rows there, so one
// walk takes queries, keys and values, and a thread's 16 values of a row are
// quantised where they are. kQ8Ahead rows are under way while one is worked on:
// 10.6 thousand tokens (32 + 8 + 8 heads of 128) take 45 us, 78% of the copy
// bandwidth; with loads between the rows 56, and 52 in blocks of 128 then; 4 rows
// ahead, 16 heads a thread and blocks of 256 or 64 are within 3 us of it. One token
// of 32 sequences takes 3.4 us.
template <int D, bool F16>
__global__ void __launch_bounds__(kQ8Threads) kv_append_q8_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int kOct = D / 16;                 // threads of a token: 8 pairs each
  constexpr int kTokens = kQ8Threads / kOct;
  __shared__ int s_q[kPagedMaxSeqs + 1], s_len[kPagedMaxSeqs];
  grid_dep_wait();
  grid_dep_launch();
  const int tid = threadIdx.x, n_kv = a.b.n_kv;
  for (int i = tid; i < a.b.n_seq; i += kQ8Threads) s_len[i] = a.b.kv_len[i];
  const int tile = blockIdx.x / a.qk_groups, grp = blockIdx.x % a.qk_groups;
  const int t = tile * kTokens + tid / kOct, oct = tid % kOct;
  const unsigned group = ((1u << kOct) - 1u) << (tid & 31 & ~(kOct - 1));   // the lanes of the token
  const int n_q = a.q ? a.b.n_heads : 0;
  const int h0 = grp * a.heads, h1 = t < a.b.n_tokens ? min(n_q + 2 * n_kv, h0 + a.heads) : h0;
  uint4 lo[kQ8Ahead], hi[kQ8Ahead];   // of the next heads, under way
  auto read = [&](int h, int u) {
    const int i = h - n_q;   // below 0: a query
    if (h >= h1) return;
    const uint16_t* src = i < 0 ? a.q + t * a.q_stride + h * D
                          : i < n_kv ? a.k + t * a.k_stride + i * D : a.v + t * a.v_stride + (i - n_kv) * D;
    lo[u] = __ldg(reinterpret_cast<const uint4*>(src + oct * 8));
    hi[u] = __ldg(reinterpret_cast<const uint4*>(src + D / 2 + oct * 8));
  };
#pragma unroll
  for (int u = 0; u < kQ8Ahead; ++u) read(h0 + u, u);
  load_q_start(a.b, s_q);
  const Place p = place_of(a.b, s_q, s_len, t, static_cast<long long>(n_kv) * q8_block_bytes(D));
  if (p.pos < 0) return;
  float cs[8], sn[8];
  if (a.rotate && h0 < n_q + n_kv) rotation(a, a.positions ? a.positions[t] : p.pos, oct, cs, sn);
  uint8_t* const page = reinterpret_cast<uint8_t*>(a.b.pool) + p.page;
#pragma unroll 1
  for (int h = h0; h < h1; h += kQ8Ahead) {
#pragma unroll
    for (int u = 0; u < kQ8Ahead; ++u) {
      const int i = h + u - n_q;
      if (h + u >= h1) continue;
      const uint4 wl = lo[u], wh = hi[u];
      read(h + u + kQ8Ahead, u);
      if (i >= 0 && p.page < 0) continue;
      float x[16];
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float2 f = unpack2<F16>((&wl.x)[w]), g = unpack2<F16>((&wh.x)[w]);
        x[2 * w] = f.x, x[2 * w + 1] = f.y, x[8 + 2 * w] = g.x, x[9 + 2 * w] = g.y;
      }
      if (a.rotate && i < n_kv) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float f = x[e], g = x[8 + e];
          x[e] = f * cs[e] - g * sn[e];
          x[8 + e] = g * cs[e] + f * sn[e];
        }
      }
      if (i < 0) {
        uint16_t* dst = a.q_out + t * a.out_stride + (h + u) * D;
        uint4 ro = wl, rh = wh;
        if (a.rotate) {
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            (&ro.x)[w] = pack2<F16>(x[2 * w], x[2 * w + 1]);
            (&rh.x)[w] = pack2<F16>(x[8 + 2 * w], x[9 + 2 * w]);
          }
        }
        *reinterpret_cast<uint4*>(dst + oct * 8) = ro;
        *reinterpret_cast<uint4*>(dst + D / 2 + oct * 8) = rh;
      } else {
        const int v = i >= n_kv;
        uint8_t* block = page + static_cast<long long>(v ? i - n_kv : i) * q8_block_bytes(D);
        write_q8<D>(x, block + (v ? q8_values_at(D) : 0) + p.slot * D,
                    reinterpret_cast<float*>(block + (v ? q8_value_scales_at(D) : q8_key_scales_at(D))) + p.slot, oct, group);
      }
    }
  }
}

template <int D, bool F16>
cudaError_t launch(AppendArgs& a, bool q8, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const long long enough = 2ll * sms;   // blocks that fill the device: few tokens are cut finer
  const int threads = q8 ? kQ8Threads : kThreads, tokens = threads / (D / 16);
  const int heads = (a.q ? a.b.n_heads : 0) + (q8 ? 2 : 1) * a.b.n_kv;
  a.qk_tiles = (a.b.n_tokens + tokens - 1) / tokens;
  a.heads = static_cast<int>(std::min<long long>(kMaxHeads, std::max<long long>(1, heads * static_cast<long long>(a.qk_tiles) / enough)));
  a.qk_groups = (heads + a.heads - 1) / a.heads;
  if (q8) {
    const long long grid = static_cast<long long>(a.qk_tiles) * a.qk_groups;
    return launch_pdl(kv_append_q8_kernel<D, F16>, dim3(static_cast<unsigned>(grid)), dim3(kQ8Threads), 0, s, a);
  }
  long long v_blocks = static_cast<long long>((a.b.n_tokens + kVTokens - 1) / kVTokens) * a.b.n_kv;
  a.v_split = v_blocks * 4 <= enough ? 4 : v_blocks * 2 <= enough ? 2 : 1;
  v_blocks *= a.v_split;
  const long long grid = static_cast<long long>(a.qk_tiles) * a.qk_groups + v_blocks;
  if (grid > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  return launch_pdl(kv_append_kernel<D, F16>, dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, s, a);
}

}  // namespace

const char* paged_check(const dflash_paged_batch* b) {
  if (!b) return "null batch";
  const int tokens = b->dtype & ~DFLASH_POOL_Q8;
  if (tokens != DFLASH_BF16 && tokens != DFLASH_FP16) return "dtype is neither DFLASH_BF16 nor DFLASH_FP16, with or without DFLASH_POOL_Q8";
  if (b->head_dim != 64 && b->head_dim != 128) return "head_dim must be 64 or 128";
  if (b->n_kv_heads < 1 || b->n_kv_heads > 128 || b->n_heads < 1 || b->n_heads % b->n_kv_heads)
    return "n_kv_heads must be 1..128 and divide n_heads";
  if (b->n_heads / b->n_kv_heads > 128) return "more than 128 query heads per kv head";
  if (b->n_seq < 0 || b->n_seq > kPagedMaxSeqs) return "n_seq must be 0..1024";
  if (b->n_tokens < 0 || b->n_tokens > (1 << 24)) return "n_tokens must be 0..2^24";
  if (b->n_seq == 0 || b->n_tokens == 0) return nullptr;
  if (!b->pool || !b->page_table || !b->q_start || !b->kv_len) return "null pointer";
  if (misaligned16(b->pool)) return "the pool must be 16-byte aligned";
  if (b->n_pages < 1) return "n_pages must be positive";
  if (b->table_pages < 1 || b->table_pages > kPagedMaxTable || b->table_stride < b->table_pages)
    return "table_pages must be 1..2^20, and table_stride at least that";
  return nullptr;
}

PagedView paged_view(const dflash_paged_batch& b) {
  PagedView v;
  v.n_heads = b.n_heads;
  v.n_kv = b.n_kv_heads;
  v.group = b.n_heads / b.n_kv_heads;
  v.n_seq = b.n_seq;
  v.n_tokens = b.n_tokens;
  v.n_pages = b.n_pages;
  v.table_pages = b.table_pages;
  v.table_stride = b.table_stride;
  v.page_table = b.page_table;
  v.q_start = b.q_start;
  v.kv_len = b.kv_len;
  v.pool = static_cast<uint16_t*>(b.pool);
  v.status = b.status;
  return v;
}

}  // namespace dfl

using namespace dfl;

extern "C" dflash_status dflash_kv_append(const dflash_paged_batch* b, const void* k, long long k_stride, const void* v,
                                          long long v_stride, const void* q, long long q_stride, void* q_out,
                                          long long q_out_stride, const int32_t* positions, float rope_base,
                                          void* stream) {
  auto refuse = [](const char* why) {
    set_unattached_error(why);
    return DFLASH_EINVAL;
  };
  if (const char* why = paged_check(b)) return refuse(why);
  if (!(rope_base == 0.f || (rope_base > 1.f && rope_base <= 1e12f))) return refuse("rope_base must be 0 (no rotation) or in (1, 1e12]");
  if ((q == nullptr) != (q_out == nullptr)) return refuse("q and q_out are given together or not at all");
  if (b->n_seq == 0 || b->n_tokens == 0) return DFLASH_OK;
  if (!k || !v) return refuse("null pointer");
  const long long kw = static_cast<long long>(b->n_kv_heads) * b->head_dim;
  const long long qw = static_cast<long long>(b->n_heads) * b->head_dim;
  if (bad_stride(k_stride, kw) || bad_stride(v_stride, kw) || (q && (bad_stride(q_stride, qw) || bad_stride(q_out_stride, qw))))
    return refuse("token strides must be multiples of 8 elements and at least a token's row");
  if (misaligned16(k) || misaligned16(v) || misaligned16(q) || misaligned16(q_out))
    return refuse("k, v, q and q_out must be 16-byte aligned");
  // each thread reads what it writes of a token's queries, and nothing else of them
  if (q && ((q != q_out || q_stride != q_out_stride) && rows_overlap(q, q_stride, qw, q_out, q_out_stride, qw, b->n_tokens)))
    return refuse("q_out must be q or not overlap it");
  if (q && (rows_overlap(k, k_stride, kw, q_out, q_out_stride, qw, b->n_tokens) ||
            rows_overlap(v, v_stride, kw, q_out, q_out_stride, qw, b->n_tokens)))
    return refuse("q_out must not overlap k or v");
  if (in_pool(*b, k, k_stride, kw) || in_pool(*b, v, v_stride, kw) ||
      (q && (in_pool(*b, q, q_stride, qw) || in_pool(*b, q_out, q_out_stride, qw))))
    return refuse("k, v, q and q_out must not lie in the pool");
  AppendArgs a;
  std::memset(&a, 0, sizeof(a));
  a.b = paged_view(*b);
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.q = static_cast<const uint16_t*>(q);
  a.q_out = static_cast<uint16_t*>(q_out);
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_stride = q_stride;
  a.out_stride = q_out_stride;
  a.positions = positions;
  a.rotate = rope_base != 0.f;
  if (a.rotate) {
    // base^(-2i/d) from two factors, since 64 powers are a quarter of the call's
    // time; those of the first pair, whose angle is the largest, are 1 / (2 pi)
    // rounded once and 1
    const double two_pi = 6.283185307179586476925286766559, base = rope_base;
    double coarse[8], fine[8];
    for (int i = 0; i < 8; ++i) {
      coarse[i] = std::pow(base, -16.0 * i / b->head_dim) / two_pi;
      fine[i] = std::pow(base, -2.0 * i / b->head_dim);
    }
    // theta_0 = 1 rad is 0.159 of a turn, so the product stays below 2^62
    for (int i = 0; i < b->head_dim / 2; ++i)
      a.turn[i] = static_cast<unsigned long long>(std::ldexp(coarse[i / 8] * fine[i % 8], 64));
  }
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  const bool q8 = b->dtype & DFLASH_POOL_Q8, f16 = b->dtype & DFLASH_FP16;
  if (b->head_dim == 128) e = f16 ? launch<128, true>(a, q8, s) : launch<128, false>(a, q8, s);
  else e = f16 ? launch<64, true>(a, q8, s) : launch<64, false>(a, q8, s);
  if (e != cudaSuccess) {
    set_unattached_error("dflash_kv_append: kernel launch failed");
    return DFLASH_ECUDA;
  }
  return DFLASH_OK;
}
