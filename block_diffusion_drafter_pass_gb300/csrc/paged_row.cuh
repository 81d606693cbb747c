// paged_row.cuh - one query row against one page of keys, by one warp in
// fp32: the definition written down, key by key, reading only what the row
// sees. Lanes take keys for the scores (slots lane and lane + 32) and head
// dims for the product with the values.
#pragma once

#include "paged.cuh"

namespace dfl {

// Bits [lo, hi) of a page's 64 slots; bounds outside 0..64 are cut.
__device__ __forceinline__ unsigned long long slot_bits(int lo, int hi) {
  lo = max(lo, 0);
  hi = min(hi, 64);
  if (lo >= hi) return 0ull;
  return (~0ull >> (64 - (hi - lo))) << lo;
}

// What a row sees of a run of keys: those below `end`, up to position hi, and
// (with a window) from lo on or among the first `sinks`.
struct RowSpan {
  int lo, hi, sinks;
};

__device__ __forceinline__ unsigned long long row_sees(const RowSpan& r, int key0, int end) {
  return slot_bits(0, min(r.hi, end - 1) - key0 + 1) & (slot_bits(r.lo - key0, 64) | slot_bits(0, r.sinks - key0));
}

template <int D>
struct RowState {
  float m, l;          // running maximum (log2 units), running sum
  float acc[D / 32];   // dims lane * D/32 ..
  __device__ __forceinline__ void clear() {
    m = -INFINITY;
    l = 0.f;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) acc[e] = 0.f;
  }
};

template <int D, bool F16>
__device__ __forceinline__ void row_page(RowState<D>& r, const uint16_t* __restrict__ q, const uint16_t* __restrict__ kp,
                                         const uint16_t* __restrict__ vp, float scale_log2, unsigned long long vis,
                                         int lane) {
  if (vis == 0) return;
  float s[2] = {-INFINITY, -INFINITY};
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int c = lane + 32 * u;
    if (!((vis >> c) & 1)) continue;
    float x = 0.f;
#pragma unroll 4
    for (int e = 0; e < D / 8; ++e) {
      const uint4 qw = __ldg(reinterpret_cast<const uint4*>(q) + e);
      const uint4 kw = *(reinterpret_cast<const uint4*>(kp + c * D) + e);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float2 a = unpack2<F16>((&qw.x)[w]), b = unpack2<F16>((&kw.x)[w]);
        x = fmaf(a.x, b.x, x);
        x = fmaf(a.y, b.y, x);
      }
    }
    s[u] = x * scale_log2;
  }
  float mx = fmaxf(s[0], s[1]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  const float nm = fmaxf(r.m, mx);
  const float ref = nm == -INFINITY ? 0.f : nm;
  const float alpha = exp2f(r.m - ref);
  float p[2], sum;
#pragma unroll
  for (int u = 0; u < 2; ++u) p[u] = ((vis >> (lane + 32 * u)) & 1) ? exp2f(s[u] - ref) : 0.f;
  sum = p[0] + p[1];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  r.l = r.l * alpha + sum;
  r.m = nm;
#pragma unroll
  for (int e = 0; e < D / 32; ++e) r.acc[e] *= alpha;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    for (int c8 = 0; c8 < 4; ++c8) {
      const int c0 = u * 32 + c8 * 8;
      uint4 w[D / 32];
#pragma unroll
      for (int e = 0; e < D / 32; ++e)
        w[e] = *reinterpret_cast<const uint4*>(vp + (lane * (D / 32) + e) * kPage + c0);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float pj = __shfl_sync(0xffffffffu, p[u], c8 * 8 + j);
        if (!((vis >> (c0 + j)) & 1)) continue;   // the same for the whole warp: what is not seen is not touched
#pragma unroll
        for (int e = 0; e < D / 32; ++e) {
          const float2 f = unpack2<F16>((&w[e].x)[j >> 1]);
          r.acc[e] = fmaf(pj, (j & 1) ? f.y : f.x, r.acc[e]);
        }
      }
    }
  }
}

}  // namespace dfl
