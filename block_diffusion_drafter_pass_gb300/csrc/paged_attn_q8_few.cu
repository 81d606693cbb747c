// paged_attn_q8_few.cu - attention over 8-bit pages for few rows (up to 32 of a
// kv head): decoding, and short blocks.
//
// The tensor cores' tile of 128 rows, and the fp16 copies of keys and values that
// it reads from shared memory, are made for many rows: with few of them
// the copies are what costs (paged_attn_q8.cu). Here every warp is by itself: it
// takes every W-th unit of 32 keys of its CTA's run, has the next halves of units
// (keys, or values) under way into a ring of its own by asynchronous copies
// while it works, and multiplies by mma.sync, whose fragments are made in
// registers. A product of code and scale never exists: codes are exact in fp16,
// key scales go onto scores and value scales onto weights in fp32, which are then
// rounded to fp16 for the product with the values, in the unit of `top` as in
// paged_attn_q8.cu: it follows the row's largest weight times value scale, of each
// 32 keys its largest weight times their largest scale where scales lie within
// 2^10, and else the largest over the keys that it sees. So 2^-21 of that still
// counts. The sum has its own reference. At an item's end
// the warps' parts are joined in shared memory, in their order.
//
// Fragments. A product over dims (scores) or keys (output) may take them in any
// order, as long as both operands do. Of a key row, lane (g, c) of the B operand
// (g = lane / 4 its column, the key; c = lane % 4) needs 4 dims a step: a 16-byte
// load of dims 16 c .. gives it 4 steps, and the queries lie in shared memory in
// that order. Scores come out with keys 2 c and 2 c + 1 of each 8 in lane c, and
// as weights that is where the A operand of the next product wants them; of the
// values lane (g, c) loads dims 16 g .. (8 g .. of heads of 64) of the 4 keys that
// a step of 16 gives it, and turns each 4 x 4 bytes over.
//
// What bounds it: up to 16 rows memory (one token of 64 sequences of 32768 keys,
// 32/8 heads of 128: 720 us, 91% of the copy bandwidth, with two CTAs an SM, as the rule
// has it, and 670 with one; one of 32 of 8192 104 us, start, joins and end included; by
// the kernel for 128 rows 1194 and 172); of 17 to 32 rows the latency of 1300 instructions a
// unit in 8 warps (8 tokens of 32 sequences of 8192 166 us instead of 177; 156 before
// sum and unit were apart). Short
// calls are chains of loads: one token over a window of 4096 keys 12.6 us (18.8).
// 12 warps an SM (8 of 32 rows) are what registers allow; 10, unevenly on four
// schedulers, took 801 us for 685 then, 14, spilling, 832.
#include <algorithm>
#include <atomic>

#include "paged_walk.cuh"

namespace dfl {
namespace {

constexpr int kUnit = 32;        // keys
constexpr float kBias = 7.f;
constexpr int kLeastE = -80;   // smaller scales count as 2^-80

template <int D, int MT, int PerSm>
struct Few {
  static constexpr int kWarps = (MT == 1 ? 12 : 8) / PerSm;
  static constexpr int kSlots = D * MT <= 128 && D == 128 ? 3 : 4;   // of a warp's ring
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kRowsMax = 16 * MT;
  // a half of a unit: 32 key rows, then all 32 key and 32 value scales, or 32 value
  // rows; rows 16 bytes apart from a multiple of 128, so that neighbours lie in other banks
  static constexpr int kRow = D + 16;
  static constexpr int kScales = kUnit * kRow, kHalf = kScales + 8 * kUnit;
  static constexpr int kQBytes = kRowsMax * D * 2;
  static constexpr int kStageOff = kBatchBytes + kQBytes;
  // The join's rows, in floats, and where four from d on lie in one: so that both
  // the lanes that hold a row's columns and those that add them meet all banks.
  static constexpr int kJoinRow = D == 128 ? D + 16 : D + 8;
  static __device__ __forceinline__ int join_at(int d) { return d ^ (d >> 5 & (D / 32 - 1)) << 2; }
  static constexpr int kSmem = kStageOff + kWarps * kSlots * kHalf;
  static_assert(kBatchBytes % 16 == 0 && kHalf % 16 == 0, "16-byte copies");
  static_assert(kWarps * kRowsMax * kJoinRow * 4 <= kWarps * kSlots * kHalf, "the join's rows lie over the units");
  static_assert(kSmem <= 220 * 1024 / PerSm, "static shared variables need the rest");
};

// 2^e for e in -128..127 (the two below 2^-126 are no normal numbers).
__device__ __forceinline__ float pow2_of(int e) { return __int_as_float(e >= -126 ? (e + 127) << 23 : 1 << (149 + e)); }

__device__ __forceinline__ void copy_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two bytes (code + 128) behind 0x64 each, 1024 + themselves in fp16, to codes.
__device__ __forceinline__ uint32_t to_codes(uint32_t x) {
  const __half2 off = __half2half2(__ushort_as_half(0x6480));   // 1152
  const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&x), off);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// What the warp's lane looked up of a unit.
struct Unit {
  int page;      // -1: missing; -2: no row sees a key of it
  int base;      // its first key
  int seq, end;  // as of its step
};

template <int D, bool F16, int MT, int PerSm>
__global__ void __launch_bounds__(Few<D, MT, PerSm>::kThreads, PerSm) paged_attn_q8_few_kernel(const __grid_constant__ PagedAttnArgs a) {
  using C = Few<D, MT, PerSm>;
  constexpr int W = C::kWarps, kThreads = C::kThreads;
  extern __shared__ __align__(16) uint8_t smem[];
  Batch& b = *reinterpret_cast<Batch*>(smem);
  uint8_t* const s_q = smem + kBatchBytes;   // [D / 16][MT][32 lanes][4 words]
  __shared__ float s_qc[C::kRowsMax];
  __shared__ float2 s_ml[W][C::kRowsMax];   // maximum and sum
  __shared__ long long s_sum[kThreads / 32];
  __shared__ Item s_first[2], s_items[2];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  if (tid == 0) {
    s_first[0].nj = 0;
    set_batch(a, b);
  }
  __syncthreads();
  grid_dep_wait();
  grid_dep_launch();
  const int run = deal_batch<kThreads>(a, b, s_sum, s_first);
  __syncthreads();
  if (tid < sizeof(Item) / 4) reinterpret_cast<int*>(s_items)[tid] = reinterpret_cast<const int*>(s_first)[tid];
  __syncthreads();
  const uint32_t ring_at = smem_u32(smem) + C::kStageOff + warp * C::kSlots * C::kHalf;
  const uint8_t* const pool = reinterpret_cast<const uint8_t*>(a.b.pool);
  const long long page_bytes = static_cast<long long>(a.b.n_kv) * q8_block_bytes(D);
  const int G = a.b.group;
  if (tid == 0) {
    int piece = 0;
    for (int before = s_items[0].nj > 0 ? s_items[0].j : 0; before > 0; before -= run) ++piece;
    a.piece[blockIdx.x] = piece;
  }
  int4 split = make_int4(0, 0, 0, 0);

#pragma unroll 1
  for (int k = 0;; ++k) {
    const Item& it = s_items[k & 1];
    const int nj = it.nj, head = it.head, rows = it.t.ntok * G;
    if (nj <= 0) break;
    if (tid == 0) next_item(b, it, s_items[(k + 1) & 1]);

    // ---- the item's queries, as paged_attn_q8.cu takes them to fp16, in the order of the A operand ----
    constexpr int kOf = D / 8;
    constexpr uint32_t kInf = F16 ? 0x7C00u : 0x7F80u;
#pragma unroll 1
    for (int i = tid; i < C::kRowsMax * kOf; i += kThreads) {   // whole warps: kRowsMax * kOf is a multiple of 32
      const int r = i / kOf, d = i % kOf * 8, j = r / G;
      uint4 w = make_uint4(0, 0, 0, 0);
      if (r < rows) w = __ldg(reinterpret_cast<const uint4*>(a.q + (it.t.t0 + j) * a.q_stride + static_cast<long long>(head * G + r - j * G) * D + d));
      uint32_t top = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t m = (&w.x)[e] & 0x7FFF7FFFu, lo = m & 0xFFFFu, hi = m >> 16;
        top = max(top, max(lo < kInf ? lo : 0u, hi < kInf ? hi : 0u));
      }
#pragma unroll
      for (int o = kOf / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      const int up = max(126 - static_cast<int>(__float_as_uint(unpack2<F16>(top).x) >> 23), -126);
      const float f = pow2_of(up);
#pragma unroll
      for (int e = 0; e < 2; ++e) {   // 4 dims each
        const int dd = d + 4 * e, step = (dd / 64) * 4 + dd % 16 / 4, cc = dd % 64 / 16;
        uint8_t* to = s_q + ((step * MT + r / 16) * 32 + (r & 7) * 4 + cc) * 16 + (r & 8 ? 4 : 0);
        const float2 x = unpack2<F16>((&w.x)[2 * e]), y = unpack2<F16>((&w.x)[2 * e + 1]);
        *reinterpret_cast<uint32_t*>(to) = pack2<true>(x.x * f, x.y * f);
        *reinterpret_cast<uint32_t*>(to + 8) = pack2<true>(y.x * f, y.y * f);
      }
      if (d == 0) s_qc[r] = a.scale_log2 * pow2_of(-up);
    }

    // ---- the rows' views: of row lane for all, of the lane's rows g and g + 8 of each 16 ----
    Row mine[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int u = 0; u < 2; ++u) mine[m][u] = row_at(b, it.t, 0, m * 16 + u * 8 + g);
    // Units from own_a to own_b of sequence `alone` (if the rows are of one), or up
    // to pre_b of the prefix, are seen whole; units above own_z, or below own_y
    // and past the first tokens, not at all.
    int own_a, own_b, pre_b, alone, own_y, own_z;
    {
      const Row x = row_at(b, it.t, 0, min(lane, C::kRowsMax - 1));
      const bool live = x.token >= 0;
      alone = __reduce_min_sync(0xffffffffu, live ? x.seq : kNoEnd);
      if (alone != __reduce_max_sync(0xffffffffu, live ? x.seq : -1)) alone = kNoEnd;
      own_a = __reduce_max_sync(0xffffffffu, live ? x.lo : 0);
      own_y = __reduce_min_sync(0xffffffffu, live ? x.lo : kNoEnd);
      own_z = __reduce_max_sync(0xffffffffu, live ? x.hi : -1);
      const int last = __reduce_min_sync(0xffffffffu, live ? x.hi : kNoEnd);
      own_b = min(last, b.len[min(alone, b.n_seq - 1)] - 1) - (kUnit - 1);
      pre_b = min(last + b.prefix_len, b.prefix_len - 1) - (kUnit - 1);
    }
    auto look_up = [&](int i) {   // the warp's i-th unit
      Unit x{-2, 0, -1, 0};
      const int u = i * W + warp;
      if (u >= 4 * nj) return x;
      StepWalk w;
      w.start(b, it.t, it.j + (u >> 2));
      x.base = w.s.base + (u & 3) * kUnit;
      x.seq = w.s.seq;
      x.end = w.s.end;
      if (x.base >= x.end) return x;
      if (x.seq >= 0 && x.seq == alone && (x.base > own_z || (x.base + kUnit <= own_y && x.base >= b.sinks))) return x;
      const int page = table_of(a, x.seq)[x.base / kPage];
      x.page = page >= 0 && page < a.b.n_pages ? page : -1;
      return x;
    };
    auto unit_of = [&](const Unit& x, int i) {   // unit i of those that the lanes looked up
      return Unit{__shfl_sync(0xffffffffu, x.page, i & 31), __shfl_sync(0xffffffffu, x.base, i & 31),
                  __shfl_sync(0xffffffffu, x.seq, i & 31), __shfl_sync(0xffffffffu, x.end, i & 31)};
    };
    auto bring = [&](int page, int base, bool keys, int slot) {   // a group of copies, whether there is something to copy or not
      if (page >= 0) {
        const uint8_t* block = pool + page * page_bytes + static_cast<long long>(head) * q8_block_bytes(D);
        const int slot0 = base % kPage;
        const uint32_t to = ring_at + slot * C::kHalf;
        constexpr int kOfRow = D / 16, kRowsAtOnce = 32 / kOfRow;
        const int r = lane / kOfRow, e = lane % kOfRow * 16;
        const uint8_t* src = block + (keys ? 0 : q8_values_at(D)) + (slot0 + r) * D + e;
#pragma unroll
        for (int i = 0; i < kUnit; i += kRowsAtOnce) copy_async16(to + (r + i) * C::kRow + e, src + i * D);
        if (keys && lane < 16)   // 8 pieces of each kind
          copy_async16(to + C::kScales + lane * 16, block + q8_key_scales_at(D) + (lane >> 3) * 4 * kPage + slot0 * 4 + (lane & 7) * 16);
      }
      copy_async_commit();
    };

    const int units = (4 * nj - warp + W - 1) / W;   // of the warp
    // Halves in a ring, keys and values in turn: up to kSlots - 1 are under way. The
    // lanes hold 32 units' pages, those of this unit and of what is to be brought.
    Unit looked = look_up(lane), ahead = looked;
    int brought = 0, to_slot = 0, slot = 0;   // halves; places to fill and to read
    auto bring_next = [&]() {
      const int i = brought >> 1;
      const bool keys = !(brought & 1);
      if (keys && i > 0 && (i & 31) == 0) ahead = look_up(i + lane);
      const int page = __shfl_sync(0xffffffffu, ahead.page, i & 31), base = __shfl_sync(0xffffffffu, ahead.base, i & 31);
      bring(page, base, keys, to_slot);
      to_slot = to_slot + 1 < C::kSlots ? to_slot + 1 : 0;
      ++brought;
    };
#pragma unroll
    for (int h = 0; h < C::kSlots - 1; ++h) bring_next();
    __syncthreads();   // the queries are there, and the next item
    // by row, log2 units, whole numbers: the reference maximum (its sum is of 2^(s - mref))
    // and the unit of its products with the values (o is of 2^(s - top) values)
    float o[MT][D / 8][4], mref[MT][2], l[MT][2], top[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
      for (int t = 0; t < D / 8; ++t) o[m][t][0] = o[m][t][1] = o[m][t][2] = o[m][t][3] = 0.f;
      mref[m][0] = mref[m][1] = top[m][0] = top[m][1] = -INFINITY;
      l[m][0] = l[m][1] = 0.f;
    }
#pragma unroll 1
    for (int i = 0; i < units; ++i) {
      if (i > 0 && (i & 31) == 0) looked = ahead;
      const Unit now = unit_of(looked, i);
      bring_next();
      if (now.page < 0) {   // both halves are empty
        bring_next();
        slot = slot + 2 < C::kSlots ? slot + 2 : slot + 2 - C::kSlots;
        if (now.page == -2) continue;
        // a row that would see a key of the page says so
        bool sees = false;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const RowSpan sp = span_of(b, mine[m][u], Step{now.seq, now.base, now.end});
            sees |= sp.hi >= 0 && static_cast<uint32_t>(row_sees(sp, now.base, now.end)) != 0;
          }
        if (sees) latch_status(a.b.status, kDevBounds);
        continue;
      }
      copy_async_wait<C::kSlots - 1>();
      __syncwarp();
      const uint32_t at = ring_at + slot * C::kHalf;
      slot = slot + 1 < C::kSlots ? slot + 1 : 0;
      // scales: those of slots past the end become 0, a value scale that is no
      // number the score of whoever sees the key; ev: the value scales are below 2^(ev + 1)
      int ev;
      bool wide;
      {
        const bool there = now.base + lane < now.end;
        float kx, vx;
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(kx) : "r"(at + C::kScales + lane * 4));
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(vx) : "r"(at + C::kScales + 4 * kUnit + lane * 4));
        const bool number = vx * 0.f == 0.f;
        if (there && !number) kx = __uint_as_float(0x7FC00000u);
        if (!there) kx = 0.f;
        kx *= 0x1p-16f;   // a score before cq: dot products with codes come to 2^14, scales of bf16 keys to 2^121
        if (!there || !number) vx = 0.f;
        // (a zero counts as the smallest: a key of all the weight may have no values)
        const uint32_t mag = __float_as_uint(vx) & 0x7FFFFFFFu;
        const Spread sv = spread_of(__reduce_max_sync(0xffffffffu, mag), __reduce_min_sync(0xffffffffu, there && number ? mag : 0x7F800000u), kLeastE);
        ev = sv.exponent;
        wide = sv.wide;
        asm volatile("st.shared.f32 [%0], %1;" ::"r"(at + C::kScales + lane * 4), "f"(kx) : "memory");
        asm volatile("st.shared.f32 [%0], %1;" ::"r"(at + C::kScales + 4 * kUnit + lane * 4), "f"(vx) : "memory");
        __syncwarp();
      }
      // ---- scores: four tiles of 8 keys ----
      float s[MT][4][4];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < 4; ++t) s[m][t][0] = s[m][t][1] = s[m][t][2] = s[m][t][3] = 0.f;
#pragma unroll
      for (int h = 0; h < D / 64; ++h) {
        uint4 kw[4];
#pragma unroll
        for (int t = 0; t < 4; ++t)
          asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(kw[t].x), "=r"(kw[t].y), "=r"(kw[t].z), "=r"(kw[t].w)
                       : "r"(at + (8 * t + g) * C::kRow + h * 64 + c * 16));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t q[MT][4];
#pragma unroll
          for (int m = 0; m < MT; ++m)
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(q[m][0]), "=r"(q[m][1]), "=r"(q[m][2]), "=r"(q[m][3])
                         : "r"(smem_u32(s_q) + (((h * 4 + e) * MT + m) * 32 + lane) * 16));
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const uint32_t w = (&kw[t].x)[e];
            const uint32_t b0 = to_codes(__byte_perm(w, 0x64646464u, 0x4140)), b1 = to_codes(__byte_perm(w, 0x64646464u, 0x4342));
#pragma unroll
            for (int m = 0; m < MT; ++m) mma_f16(s[m][t], q[m], b0, b1);
          }
        }
      }
      // ---- weights ----
      float2 ks[4], vs[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(ks[t].x), "=f"(ks[t].y) : "r"(at + C::kScales + (8 * t + 2 * c) * 4));
        asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(vs[t].x), "=f"(vs[t].y) : "r"(at + C::kScales + 4 * kUnit + (8 * t + 2 * c) * 4));
      }
      const bool masked = now.seq < 0 ? now.base > pre_b : now.seq != alone || now.base < own_a || now.base > own_b;
      uint32_t p[MT][4][2];   // packed weights of tile t: rows g, g + 8
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int u = 0; u < 2; ++u) {
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            s[m][t][2 * u] *= ks[t].x;
            s[m][t][2 * u + 1] *= ks[t].y;
          }
          if (masked) {
            const RowSpan sp = span_of(b, mine[m][u], Step{now.seq, now.base, now.end});
            const uint32_t vis = sp.hi >= 0 ? static_cast<uint32_t>(row_sees(sp, now.base, now.end)) : 0u;
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              s[m][t][2 * u] = vis >> (8 * t + 2 * c) & 1 ? s[m][t][2 * u] : -INFINITY;
              s[m][t][2 * u + 1] = vis >> (8 * t + 2 * c + 1) & 1 ? s[m][t][2 * u + 1] : -INFINITY;
            }
          }
#pragma unroll
          for (int t = 0; t < 4; ++t) mx[u] = max3(mx[u], s[m][t][2 * u], s[m][t][2 * u + 1]);
          mx[u] = fmaxf(mx[u], __shfl_xor_sync(0xffffffffu, mx[u], 1));
          mx[u] = fmaxf(mx[u], __shfl_xor_sync(0xffffffffu, mx[u], 2));
        }
        float alpha[2] = {1.f, 1.f}, cq[2], most[2];
        bool grows = false;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          cq[u] = fminf(fmaxf(s_qc[m * 16 + u * 8 + g] * 0x1p16f, 0x1p-126f), 0x1p127f);
          mx[u] *= cq[u];
          most[u] = mx[u] + static_cast<float>(ev + 1);   // the row's largest weight times value scale, at most
        }
        if (wide) {   // of what it sees, key by key
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            most[u] = -INFINITY;
#pragma unroll
            for (int t = 0; t < 4; ++t)
              most[u] = max3(most[u], fmaf(s[m][t][2 * u], cq[u], scale_log2_bound(vs[t].x)),
                             fmaf(s[m][t][2 * u + 1], cq[u], scale_log2_bound(vs[t].y)));
            most[u] = fmaxf(most[u], __shfl_xor_sync(0xffffffffu, most[u], 1));
            most[u] = fmaxf(most[u], __shfl_xor_sync(0xffffffffu, most[u], 2));
          }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          if (mx[u] > mref[m][u] + kRescaleLog2) {   // each row by itself
            const float nm = ceilf(mx[u]);
            l[m][u] *= ex2(mref[m][u] - nm);
            mref[m][u] = nm;
          }
          if (most[u] > top[m][u] + (kBias + kRescaleLog2)) {
            const float nt = ceilf(most[u]) - kBias;
            alpha[u] = ex2(top[m][u] - nt);
            top[m][u] = nt;
            grows = true;
          }
        }
        if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
          for (int t = 0; t < D / 8; ++t) {
            o[m][t][0] *= alpha[0], o[m][t][1] *= alpha[0];
            o[m][t][2] *= alpha[1], o[m][t][3] *= alpha[1];
          }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          // (mref is at most 106 above top, since no key counts for less than 2^-90 of its weight there)
          const float neg = mref[m][u] == -INFINITY ? 0.f : -mref[m][u];
          const float by = top[m][u] == -INFINITY ? 0.f : ex2(mref[m][u] - top[m][u]);
          float sum = 0.f;
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const float x = ex2(fmaf(s[m][t][2 * u], cq[u], neg)), y = ex2(fmaf(s[m][t][2 * u + 1], cq[u], neg));
            sum += x + y;
            p[m][t][u] = pack2<true>(x * by * vs[t].x, y * by * vs[t].y);
          }
          l[m][u] += sum;
        }
      }
      // ---- output: two steps of 16 keys ----
      __syncwarp();   // the keys' place is read
      bring_next();
      copy_async_wait<C::kSlots - 1>();
      __syncwarp();
      const uint32_t values_at = ring_at + slot * C::kHalf;
      slot = slot + 1 < C::kSlots ? slot + 1 : 0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        constexpr int kWords = D / 32;   // of a key's dims for this lane
        uint32_t v[4][kWords];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int key = 16 * h + 8 * (e >> 1) + 2 * c + (e & 1);
          const uint32_t from = values_at + key * C::kRow + g * (D / 8);
          if constexpr (D == 128) asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v[e][0]), "=r"(v[e][1]), "=r"(v[e][2]), "=r"(v[e][3]) : "r"(from));
          else asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v[e][0]), "=r"(v[e][1]) : "r"(from));
        }
#pragma unroll
        for (int q = 0; q < kWords; ++q) {
          const uint32_t t0 = __byte_perm(v[0][q], v[1][q], 0x5140), t1 = __byte_perm(v[0][q], v[1][q], 0x7362);
          const uint32_t u0 = __byte_perm(v[2][q], v[3][q], 0x5140), u1 = __byte_perm(v[2][q], v[3][q], 0x7362);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t b0 = to_codes(__byte_perm(e < 2 ? t0 : t1, 0x64646464u, e & 1 ? 0x4342 : 0x4140));
            const uint32_t b1 = to_codes(__byte_perm(e < 2 ? u0 : u1, 0x64646464u, e & 1 ? 0x4342 : 0x4140));
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              const uint32_t w[4] = {p[m][2 * h][0], p[m][2 * h][1], p[m][2 * h + 1][0], p[m][2 * h + 1][1]};
              mma_f16(o[m][4 * q + e], w, b0, b1);
            }
          }
        }
      }
      __syncwarp();   // the unit's place is read
    }

    // ---- the warps' parts joined ----
    copy_async_wait<0>();   // (of what is behind the item's end, nothing)
    __syncthreads();
    float* const s_o = reinterpret_cast<float*>(smem + C::kStageOff);   // [W][kRowsMax][kJoinRow]
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float x = l[m][u];
        x += __shfl_xor_sync(0xffffffffu, x, 1);
        x += __shfl_xor_sync(0xffffffffu, x, 2);
        const int r = m * 16 + u * 8 + g;
        const float2 whole = joined_form(mref[m][u], x);
        const float f = top[m][u] == -INFINITY ? 0.f : ex2(top[m][u] - whole.x);   // o in its terms
        if (c == 0) s_ml[warp][r] = whole;
        float* to = s_o + (warp * C::kRowsMax + r) * C::kJoinRow;   // dims of columns 2 c, then 2 c + 1
        if (units <= 0) continue;
#pragma unroll
        for (int t = 0; t < D / 8; t += 4) {
          const int d = 2 * c * (D / 8) + t;
          *reinterpret_cast<float4*>(to + C::join_at(d)) = make_float4(o[m][t][2 * u] * f, o[m][t + 1][2 * u] * f, o[m][t + 2][2 * u] * f, o[m][t + 3][2 * u] * f);
          *reinterpret_cast<float4*>(to + C::join_at(d + D / 8)) =
              make_float4(o[m][t][2 * u + 1] * f, o[m][t + 1][2 * u + 1] * f, o[m][t + 2][2 * u + 1] * f, o[m][t + 3][2 * u + 1] * f);
        }
      }
    }
    __syncthreads();
    const bool whole = nj == it.t.n;
    const int parts = min(W, 4 * nj);   // warps that had units
#pragma unroll 1
    for (int i = tid; i < rows * (D / 4); i += kThreads) {
      const int r = i / (D / 4), d = i % (D / 4) * 4;
      float top = -INFINITY, sum = 0.f;
#pragma unroll 4
      for (int w = 0; w < parts; ++w) top = fmaxf(top, s_ml[w][r].x);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int w = 0; w < parts; ++w) {
        const float2 ml = s_ml[w][r];
        const float f = ml.x == -INFINITY ? 0.f : ex2(ml.x - top);
        const float4 x = *reinterpret_cast<const float4*>(s_o + (w * C::kRowsMax + r) * C::kJoinRow + C::join_at(d));
        sum = fmaf(f, ml.y, sum);
        acc.x = fmaf(f, x.x, acc.x), acc.y = fmaf(f, x.y, acc.y), acc.z = fmaf(f, x.z, acc.z), acc.w = fmaf(f, x.w, acc.w);
      }
      if (whole && a.part == 1) {
        const size_t at = static_cast<size_t>(it.t.t0 + r / G) * a.b.n_heads + head * G + r % G;
        *reinterpret_cast<float4*>(a.own_o + at * D + d) = acc;
        if (d == 0) a.own_ml[at] = make_float2(top, sum);
      } else if (whole) {
        const float f = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
        const int j = r / G;
        uint16_t* out = out_row(a, it.t.t0 + j, head, r - j * G, D) + d;
        *reinterpret_cast<uint2*>(out) = make_uint2(pack2<F16>(acc.x * f, acc.y * f), pack2<F16>(acc.z * f, acc.w * f));
      } else {
        const size_t pr = partial_row(a, it, 0, r);
        *reinterpret_cast<float4*>(a.part_o + pr * D + d) = acc;
        if (d == 0) a.part_ml[pr] = make_float2(top, sum);
      }
    }
    if (it.j == 0 && !whole) {   // the run ends here: the rest is the next CTAs'
      int pieces = 1;
      for (int left = it.t.n - nj; left > 0; left -= run) ++pieces;
      split = make_int4(it.t.t0, it.t.ntok, head, pieces);
    }
    __syncthreads();   // the join's rows and the queries are read
  }
  if (tid == 0) a.split[blockIdx.x] = split;
}

template <int D, bool F16, int MT, int PerSm>
cudaError_t launch(const PagedAttnArgs& a, int device, int ctas, cudaStream_t s) {
  using C = Few<D, MT, PerSm>;
  // the shared-memory limit is set once per device (setting it again changes nothing)
  static std::atomic<uint64_t> set{0};
  if (device > 63 || !(set.load(std::memory_order_acquire) >> device & 1)) {
    const cudaError_t e = cudaFuncSetAttribute(paged_attn_q8_few_kernel<D, F16, MT, PerSm>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    if (device < 64) set.fetch_or(uint64_t(1) << device, std::memory_order_release);
  }
  return launch_pdl(paged_attn_q8_few_kernel<D, F16, MT, PerSm>, dim3(ctas), dim3(C::kThreads), C::kSmem, s, a);
}

template <int D, bool F16>
cudaError_t pick(const PagedAttnArgs& a, const Q8Few& few, int device, int ctas, cudaStream_t s) {
  if (few.rows > 16) return launch<D, F16, 2, 2>(a, device, ctas, s);
  return few.per_sm == 2 ? launch<D, F16, 1, 2>(a, device, ctas, s) : launch<D, F16, 1, 1>(a, device, ctas, s);
}

}  // namespace

cudaError_t launch_paged_attn_q8_few(const PagedAttnArgs& a, int head_dim, bool f16, const Q8Few& few, int device, int ctas, cudaStream_t s) {
  if (head_dim == 128) return f16 ? pick<128, true>(a, few, device, ctas, s) : pick<128, false>(a, few, device, ctas, s);
  return f16 ? pick<64, true>(a, few, device, ctas, s) : pick<64, false>(a, few, device, ctas, s);
}

}  // namespace dfl
