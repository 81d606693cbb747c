// paged_attn_q8.cu - the attention of paged_attn.cu over 8-bit pages: the same
// rows, masks, prefixes, tiles and steps, with keys and values that stand for
// code * scale.
//
// Row q (times the softmax scale), key j with codes c_j and scale a_j, value
// with codes d_j and scale b_j:
//     s_j = q . (a_j c_j),   o = sum_j 2^(s_j - m) b_j d_j / sum_j 2^(s_j - m).
// The products are of fp16 whatever the tokens' type. Queries are taken to it
// behind a power of two that puts the row's largest value between 1/2 and 1
// (values below 2^-13 of that are rounded in steps of 2^-24, all others of bf16
// are exact). Keys and values are a code times its scale, behind a power of two
// 2^(7 - e) that all 128 of a step share (its largest scale comes to lie between 2^7
// and 2^8), rounded to fp16 once, or for tokens of bf16, whose own steps are 8 times
// as large, twice: the scale, too. Found over 2000 keys of scores of deviation 1.5:
// 0.0005 of the output's norm in fp16 (0.0011 with a rounded scale; a plain fp32
// computation rounded once at the end 0.0002), 0.0020 in bf16 (0.0017 with whole
// scales; plain 0.0017), where whole scales took 287 us instead of 278 for 16
// tokens of 32 sequences behind 32768; quantising the same keys and values moves the
// output by 0.013. (Scales multiplied onto scores and weights in fp32 instead are exact, but
// each row then needs all 256 of a step: 364 us instead of 322, then.)
// The step's scales must lie within 2^10 of each other for that (a key scale of zero
// apart, but not a value scale of zero beside others). In a step of wider ones each key
// has a power of two of its own, and the softmax multiplies the row's scores and
// weights by these, in a second pass over the scores: no key's scale takes bits from
// another's.
// Weights are rounded to fp16 for the product with the values, in its best place:
// as 2^(s - T + e) for a value exponent e, T (`top`) at least the row's largest s + e
// less 15 so far, of which s is its largest score in a step and e the step's exponent
// (in a wide step s + e is of one key that the row sees). So they stay below 2^15, and
// 2^-21 of the row's largest weight times value scale still counts, 2^-31 where
// scales are alike. Their sum is in fp32 by a reference m of its own, since keys of
// small or no values count there, too. m and T are whole numbers, and what is left of an
// item is given on by m: the sum between 1 and 2, and O 2^(T - m).
//
// Per CTA: a warp walks the steps, looks up their pages and brings each half
// (128 keys, or their values) and its scales by bulk copies; a warp turns scales
// into fp16 pairs and exponents; 8 warps, in two teams that take every other half,
// put codes as fp16 into the ring that the products read (and the queries of
// each item, scaled); two warps issue the tcgen05.mma of a stream each and eight do
// the softmax, as in paged_attn.cu. Values lie in rows of a token like keys; the
// product takes them as its MN-major operand. Hidden or missing keys need no care
// in the products: every code is finite, and weights of hidden keys are zero
// before their scale. So no row has to be done again.
//
// What bounds it: a step's chain (scores, weights, product, next scores), with
// eight more warps on the softmax's schedulers than 16-bit pages need. A
// pair's step took 2.4 us, 4600 cycles of which the tensor pipe is active for 44%
// (3300 and 57% there); issue slots are 54% taken, shared memory's load/store pipe
// 36%. 16 tokens of 32 sequences of 1024 to 8192
// keys (32/8 heads of 128) take 120 us (floor 47.5), of one over 262144 keys 165
// (3.4 TB/s), 8.7 thousand new tokens with a window of 2048 398, 16 of 32 sequences
// behind 32768 284. Instruction fetch is part of it: with five roles at work a warp is
// held up by it for every instruction issued (1.0 of 11 stalled warps, ncu), so the
// same rare code (wide steps, an item's successor) costs from nothing to 14% of these
// times by its length and by how often it is laid out: prompts 386 us without it, 438
// unrolled and in line, 400 as short loops with the products' warps' three copies of
// the item's successor made one.
// What was tried and is slower: halves in rounds of two with their scales, one wait
// for each; codes by the converting warps' own loads from global memory, without
// the first ring and with room for a fourth half of fp16 (130 us instead of 119, 190
// instead of 168, 433 instead of 389, 338 instead of 281 in these four cases: with
// registers for the loads in flight the softmax spills, without them the loads
// do); bytes as fp16's smallest numbers, times the scale and plus -128 times it in one
// multiply-add, 4 instructions for 4 codes instead of 6 (121, 165, 379, 271 for 118,
// 164, 377, 277, and scales lose bits at 2^12); one team of converting warps for
// every half (141 us instead of 137 and 380 instead of 364 in the first and last
// case, then).
#include <algorithm>
#include <atomic>

#define DFL_WALK_CALL __forceinline__
#include "paged_q8_rings.h"
#include "paged_walk.cuh"

namespace dfl {
namespace {

constexpr int kWalkWarp = 0, kMmaWarp0 = 1, kScaleWarp = 3;   // first: the schedulers seem to prefer older warps
constexpr int kSoftWarp0 = 4;                                 // eight: TMEM lanes go by warp % 4
constexpr int kConvWarp0 = 12, kConvWarps = 8;
constexpr int kThreads = 20 * 32;
// Registers of a thread, by warpgroup: the launch's (96, as the kernel's bounds
// make it) are dealt anew.
constexpr int kLaunchRegs = 96, kSoftRegs = 144, kConvRegs = 64, kRestRegs = 64;
static_assert(2 * kSoftRegs + 2 * kConvRegs + kRestRegs <= 5 * kLaunchRegs, "setmaxnreg waits for registers that the launch must have");
static_assert(kSoftRegs >= kLaunchRegs && kConvRegs <= kLaunchRegs && kRestRegs <= kLaunchRegs, "inc must go up and dec down");
constexpr int kAhead = 16;       // steps that the walk looks up at a time
constexpr int kScalesAhead = 2;  // steps that scales are ahead of their keys
// The walk is ahead of the softmax by these, the halves of both rings and the
// scales' lead.
constexpr int kStepRing = 32;
constexpr float kBias = 7.f;
constexpr int kLeastE = -80;   // smaller scales count as 2^-80
// In a wide step (kNear) each key has an exponent of its own, behind which its code *
// scale is rounded just so; scores and weights are multiplied by the powers of two
// then, each row's for what it sees. So one key's scale takes no bits from another's.
constexpr int kLeastOwnE = -90, kWide = 1024;   // kWide stands for a wide step's value exponent, which is 0 then
// A step whose largest contribution lies that far below the unit of O is summed by
// itself: the exponentials of its weights in that unit would leave fp32.
constexpr float kFar = 60.f;

// Notice of an item's queries; nj = 0: the run's end.
struct Notice {
  int nj, pair, head, t0, ntok;
  int unused[3];
};

template <int D>
struct Cfg {
  static constexpr int kBox = kRows * 128;                  // 128 rows of 64 elements, swizzled
  static constexpr int kHalf = (D / 64) * kBox;             // a step's keys, or its values, or a stream's queries
  static constexpr int kSlots = D == 128 ? 3 : 6;           // halves as fp16
  // Raw halves: codes [128][d]. The last two places lie where the second
  // stream's queries go, so only tiles without those use them.
  static constexpr int kRaw = kStepKeys * D;
  static constexpr int kRawSlots = D == 128 ? 4 : 6, kRawPair = kRawSlots - 2;
  static constexpr int kQ1Off = kHalf;
  static constexpr int kRawOff = kQ1Off + 2 * kRaw;         // of place 0; the last two before it
  static constexpr int kRingOff = kRawOff + kRawPair * kRaw;
  static constexpr int kIntOff = kRingOff + kSlots * kHalf;
  // Steps whose scales are held: while the softmax is at step j, whose values the
  // rings then begin with, kSlots + kRawSlots halves from there on may be in them,
  // and the scales of kScalesAhead steps after the next half's.
  static constexpr int kScaleRing = D == 128 ? 8 : 16;
  static_assert((kSlots + kRawSlots - 1) / 2 + kScalesAhead + 3 <= kScaleRing, "scales that are still read");
  static_assert((kSlots + kRawSlots - 1) / 2 + kScalesAhead + 3 + kAhead <= kStepRing, "pages that are still read");
  // A step's scales: per page those of its keys and of its values, as they come
  // (fp32), then as two fp16 each.
  static constexpr int kScaleOff = kIntOff + kBatchBytes;
  // Of a wide step, each key's exponents, a byte each: [128] of the key scales (less
  // 32, + 127), [128] of the value scales (+ 127).
  static constexpr int kExpOff = kScaleOff + kScaleRing * 1024;
  static constexpr int kSmem = kExpOff + kScaleRing * 256 + 1024;
  static_assert(2 * kRaw >= kHalf && kRaw % 1024 == 0, "queries over raw places, halves in whole swizzle atoms");
  static_assert(kSmem <= 226 * 1024 - 5120, "static shared variables need the rest");
  static constexpr int kPieces = D / 16;                    // 16 bytes of a half for each converting thread
  static __device__ __forceinline__ int raw_at(int place) {
    return place < kRawPair ? kRawOff + place * kRaw : kQ1Off + (place - kRawPair) * kRaw;
  }
};

__device__ __forceinline__ void store_shared16(uint32_t at, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

__device__ __forceinline__ uint4 load_shared_codes(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
  return v;
}

__device__ __forceinline__ uint32_t load_shared_u32(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at));
  return v;
}

__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {   // bulk_load
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(bar)
               : "memory");
}

// Four codes (bytes, + 128) times a scale, as fp16: behind the byte 0x64 a byte
// is 1024 + itself. The scale is its fp16 twice, or (kTwo) its fp16 and what that
// leaves, so that only the product is rounded.
template <bool kTwo>
__device__ __forceinline__ uint2 codes_to_f16(uint32_t w, __half2 scale) {
  const uint32_t lo = __byte_perm(w, 0x64646464u, 0x4140), hi = __byte_perm(w, 0x64646464u, 0x4342);
  const __half2 off = __half2half2(__ushort_as_half(0x6480));   // 1152
  const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&lo), off), y = __hsub2(*reinterpret_cast<const __half2*>(&hi), off);
  const __half2 most = kTwo ? __low2half2(scale) : scale, rest = __high2half2(scale);
  const __half2 a = kTwo ? __hfma2(x, most, __hmul2(x, rest)) : __hmul2(x, most);
  const __half2 b = kTwo ? __hfma2(y, most, __hmul2(y, rest)) : __hmul2(y, most);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

template <bool kTwo>
__device__ __forceinline__ uint32_t scale_of(float x) {
  const float most = kTwo ? __half2float(__float2half_rn(x)) : x;
  return pack2<true>(most, kTwo ? x - most : x);
}

// Of a step's scales, of which each lane has four: their finite ones' spread. Zeros
// count where the mask has a bit (there, a key of all the weight may have no values).
__device__ __forceinline__ Spread step_spread(const float (&x)[4], uint32_t zeros) {
  uint32_t top = 0, low = 0x7F800000u;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t mag = __float_as_uint(x[e]) & 0x7FFFFFFFu;
    top = mag < 0x7F800000u ? max(top, mag) : top;
    low = mag != 0 || (zeros >> e & 1) ? min(low, mag) : low;
  }
  return spread_of(__reduce_max_sync(0xffffffffu, top), __reduce_min_sync(0xffffffffu, low), kLeastE);
}

// The exponent of one scale, of a finite one in -90 .. 127.
__device__ __forceinline__ int own_exponent(float x) {
  return min(max(static_cast<int>(__float_as_uint(x) >> 23 & 255u) - 127, kLeastOwnE), 127);
}

__device__ __forceinline__ float own_log2(uint32_t byte) { return static_cast<float>(static_cast<int>(byte) - 127); }

// A few columns of tensor memory at a time, for what is seldom done: its code shall be short.
__device__ __forceinline__ void tmem_ld4(uint32_t at, float (&v)[4]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];\n\ttcgen05.wait::ld.sync.aligned;"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void tmem_st4(uint32_t at, const float (&v)[4]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]) : "memory");
}
__device__ __forceinline__ void tmem_st2(uint32_t at, uint32_t x, uint32_t y) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%0], {%1, %2};" ::"r"(at), "r"(x), "r"(y) : "memory");
}

// Descriptor of values as they lie in the ring, MN-major with 128-byte swizzle:
// groups of 64 dims a box apart, groups of 8 keys 1024 bytes apart.
template <int D>
__device__ __forceinline__ uint32_t vdesc_low(uint32_t saddr) {
  return ((saddr & 0x3FFFFu) >> 4) | (static_cast<uint32_t>(Cfg<D>::kBox >> 4) << 16);
}

// A row's power of two 2^(e - 126), e the biased exponent of its largest value.
__device__ __forceinline__ float pow2_of(int e) { return __int_as_float((e + 127) << 23); }   // -126..127

// An item's queries into shared memory as fp16, by the converting warps: a row
// times the power of two that puts its largest finite value between 1/2 and 1
// (its infinities and NaN stay what they are), and s_qc what its dot products are
// multiplied by for that. No branch depends on the values: rows that fp16 holds
// taken as they are, behind votes and shuffles in a branch, made prompts 3% faster,
// and then an illegal instruction of batches whose rows differ, in calls whose CTAs
// had one step each (so no ring was gone round) and with the same addresses, barriers
// and dealt registers as here. Reading found no cause.
template <int D, bool F16>
__device__ __forceinline__ void bring_queries(const PagedAttnArgs& a, const Notice& r, uint32_t q_at, float* s_qc, int ct) {
  constexpr int kOf = D / 8, kPass = kConvWarps * 32 / kOf, kAtOnce = 4;   // lanes of a row, rows at a time
  constexpr uint32_t kInf = F16 ? 0x7C00u : 0x7F80u;
  const int c = ct % kOf, G = a.b.group, stream_rows = a.stream_tokens * G;
  const int n = (r.pair ? 2 : 1) * stream_rows, end = r.t0 + r.ntok;
  const int dt = kPass / G, dg = kPass - dt * G;
  int token = r.t0 + ct / kOf / G, g = ct / kOf % G;   // a stream's tokens follow the other's
#pragma unroll 1
  for (int i0 = ct / kOf; i0 - ct / kOf < n; i0 += kPass * kAtOnce) {
    uint4 w[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      w[u] = make_uint4(0, 0, 0, 0);
      if (i0 + u * kPass < n && token < end)
        w[u] = __ldg(reinterpret_cast<const uint4*>(a.q + token * a.q_stride + static_cast<long long>(r.head * G + g) * D) + c);
      token += dt;
      g += dg;
      if (g >= G) g -= G, ++token;
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int i = i0 + u * kPass;
      // magnitudes order as their bits
      uint32_t top = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t m = (&w[u].x)[e] & 0x7FFF7FFFu;
        top = __vmaxu2(top, m & __vcmpltu2(m, kInf << 16 | kInf));   // of the finite ones
      }
      top = max(top & 0xFFFFu, top >> 16);
#pragma unroll
      for (int o = kOf / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      // (of the largest bf16 values 2^-126 leaves 4)
      const int up = max(126 - static_cast<int>(__float_as_uint(unpack2<F16>(top).x) >> 23), -126);
      const float f = pow2_of(up);
      uint4 h;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 x = unpack2<F16>((&w[u].x)[k]);
        (&h.x)[k] = pack2<true>(x.x * f, x.y * f);
      }
      if (i < n) {
        const int stream = i >= stream_rows, row = i - stream * stream_rows;
        store_shared16(q_at + stream * Cfg<D>::kQ1Off + (c >> 3) * Cfg<D>::kBox + row * 128 + (((c & 7) ^ (row & 7)) << 4), h);
        if (c == 0) s_qc[stream * kRows + row] = a.scale_log2 * pow2_of(-up);
      }
    }
  }
}

// Step j of an item: its pages, its keys, and in bits 2, 3 which streams of a pair take it.
__device__ __forceinline__ int4 look_up(const PagedAttnArgs& a, const Batch& b, const Item& it, int j) {
  StepWalk w;
  w.start(b, it.t, it.j + j);
  const int32_t* table = table_of(a, w.s.seq) + w.s.base / kPage;
  return make_int4(w.s.base < w.s.end ? table[0] : -1, w.s.base + kPage < w.s.end ? table[1] : -1, w.s.end - w.s.base,
                   it.pair ? pair_takes(b, it.t, w.s.seq, w.s.base) << 2 : 0);
}

struct NoRedo {
  static constexpr bool kOn = false;
};

template <int D, bool F16>
__global__ void __launch_bounds__(kThreads, 1) paged_attn_q8_kernel(const __grid_constant__ PagedAttnArgs a) {
  using C = Cfg<D>;
  constexpr int S = C::kSlots, kScaleRing = C::kScaleRing;
  constexpr uint32_t kIdescS = idesc_f16_f32(kRows, kStepKeys);
  constexpr uint32_t kIdescO = idesc_f16_f32(kRows, D) | (1u << 16);   // B is MN-major
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Batch& b = *reinterpret_cast<Batch*>(smem + C::kIntOff);
  __shared__ __align__(16) Notice s_notice[2];
  __shared__ __align__(8) int2 s_unit[kScaleRing];   // exponents of a step's key and value scales, or (32, kWide)
  __shared__ float s_qc[2][2 * kRows];     // by item: what a row's dot products are multiplied by
  __shared__ __align__(8) uint64_t raw_full[C::kRawSlots], raw_empty[C::kRawSlots], note_full[2], note_empty[2], conv_meet;
  __shared__ __align__(8) uint64_t scale_raw[kScaleRing], scale_full[kScaleRing];
  __shared__ __align__(8) uint64_t kv_full[2][S], kv_empty[2 * S];   // full: by stream, empty: paged_q8_rings.h
  __shared__ __align__(8) uint64_t q_full, q_empty, mma_done;
  __shared__ __align__(8) uint64_t s_full[2], p_full[2][2], o_done[2], turn[2];   // p_full: by page of the step
  __shared__ JoinUnits join;
  __shared__ __align__(16) int4 s_steps[kStepRing];
  __shared__ uint32_t s_step[kStepRing];
  __shared__ long long s_sum[kThreads / 32];
  __shared__ Item s_first[2];   // the CTA's first item (and where its run begins)
  __shared__ Item s_items[11][2];   // an item and the one after it: softmax warps, walk, products
  __shared__ uint32_t tmem_slot;
  __shared__ int s_progress;
  __shared__ int s_never;   // 0: the progress of waits that must not be cut short

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < C::kRawSlots; ++s) {
      mbar_init(&raw_full[s], 1);
      mbar_init(&raw_empty[s], kConvWarps / 2);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&note_full[s], 1);
      mbar_init(&note_empty[s], kConvWarps + 1);
    }
    for (int s = 0; s < kScaleRing; ++s) {
      mbar_init(&scale_raw[s], 1);
      mbar_init(&scale_full[s], 1);
    }
    mbar_init(&conv_meet, kConvWarps);
    for (int s = 0; s < S; ++s) {
      mbar_init(&kv_full[0][s], kConvWarps / 2);
      mbar_init(&kv_full[1][s], kConvWarps / 2);
    }
    for (int s = 0; s < 2 * S; ++s) mbar_init(&kv_empty[s], 2);   // both streams
    mbar_init(&q_full, kConvWarps);
    mbar_init(&q_empty, 2);
    mbar_init(&mma_done, 2);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&s_full[s], 1);
      mbar_init(&p_full[s][0], 4);
      mbar_init(&p_full[s][1], 4);
      mbar_init(&o_done[s], 1);
      mbar_init(&turn[s], 1);
    }
    mbar_init(&join.x_ml, 8);
    mbar_init(&join.x_bad, 8);
    s_progress = a.wait_tries > 0 ? 0 : kGaveUp;
    s_first[0].nj = 0;
    s_never = 0;
    set_batch(a, b);
    fence_mbar_init();
  }
  if (tid < kStepRing) s_step[tid] = 0;   // no step's note (an earlier CTA's may lie here)
  if (warp == kMmaWarp0) tmem_alloc(&tmem_slot, kTmemCols);
  grid_dep_wait();
  grid_dep_launch();
  const int run = deal_batch<kThreads>(a, b, s_sum, s_first);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;

  const bool converts = warp >= kConvWarp0;
  const bool walks = !converts && warp != kScaleWarp;   // has items of its own
  Item* const items = s_items[!walks ? 0 : warp < kSoftWarp0 ? warp : warp - 1];   // written by lane 0
  if (walks && lane < sizeof(Item) / 4) reinterpret_cast<int*>(items)[lane] = reinterpret_cast<const int*>(s_first)[lane];
  __syncwarp();
  const uint32_t progress_at = smem_u32(&s_progress), never_at = smem_u32(&s_never);
  const uint32_t wait_tries = a.wait_tries;
  auto give_up = [&]() {
    atomicOr(&s_progress, kGaveUp);
    latch_status(a.b.status, kDevTimeout);
  };
  // An item goes in rounds j = -lead .. nj-1: round j multiplies P of step j
  // with its values and issues the scores of step j + lead, so the ring holds,
  // in turn, the values of step j and the keys of step j + lead. lead is 1 for
  // a pair (both streams take every step) and 2 for an alternating tile
  // (stream s takes the steps of parity s).

  if (warp < kSoftWarp0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRestRegs));
    if (warp == kWalkWarp) {
      // ---------------- the walk over keys and values, and their copies ----------------
      // The whole warp: a lane looks up a step (kAhead steps at a time, the next
      // while these are brought), and a half's copies go out from a lane each. One
      // lane for all of it took 3000 cycles a step, 2.1 times what memory does.
      const uint32_t full_at = smem_u32(raw_full), empty_at = smem_u32(raw_empty), base_at = smem_u32(smem);
      const uint8_t* const pool = reinterpret_cast<const uint8_t*>(a.b.pool);
      const long long page_bytes = static_cast<long long>(a.b.n_kv) * q8_block_bytes(D);
      int at = 0, steps = 0, k = 0;      // place in the raw ring, steps of the items before this one, items
      int places = C::kRawSlots;         // places in use: the pair's, or all
      int keyed = 0;                     // steps whose scales are on their way
      uint32_t used = 0, sent = 0;       // by place: parity of its records, whether there are copies to wait for at the end
      bool ok = true;
      int4 split = make_int4(0, 0, 0, 0), found = make_int4(-1, -1, 0, 0);   // found: pages, keys, note bits of the lane's step
      int piece = 0;
#pragma unroll 1
      for (int before = items[0].nj > 0 ? items[0].j : 0; before > 0; before -= run) ++piece;
      auto wait = [&](uint32_t bar, uint32_t parity) {
        if (ok) ok = __all_sync(0xffffffffu, bar_wait(bar, parity, progress_at, wait_tries));
        return ok;
      };
      auto notice = [&](const Notice& n) {
        if (!wait(smem_u32(note_empty) + (k & 1) * 8, (k >> 1 & 1) ^ 1)) return false;
        if (lane == 0) {
          s_notice[k & 1] = n;
          bar_arrive(smem_u32(note_full) + (k & 1) * 8);
        }
        return true;
      };
      auto go_on = [&]() {
        used ^= 1u << at;
        at = at + 1 < places ? at + 1 : 0;
      };
      if (lane < kAhead && lane < items[0].nj) found = look_up(a, b, items[0], lane);
#pragma unroll 1
      while (true) {
        const Item& it = items[k & 1];
        const Item& after = items[(k + 1) & 1];
        const int nj = it.nj, pair = it.pair, head = it.head, lead = pair ? 1 : 2;
        if (nj <= 0) break;
        __syncwarp();
        if (lane == 0) next_item(b, it, items[(k + 1) & 1]);
        __syncwarp();
        const int was = places;
        places = pair ? C::kRawPair : C::kRawSlots;
        // Behind a pair's queries: their place is free when its last scores are done. A
        // parity tells a phase from its neighbours only, and all of a pair of one step may
        // be on its way before the scores of the item before it are done: then the pair's
        // phase looks over. So first its queries must be in: who brings them has waited for those.
        if (places > was) {
          wait(smem_u32(note_empty) + ((k - 1) & 1) * 8, (k - 1) >> 1 & 1);
          wait(smem_u32(&q_empty), (k - 1) & 1);
        }
        if (at >= places) at = 0;
        if (!ok || !notice(Notice{nj, pair, head, it.t.t0, it.t.ntok, {}})) break;
        // Scales go kScalesAhead steps ahead of their keys: a warp has work with them.
        auto bring_scales = [&](int j) {
          if (j % kAhead == 0) {
            int4 f = found;
            if (lane < kAhead && j + lane < nj) {
              if (f.x < 0 || f.x >= a.b.n_pages) f.x = -1, f.w |= 1;
              if (f.y < 0 || f.y >= a.b.n_pages) f.y = -1, f.w |= 2;
              s_steps[(steps + j + lane) % kStepRing] = f;
              s_step[(steps + j + lane) % kStepRing] = step_note(steps + j + lane, f.w);
            }
            const bool same = j + kAhead < nj;   // else the next item's first
            const Item& of = same ? it : after;
            const int of_j = (same ? j + kAhead : 0) + lane;
            if (lane < kAhead && of_j < of.nj) found = look_up(a, b, of, of_j);
            __syncwarp();
          }
          const int4 f = s_steps[(steps + j) % kStepRing];
          const int slot = (steps + j) % kScaleRing, page = lane ? f.y : f.x;
          const bool has0 = f.x >= 0 && f.z > 0, has1 = f.y >= 0 && f.z > kPage;
          const uint32_t bar = smem_u32(scale_raw) + slot * 8;
          if (lane == 0)
            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"((has0 ? 512 : 0) + (has1 ? 512 : 0)) : "memory");
          __syncwarp();
          if (lane < 2 && (lane ? has1 : has0))
            bulk_copy(base_at + C::kScaleOff + slot * 1024 + lane * 512,
                      pool + page * page_bytes + static_cast<long long>(head) * q8_block_bytes(D) + q8_key_scales_at(D), 512, bar);
          ++keyed;
        };
#pragma unroll 1
        for (int i = 1 - 2 * lead - 2 * kScalesAhead; i < 2 * nj; ++i) {   // round i >> 1: values, then scales and keys
          const bool keys = i & 1;
          const int j = (i >> 1) + (keys ? lead : 0);
          if (keys && j + kScalesAhead < nj) bring_scales(j + kScalesAhead);
          if (j < 0 || j >= nj) continue;
          if (!wait(empty_at + at * 8, (used >> at & 1) ^ 1)) break;
          const int4 f = s_steps[(steps + j) % kStepRing];
          // a lane for each page's keys that exist
          const int rows0 = f.x < 0 ? 0 : min(max(f.z, 0), kPage), rows1 = f.y < 0 ? 0 : min(max(f.z - kPage, 0), kPage);
          const int rows = lane ? rows1 : rows0;
          const uint32_t bar = full_at + at * 8;
          if (lane == 0)
            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"((rows0 + rows1) * D) : "memory");
          __syncwarp();
          if (lane < 2 && rows > 0)
            bulk_copy(base_at + C::raw_at(at) + lane * kPage * D,
                      pool + (lane ? f.y : f.x) * page_bytes + static_cast<long long>(head) * q8_block_bytes(D) + (keys ? 0 : q8_values_at(D)),
                      rows * D, bar);
          sent |= 1u << at;
          go_on();
        }
        if (!ok) break;
        steps += nj;
        if (it.j == 0 && nj < it.t.n) {   // the run ends here: the rest is the next CTAs'
          int pieces = 1;
#pragma unroll 1
          for (int left = it.t.n - nj; left > 0; left -= run) ++pieces;
          split = make_int4(it.t.t0, it.t.ntok, it.head, pieces);
        }
        ++k;
      }
      if (ok) notice(Notice{});
      if (!ok) give_up();
      if (lane == 0) {
        a.split[blockIdx.x] = split;
        a.piece[blockIdx.x] = piece;
      }
      // copies still in flight complete before shared memory is released
#pragma unroll 1
      for (int p = 0; p < C::kRawSlots; ++p)
        if (sent >> p & 1) bar_wait(full_at + p * 8, (used >> p & 1) ^ 1, never_at, kWaitTries);
#pragma unroll 1
      for (int t = max(0, keyed - kScaleRing); t < keyed; ++t)
        bar_wait(smem_u32(scale_raw) + t % kScaleRing * 8, t / kScaleRing & 1, never_at, kWaitTries);
    } else if (warp == kScaleWarp) {
      // ---------------- scales ----------------
      // A step's exponents, and its scales as what the codes are multiplied by;
      // those of keys that are not there become 0.
      const uint32_t base_at = smem_u32(smem);
      bool ok = true;
      auto wait = [&](uint32_t bar, uint32_t parity) {
        if (ok) ok = __all_sync(0xffffffffu, bar_wait(bar, parity, progress_at, wait_tries));
        return ok;
      };
      int steps = 0;   // of the items before this one
#pragma unroll 1
      for (int k = 0;; ++k) {
        if (!wait(smem_u32(note_full) + (k & 1) * 8, k >> 1 & 1)) break;
        const int nj = s_notice[k & 1].nj;
        __syncwarp();
        if (nj == 0) break;
        if (lane == 0) bar_arrive(smem_u32(note_empty) + (k & 1) * 8);
#pragma unroll 1
        for (int j = 0; j < nj; ++j, ++steps) {
          const int slot = steps % kScaleRing;
          if (!wait(smem_u32(scale_raw) + slot * 8, steps / kScaleRing & 1)) break;
          const int4 f = s_steps[steps % kStepRing];
          const uint32_t at = base_at + C::kScaleOff + slot * 1024 + lane * 4;   // of keys lane + 32 e
          auto load = [&](int e, const int4& f, float& x, float& y) {
            const bool there = lane + 32 * e < f.z && !(f.w >> (e >> 1) & 1);
            const uint32_t from = at + (e >> 1) * 512 + (e & 1) * 128;
            x = there ? __uint_as_float(load_shared_u32(from)) : 0.f;
            y = there ? __uint_as_float(load_shared_u32(from + 256)) : 0.f;
            return there ? 1u << e : 0u;
          };
          float x[4], y[4];
          uint32_t there = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) there |= load(e, f, x[e], y[e]);
          const Spread sx = step_spread(x, 0), sy = step_spread(y, there);
          const int ex = sx.exponent, ey = sy.exponent;
          const bool wide = sx.wide || sy.wide;
          if (lane == 0) s_unit[slot] = wide ? make_int2(32, kWide) : make_int2(ex, ey);
          auto put = [&](int e, float x, float y, int ek, int ev) {
            // A value scale that is no number becomes the score of whoever sees the
            // key: as a factor of a weight it would reach rows that do not.
            const bool number = y * 0.f == 0.f;
            const float kx = number ? x * pow2_of(7 - ek) : __uint_as_float(0x7FC00000u), vx = number ? y * pow2_of(7 - ev) : 0.f;
            const uint32_t to = at + (e >> 1) * 512 + (e & 1) * 128;
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(to), "r"(scale_of<F16>(kx)) : "memory");
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(to + 256), "r"(scale_of<F16>(vx)) : "memory");
          };
          if (__builtin_expect(!wide, 1)) {
#pragma unroll
            for (int e = 0; e < 4; ++e) put(e, x[e], y[e], ex, ey);
          } else {
#pragma unroll 1
            for (int e = 0; e < 4; ++e) {   // (read again: registers have no index)
              float kx, vx;
              load(e, f, kx, vx);
              const int ek = own_exponent(kx), ev = own_exponent(vx);
              uint8_t* const exps = smem + C::kExpOff + slot * 256 + lane + 32 * e;
              exps[0] = static_cast<uint8_t>(ek + 95);   // (scores stay in range: these are 2^22 at most before)
              exps[128] = static_cast<uint8_t>(ev + 127);
              put(e, kx, vx, ek, ev);
            }
          }
          fence_proxy_async_smem();   // the next copies into this place are the async proxy's
          __syncwarp();
          if (lane == 0) bar_arrive(smem_u32(scale_full) + slot * 8);
        }
        if (!ok) break;
      }
      if (!ok) give_up();
    } else {
      // ---------------- products of one stream ----------------
      // As in paged_attn.cu: the warp goes through this as one, with one elected
      // lane in front of the instructions. Each stream has its own barriers of
      // halves that came, so that one with alternating steps need not follow the
      // other's; a half's place is free when two products (or one, committed
      // twice) have read it.
      const int s = warp_uniform(warp - kMmaWarp0);
      const bool one = elect_one();
      const uint32_t q_low = sdesc_low(smem_u32(smem)), ring_low = q_low + (C::kRingOff >> 4);
      const uint32_t vring_low = vdesc_low<D>(smem_u32(smem)) + (C::kRingOff >> 4);
      const uint32_t full_at = smem_u32(&kv_full[s][0]), empty_at = smem_u32(kv_empty);
      const uint32_t s_at = smem_u32(&s_full[0]) + s * 8, p_at = smem_u32(&p_full[0][0]) + s * 16;
      const uint32_t turn_at = smem_u32(&turn[0]) + s * 8, pass_at = smem_u32(&turn[0]) + (s ^ 1) * 8;
      const uint32_t tm = warp_uniform(tmem);
      const uint32_t s_col = tm + s * kStepKeys, o_col = tm + kOCol + s * D;
      int c = 0, steps = 0, k = 0, np = 0, turns = 0;   // ring halves, steps, items, P tiles, rounds of pairs
      uint32_t got = 0;                                 // by ring slot: parity of the halves that came for this stream
      bool ok = true;
      auto wait = [&](uint32_t bar, uint32_t parity) {
        if (ok) ok = __all_sync(0xffffffffu, bar_wait(bar, parity, progress_at, wait_tries));
        return ok;
      };
      auto empty_of = [&](int half) { return empty_at + read_bar(half, S) * 8; };
      auto scores = [&](uint32_t q_at, int half) {   // S = Q K^T
        const uint32_t k_at = ring_low + half % S * (C::kHalf >> 4);
        if (one) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = ((kk >> 2) * C::kBox + (kk & 3) * 32) >> 4;
            tc_mma_bf16(s_col, sdesc_of(q_at + off), sdesc_of(k_at + off), kIdescS, kk > 0);
          }
          bar_commit(s_at);
          bar_commit(empty_of(half));
        }
      };
      auto product = [&](int half, uint32_t add) {   // O (+)= P V: the first page's weights while the second's are still made
        const uint32_t v_at = vring_low + half % S * (C::kHalf >> 4);
        if (one) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc_mma_bf16_ts(o_col, s_col + kk * 8, sdesc_of(v_at + (kk * 2048 >> 4)), kIdescO, kk > 0 ? 1u : add);
        }
        __syncwarp();
        if (!wait(p_at + 8, np & 1)) return;
        tc_fence_after();
        if (one) {
#pragma unroll
          for (int kk = 4; kk < 8; ++kk)
            tc_mma_bf16_ts(o_col, s_col + kk * 8, sdesc_of(v_at + (kk * 2048 >> 4)), kIdescO, 1u);
          bar_commit(empty_of(half));
        }
      };
      while (true) {
        const Item& it = items[k & 1];
        const int pair = warp_uniform(it.pair), nj = warp_uniform(it.nj);
        if (nj <= 0) break;
        __syncwarp();
        if (lane == 0) next_item(b, it, items[(k + 1) & 1]);   // while the queries come; in one place, since code costs where it lies
        __syncwarp();
        wait(smem_u32(&q_full), k & 1);
        ++k;
        uint32_t add = 0;
        if (!pair) {
          // its steps s, s + 2, ...: the first's scores, then a step's product and
          // the scores of the step after the next, in the order of the ring's halves
          const int first = min(2, nj);   // keys before the first values
          int j = s;
          uint32_t next = j < nj ? c + j : 0;   // half with the keys of step j
          while (ok && j < nj + 2) {
            if (j < nj) {
              const int slot = next % S;
              if (!wait(full_at + slot * 8, got >> slot & 1)) break;
              got ^= 1u << slot;
              tc_fence_after();
              scores(q_low, next);
              if (one) bar_commit(empty_of(next));
            }
            if (j >= nj - 2 && j < nj) {   // the last scores
              if (one) bar_commit(smem_u32(&q_empty));
              __syncwarp();
            }
            const int jv = j;   // its weights are due
            if (jv >= nj) break;
            const int half = c + first + jv + min(jv, max(nj - 2, 0)), slot = half % S;
            if (!wait(full_at + slot * 8, got >> slot & 1) || !wait(p_at, np & 1)) break;
            got ^= 1u << slot;
            tc_fence_after();
            product(half, add);
            if (!ok) break;
            if (one) bar_commit(empty_of(half));
            add = 1;
            ++np;
            __syncwarp();
            j += 2;
            next = half + 1;
          }
          if (s >= nj) {   // no step of its own
            if (one) bar_commit(smem_u32(&q_empty));
            __syncwarp();
          }
          c += 2 * nj;
        } else {
          // every step, in turns: in each round the product of the step's weights
          // with its values and the scores of the next, where the stream takes them
          const uint32_t q_at = q_low + s * (C::kQ1Off >> 4);
          uint32_t takes = 0;   // bit 0: the stream takes step j, bit 1: the next
#pragma unroll 1
          for (int j = -1; j < nj && ok; ++j) {
            const int pv = j >= 0, more = j + 1 < nj;
            const int ck = c + pv, vslot = c % S, kslot = ck % S;
            // one lane for each thing to wait for, so that the waits are one
            const uint32_t early = more ? note_early<kStepRing>(s_step, steps) : 0u;
            {
              bool need = lane == 0 && pv;
              uint32_t bar = full_at + vslot * 8, parity = got >> vslot & 1;
              if (lane == 1) need = more, bar = full_at + kslot * 8, parity = got >> kslot & 1;
              if (lane == 2) need = pv, bar = p_at, parity = np & 1;
              if (lane == 3) need = s == 1 || turns > 0, bar = turn_at, parity = (s == 1 ? turns : turns - 1) & 1;
              int polls = kWaitPolls, seen = 0;
              while (!__all_sync(0xffffffffu, !need || bar_test(bar, parity))) {
                const int progress = warp_uniform(*const_cast<const volatile int*>(&s_progress));
                if (progress != seen) polls = kWaitPolls;
                seen = progress;
                if (progress < 0 || --polls == 0) {
                  ok = false;
                  break;
                }
              }
            }
            ++turns;
            if (!ok) break;
            if (pv) got ^= 1u << vslot;
            if (more) got ^= 1u << kslot;
            const uint32_t take = more ? warp_uniform(note_of<kStepRing>(s_step, steps, early) >> (2 + s) & 1) : 0u;
            tc_fence_after();
            if (takes & 1) {
              product(c, add);
              if (!ok) break;
              add = 1;
            } else if (pv) {
              if (!wait(p_at + 8, np & 1)) break;
              if (one) bar_arrive(empty_of(c));
            }
            np += pv;
            __syncwarp();
            if (one) bar_arrive(pass_at);   // the other stream's waits pass under these products
            if (take) {
              scores(q_at, ck);
            } else if (more && one) {
              bar_arrive(s_at);   // the softmax follows every step of a pair
              bar_arrive(empty_of(ck));
            }
            if (one && j + 2 == nj) bar_commit(smem_u32(&q_empty));   // the item's queries are not needed any more
            __syncwarp();
            c = ck + more;
            steps += more;
            takes = take;
          }
        }
        if (!pair) steps += nj;
        if (!ok) {
          give_up();
          break;
        }
        if (add && one) bar_commit(smem_u32(&o_done[0]) + s * 8);   // only then does the softmax wait for it
      }
      // every issued product completes before TMEM and shared memory are released
      if (one) bar_commit(smem_u32(&mma_done));
      bar_wait(smem_u32(&mma_done), 0, never_at, kWaitTries);
    }
  } else if (converts) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kConvRegs));
    // ---------------- codes to fp16 ----------------
    // Two teams of four warps take every other half, so that one's waits pass
    // under the other's work. A lane takes 16 bytes of a row at a time, in an
    // order in which 8 neighbours meet all 8 bank groups both of the rows that
    // they read and of the swizzled rows that they write.
    constexpr int P = C::kPieces, kRowsOf = kStepKeys / P;   // rows of a piece
    const int ct = tid - kConvWarp0 * 32, team = ct >> 7, tt = ct & 127;
    const int box = D == 128 ? lane >> 2 & 1 : 0, chunk = lane & 3;
    const int row0 = D == 128 ? (tt >> 5) * 4 + (lane >> 4) * 2 + (box ^ (lane >> 3 & 1)) : tt >> 2;
    const uint32_t full_at = smem_u32(raw_full), empty_at = smem_u32(raw_empty), base_at = smem_u32(smem);
    const uint32_t from = row0 * D + box * 64 + chunk * 16;
    const uint32_t to = box * C::kBox + row0 * 128 + ((chunk * 2 ^ (row0 & 7)) << 4);   // its neighbour: ^ 16
    int at = 0, c = 0, steps = 0;   // place in the raw ring, halves, steps of the items before this one
    uint32_t used = 0;              // by place: parity of its halves
    bool ok = true;
    auto wait = [&](uint32_t bar, uint32_t parity) {
      if (ok) ok = __all_sync(0xffffffffu, bar_wait(bar, parity, progress_at, wait_tries));
      return ok;
    };
#pragma unroll 1
    for (int k = 0;; ++k) {
      if (!wait(smem_u32(note_full) + (k & 1) * 8, k >> 1 & 1)) break;
      const Notice& n = s_notice[k & 1];
      const int nj = n.nj, pair = n.pair, lead = pair ? 1 : 2;
      if (nj == 0) break;
      const int places = pair ? C::kRawPair : C::kRawSlots;
      if (at >= places) at = 0;
      if (k > 0) wait(smem_u32(&q_empty), (k - 1) & 1);
      // the second stream's queries lie over raw places that the other warps may still read
      if (lane == 0) bar_arrive(smem_u32(&conv_meet));
      if (!wait(smem_u32(&conv_meet), k & 1)) break;
      bring_queries<D, F16>(a, n, base_at, s_qc[k & 1], ct);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        bar_arrive(smem_u32(&q_full));
        bar_arrive(smem_u32(note_empty) + (k & 1) * 8);
      }
#pragma unroll 1
      for (int i = 1 - 2 * lead; i < 2 * nj; ++i) {   // as the walk does
        const bool keys = i & 1;
        const int j = (i >> 1) + (keys ? lead : 0);
        if (j < 0 || j >= nj) continue;
        const int place = at, half = c++, parity = used >> at & 1;
        used ^= 1u << at;
        at = at + 1 < places ? at + 1 : 0;
        if ((half & 1) != team) continue;
        if (!wait(full_at + place * 8, parity)) break;
        const uint32_t src = base_at + C::raw_at(place) + from, dst = base_at + C::kRingOff + half % S * C::kHalf + to;
        const int slot = (steps + j) % kScaleRing;
        if (!wait(smem_u32(scale_full) + slot * 8, (steps + j) / kScaleRing & 1)) break;
        // all loads first: a load takes 300 cycles
        const uint32_t scales = base_at + C::kScaleOff + slot * 1024 + (keys ? 0 : 256) + row0 * 4;
        uint4 code[P];
        uint32_t scale[P];
#pragma unroll
        for (int p = 0; p < P; ++p) {
          code[p] = load_shared_codes(src + p * kRowsOf * D);
          scale[p] = load_shared_u32(scales + (p * kRowsOf / kPage) * 512 + p * kRowsOf % kPage * 4);
        }
        if (half >= S && !wait(smem_u32(kv_empty) + free_bar(half, S) * 8, free_parity(half, S))) break;
#pragma unroll
        for (int p = 0; p < P; ++p) {
          const uint4 w = code[p];
          const __half2 by = *reinterpret_cast<const __half2*>(&scale[p]);
          const uint2 h0 = codes_to_f16<F16>(w.x, by), h1 = codes_to_f16<F16>(w.y, by);
          const uint2 h2 = codes_to_f16<F16>(w.z, by), h3 = codes_to_f16<F16>(w.w, by);
          store_shared16(dst + p * kRowsOf * 128, make_uint4(h0.x, h0.y, h1.x, h1.y));
          store_shared16((dst ^ 16) + p * kRowsOf * 128, make_uint4(h2.x, h2.y, h3.x, h3.y));
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          bar_arrive(empty_at + place * 8);
          if (pair || !(j & 1)) bar_arrive(smem_u32(&kv_full[0][half % S]));
          if (pair || (j & 1)) bar_arrive(smem_u32(&kv_full[1][half % S]));
        }
      }
      if (!ok) break;
      steps += nj;
    }
    if (!ok) give_up();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    // ---------------- softmax and output ----------------
    const int stream = (warp - kSoftWarp0) >> 2, quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t lane_tmem = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t s_tmem = lane_tmem + stream * kStepKeys;
    const uint32_t o_tmem = lane_tmem + kOCol + stream * D;
    int ns = 0;         // S tiles taken by this stream
    int nx = 0;         // alternating tiles ended
    int outs = 0;       // items with products of this stream
    int k = 0;
    int step0 = 0;      // steps of the CTA's items before this one
    const int prefix_len = b.prefix_len, sinks = b.sinks;
    bool ok = true;
    // waits taken by all 32 lanes together, so the warp-collective TMEM
    // accesses after them never diverge (also when a wait runs out)
    auto warp_wait = [&](uint64_t* bar, uint32_t parity) {
      if (ok) ok = __all_sync(0xffffffffu, bar_wait(smem_u32(bar), parity, progress_at, wait_tries));
      tc_fence_after();
    };
    while (true) {
      const Item& it = items[k & 1];
      if (it.nj <= 0) break;
      __syncwarp();
      if (lane == 0) next_item(b, it, items[++k & 1]);
      k = __shfl_sync(0xffffffffu, k, 0);
      const Row row = row_at(b, it.t, it.pair ? stream : 0, r);
      // log2 units, whole numbers: the row's reference maximum (its sum is of 2^(s - mref)),
      // and the unit of its products with the values (O is of 2^(s - top) values 2^7)
      float mref = -INFINITY, l = 0.f, top = -INFINITY;
      float cq = 0.f;                    // of the row's dot products
      int done = 0;                      // steps of this item that this stream took
      StepWalk w;
      w.start(b, it.t, it.j);
      const int pair = it.pair, nj = it.nj;
      // Of an alternating tile of few rows the stream's first warp arrives for
      // those that have none, and these pass over the steps.
      const int idle = pair ? 0 : 4 - (it.t.ntok * b.group + 31) / 32;
      const uint32_t arrivals = quarter == 0 ? 1 + idle : 1;
      auto weights_there = [&](int u) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(&p_full[stream][u])), "r"(arrivals) : "memory");
      };
      // The references for a step whose largest score is mx and that adds `need` to O
      // at most (log2 units). Each row by itself, so that it does not depend on its neighbours.
      auto raise = [&](float mx, float need) {
        if (mx > mref + kRescaleLog2) {
          const float nm = ceilf(mx);
          l *= ex2(mref - nm);
          mref = nm;
        }
        const bool grows = need > top + (kBias + kRescaleLog2);
        const float nt = grows ? ceilf(need) - kBias : top;
        const float alpha = grows ? ex2(top - nt) : 1.f;
        top = nt;
        if (done == 0 || !__any_sync(0xffffffffu, grows)) return;
        // O holds the stream's products so far: they were issued before
        // the product whose scores these are, and end in that order
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 16) {
          float o[16];
          uint32_t bits[16];
          tmem_ld16(o_tmem + c0, o);
#pragma unroll
          for (int c = 0; c < 16; ++c) bits[c] = __float_as_uint(o[c] * alpha);
          tmem_st_u16(o_tmem + c0, bits);
        }
        tmem_wait_st();
      };
      // A step's weights 2^(s + neg), and their sum, for rows that are `alone` by the sum's own
      // reference. exps: where a wide step's value exponents lie, which belong to the weights, or 0.
      // Of the other rows sums are added in the order in which they are elsewhere.
      auto weigh_apart = [&](float cs, float neg, bool alone, uint32_t exps) {
        const float base = alone ? (mref == -INFINITY ? 0.f : -mref) : neg;
        float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
        for (int c0 = 0; c0 < kStepKeys; c0 += 4) {   // P over scores that are read
          float x[4], w[4];
          tmem_ld4(s_tmem + c0, x);
          const uint32_t own = exps ? load_shared_u32(exps + c0) : 0x7F7F7F7Fu;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            part[e] += ex2_here(fmaf(x[e], cs, base));
            w[e] = ex2_here(fmaf(x[e], cs, own_log2(own >> 8 * e & 255u) + neg));
          }
          tmem_st2(s_tmem + c0 / 2, pack2<true>(w[0], w[1]), pack2<true>(w[2], w[3]));
        }
        tmem_wait_st();
        weights_there(0);
        weights_there(1);
        return (part[0] + part[2]) + (part[1] + part[3]);
      };
      auto exps_at = [&](int j) { return smem_u32(smem) + C::kExpOff + (step0 + j) % kScaleRing * 256; };
      // Steps that begin at own_a .. own_b of sequence `alone` (if the warp's rows
      // are of one), or up to pre_b of the prefix: every row sees all their keys.
      int own_a, own_b, pre_b, alone;
      {
        const bool live = row.token >= 0;
        alone = __reduce_min_sync(0xffffffffu, live ? row.seq : kNoEnd);
        if (alone != __reduce_max_sync(0xffffffffu, live ? row.seq : -1)) alone = kNoEnd;
        own_a = __reduce_max_sync(0xffffffffu, live ? row.lo : 0);
        const int last = __reduce_min_sync(0xffffffffu, live ? row.hi : kNoEnd);
        own_b = min(last, b.len[min(alone, b.n_seq - 1)] - 1) - (kStepKeys - 1);
        pre_b = min(last + prefix_len, prefix_len - 1) - (kStepKeys - 1);
      }
      if (quarter >= 4 - idle) {
        done = (nj + 1 - stream) / 2;
        ns += done;
      }
      for (int j = quarter >= 4 - idle ? nj : 0; j < nj; ++j, w.next(b, it.t)) {
        if (!pair && (j & 1) != stream) continue;
        const uint32_t early = note_early<kStepRing>(s_step, step0 + j);
        warp_wait(&s_full[stream], ns & 1);
        if (!ok) break;
        const int flags = note_of<kStepRing>(s_step, step0 + j, early);
        if (pair && !(flags >> (2 + stream) & 1)) {   // no row of the stream sees the step
          __syncwarp();
          if (lane < 2) mbar_arrive(&p_full[stream][lane]);
          ++ns;
          continue;
        }
        if (done == 0) cq = s_qc[(k - 1) & 1][(pair ? stream * kRows : 0) + r];
        const int gone = flags & 3;
        const bool masked = gone != 0 || (w.s.seq < 0 ? w.s.base > pre_b : w.s.seq != alone || w.s.base < own_a || w.s.base > own_b);
        if (masked) {
          // columns [0, c_hi) less those in [c_sink, c_lo) are seen
          const RowSpan sp = row.token < 0 || (w.s.seq >= 0 && w.s.seq != row.seq) ? RowSpan{0, -1, 0}
                             : w.s.seq < 0 ? RowSpan{0, row.hi + prefix_len, 0} : RowSpan{row.lo, row.hi, sinks};
          const int c_hi = min(sp.hi, w.s.end - 1) - w.s.base + 1;
          const int c_lo = sp.lo - w.s.base, c_sink = sp.sinks - w.s.base;
          const bool none = c_hi <= 0 || (c_lo >= min(c_hi, kStepKeys) && c_sink <= 0);
          if (__all_sync(0xffffffffu, none)) {
            const uint32_t zero[16] = {};
#pragma unroll 1
            for (int c0 = 0; c0 < kStepKeys / 2; c0 += 16) tmem_st_u16(s_tmem + c0, zero);
            tmem_wait_st();
            weights_there(0);
            weights_there(1);
            ++done;
            ++ns;
            continue;
          }
          if (gone != 0) report_gone(a.b.status, gone, c_lo, c_hi, c_sink);
          // scores of keys that the row does not see become -inf in place
#pragma unroll 1
          for (int c0 = 0; c0 < kStepKeys; c0 += 32) {
            const unsigned long long seen = slot_bits(0, c_hi - c0) & (slot_bits(c_lo - c0, 64) | slot_bits(0, c_sink - c0));
            const uint32_t vis = gone >> (c0 / kPage) & 1 ? 0u : static_cast<uint32_t>(seen);
            float x[32];
            tmem_ld32(s_tmem + c0, x);
#pragma unroll
            for (int c = 0; c < 32; ++c) x[c] = vis >> c & 1 ? x[c] : -INFINITY;
            tmem_st32(s_tmem + c0, x);
          }
          tmem_wait_st();
        }
        {
          // the step's factor of dot products, with room for -inf at both ends
          const int2 un = s_unit[(step0 + j) % kScaleRing];
          const float cs = fminf(fmaxf(cq * pow2_of(un.x - 7), 0x1p-126f), 0x1p127f);
          // a half of the scores (one page) at a time: the second for its
          // maximum, the first for its maximum and weights, the second again
          float sv[64];
          auto load = [&](int u) { tmem_ld64(s_tmem + u * kPage, sv); };
          load(1);
          float mx = row_max(sv);
          load(0);
          mx = fmaxf(mx, row_max(sv)) * cs;
          // what the step adds to O, at most: its scales count as the largest of them
          const float ey = static_cast<float>(un.y);
          float need = mx + ey;
          bool alone = row.token >= 0 && need < top - kFar && mx > -INFINITY;   // far below the unit
          bool apart = false;
          if (__any_sync(0xffffffffu, mx > mref + kRescaleLog2 || need > top + (kBias + kRescaleLog2) || alone || un.y == kWide)) {
            if (un.y == kWide) {   // scores are multiplied by their keys' powers of two in place
              need = mx = -INFINITY;   // the largest weight times value scale that the row sees, and score
              alone = true;
#pragma unroll 1
              for (int c0 = 0; c0 < kStepKeys; c0 += 4) {
                float x[4];
                tmem_ld4(s_tmem + c0, x);
                const uint32_t of_k = load_shared_u32(exps_at(j) + c0), of_v = load_shared_u32(exps_at(j) + 128 + c0);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  x[e] *= __uint_as_float((of_k >> 8 * e & 255u) << 23);
                  mx = fmaxf(mx, x[e] * cs);
                  need = fmaxf(need, fmaf(x[e], cs, own_log2(of_v >> 8 * e & 255u)));
                }
                tmem_st4(s_tmem + c0, x);
              }
              tmem_wait_st();
            }
            raise(mx, need);
            apart = __any_sync(0xffffffffu, alone);
          }
          // weights are 2^(s - ref), which times the step's values are in the unit of O
          const float ref = top - (un.y == kWide ? 0.f : ey), neg = top == -INFINITY ? 0.f : -ref;
          if (__builtin_expect(apart, 0)) {
            l = fmaf(weigh_apart(cs, neg, alone, un.y == kWide ? exps_at(j) + 128 : 0), alone ? 1.f : ex2(fminf(ref - mref, 100.f)), l);
          } else {
            float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
            for (int u = 0; u < 2; ++u) {   // P replaces scores that are in registers by then
              if (u == 1) load(1);
#pragma unroll
              for (int h = 0; h < 64; h += 32) {
                uint32_t pk[16];
#pragma unroll
                for (int c = h; c < h + 32; c += 2) {
                  const float2 e = fma2(make_float2(sv[c], sv[c + 1]), make_float2(cs, cs), make_float2(neg, neg));
                  sv[c] = ex2_here(e.x);
                  sv[c + 1] = ex2_here(e.y);
                }
#pragma unroll
                for (int c = 0; c < 16; ++c) pk[c] = pack2<true>(sv[h + 2 * c], sv[h + 2 * c + 1]);
#pragma unroll
                for (int c = 0; c < 16; ++c) sum[c & 1] = add2(sum[c & 1], make_float2(sv[h + 2 * c], sv[h + 2 * c + 1]));
                tmem_st_u16(s_tmem + u * (kPage / 2) + h / 2, pk);
              }
              tmem_wait_st();
              weights_there(u);
            }
            // (ref - mref is at most kFar + kRescaleLog2 where there are weights)
            l = fmaf((sum[0].x + sum[1].x) + (sum[0].y + sum[1].y), ex2(fminf(ref - mref, 100.f)), l);
          }
        }
        ++done;
        ++ns;
        if (!ok) break;
      }
      if (!ok) break;
      step0 += it.nj;
      if (done > 0) warp_wait(&o_done[stream], outs++ & 1);
      if (!ok) break;

      const float2 whole = joined_form(mref, l);
      const float unit = top == -INFINITY ? 0.f : ex2(top - 7.f - whole.x);
      ok = finish_item<D, F16, NoRedo>(a, b, it, join, stream, tmem, row.token, whole.x, whole.y, unit, done > 0, nx & 1, progress_at);
      nx += !it.pair;
      if (!ok) break;
    }
    if (!ok) give_up();
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp0) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D, bool F16>
cudaError_t launch(const PagedAttnArgs& a, int device, int ctas, cudaStream_t s) {
  // the shared-memory limit is set once per device (setting it again changes nothing)
  static std::atomic<uint64_t> set{0};
  if (device > 63 || !(set.load(std::memory_order_acquire) >> device & 1)) {
    const cudaError_t e = cudaFuncSetAttribute(paged_attn_q8_kernel<D, F16>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kSmem);
    if (e != cudaSuccess) return e;
    if (device < 64) set.fetch_or(uint64_t(1) << device, std::memory_order_release);
  }
  return launch_pdl(paged_attn_q8_kernel<D, F16>, dim3(ctas), dim3(kThreads), Cfg<D>::kSmem, s, a);
}

}  // namespace

cudaError_t launch_paged_attn_q8(const PagedAttnArgs& a, int head_dim, bool f16, int device, int ctas, cudaStream_t s) {
  if (head_dim == 128) return f16 ? launch<128, true>(a, device, ctas, s) : launch<128, false>(a, device, ctas, s);
  return f16 ? launch<64, true>(a, device, ctas, s) : launch<64, false>(a, device, ctas, s);
}

}  // namespace dfl
