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
// Work. The rows of a kv head (group query heads of each token) are cut into
// tiles of up to 2 x 128 rows: a tile's tokens are one sequence's, or behind a
// shared prefix neighbours of any sequences, so that the prefix is read once
// for all of them. A tile walks steps of 128 keys (two pages): of its own
// cache the pages that some row sees (first tokens, then the window); behind a
// prefix the prefix and then the cache of each of its sequences in turn, where
// the other sequences' rows see nothing. All steps of all (tile, kv head) in
// one line are dealt to the CTAs in equal runs, so long rows are split over
// the keys as far as needed and no CTA waits for a longer one; a tile that
// ends in another CTA leaves unnormalised partials (O, maximum, sum), which
// paged_combine_kernel joins. Every CTA finds its run from the lengths on the
// device, so a captured launch follows them.
//
// Per CTA: warp 0 brings keys and values by TMA into a ring of step halves (128
// keys, or their values transposed). Two streams, each with its own S/P and O in
// tensor memory, have one warp that issues their tcgen05.mma (one for both left
// the tensor cores waiting for its bookkeeping; the first of them also brings
// the queries) and four softmax warps. A tile of more than 128 rows gives each
// stream 128 rows, and both read the same keys ("pair"); a smaller tile gives
// both streams the same rows and every other step ("alternate": a split over
// the keys inside the CTA, joined at its end). Either way one stream's products
// run while the other's softmax does. With alternating tiles only, keys are
// loaded twice as often and a step's hand-overs serve half the rows: 299 against
// 210 us for 16 tokens of 32 sequences behind 32768, 352 against 280 for the
// prefill below, 87 against 81 for one token of 64 sequences. Rows that fit one
// stream have no second half to pair.
//
// Bounds and measurements (32/8 heads of 128, bf16, device time; floor: the
// keys and values read once at the measured copy bandwidth, or the products at
// the measured bf16 rate): 16 tokens over 262144 keys 162 us, floor 158 (memory);
// 16 tokens of 32 sequences of 1024 to 8192 keys 112 us, floor 91 (memory, and
// about 4 us each for the start, the joins and the items' ends); prefill of 8700
// tokens with a window of 2048 280 us, floor 135 (products; items' ends and masks
// take a quarter); one token of 64 sequences behind 32768 keys 81 us, floor 40;
// 16 tokens of 32 behind 32768 keys 210 us, floor 144 (products, 1320 TFLOP/s).
// With heads of 64 a half step is 16 KB, and what the producer's one lane does
// for each counts more than memory: 16 tokens over 262144 keys 143 us, floor 79
// (157 when that lane also asked which rows miss a page). In the product-bound
// cases a step of a pair takes 3300 cycles for 2048 of tensor work: scores ->
// maximum -> weights -> P V -> the next scores is one chain per stream, mostly
// hand-overs (with the exponentials, the sums and 7/8 of the products taken out
// the last case still takes 200 us), and with heads of 128 tensor memory (two S
// and two O of 128 columns) holds no second S to break it. What was tried against
// that and lost, for that case: scores page by page into the place whose weights
// were just multiplied (230 us: a product over 64 keys takes 3/4 of one over 128,
// and the softmax waits twice), or only the second page's ahead (234), weights
// page by page without the second page's maximum (216), products without turns
// (265), two softmax warps per row (315: the scalar work of a step is per warp),
// the two streams' own caches step by step in turn (209, and 2 to 3% more where
// own caches are long).
#include <cuda.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>

#include "paged_walk.cuh"

namespace dfl {
namespace {

constexpr int kThreads = 352;         // producer, 2 x MMA, 2 x 4 softmax warps
constexpr int kSoftWarp0 = 3;
// The producer is at most the ring's 8 halves of values and 2 steps of keys
// ahead of the softmax (a step's values are not overwritten before its P).
constexpr int kStepRing = 16;
constexpr int kIdsAhead = 2, kIdRing = 16;   // steps

struct PagedMaps {
  CUtensorMap k, v, q;
};

template <int D>
struct Cfg {
  static constexpr int kBox = kRows * 128;                  // 128 rows of 64 elements, swizzled
  static constexpr int kHalf = (D / 64) * kBox;             // a step's keys, or its values
  static constexpr int kSlots = D == 128 ? 4 : 8;
  static constexpr int kQBytes = 2 * kHalf;                 // queries of both streams
  static constexpr int kIntOff = kQBytes + kSlots * kHalf;
  static constexpr int kSmem = kIntOff + kBatchBytes + 1024;
  static_assert(kSmem <= 227 * 1024 - 4096, "static shared variables need the rest");
};

// One row of an item again, read key by key by one warp, and written over what
// the products gave: they met a non-finite value, which may have come from a
// place that the row does not see (0 times infinity or NaN).
template <int D, bool F16>
__device__ __noinline__ void redo_row(const PagedAttnArgs& a, const Batch& b, const Item& it, int stream, int r,
                                      uint32_t progress) {
  const int lane = threadIdx.x & 31, rows_of = it.pair ? stream : 0;
  const Row x = row_at(b, it.t, rows_of, r);
  const int g = r % a.b.group;
  const uint16_t* q = a.q + x.token * a.q_stride + static_cast<long long>(it.head * a.b.group + g) * D;
  const size_t page_elems = static_cast<size_t>(2) * a.b.n_kv * kPage * D;
  RowState<D> st;
  st.clear();
  StepWalk w;
  w.start(b, it.t, it.j);
  for (int j = 0; j < it.nj; ++j, w.next(b, it.t)) {
    const RowSpan sp = span_of(b, x, w.s);
    for (int u = 0; u < 2; ++u) {
      const int key0 = w.s.base + u * kPage;
      const unsigned long long vis = sp.hi >= 0 ? row_sees(sp, key0, w.s.end) : 0ull;
      if (vis == 0) continue;
      const int page = table_of(a, w.s.seq)[key0 / kPage];
      if (page < 0 || page >= a.b.n_pages) continue;
      const uint16_t* kp = a.b.pool + page * page_elems + static_cast<size_t>(it.head) * kPage * D;
      row_page<D, F16>(st, q, kp, kp + static_cast<size_t>(a.b.n_kv) * kPage * D, a.scale_log2, vis, lane);
      if (lane == 0) asm volatile("red.shared.add.u32 [%0], 1;" ::"r"(progress) : "memory");
    }
  }
  if (it.nj == it.t.n) {
    const float f = st.l > 0.f || st.l != st.l ? 1.f / st.l : 0.f;
    uint16_t* o = out_row(a, x.token, it.head, g, D) + lane * (D / 32);
#pragma unroll
    for (int e = 0; e < D / 32; e += 2)
      *reinterpret_cast<uint32_t*>(o + e) = pack2<F16>(st.acc[e] * f, st.acc[e + 1] * f);
  } else {
    const size_t pr = partial_row(a, it, stream, r);
#pragma unroll
    for (int e = 0; e < D / 32; ++e) a.part_o[pr * D + lane * (D / 32) + e] = st.acc[e];
    if (lane == 0) a.part_ml[pr] = make_float2(st.m, st.l);
  }
}

template <int D, bool F16>
struct Redo {
  static constexpr bool kOn = true;
  static __device__ __forceinline__ void row(const PagedAttnArgs& a, const Batch& b, const Item& it, int stream, int r,
                                             uint32_t progress) {
    redo_row<D, F16>(a, b, it, stream, r, progress);
  }
};

// Slots past a length may hold any bits. Their weights are zero, but 0 times
// infinity or NaN would spoil every row of the tile, so where a run of keys ends
// inside a page, the values behind it are cleared before their product: those of
// a step from its key `cut` to the end of that page (per page D rows of 64 slots,
// 128 bytes, swizzled), in half `c` of the ring. By the four softmax warps of a
// stream, a row for each thread, while their scores are made: in the issuing
// warps the same cost 3% of a windowed prefill, in the producer's or in a warp of
// its own 2 to 7% of all long cases. Here it costs 1% of that prefill, half a
// microsecond of the shortest calls and 2 of one token of 64 sequences behind a
// prefix. (Left to redo_row, 16 tokens of 32 sequences of 1024 to 8192 keys with
// NaN behind their ends took 36 ms instead of 0.11.) s_bar: a barrier to wait for
// first, or 0. False when a wait ran out.
template <int D>
__device__ __noinline__ bool cut_values(uint32_t ring, uint32_t full_at, uint32_t progress, uint32_t tries, int c,
                                           int cut, uint32_t s_bar, uint32_t s_parity) {
  constexpr int S = Cfg<D>::kSlots;
  bool ok = s_bar == 0 || bar_wait(s_bar, s_parity, progress, tries);
  ok = ok && bar_wait(full_at + c % S * 8, c / S & 1, progress, tries);
  if (!__all_sync(0xffffffffu, ok)) return false;
  const int r = (threadIdx.x - kSoftWarp0 * 32) % kRows, keep = cut % kPage;
  if (r < D) {
    const uint32_t row = ring + c % S * Cfg<D>::kHalf + cut / kPage * (D * 128) + r * 128;
#pragma unroll 1
    for (int e = keep; e < kPage;) {
      const uint32_t at = row + (((e >> 3) ^ (r & 7)) << 4) + (e & 7) * 2;
      if (e % 8) {
        asm volatile("st.shared.b16 [%0], %1;" ::"r"(at), "h"(static_cast<uint16_t>(0)) : "memory");
        ++e;
      } else {
        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(at), "r"(0u) : "memory");
        e += 8;
      }
    }
    fence_proxy_async_smem();
  }
  return true;
}

template <int D, bool F16>
__global__ void __launch_bounds__(kThreads, 1)
    paged_attn_kernel(const __grid_constant__ PagedMaps maps, const __grid_constant__ PagedAttnArgs a) {
  using C = Cfg<D>;
  constexpr int S = C::kSlots;
  // fp16 has no weights below 2^-24: a row's largest is put at 2^7 (and may
  // stand at 2^15 before O is rescaled), so that weights 2^-31 of it still count
  constexpr float kBias = F16 ? 7.f : 0.f;
  constexpr uint32_t kIdescS = F16 ? idesc_f16_f32(kRows, kStepKeys) : idesc_bf16_f32(kRows, kStepKeys);
  constexpr uint32_t kIdescO = F16 ? idesc_f16_f32(kRows, D) : idesc_bf16_f32(kRows, D);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Batch& b = *reinterpret_cast<Batch*>(smem + C::kIntOff);
  __shared__ __align__(8) uint64_t kv_full[S], kv_empty[S];
  __shared__ __align__(8) uint64_t q_full, q_empty, mma_done;
  __shared__ __align__(8) uint64_t s_full[2], p_full[2][2], o_done[2], turn[2];   // p_full: by page of the step
  __shared__ Join join;
  __shared__ int s_page[kIdRing][2];
  __shared__ uint32_t s_step[kStepRing];
  __shared__ long long s_sum[kThreads / 32];
  __shared__ Item s_first[2];   // the CTA's first item (and where its run begins)
  __shared__ Item s_items[kThreads / 32][2];   // each warp's item and the one after it
  __shared__ uint32_t tmem_slot;
  __shared__ int s_progress;
  __shared__ int s_never;   // 0: the progress of waits that must not be cut short

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.b.group;
  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&kv_full[s], 1);
      mbar_init(&kv_empty[s], 2);   // both streams
    }
    mbar_init(&q_full, 1);
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
    tma_prefetch_desc(&maps.k);
    tma_prefetch_desc(&maps.v);
    tma_prefetch_desc(&maps.q);
  }
  if (tid < kStepRing) s_step[tid] = 0;   // no step's note (an earlier CTA's may lie here)
  if (warp == 1) tmem_alloc(&tmem_slot, kTmemCols);
  grid_dep_wait();
  grid_dep_launch();

  // ---- the batch's shape, and this CTA's run of places ----
  const int run = deal_batch<kThreads>(a, b, s_sum, s_first);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;

  Item* const items = s_items[warp];   // written by lane 0
  if (lane < sizeof(Item) / 4) reinterpret_cast<int*>(items)[lane] = reinterpret_cast<const int*>(s_first)[lane];
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
  // The loops here are kept rolled where they can be: an item's path is walked
  // a few times by each warp, so code that does not stay in the instruction
  // caches costs more than the loops (unrolled over all 128 scores, the first
  // and last steps of an item took 3 to 7 us each instead of 1).

  if (warp == 0) {
    // ---------------- keys and values ----------------
    if (lane == 0) {
      const uint32_t full_at = smem_u32(kv_full), empty_at = smem_u32(kv_empty), ring = smem_u32(smem) + C::kQBytes;
      int c = 0, steps = 0;   // ring halves, steps whose keys were brought
      bool ok = true;
      int4 split = make_int4(0, 0, 0, 0);
      int piece = 0;
#pragma unroll 1
      for (int before = items[0].nj > 0 ? items[0].j : 0; before > 0; before -= run) ++piece;
      for (int k = 0; items[k & 1].nj > 0; ++k) {
        const Item& it = items[k & 1];
        next_item(b, it, items[(k + 1) & 1]);
        const int lead = it.pair ? 1 : 2, nj = it.nj;
        // Page ids are copied kIdsAhead steps before their keys are due, so no
        // load waits for one.
        StepWalk wf, wk;   // of the ids, of the keys
        wf.start(b, it.t, it.j);
        wk = wf;
        const int step0 = steps;
#pragma unroll 1
        for (int i = -2 * (lead + kIdsAhead); i < 2 * nj; ++i) {   // round i >> 1: values, then ids and keys
          const bool keys = i & 1;
          const int j = (i >> 1) + (keys ? lead : 0);
          if (keys) {
            const int jf = j + kIdsAhead;
            if (jf < nj) {
              const int32_t* table = table_of(a, wf.s.seq);
              int* dst = s_page[(step0 + jf) % kIdRing];
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                const int key0 = wf.s.base + u * kPage;
                if (key0 < wf.s.end) copy_async4(dst + u, table + key0 / kPage);
                else dst[u] = -1;
              }
              wf.next(b, it.t);
            }
            copy_async_commit();
            copy_async_wait<kIdsAhead>();
          }
          if (j < 0 || j >= nj) continue;
          const int slot = c % S;
          ok = bar_wait(empty_at + slot * 8, (c / S & 1) ^ 1, progress_at, wait_tries);
          if (!ok) break;
          const uint32_t dst = ring + slot * C::kHalf, bar = full_at + slot * 8;
          // a page past the sequence's end, or none of the pool's, reads as
          // zeros: from behind the pool's last page
          int page[2], gone = 0;
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            page[u] = s_page[(step0 + j) % kIdRing][u];
            if (page[u] >= 0 && page[u] < a.b.n_pages) continue;
            page[u] = a.b.n_pages;
            gone |= 1 << u;
          }
          if (keys) {
            int flags = gone;
            if (it.pair) flags |= pair_takes(b, it.t, wk.s.seq, wk.s.base) << 2;
            wk.next(b, it.t);
            const uint32_t note = step_note(steps, flags);
            *const_cast<volatile uint32_t*>(s_step + steps++ % kStepRing) = note;
          }
          asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(C::kHalf) : "memory");
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            if (keys) {
#pragma unroll
              for (int bx = 0; bx < D / 64; ++bx)
                box_load(dst + bx * C::kBox + u * (C::kBox / 2), &maps.k, bar, bx * 64, it.head * kPage, page[u]);
            } else {
              box_load(dst + u * (C::kHalf / 2), &maps.v, bar, 0, it.head * D, page[u]);
            }
          }
          ++c;
        }
        if (!ok) {
          give_up();
          break;
        }
        if (it.j == 0 && nj < it.t.n) {   // the run ends here: the rest is the next CTAs'
          int pieces = 1;
#pragma unroll 1
          for (int left = it.t.n - nj; left > 0; left -= run) ++pieces;
          split = make_int4(it.t.t0, it.t.ntok, it.head, pieces);
        }
      }
      a.split[blockIdx.x] = split;
      a.piece[blockIdx.x] = piece;
      // copies still in flight complete before shared memory is released
      copy_async_wait<0>();
#pragma unroll 1
      for (int j = max(0, c - S); j < c; ++j) bar_wait(full_at + (j % S) * 8, j / S & 1, never_at, kWaitTries);
    }
  } else if (warp < kSoftWarp0) {
    // ---------------- products of one stream ----------------
    // In each round the product of the step's weights with its values and the
    // scores of the step `lead` later, where the stream takes them. Each stream
    // waits for every half and arrives for it, its own or not: a stream that
    // passed over halves could meet a barrier a whole turn of the ring away.
    // The warp goes through this as one, with one elected lane in front of the
    // instructions, so that descriptors stay in uniform registers: with one
    // lane alone in here a product took 98 cycles to issue beside the softmax
    // warps, against 64 to run.
    const int s = warp_uniform(warp - 1);
    const bool one = elect_one();
    const uint32_t q_low = sdesc_low(smem_u32(smem)), ring_low = q_low + (C::kQBytes >> 4);
    const uint32_t full_at = smem_u32(kv_full), empty_at = smem_u32(kv_empty);
    const uint32_t s_at = smem_u32(&s_full[0]) + s * 8, p_at = smem_u32(&p_full[0][0]) + s * 16;
    const uint32_t turn_at = smem_u32(&turn[0]) + s * 8, pass_at = smem_u32(&turn[0]) + (s ^ 1) * 8;
    const uint32_t tm = warp_uniform(tmem);
    const uint32_t s_col = tm + s * kStepKeys, o_col = tm + kOCol + s * D;
    int c = 0, steps = 0, k = 0, np = 0, turns = 0;   // ring halves, steps with scores, items, P tiles, rounds of pairs
    int brought = 0;    // items whose queries were called for
    bool ok = true;
    auto wait = [&](uint32_t bar, uint32_t parity) {
      if (ok) ok = __all_sync(0xffffffffu, bar_wait(bar, parity, progress_at, wait_tries));
    };
    auto bring_q = [&](const Item& it) {   // an item's queries
      if (ok && one) {
        const uint32_t bar = smem_u32(&q_full);
        const int n = it.pair ? 2 : 1;
        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar),
                     "r"(n * (D / 64) * a.stream_tokens * G * 128)
                     : "memory");
#pragma unroll 1
        for (int i = 0; i < n * (D / 64); ++i) {
          const int st = i / (D / 64), bx = i % (D / 64);
          box_load(smem_u32(smem) + st * C::kHalf + bx * C::kBox, &maps.q, bar, bx * 64, it.head * G,
                   it.t.t0 + st * a.stream_tokens);
        }
      }
      brought += ok;
      __syncwarp();
    };
    if (s == 0 && items[0].nj > 0) bring_q(items[0]);
    while (true) {
      const Item& it = items[k & 1];
      const int pair = warp_uniform(it.pair), nj = warp_uniform(it.nj), lead = pair ? 1 : 2;
      if (nj <= 0) break;
      __syncwarp();
      const uint32_t q_at = q_low + (pair ? s * (C::kHalf >> 4) : 0);
      wait(smem_u32(&q_full), k & 1);
      ++k;
      uint32_t add = 0;
      uint32_t takes = 0;   // bit i: the stream takes step j + i
#pragma unroll 1
      for (int j = -lead; j < nj && ok; ++j) {
        const int pv = j >= 0, more = j + lead < nj;
        if (j == nj - lead) {   // the scores are all issued: on to the next item's queries
          if (lane == 0) next_item(b, it, items[k & 1]);
          __syncwarp();
          if (s == 0 && items[k & 1].nj > 0) {
            wait(smem_u32(&q_empty), (k - 1) & 1);
            bring_q(items[k & 1]);
          }
        }
        const int ck = c + pv, vslot = c % S, kslot = ck % S;
        // One lane for each thing to wait for, so that the waits are one (in a
        // row they were 300 cycles each: the products keep shared memory busy).
        // Of a pair, whose steps are long, that is everything but the second
        // page's weights, and its streams take turns: their products in one
        // block each, so that one stream's run while the other's softmax does.
        // An alternating tile's values go back as soon as they can.
        const bool weights = pair ? pv : takes & 1;   // the softmax has arrived, or will
        uint32_t early = 0;
        {
          if (pair && more) early = note_early<kStepRing>(s_step, steps);
          bool need = lane == 0 && pv;
          uint32_t bar = full_at + vslot * 8, parity = c / S & 1;
          if (lane == 1) need = pair && more, bar = full_at + kslot * 8, parity = ck / S & 1;
          if (lane == 2) need = weights, bar = p_at, parity = np & 1;
          if (lane == 3) need = pair && (s == 1 || turns > 0), bar = turn_at, parity = (s == 1 ? turns : turns - 1) & 1;
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
        turns += pair;
        if (!ok) break;
        uint32_t take = ((j + lead) & 1) == s && more;
        if (pair && more) take = warp_uniform(note_of<kStepRing>(s_step, steps, early) >> (2 + s) & 1);
        tc_fence_after();
        if (takes & 1) {   // O (+)= P V
          const uint32_t v_at = ring_low + vslot * (C::kHalf >> 4);
          // the first page's weights while the second's are still made
          if (one) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              tc_mma_bf16_ts(o_col, s_col + kk * 8, sdesc_of(v_at + (kk * 32 >> 4)), kIdescO, kk > 0 ? 1u : add);
          }
          __syncwarp();
          wait(p_at + 8, np & 1);
          if (!ok) break;
          tc_fence_after();
          if (one) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              tc_mma_bf16_ts(o_col, s_col + 32 + kk * 8, sdesc_of(v_at + ((C::kHalf / 2 + kk * 32) >> 4)), kIdescO, 1u);
            bar_commit(empty_at + vslot * 8);
          }
          add = 1;
        } else if (pv) {
          if (weights) wait(p_at + 8, np & 1);
          if (one) bar_arrive(empty_at + vslot * 8);
        }
        np += weights;
        __syncwarp();
        if (!pair && more) {
          wait(full_at + kslot * 8, ck / S & 1);
          if (!ok) break;
        }
        if (pair && one) bar_arrive(pass_at);   // the other stream's waits pass under these products
        if (take) {   // S = Q K^T
          const uint32_t k_at = ring_low + kslot * (C::kHalf >> 4);
          if (one) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = ((kk >> 2) * C::kBox + (kk & 3) * 32) >> 4;
              tc_mma_bf16(s_col, sdesc_of(q_at + off), sdesc_of(k_at + off), kIdescS, kk > 0);
            }
            bar_commit(s_at);
            bar_commit(empty_at + kslot * 8);
          }
          takes |= 1u << lead;
        } else if (more && one) {
          if (pair) bar_arrive(s_at);   // the softmax follows every step of a pair
          bar_arrive(empty_at + kslot * 8);
        }
        if (one) {
          if (more && j + lead + 1 == nj) bar_commit(smem_u32(&q_empty));   // the item's queries are not needed any more
        }
        __syncwarp();
        c = ck + more;
        steps += more;
        takes >>= 1;
      }
      if (!ok) {
        give_up();
        break;
      }
      if (add && one) bar_commit(smem_u32(&o_done[0]) + s * 8);   // only then does the softmax wait for it
    }
    // every issued product completes before TMEM and shared memory are released
    if (one) bar_commit(smem_u32(&mma_done));
    bar_wait(smem_u32(&mma_done), 0, never_at, kWaitTries);
    if (brought > 0) bar_wait(smem_u32(&q_full), (brought - 1) & 1, never_at, kWaitTries);   // and every copy arrives
  } else {
    // ---------------- softmax and output ----------------
    const int stream = warp >= kSoftWarp0 + 4 ? 1 : 0;
    const int quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t lane_tmem = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t s_tmem = lane_tmem + stream * kStepKeys;
    const uint32_t o_tmem = lane_tmem + kOCol + stream * D;
    const float sl2 = a.scale_log2;
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
    auto warp_arrive = [&](uint64_t* bar) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    while (true) {
      const Item& it = items[k & 1];
      if (it.nj <= 0) break;
      __syncwarp();
      if (lane == 0) next_item(b, it, items[++k & 1]);
      k = __shfl_sync(0xffffffffu, k, 0);
      const Row row = row_at(b, it.t, it.pair ? stream : 0, r);
      float mref = -INFINITY, l = 0.f;   // the row's reference maximum (log2 units, less the bias), sum
      int done = 0;                      // steps of this item that this stream took
      StepWalk w;
      w.start(b, it.t, it.j);
      const int pair = it.pair, nj = it.nj;
      for (int j = 0; j < nj; ++j, w.next(b, it.t)) {
        if (!pair && (j & 1) != stream) continue;
        const uint32_t rest = w.s.end - w.s.base;
        if (rest < kStepKeys && rest % kPage != 0 && (!pair || stream == 0)) {
          // Of a pair the first stream's warps do it: its products' turn comes
          // before the other's. In the ring an item's keys lead its values by 1
          // step (pair) or 2, and the half that lay in the values' place must have
          // come, or its barrier's phase would be taken for theirs: with 8 halves,
          // or in a pair, the scores seen last say so, else the ones to come.
          const int c = 2 * step0 + j + min(j + (pair ? 1 : 2), nj);
          ok = cut_values<D>(smem_u32(smem) + C::kQBytes, smem_u32(kv_full), progress_at, wait_tries, c, rest,
                             S == 4 && !pair ? smem_u32(&s_full[stream]) : 0, ns & 1);
          if (!ok) break;
        }
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
          warp_arrive(&p_full[stream][0]);
          warp_arrive(&p_full[stream][1]);
        } else {
          const int gone = flags & 3;
          if (gone != 0 || !__all_sync(0xffffffffu, c_hi >= kStepKeys && (c_lo <= 0 || c_sink >= kStepKeys))) {
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
          // a half of the scores (one page) at a time: the second for its
          // maximum, the first for its maximum and weights, the second again
          float sv[64];
          auto load = [&](int u) { tmem_ld64(s_tmem + u * kPage, sv); };
          load(1);
          float mx = row_max(sv);
          load(0);
          mx = fmaxf(mx, row_max(sv)) * sl2 - kBias;
          if (__any_sync(0xffffffffu, mx > mref + kRescaleLog2)) {
            const float nm = fmaxf(mref, mx);
            const float alpha = nm == -INFINITY ? 1.f : ex2(mref - nm);
            l *= alpha;
            mref = nm;
            if (done > 0) {
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
            }
          }
          const float neg = mref == -INFINITY ? 0.f : -mref;
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
          for (int u = 0; u < 2; ++u) {   // P replaces scores that are in registers by then
            if (u == 1) load(1);
            uint32_t pk[32];
            // ex2.approx is off by 2^-22 of a weight at most and takes those below
            // 2^-126 for zero. For the product weights are rounded to the values'
            // type, since its two operands have one (the sum takes them in fp32):
            // half a step of each, which makes the error against 64 bits 0.0023
            // instead of the 0.0017 of rounding the output alone (fp16: 0.0003 and
            // 0.0002). Weights in two parts would double the product.
            // exponentials, then packing, then sums: the three in turn for each
            // pair cost 5.7 instead of 5.2 cycles a value (two warps a scheduler)
#pragma unroll
            for (int c = 0; c < 32; ++c) {
              const float2 e = fma2(make_float2(sv[2 * c], sv[2 * c + 1]), make_float2(sl2, sl2), make_float2(neg, neg));
              sv[2 * c] = ex2_here(e.x);
              sv[2 * c + 1] = ex2_here(e.y);
            }
#pragma unroll
            for (int c = 0; c < 32; ++c) pk[c] = pack2<F16>(sv[2 * c], sv[2 * c + 1]);
#pragma unroll
            for (int c = 0; c < 32; ++c) sum[c & 1] = add2(sum[c & 1], make_float2(sv[2 * c], sv[2 * c + 1]));
            tmem_st_u32(s_tmem + u * (kPage / 2), pk);
            tmem_wait_st();
            warp_arrive(&p_full[stream][u]);
          }
          l += (sum[0].x + sum[1].x) + (sum[0].y + sum[1].y);
        }
        ++done;
        ++ns;
        if (!ok) break;
      }
      if (!ok) break;
      step0 += it.nj;
      if (done > 0) warp_wait(&o_done[stream], outs++ & 1);
      if (!ok) break;

      ok = finish_item<D, F16, Redo<D, F16>>(a, b, it, join, stream, tmem, row.token, mref, l, 1.f, done > 0, nx & 1, progress_at);
      nx += !it.pair;
      if (!ok) break;
    }
    if (!ok) give_up();
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Join the pieces of the tiles that the main kernel split: piece 0 lies in slot
// 1 of the CTA c that began the tile, piece p in slot 0 of CTA c + p. Every CTA
// that holds a piece has blocks here which take their share of the tile's rows
// (a tile in many pieces, whose rows cost more, gets more of them). One warp per
// row; a row's pieces are read kAtOnce at a time, all under way together.
constexpr int kCombineWarps = 8, kAtOnce = 8, kCombineBlocks = 8;

template <int D, bool F16>
__global__ void __launch_bounds__(kCombineWarps * 32) paged_combine_kernel(const __grid_constant__ PagedAttnArgs a) {
  constexpr int kPer = D / 32;
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31, G = a.b.group, stream_rows = a.stream_tokens * G;
  const int last_piece = a.piece[blockIdx.x];
#pragma unroll 1
  for (int own = last_piece > 0 ? 0 : 1; own < 2; ++own) {
    const int share = own ? 0 : last_piece, cta = blockIdx.x - share;
    const int4 sp = a.split[cta];   // first token, tokens, kv head, pieces
    const int n = sp.w;
#pragma unroll 1
    for (int i = (blockIdx.y * kCombineWarps + (threadIdx.x >> 5)) * n + share; n > 0 && i < sp.y * G;
         i += gridDim.y * kCombineWarps * n) {
      const int row = i < stream_rows ? i : kRows + i - stream_rows;
      const size_t first = (static_cast<size_t>(cta) * 2 + 1) * a.rows_cap + row;
      const size_t step = static_cast<size_t>(2) * a.rows_cap;
      auto at = [&](int p) { return p == 0 ? first : first + p * step - a.rows_cap; };
      float top = -INFINITY, l = 0.f, acc[kPer];
#pragma unroll
      for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
#pragma unroll 1
      for (int p0 = 0; p0 < n; p0 += kAtOnce) {
        float2 ml[kAtOnce];
        float2 v[kAtOnce][kPer / 2];
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
          ml[u] = make_float2(-INFINITY, 0.f);
#pragma unroll
          for (int e = 0; e < kPer / 2; ++e) v[u][e] = make_float2(0.f, 0.f);
          if (p0 + u < n) {
            ml[u] = __ldcg(a.part_ml + at(p0 + u));
            const float2* src = reinterpret_cast<const float2*>(a.part_o + at(p0 + u) * D + lane * kPer);
#pragma unroll
            for (int e = 0; e < kPer / 2; ++e) v[u][e] = __ldcg(src + e);
          }
        }
        float nt = top;
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) nt = fmaxf(nt, ml[u].x);
        const float ref = nt == -INFINITY ? 0.f : nt, old = ex2(top - ref);
        top = nt;
        l *= old;
#pragma unroll
        for (int e = 0; e < kPer; ++e) acc[e] *= old;
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
          const float w = ex2(ml[u].x - ref);
          l = fmaf(w, ml[u].y, l);
#pragma unroll
          for (int e = 0; e < kPer / 2; ++e) {
            acc[2 * e] = fmaf(w, v[u][e].x, acc[2 * e]);
            acc[2 * e + 1] = fmaf(w, v[u][e].y, acc[2 * e + 1]);
          }
        }
      }
      const int j = i / G;
      if (a.part == 1) {   // of the own caches: for the prefix's part
        const size_t to = static_cast<size_t>(sp.x + j) * a.b.n_heads + sp.z * G + i - j * G;
#pragma unroll
        for (int e = 0; e < kPer; e += 2) *reinterpret_cast<float2*>(a.own_o + to * D + lane * kPer + e) = make_float2(acc[e], acc[e + 1]);
        if (lane == 0) a.own_ml[to] = make_float2(top, l);
        continue;
      }
      const float f = l > 0.f || l != l ? 1.f / l : 0.f;
      uint16_t* out = out_row(a, sp.x + j, sp.z, i - j * G, D) + lane * kPer;
#pragma unroll
      for (int e = 0; e < kPer; e += 2)
        *reinterpret_cast<uint32_t*>(out + e) = pack2<F16>(acc[e] * f, acc[e + 1] * f);
    }
  }
}

const char* attn_check(const dflash_paged_batch* b, const void* q, long long q_stride, const void* out,
                       long long out_stride, float scale) {
  if (const char* why = paged_check(b)) return why;
  // the exponents are taken to base 2, by a factor of scale * log2(e)
  if (!(scale > 0.f && scale <= 0x1p127f)) return "scale must be in (0, 2^127]";
  if (b->n_seq == 0 || b->n_tokens == 0) return nullptr;
  const long long width = static_cast<long long>(b->n_heads) * b->head_dim;
  if (!q || !out) return "null pointer";
  if (bad_stride(q_stride, width) || bad_stride(out_stride, width))
    return "token strides must be multiples of 8 elements and at least a token's row";
  if (misaligned16(q) || misaligned16(out)) return "q and out must be 16-byte aligned";
  if (rows_overlap(q, q_stride, width, out, out_stride, width, b->n_tokens)) return "out must not overlap q";
  if (in_pool(*b, out, out_stride, width)) return "out must not lie in the pool";
  return nullptr;
}

// The tile's shape and the workspace's layout for a batch.
struct Plan {
  Q8Few few;
  int device, ctas, stream_tokens, tile_tokens, rows_cap;
  bool own;   // behind a prefix: the own caches apart (`few` is theirs then)
  size_t piece_off, ml_off, o_off, own_ml_off, own_o_off, bytes;   // the split records come first
};

// Whether a batch over 8-bit pages is one for the kernel of few rows (that many
// of a kv head for each sequence on average: tiles hold no more, so longer blocks
// are cut), and how. At 32 rows it takes 166 us instead of 177 (8 tokens of 32
// sequences of 8192 keys, 4 heads a kv head); 64 would read the keys twice. Short
// caches of 17 to 32 rows are read twice by two tiles of 16, whose steps are
// shorter chains (8 tokens over 4096 keys 14.2 us instead of 17.7, of 8 sequences
// over 1024 22.4 instead of 24.3, of 16 over 2048 the same, of 48 over 1024 62
// instead of 58; tables wider than the caches leave it at 32 rows). Two
// CTAs an SM let one's ends pass under the other's work (8 tokens of 16 sequences of
// 2048 keys 40 us instead of 43, 128 single ones of 2048 109 instead of 129; but 64 of
// 32768 720 instead of 670, 8 tokens of 8 of 256 16.3 instead of 12.5); one for
// each, of all its warps, is better with few tiles (a token over 4096 keys 12.2 us
// instead of 13.2; with 16 tiles 14.2 instead of 13.7).
// What the average hides: a long block among single tokens or empty entries is cut
// into tiles of so many rows, which each read its whole cache, at most as often as the
// batch has sequences. 160 single tokens and a block of 1024, all over 8192 keys, take
// 1300 us (446 and 158 in two calls; over 16-bit pages 1178), 63 and a block of 200
// 420 (191 and 62; 470), a block of 4096 among 1023 empty entries 2046 (alone 424; 329).
// The lengths that tell are on the device; the caller can give such a block its own call.
Q8Few few_rows(const dflash_paged_batch& b, bool shared) {
  const int group = b.n_heads / b.n_kv_heads;
  const long long rows = static_cast<long long>(b.n_tokens) * group, tiles = shared ? 1 : b.n_seq;
  const long long keys = tiles * b.n_kv_heads * kPage * b.table_pages;   // at most, all heads together
  Q8Few few{0, 1};
  if (!(b.dtype & DFLASH_POOL_Q8)) return few;
  if (group <= 16 && rows <= 16 * tiles) few.rows = 16;
  else if (group <= 32 && rows <= 32 * tiles) few.rows = group <= 16 && !shared && keys <= 1 << 18 ? 16 : 32;
  if (few.rows == 32 || (few.rows == 16 && tiles * b.n_kv_heads > 8)) few.per_sm = 2;
  return few;
}

// Behind a prefix a tile of 128 rows meets the own cache of each of its sequences
// with the rows of one. Of many short blocks with long own caches these steps are
// most of the work, and are taken apart from the prefix, by the kernel of few rows.
// The rule sees the page tables' width, not the lengths: single tokens behind 2048
// take 110 us instead of 158 (64 sequences, own caches of 2048) and 163 instead of
// 285 (128 of 2048), about the same at 1024 pages (98 and 101: 128 of 512), and
// less would cost (67 instead of 65: 64 of 512; wide tables of short caches, 56
// instead of 39: 64 of 64). Below 64 sequences it is never done, also where it would
// pay (139 us instead of 208: 32 of 8192; 50 instead of 46: 16 of 2048).
constexpr int kOwnTokens = 1024;   // (the workspace holds their part in fp32)
bool own_apart(const dflash_paged_batch& b) {
  return b.n_seq >= 64 && b.n_tokens <= kOwnTokens && static_cast<long long>(b.n_seq) * b.table_pages > 1024 && few_rows(b, true).rows == 0 && few_rows(b, false).rows > 0;
}

bool make_plan(const dflash_paged_batch& b, bool shared, Plan& p) {
  if (cudaGetDevice(&p.device) != cudaSuccess ||
      cudaDeviceGetAttribute(&p.ctas, cudaDevAttrMultiProcessorCount, p.device) != cudaSuccess)
    return false;
  const int group = b.n_heads / b.n_kv_heads;
  p.stream_tokens = kRows / group;
  p.tile_tokens = 2 * p.stream_tokens;
  p.rows_cap = b.n_tokens > p.stream_tokens ? 2 * kRows : std::min(kRows, b.n_tokens * group);
  p.own = shared && own_apart(b);
  p.few = few_rows(b, shared && !p.own);
  // the same for every batch of so many tokens: over 8-bit pages there may be two
  // CTAs an SM, and own caches apart
  const bool q8 = b.dtype & DFLASH_POOL_Q8;
  const int ctas = q8 ? 2 * p.ctas : p.ctas;
  const size_t own_rows = q8 ? static_cast<size_t>(std::min(b.n_tokens, kOwnTokens)) * b.n_heads : 0;
  auto up = [](size_t n) { return (n + 255) & ~size_t(255); };
  p.piece_off = up(sizeof(int4) * ctas);
  p.ml_off = p.piece_off + up(sizeof(int) * ctas);
  p.o_off = p.ml_off + up(sizeof(float2) * 2 * ctas * p.rows_cap);
  p.bytes = p.o_off + sizeof(float) * 2 * ctas * p.rows_cap * b.head_dim;
  p.own_ml_off = up(p.bytes);
  p.own_o_off = p.own_ml_off + up(sizeof(float2) * own_rows);
  if (own_rows) p.bytes = p.own_o_off + sizeof(float) * own_rows * b.head_dim;
  return true;
}

cudaError_t launch_combine(const PagedAttnArgs& a, int d, bool f16, const Plan& p, int ctas, cudaStream_t s) {
  const dim3 grid(ctas, std::min(kCombineBlocks, (p.rows_cap + kCombineWarps - 1) / kCombineWarps));
  auto go = [&](auto kernel) { return launch_pdl(kernel, grid, dim3(kCombineWarps * 32), 0, s, a); };
  if (d == 128) return f16 ? go(paged_combine_kernel<128, true>) : go(paged_combine_kernel<128, false>);
  return f16 ? go(paged_combine_kernel<64, true>) : go(paged_combine_kernel<64, false>);
}

template <int D, bool F16>
cudaError_t launch(const PagedMaps& maps, const PagedAttnArgs& a, const Plan& p, cudaStream_t s) {
  // the shared-memory limit is set once per device (setting it again changes nothing)
  static std::atomic<uint64_t> set{0};
  cudaError_t e = cudaSuccess;
  if (p.device > 63 || !(set.load(std::memory_order_acquire) >> p.device & 1)) {
    e = cudaFuncSetAttribute(paged_attn_kernel<D, F16>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kSmem);
    if (e != cudaSuccess) return e;
    if (p.device < 64) set.fetch_or(uint64_t(1) << p.device, std::memory_order_release);
  }
  e = launch_pdl(paged_attn_kernel<D, F16>, dim3(p.ctas), dim3(kThreads), Cfg<D>::kSmem, s, maps, a);
  return e == cudaSuccess ? launch_combine(a, D, F16, p, p.ctas, s) : e;
}

std::atomic<int> g_wait_tries{kWaitTries};

dflash_status refuse(const char* why) {
  set_unattached_error(why);
  return DFLASH_EINVAL;
}

dflash_status fail_cuda(const char* why) {
  set_unattached_error(why);
  return DFLASH_ECUDA;
}

dflash_status run(const dflash_paged_batch& b, PagedAttnArgs& a, void* workspace, size_t workspace_bytes, void* stream) {
  Plan p;
  if (!make_plan(b, a.shared, p)) return fail_cuda("paged attention: no CUDA device");
  if (!workspace || reinterpret_cast<uintptr_t>(workspace) & 31 || workspace_bytes < p.bytes)
    return refuse("the workspace is null, not 32-byte aligned or smaller than dflash_paged_attn_workspace says");
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.stream_tokens = p.stream_tokens;
  a.tile_tokens = p.tile_tokens;
  a.rows_cap = p.rows_cap;
  a.split = reinterpret_cast<int4*>(ws);
  a.piece = reinterpret_cast<int*>(ws + p.piece_off);
  a.part_ml = reinterpret_cast<float2*>(ws + p.ml_off);
  a.part_o = reinterpret_cast<float*>(ws + p.o_off);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (b.dtype & DFLASH_POOL_Q8) {
    const bool f16 = b.dtype & DFLASH_FP16;
    cudaError_t e = cudaSuccess;
    if (p.few.rows > 0) {
      PagedAttnArgs f = a;
      f.stream_tokens = f.tile_tokens = p.few.rows / a.b.group;
      if (p.own) {
        f.shared = f.prefix_len = 0;
        p.own = a.prefix_len > 0;   // else there is nothing but the own caches
      }
      if (p.own) {
        f.part = 1;
        f.own_ml = a.own_ml = reinterpret_cast<float2*>(ws + p.own_ml_off);
        f.own_o = a.own_o = reinterpret_cast<float*>(ws + p.own_o_off);
        a.part = 2;
      }
      e = launch_paged_attn_q8_few(f, b.head_dim, f16, p.few, p.device, p.few.per_sm * p.ctas, s);
      if (e == cudaSuccess) e = launch_combine(f, b.head_dim, f16, p, p.few.per_sm * p.ctas, s);
    }
    if (e == cudaSuccess && (p.few.rows == 0 || p.own)) {
      e = launch_paged_attn_q8(a, b.head_dim, f16, p.device, p.ctas, s);
      if (e == cudaSuccess) e = launch_combine(a, b.head_dim, f16, p, p.ctas, s);
    }
    return e == cudaSuccess ? DFLASH_OK : fail_cuda("paged attention: kernel launch failed");
  }
  const uint64_t d = b.head_dim, n_kv = b.n_kv_heads, pages = b.n_pages;
  const uint64_t page_bytes = 2 * n_kv * kPage * d * 2;
  PagedMaps maps;
  // keys: rows of d elements, a page's rows head after head; values: rows of
  // the page's 64 slots; queries: [token][head][d]
  if (!encode_box_3d(&maps.k, b.pool, {d, kPage * n_kv, pages}, {d * 2, page_bytes}, {64, kPage, 1}) ||
      !encode_box_3d(&maps.v, static_cast<uint8_t*>(b.pool) + page_bytes / 2, {kPage, d * n_kv, pages},
                     {kPage * 2, page_bytes}, {64, static_cast<uint32_t>(d), 1}) ||
      !encode_box_3d(&maps.q, a.q, {d, static_cast<uint64_t>(b.n_heads), static_cast<uint64_t>(b.n_tokens)},
                     {d * 2, static_cast<uint64_t>(a.q_stride) * 2},
                     {64, static_cast<uint32_t>(a.b.group), static_cast<uint32_t>(p.stream_tokens)}))
    return fail_cuda("paged attention: cannot describe the pool or the queries for TMA");
  cudaError_t e;
  if (b.head_dim == 128) e = b.dtype == DFLASH_FP16 ? launch<128, true>(maps, a, p, s) : launch<128, false>(maps, a, p, s);
  else e = b.dtype == DFLASH_FP16 ? launch<64, true>(maps, a, p, s) : launch<64, false>(maps, a, p, s);
  return e == cudaSuccess ? DFLASH_OK : fail_cuda("paged attention: kernel launch failed");
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
  a.wait_tries = g_wait_tries.load(std::memory_order_relaxed);
  return a;
}

}  // namespace
}  // namespace dfl

using namespace dfl;

extern "C" dflash_status dflash_paged_attn_workspace(const dflash_paged_batch* b, size_t* bytes) {
  if (!bytes) return refuse("null pointer");
  *bytes = 0;
  if (const char* why = paged_check(b)) return refuse(why);
  if (b->n_seq == 0 || b->n_tokens == 0) return DFLASH_OK;
  Plan p;
  if (!make_plan(*b, false, p)) return fail_cuda("paged attention: no CUDA device");
  *bytes = p.bytes;
  return DFLASH_OK;
}

extern "C" dflash_status dflash_paged_attn(const dflash_paged_batch* b, const void* q, long long q_stride, void* out,
                                           long long out_stride, int window, int sinks, int causal, float scale,
                                           void* workspace, size_t workspace_bytes, void* stream) {
  if (const char* why = attn_check(b, q, q_stride, out, out_stride, scale)) return refuse(why);
  if (window < 0 || sinks < 0) return refuse("window and sinks must not be negative");
  if (b->n_seq == 0 || b->n_tokens == 0) return DFLASH_OK;
  PagedAttnArgs a = attn_args(*b, q, q_stride, out, out_stride, causal, scale);
  // positions stay below 2^30, so wider spans see the same
  a.window = std::min(window, 1 << 30);
  a.sinks = window > 0 ? std::min(sinks, 1 << 30) : 0;
  return run(*b, a, workspace, workspace_bytes, stream);
}

extern "C" dflash_status dflash_shared_prefix_attn(const dflash_paged_batch* b, const int32_t* prefix_table,
                                                   int prefix_len, const void* q, long long q_stride, void* out,
                                                   long long out_stride, int causal, float scale, void* workspace,
                                                   size_t workspace_bytes, void* stream) {
  if (const char* why = attn_check(b, q, q_stride, out, out_stride, scale)) return refuse(why);
  if (prefix_len < 0 || prefix_len > kPage * kPagedMaxTable) return refuse("prefix_len must be 0..2^26");
  if (b->n_seq == 0 || b->n_tokens == 0) return DFLASH_OK;
  if (prefix_len > 0 && !prefix_table) return refuse("null pointer");
  PagedAttnArgs a = attn_args(*b, q, q_stride, out, out_stride, causal, scale);
  a.prefix_table = prefix_table;
  a.prefix_len = prefix_len;
  a.shared = 1;
  return run(*b, a, workspace, workspace_bytes, stream);
}

extern "C" dflash_status dflash_debug_paged_wait_tries(int tries) {
  if (tries < 0 || tries > kWaitTries) return refuse("tries must be 0..2^23");
  g_wait_tries.store(tries, std::memory_order_relaxed);
  return DFLASH_OK;
}
