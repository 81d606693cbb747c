// paged_walk.cuh - what the attention kernels over a caller's page pool share
// (16-bit pages: paged_attn.cu, 8-bit pages: paged_attn_q8.cu, few rows of these:
// paged_attn_q8_few.cu): the batch in
// shared memory, its tiles and their steps of 128 keys, how they are dealt to
// the CTAs, what a row sees, the waits, and an item's end. How the work is cut
// is said at the head of paged_attn.cu.
#pragma once

#include <cuda.h>

#include "paged.cuh"
#include "paged_deal.h"
#include "paged_row.cuh"

// Functions that are not worth their place in line, unless the kernel deals its
// registers to its warps by setmaxnreg, under which ptxas takes no calls.
#ifndef DFL_WALK_CALL
#define DFL_WALK_CALL __noinline__
#endif

namespace dfl {

constexpr int kStepKeys = 2 * kPage;
constexpr int kRows = 128;            // rows of a stream: the MMA's M
// What an item costs beside its steps, in steps (dealing only). With 2, uneven
// short blocks take 27.5 us instead of 25.5, uneven blocks behind a prefix of
// 5000 64.3 instead of 62.8 and one long sequence 170 instead of 162 (its runs
// then end a little off the heads' ends); with 8, 26.8, 66.2 and 177.
constexpr int kItemSteps = 4;
constexpr int kNoEnd = 1 << 30;       // above every position
constexpr float kRescaleLog2 = 8.f;   // rescale O when a row's maximum grows by more than 2^8

struct PagedAttnArgs {
  PagedView b;
  const int32_t* prefix_table;
  int prefix_len;
  int shared;                  // tiles span sequences, behind prefix_len shared tokens
  // 8-bit pages: a batch behind a prefix may be taken in two parts, the sequences'
  // own caches into own_o [token][head][d] and own_ml (maximum and sum), and then
  // the prefix alone, which joins them
  int part;                    // 0: all in one, 1: the own caches, 2: the prefix
  float* own_o;
  float2* own_ml;
  const uint16_t* q;
  long long q_stride;
  uint16_t* out;
  long long out_stride;
  int window, sinks, causal;
  float scale_log2;
  int wait_tries;              // of a wait in the kernel (bar_wait); 0: every one that has to wait gives up
  int stream_tokens;           // tokens of one stream's 128 rows
  int tile_tokens;             // tokens of a tile: one or two streams
  // partials: two slots per CTA (0: a tile begun by an earlier CTA, 1: a tile
  // that a later CTA ends), rows_cap rows each
  int rows_cap;
  float* part_o;               // [cta][2][rows_cap][d]
  float2* part_ml;             // [cta][2][rows_cap] maximum (log2 units), sum
  int4* split;                 // [cta] tile begun here and ended elsewhere: first token, tokens, kv head, pieces (0: none)
  int* piece;                  // [cta] which piece of a tile begun by an earlier CTA it holds (0: none)
};

// The kernel over 8-bit pages (paged_attn_q8.cu); the partials are joined by the caller.
cudaError_t launch_paged_attn_q8(const PagedAttnArgs& a, int head_dim, bool f16, int device, int ctas, cudaStream_t s);
// The one for few rows (paged_attn_q8_few.cu): tiles of up to `rows` of them (16
// or 32; 0: not for this batch) in one stream, and `per_sm` CTAs an SM.
struct Q8Few {
  int rows, per_sm;
};
cudaError_t launch_paged_attn_q8_few(const PagedAttnArgs& a, int head_dim, bool f16, const Q8Few& few, int device, int ctas, cudaStream_t s);

namespace {

// Tensor memory: the columns of the streams' S (P over its first 64), then their O.
constexpr uint32_t kOCol = 2 * kStepKeys;
constexpr uint32_t kTmemCols = 512;

constexpr int kBatchBytes = 4 * (3 * kPagedMaxSeqs + 16);

// A shared-memory descriptor (sdesc_kmajor_sw128) in two halves: the upper one
// is the same for every tile, and addresses step within the lower one.
__device__ __forceinline__ uint32_t sdesc_low(uint32_t saddr) { return ((saddr & 0x3FFFFu) >> 4) | (1u << 16); }
__device__ __forceinline__ uint64_t sdesc_of(uint32_t low) {
  constexpr uint32_t kHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
  return (static_cast<uint64_t>(kHigh) << 32) | low;
}

// 2^x, not moved by the compiler.
__device__ __forceinline__ float ex2_here(float x) {
  float y;
  asm volatile("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ unsigned long long bits2(float2 v) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(v.x), "f"(v.y));
  return r;
}
__device__ __forceinline__ float2 floats2(unsigned long long v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 x, float2 y, float2 z) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits2(x)), "l"(bits2(y)), "l"(bits2(z)));
  return floats2(r);
}
__device__ __forceinline__ float2 add2(float2 x, float2 y) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(x)), "l"(bits2(y)));
  return floats2(r);
}

// What the walk over the work needs, in shared memory: functions that are
// called take it by reference, and a reference to registers or parameters
// would put those into local memory.
struct Batch {
  int shared, causal, window, sinks, prefix_len, prefix_only;
  int stream_tokens, tile_tokens;
  int n_seq, n_kv, group;
  int q[kPagedMaxSeqs + 1];      // the bounds of the sequences' tokens (bent into range)
  int len[kPagedMaxSeqs];        // their cached tokens
  int base[kPagedMaxSeqs + 1];   // own cache: tiles before a sequence; shared: own-cache steps before it
};

static_assert(sizeof(Batch) <= kBatchBytes, "room for the batch");

struct Tile {
  int t0, ntok;         // tokens
  int seq0, seq1;       // sequences of the first and last token
  int n;                // steps, at least 1 (a tile that sees nothing has a step without a visible key)
  int head_steps;       // own cache: steps over the first tokens; shared: over the prefix
  int window_step;      // own cache: the step index after those
};

__device__ __forceinline__ int steps_of(int keys) { return keys > 0 ? (keys + kStepKeys - 1) / kStepKeys : 0; }

__device__ __forceinline__ Tile tile_at(const Batch& b, int tile) {
  Tile r;
  if (b.shared) {
    r.t0 = b.q[0] + tile * b.tile_tokens;
    r.ntok = min(b.tile_tokens, b.q[b.n_seq] - r.t0);
    const int last = r.t0 + r.ntok - 1;
    r.seq0 = seq_of_token(b.q, b.n_seq, r.t0);
    r.seq1 = seq_of_token(b.q, b.n_seq, last);
    r.head_steps = steps_of(b.prefix_len);
    r.window_step = 0;
    // the last sequence may go on behind the tile: its keys up to the tile's last row
    const int end = b.causal ? b.len[r.seq1] - (b.q[r.seq1 + 1] - 1 - last) : b.len[r.seq1];
    r.n = max(1, b.prefix_only ? r.head_steps : r.head_steps + b.base[r.seq1] - b.base[r.seq0] + steps_of(end));
    return r;
  }
  int lo = 0, hi = b.n_seq - 1;   // the last sequence whose tiles start at or before this one
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (b.base[mid] <= tile) lo = mid;
    else hi = mid - 1;
  }
  r.seq0 = r.seq1 = lo;
  r.t0 = b.q[lo] + (tile - b.base[lo]) * b.tile_tokens;
  r.ntok = min(b.tile_tokens, b.q[lo + 1] - r.t0);
  const int pos0 = b.len[lo] - (b.q[lo + 1] - r.t0);
  const int end = b.causal ? pos0 + r.ntok : b.len[lo];
  const int w1 = steps_of(end);
  const int w0 = b.window > 0 ? min(max(0, pos0 - b.window + 1) / kStepKeys, w1) : 0;
  r.head_steps = min(steps_of(b.sinks), w0);
  r.window_step = w0;
  r.n = max(1, r.head_steps + w1 - w0);
  return r;
}

// One step: 128 keys from `base` of a sequence's cache (seq >= 0) or of the
// prefix (seq = -1), of which those below `end` exist.
struct Step {
  int seq, base, end;
};

// The steps of a tile in order, from any of them on.
struct StepWalk {
  Step s;
  int left;   // steps left in this run of keys
  __device__ __forceinline__ void start(const Batch& b, const Tile& t, int j) {
    if (b.shared) {
      if (j < t.head_steps) {
        s = Step{-1, j * kStepKeys, b.prefix_len};
        left = t.head_steps - j;
        return;
      }
      const int want = b.base[t.seq0] + j - t.head_steps;
      int lo = t.seq0, hi = t.seq1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (b.base[mid] <= want) lo = mid;
        else hi = mid - 1;
      }
      s = Step{lo, (want - b.base[lo]) * kStepKeys, b.len[lo]};
      left = lo < t.seq1 ? b.base[lo + 1] - want : INT32_MAX;
      return;
    }
    const bool head = j < t.head_steps;
    s = Step{t.seq0, (head ? j : t.window_step + j - t.head_steps) * kStepKeys, b.len[t.seq0]};
    left = head ? t.head_steps - j : INT32_MAX;
  }
  __device__ __forceinline__ void next(const Batch& b, const Tile& t) {
    s.base += kStepKeys;
    if (--left > 0) return;
    if (!b.shared) {
      s.base = t.window_step * kStepKeys;
      left = INT32_MAX;
      return;
    }
    int i = s.seq < 0 ? t.seq0 : s.seq + 1;
    while (i < t.seq1 && b.base[i + 1] == b.base[i]) ++i;
    s = Step{i, 0, b.len[i]};
    left = i < t.seq1 ? b.base[i + 1] - b.base[i] : INT32_MAX;
  }
};

// Whether some row of the tokens [ta, tb) of a tile sees a key of the step.
__device__ __forceinline__ bool step_counts(const Batch& b, int seq, int base, int ta, int tb) {
  if (seq < 0) return true;
  const int q0 = b.q[seq], q1 = b.q[seq + 1];
  const int first = max(ta, q0), last = min(tb, q1) - 1;
  if (first > last) return false;
  const int shift = b.len[seq] - q1;   // position of token t: t + shift
  if (b.causal && base > last + shift) return false;
  if (b.window > 0 && base + kStepKeys - 1 < first + shift - b.window + 1 && base >= b.sinks) return false;
  return true;
}

// Bit s: stream s of a pair takes the step.
__device__ DFL_WALK_CALL int pair_takes(const Batch& b, const Tile& t, int seq, int base) {
  const int mid = t.t0 + b.stream_tokens;
  return (step_counts(b, seq, base, t.t0, mid) ? 1 : 0) | (step_counts(b, seq, base, mid, t.t0 + t.ntok) ? 2 : 0);
}

// The producer's note on a step: bit u, page u is not there; bit 2 + s, stream s
// of a pair takes the step; from bit 4 on the step's number + 1, so that a
// reader may look for it before the barrier that says it is there (while the
// products read shared memory a load takes 300 cycles, which is better spent
// beside the wait than after it).
__device__ __forceinline__ uint32_t step_note(int step, int bits) { return (static_cast<uint32_t>(step) + 1) << 4 | bits; }
template <int kRing>
__device__ __forceinline__ uint32_t note_early(const uint32_t* s_step, int step) {
  return *const_cast<const volatile uint32_t*>(s_step + step % kRing);
}
// After the barrier, what was read before it or else the note itself.
template <int kRing>
__device__ __forceinline__ uint32_t note_of(const uint32_t* s_step, int step, uint32_t early) {
  return early >> 4 == static_cast<uint32_t>(step) + 1 ? early : note_early<kRing>(s_step, step);
}

// The row of one softmax thread: what it sees of its sequence's cache, and (of
// a shared prefix) prefix_len more.
struct Row {
  int token, seq;   // token < 0: no row
  int lo, hi;
};

__device__ __forceinline__ Row row_at(const Batch& b, const Tile& t, int stream, int r) {
  Row x;
  const int j = r / b.group, token = t.t0 + stream * b.stream_tokens + j;
  x.token = j < b.stream_tokens && token < t.t0 + t.ntok ? token : -1;
  x.seq = t.seq0 == t.seq1 || x.token < 0 ? t.seq0 : seq_of_token(b.q, b.n_seq, x.token);
  const int pos = b.len[x.seq] - b.q[x.seq + 1] + x.token;
  x.lo = b.window > 0 ? max(0, pos - b.window + 1) : 0;
  x.hi = b.causal ? pos : kNoEnd;
  return x;
}

// Its span of a step's run of keys (empty: hi < 0).
__device__ __forceinline__ RowSpan span_of(const Batch& b, const Row& x, const Step& s) {
  if (x.token < 0 || (s.seq >= 0 && s.seq != x.seq)) return RowSpan{0, -1, 0};
  if (s.seq < 0) return RowSpan{0, x.hi + b.prefix_len, 0};
  return RowSpan{x.lo, x.hi, b.sinks};
}

__device__ __forceinline__ const int32_t* table_of(const PagedAttnArgs& a, int seq) {
  return seq < 0 ? a.prefix_table : a.b.page_table + seq * a.b.table_stride;
}

// An item: steps [j, j + nj) of one tile and kv head. Every role walks the
// CTA's items in the same order; each warp keeps its own in shared memory.
// In the line that is dealt to the CTAs a tile and head takes kItemSteps
// places for what it costs at its begin and end, then one for each step; a run
// that ends within those leaves the item to the next CTA.
struct Item {
  Tile t;
  int tile, head, j, nj;
  int pair;         // each stream has its own 128 rows (else: the same rows, every other step)
  int place;        // the run's place within this tile and head
  int todo;         // places of the CTA from this item on
};

__device__ __forceinline__ int places_of(int steps) { return steps + kItemSteps; }

// The item at the run's place; nj <= 0 when the run ends before its steps.
__device__ __forceinline__ void cut_item(Item& it) {
  const int take = min(it.todo, places_of(it.t.n) - it.place);
  it.j = max(it.place - kItemSteps, 0);
  it.nj = it.place + take - kItemSteps - it.j;
  it.todo -= take;
}

// The run's item after `was` (its first: was.tile holds ~tile); nj = 0: none.
__device__ DFL_WALK_CALL void next_item(const Batch& b, const Item& was, Item& it) {
  it = was;
  it.nj = 0;
  if (it.todo <= 0) return;
  bool other = it.tile < 0;
  if (other) {
    it.tile = ~it.tile;
  } else {
    it.place = 0;
    if (++it.head == b.n_kv) {
      it.head = 0;
      ++it.tile;
      other = true;
    }
  }
  if (other) {
    it.t = tile_at(b, it.tile);
    it.pair = it.t.ntok > b.stream_tokens;
  }
  cut_item(it);
}

// Row of a partial: [cta][slot][rows_cap], slot 1 for a tile that begins here.
__device__ __forceinline__ size_t partial_row(const PagedAttnArgs& a, const Item& it, int stream, int r) {
  return (static_cast<size_t>(blockIdx.x) * 2 + (it.j == 0 ? 1 : 0)) * a.rows_cap + (it.pair ? stream * kRows : 0) + r;
}

__device__ __forceinline__ uint16_t* out_row(const PagedAttnArgs& a, int token, int kvh, int g, int d) {
  return a.out + token * a.out_stride + static_cast<long long>(kvh * a.b.group + g) * d;
}

// Waits of a CTA give up together: its word of progress is negative from then
// on. Before, it counts the pages of rows that are done again (redo_row), which
// take as long as the rows have keys: the others wait on while they go on.
constexpr int kGaveUp = INT32_MIN;
constexpr int kWaitTries = 1 << 23;   // of a microsecond at most
constexpr int kWaitPolls = 1 << 27;   // where barriers are polled

// Barriers by shared-window address. The wait is a loop of a few instructions
// in place (a called or clocked one costs every role's round a hundred and
// more): each try gives up after a microsecond at the latest, and the wait after
// `tries` of them between which *progress did not change, or when that is
// negative. False when it gave up.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, uint32_t progress, uint32_t tries) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b32 n, f, w;\n\tmov.b32 n, %4;\n\tmov.b32 w, 0;\n"
      "again:\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 1000;\n\t"
      "@p bra done;\n\t"
      "ld.volatile.shared.b32 f, [%3];\n\t"
      "setp.lt.s32 p, f, 0;\n\t"
      "@p bra fail;\n\t"
      "setp.ne.b32 p, f, w;\n\t"
      "@p mov.b32 n, %4;\n\t"
      "mov.b32 w, f;\n\t"
      "sub.u32 n, n, 1;\n\t"
      "setp.ne.u32 p, n, 0;\n\t"
      "@p bra again;\n"
      "fail:\n\tmov.b32 %0, 0;\n\tbra over;\n"
      "done:\n\tmov.b32 %0, 1;\n"
      "over:\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(progress), "r"(tries)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ bool bar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void bar_commit(uint32_t bar) {   // tc_commit
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// The warp's lane 0's value, as one that the compiler knows to be the warp's.
template <typename T>
__device__ __forceinline__ T warp_uniform(T v) {
  return __shfl_sync(0xffffffffu, v, 0);
}

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// tma_load_3d by shared-window addresses.
__device__ __forceinline__ void box_load(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// Sum over the threads before this one; `all`: over all. s_sum holds one for
// each warp and is free again behind the next barrier.
template <int kThreads>
__device__ __forceinline__ long long block_scan(long long v, long long* s_sum, long long& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long x = v;
#pragma unroll 1
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) s_sum[warp] = x;
  __syncthreads();
  long long before = x - v;
  all = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    const long long of = s_sum[w];
    if (w < warp) before += of;
    all += of;
  }
  return before;
}

__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// What deal_batch and the walk read of the arguments; one thread.
__device__ __forceinline__ void set_batch(const PagedAttnArgs& a, Batch& b) {
  b.shared = a.shared;
  b.causal = a.causal;
  b.window = a.window;
  b.sinks = a.sinks;
  b.prefix_len = a.prefix_len;
  b.prefix_only = a.part == 2;
  b.stream_tokens = a.stream_tokens;
  b.tile_tokens = a.tile_tokens;
  b.n_seq = a.b.n_seq;
  b.n_kv = a.b.n_kv;
  b.group = a.b.group;
}

// The batch into shared memory and this CTA's run of places: s_first[0] becomes
// its first item (nj is 0 before and stays it when there is none). Returns the
// places of a run. All kThreads threads call it; a barrier must follow.
template <int kThreads>
__device__ __forceinline__ int deal_batch(const PagedAttnArgs& a, Batch& b, long long* s_sum, Item* s_first) {
  const int tid = threadIdx.x, n_seq = a.b.n_seq, n_kv = a.b.n_kv;
  int raw_len = tid < n_seq ? a.b.kv_len[tid] : 0;   // under way with the bounds
  load_q_start(a.b, b.q);
  int total = 0;
#pragma unroll 1
  for (int i = tid, i0 = 0; i0 < n_seq; i0 += kThreads, i += kThreads) {
    int v = 0;
    if (i < n_seq) {
      const int nq = b.q[i + 1] - b.q[i], len = cached_tokens(a.b, i0 ? a.b.kv_len[i] : raw_len);
      b.len[i] = len;
      if (a.shared) v = nq > 0 ? steps_of(len) : 0;
      else v = (nq + a.tile_tokens - 1) / a.tile_tokens;
    }
    long long part;
    const int before = total + static_cast<int>(block_scan<kThreads>(v, s_sum, part));
    if (i < n_seq) b.base[i] = before;
    total += static_cast<int>(part);
    __syncthreads();   // the sums are read
  }
  if (tid == 0) b.base[n_seq] = total;
  __syncthreads();
  const int n_tiles = a.shared ? (b.q[n_seq] - b.q[0] + a.tile_tokens - 1) / a.tile_tokens : total;
  const int per = (n_tiles + kThreads - 1) / kThreads;
  const int tile_a = min(tid * per, n_tiles), tile_b = min(tile_a + per, n_tiles);
  long long mine = 0;
  int n = 0;   // places of one kv head of this thread's first tile
#pragma unroll 1
  for (int t = tile_b - 1; t >= tile_a; --t) {
    n = places_of(tile_at(b, t).n);
    mine += static_cast<long long>(n) * n_kv;
  }
  long long all;
  const long long before = block_scan<kThreads>(mine, s_sum, all);
  if (!deal_fits(all, gridDim.x)) {
    if (tid == 0) latch_status(a.b.status, kDevBounds);
    all = 0;
  }
  const int run = deal_run(all, gridDim.x);
  const long long x0 = static_cast<long long>(run) * blockIdx.x;
  const int x_len = static_cast<int>(max(0ll, min(static_cast<long long>(run), all - x0)));
  if (x_len > 0 && x0 >= before && x0 < before + mine) {   // one thread: the run begins in its tiles
    long long rem = x0 - before;
    Item& begin = s_first[1];
    begin.tile = tile_a;
#pragma unroll 1
    while (rem >= static_cast<long long>(n) * n_kv) {
      rem -= static_cast<long long>(n) * n_kv;
      n = places_of(tile_at(b, ++begin.tile).n);
    }
    begin.head = 0;
#pragma unroll 1
    for (; rem >= n; rem -= n) ++begin.head;
    begin.tile = ~begin.tile;
    begin.place = static_cast<int>(rem);
    begin.todo = x_len;
    next_item(b, begin, s_first[0]);
  }
  return run;
}

// Sets the status when a row would see a key of a page that is not there (bit u
// of gone: page u of the step); pages in front of the window or past the end may
// have been given back. Here since the row knows what it sees, and since the
// producer is a chain of steps in one lane: asked there, 16 tokens over 262144
// keys took 166 us instead of 162 (with heads of 64: 157 instead of 144).
__device__ DFL_WALK_CALL void report_gone(int* status, int gone, int c_lo, int c_hi, int c_sink) {
#pragma unroll 1
  for (int u = 0; u < 2; ++u) {
    const int c0 = u * kPage;
    const unsigned long long seen = slot_bits(0, c_hi - c0) & (slot_bits(c_lo - c0, 64) | slot_bits(0, c_sink - c0));
    if ((gone >> u & 1) && seen) latch_status(status, kDevBounds);
  }
}

// What the two softmax groups exchange at an alternating tile's end.
struct Join {
  uint64_t x_ml, x_bad;
  float2 ml[2][kRows];
  uint8_t bad[kRows];
};

// The same where O has a unit of its own.
struct JoinUnits : Join {
  float unit[2][kRows];
};

// log2 of a value scale's size from its bits, at least and by less than 0.09 too
// much; of smaller scales than 2^-90, and of zeros, -90.
__device__ __forceinline__ float scale_log2_bound(float scale) {
  return fmaxf(fmaf(static_cast<float>(__float_as_uint(scale) & 0x7FFFFFFFu), 0x1p-23f, -126.9138f), -90.f);
}

// Scales (of 128 keys, or of 32) are wide when they lie further apart than this many
// powers of two: each counts by itself then, for the rows that see its key.
constexpr int kNear = 10;
// Of the largest and the smallest of finite magnitudes, as bits (0x7F800000: there is no
// smallest), the largest's exponent, at least `least`, and whether they are wide. Scales
// that are all zero are not.
struct Spread {
  int exponent;
  bool wide;
};
__device__ __forceinline__ Spread spread_of(uint32_t top, uint32_t low, int least) {
  Spread r;
  r.exponent = max(static_cast<int>(top >> 23) - 127, least);
  r.wide = top != 0 && static_cast<int>(low >> 23) - 127 < r.exponent - kNear;
  return r;
}

// A sum of weights and its reference, for others to join: the sum between 1 and 2,
// so that a sum's product with a mean value stays in range where the value does.
__device__ __forceinline__ float2 joined_form(float mref, float l) {
  const int e = l > 0.f && l < INFINITY ? static_cast<int>(__float_as_uint(l) >> 23) - 127 : 0;
  return make_float2(mref + static_cast<float>(e), l * __int_as_float((127 - e) << 23));
}

// A stream's part of an item's end: O out of tensor memory, joined with the
// other stream's where both have the same rows, to `out` when the item is the
// whole tile, else to the partials. O times `unit` is in the terms of mref and l.
// False when a wait ran out. (A function of its own so that its registers are not
// the softmax loop's.)
template <int D, bool F16, class Again, class J>
__device__ DFL_WALK_CALL bool finish_item(const PagedAttnArgs& a, const Batch& b, const Item& it, J& join, int stream,
                                         uint32_t tmem, int token, float mref, float l, float unit, bool products,
                                         int parity, uint32_t progress) {
  const int lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) & 3, r = quarter * 32 + lane;
  const uint32_t lane_tmem = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
  auto meet = [&](uint64_t* bar) {   // of the two groups' eight warps
    tc_fence_before();
    __syncwarp();
    if (lane == 0) bar_arrive(smem_u32(bar));
    const bool ok = __all_sync(0xffffffffu, bar_wait(smem_u32(bar), parity, progress, a.wait_tries));
    tc_fence_after();
    return ok;
  };
  const bool whole = it.nj == it.t.n;
  const bool live = token >= 0;
  const size_t prow = partial_row(a, it, stream, r);
  // a warp's store touches a line for each of its rows: 32 bytes at a time
  // halves them (rows of partials and, where the caller's are aligned so, of out)
  const bool wide = ((reinterpret_cast<uintptr_t>(a.out) | static_cast<uintptr_t>(a.out_stride * 2)) & 31) == 0;
  char* const to = whole ? reinterpret_cast<char*>(out_row(a, token, it.head, r % b.group, D))
                         : reinterpret_cast<char*>(a.part_o + prow * D);
  // A pair's stream has its rows' whole sums in its O. Of an alternating
  // tile both streams hold a part of every row's: the groups exchange
  // maxima and sums, and each joins half of the columns.
  float w0 = Again::kOn ? 1.f : unit, w1 = 0.f, top = mref, lj = l;   // out = w0 * O of stream s0 + w1 * O of stream 1
  int col = 0, col_end = D, s0 = stream;
  bool use0 = products && l != 0.f, use1 = false;   // a stream without a visible key has no O to read
  if (!it.pair) {
    if (stream == 0) join.bad[r] = 0;
    join.ml[stream][r] = make_float2(mref, l);
    if constexpr (!Again::kOn) join.unit[stream][r] = unit;
    if (!meet(&join.x_ml)) return false;
    const float2 m0 = join.ml[0][r], m1 = join.ml[1][r];
    top = fmaxf(m0.x, m1.x);
    w0 = m0.x == -INFINITY ? 0.f : ex2(m0.x - top);
    w1 = m1.x == -INFINITY ? 0.f : ex2(m1.x - top);
    lj = m0.y * w0 + m1.y * w1;
    if constexpr (!Again::kOn) w0 *= join.unit[0][r], w1 *= join.unit[1][r];
    use0 = m0.y != 0.f;
    use1 = m1.y != 0.f;
    s0 = 0;
    col = stream * (D / 2);
    col_end = col + D / 2;
  }
  // what the row sees of its sequence's own cache, joined by the prefix's first piece
  float w2 = 0.f;
  const float* own = nullptr;
  if constexpr (!Again::kOn) {
    if (a.part == 2 && it.j == 0 && live) {
      const size_t at = static_cast<size_t>(token) * a.b.n_heads + it.head * b.group + r % b.group;
      const float2 m = __ldcg(a.own_ml + at);
      const float both = fmaxf(top, m.x), f = top == -INFINITY ? 0.f : ex2(top - both);
      w2 = m.x == -INFINITY ? 0.f : ex2(m.x - both);
      top = both;
      w0 *= f;
      w1 *= f;
      lj = fmaf(lj, f, m.y * w2);
      own = a.own_o + at * D;
    }
  }
  if (whole) {
    const float f = lj > 0.f || lj != lj ? 1.f / lj : 0.f;
    w0 *= f;
    w1 *= f;
    w2 *= f;
  }
  const bool any0 = __any_sync(0xffffffffu, use0), any1 = __any_sync(0xffffffffu, use1);
  float check = 0.f;   // NaN once a stored value is not finite
  // sixteen columns at a time: this runs once an item, so it costs what its
  // instructions cost to fetch, and more of them at a time were slower
#pragma unroll 1
  for (; col < col_end; col += 16) {
    float o[16];
    if (any0) tmem_ld16(lane_tmem + kOCol + s0 * D + col, o);
#pragma unroll
    for (int c = 0; c < 16; ++c) o[c] = use0 ? o[c] * w0 : 0.f;
    if (any1) {
      float o1[16];
      tmem_ld16(lane_tmem + kOCol + D + col, o1);
#pragma unroll
      for (int c = 0; c < 16; ++c) o[c] = use1 ? fmaf(o1[c], w1, o[c]) : o[c];
    }
#pragma unroll
    for (int c = 0; c < 16 && !Again::kOn; c += 4) {
      if (!own) continue;
      const float4 x = __ldcg(reinterpret_cast<const float4*>(own + col + c));
      o[c] = fmaf(x.x, w2, o[c]), o[c + 1] = fmaf(x.y, w2, o[c + 1]), o[c + 2] = fmaf(x.z, w2, o[c + 2]), o[c + 3] = fmaf(x.w, w2, o[c + 3]);
    }
#pragma unroll
    for (int c = 0; c < 16 && Again::kOn; ++c) check = fmaf(o[c], 0.f, check);
    if (live && whole) {
      uint32_t w[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) w[c] = pack2<F16>(o[2 * c], o[2 * c + 1]);
      char* const p = to + col * 2;
      if (wide) {
        store32(p, w);
      } else {
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        *reinterpret_cast<uint4*>(p + 16) = make_uint4(w[4], w[5], w[6], w[7]);
      }
    } else if (live) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t w[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) w[c] = __float_as_uint(o[8 * h + c]);
        store32(to + (col + 8 * h) * 4, w);
      }
    }
    __syncwarp();   // the next loads are the warp's
  }
  if (live && !whole && (it.pair || stream == 0)) a.part_ml[prow] = make_float2(top, lj);
  if (!it.pair) {
    if (live && check != 0.f) join.bad[r] = 1;
    // also: both groups have read both O before either's next P lets O be overwritten
    if (!meet(&join.x_bad)) return false;
    check = stream == 0 && join.bad[r] ? 1.f : 0.f;
  }
  // rows that met a non-finite value: again, from what they see
  if constexpr (Again::kOn)
  for (uint32_t bad = __ballot_sync(0xffffffffu, live && check != 0.f); bad; bad &= bad - 1)
    Again::row(a, b, it, stream, quarter * 32 + __ffs(bad) - 1, progress);
  return true;
}

}  // namespace
}  // namespace dfl
