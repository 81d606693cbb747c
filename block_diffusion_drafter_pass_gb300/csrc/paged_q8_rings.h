// paged_q8_rings.h - which barrier says that a half of the fp16 ring has been read
// (paged_attn_q8.cu), in plain C++, so that it is checked on the host.
//
// A wait on a barrier's parity tells a phase from its neighbours only, so who waits
// has to know already that the phase before the last is over. Two teams take every
// other half, and of a ring of `slots` halves the one that writes half h waits until
// half h - slots is read. With one barrier a slot and an odd number of slots a team
// would come by each only every second phase. With two, for the halves that a slot
// holds in turn, every team's visits to a barrier are consecutive phases of it.
#pragma once

#ifdef __CUDACC__
#define DFL_RING_FN __host__ __device__ __forceinline__
#else
#define DFL_RING_FN inline
#endif

namespace dfl {

// The barrier that half h's readers arrive on, of 2 * slots.
DFL_RING_FN constexpr int read_bar(int half, int slots) { return half % (2 * slots); }

// Before half h is written: the barrier of half h - slots, and the parity of its
// phase (h >= slots; the first `slots` halves wait for nothing).
DFL_RING_FN constexpr int free_bar(int half, int slots) { return read_bar(half - slots, slots); }
DFL_RING_FN constexpr int free_parity(int half, int slots) { return (half - slots) / (2 * slots) & 1; }

}  // namespace dfl
