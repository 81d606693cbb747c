// paged_deal.h - how the attention's places are dealt to the CTAs (plain C++,
// so that it is checked on the host).
#pragma once

#ifdef __CUDACC__
#define DFL_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define DFL_HOST_DEVICE inline
#endif

namespace dfl {

// Whether `all` places can be dealt: runs of up to 2^29 of them (a quarter of an
// hour of work at least), so that twice a run's steps, the halves of the ring,
// are an int.
DFL_HOST_DEVICE bool deal_fits(long long all, int ctas) { return all >> 29 < ctas; }

// Places of a CTA's run: CTA c of `ctas` takes [c * run, (c + 1) * run). Of more
// than 2^31 in all the run is rounded up a little, which spares a division of 64
// bits.
DFL_HOST_DEVICE int deal_run(long long all, int ctas) {
#ifdef __CUDA_ARCH__
  const int zeros = __clzll(all);
#else
  const int zeros = all ? __builtin_clzll(all) : 64;
#endif
  const int up = all >> 31 ? 33 - zeros : 0;
  const unsigned n = ctas;
  return static_cast<int>((static_cast<unsigned>(all >> up) + (up ? n : n - 1)) / n) << up;
}

}  // namespace dfl
