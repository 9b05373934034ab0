// The kernels' bounded wait, as plain C++ so that a host test can run it.
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define VIDATTN_WAIT_FN __device__ __forceinline__
#else
#define VIDATTN_WAIT_FN inline
#endif

namespace vidattn {

enum class WaitEnd { kPhase, kGone, kTimeout };

// poll(): has the phase passed?  gone(): has this CTA, or any of the launch,
// given up?  now(): nanoseconds.  The limit counts from `since`, or, where that
// is 0, from the first look at the clock.
//
// A wait for other warps ends with them (gone).  kDrain, for copies and products
// that are in flight when the CTA is about to leave: it ends at its phase or at
// the limit, and whatever has gone wrong elsewhere does not end it, because
// shared and tensor memory may not be released under them.
template <bool kDrain, class Poll, class Gone, class Now>
VIDATTN_WAIT_FN WaitEnd bounded_wait(Poll poll, Gone gone, Now now, uint64_t limit_ns,
                                     uint64_t since = 0) {
  if (poll()) return WaitEnd::kPhase;
  for (uint32_t it = 1;; ++it) {
    if (poll()) return WaitEnd::kPhase;
    if ((it & 255u) != 0) continue;
    if (!kDrain && gone()) return WaitEnd::kGone;
    const uint64_t t = now();
    if (since == 0) since = t;
    if (t - since > limit_ns) return WaitEnd::kTimeout;
  }
}

}  // namespace vidattn
