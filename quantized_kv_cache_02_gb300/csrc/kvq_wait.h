// A wait bounded in time, apart from what it waits on and from the clock it
// reads, so that the order of its looks can be checked on the host.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define KVQ_WAIT_INLINE __device__ __forceinline__
#else
#define KVQ_WAIT_INLINE inline
#endif

namespace kvq {

// True once ready() is; false once stop() is, or when ``limit`` units of now()
// have passed since its first reading.  The caller may have stood still between
// a look and the clock for longer than the limit, with the phase completed
// meanwhile: the clock only ever ends the wait behind one more look.
template <typename Ready, typename Stop, typename Now>
KVQ_WAIT_INLINE bool bounded_wait(Ready ready, Stop stop, Now now, uint64_t limit) {
  if (ready()) return true;
  uint64_t begun = 0;
  for (uint32_t it = 1;; ++it) {
    if (ready()) return true;
    if (stop()) return false;
    if ((it & 63) == 0) {
      const uint64_t t = now();
      if (begun == 0) begun = t;
      if (t - begun > limit) return ready();
    }
  }
}

}  // namespace kvq
