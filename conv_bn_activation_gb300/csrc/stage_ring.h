// Which phases of a ring of copies a warp has waited for, for kernels that
// issue the copies of step + stages - 1 before they wait for those of `step`.
// A bit is turned by a wait that ended well only: after one that ran out, it
// still names the phase that those copies complete.
#pragma once

#ifdef __CUDACC__
#define CB_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define CB_HOST_DEVICE inline
#endif

namespace cb {

template <int STAGES>
struct StageRing {
  unsigned phases = 0;  // bit s: the parity that stage s is waited for with
  CB_HOST_DEVICE unsigned parity(int stage) const { return (phases >> stage) & 1u; }
  CB_HOST_DEVICE void waited(int stage) { phases ^= 1u << stage; }
  // The stages whose copies are in flight when the wait for `step`, in `stage`, has run out: f(stage, parity).
  template <class F>
  CB_HOST_DEVICE void in_flight(int stage, int step, int steps, F f) const {
    for (int s = 0; s < STAGES && step + s < steps; ++s) {
      const int at = stage + s < STAGES ? stage + s : stage + s - STAGES;
      f(at, parity(at));
    }
  }
};

}  // namespace cb
