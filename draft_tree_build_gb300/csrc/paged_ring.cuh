// The ring of tiles of a shared-prefix attention CTA: what the two warps that fill
// it wait for.  Plain arithmetic and order, for the host as well.
//
// Key tile t of the share is place 2 t, its value tile place 2 t + 1; place x is in
// stage x % kStages, whose barriers (full, empty) pass a phase a place.  A barrier is
// waited for by its phase's parity, so that whoever waits must have seen the phase
// before, or be what the phase after needs: else two more phases may have passed,
// and the parity means one that is still to come.
//
// The first keys go alone: all SMs fill their rings at once, and products begin 1 us
// sooner.  The key warp, without which stage 0 is not filled again, sees them land in
// full[0].  The value warp may be slow to begin, and two phases of full[0] pass without
// any value (the first scores are all that stage 0 waits for): it has a barrier of its
// own, `begun`, which completes once.
#pragma once

#include <cuda_runtime.h>

namespace bastion {

template <int kStages>
struct Ring {
  static __host__ __device__ __forceinline__ int stage(int x) { return x % kStages; }
  static __host__ __device__ __forceinline__ unsigned full_parity(int x) { return (unsigned)(x / kStages) & 1u; }
  static __host__ __device__ __forceinline__ unsigned empty_parity(int x) { return full_parity(x) ^ 1u; }

  // What comes before place x is filled; false: a wait ran out, and it must not be.
  template <typename Bars>
  static __host__ __device__ __forceinline__ bool before(Bars &b, int x) {
    if (x == 1 && !b.wait_begun()) return false;
    if (x == 2) {
      if (!b.wait_full(0, 0u)) return false;
      b.arrive_begun();
    }
    return b.wait_empty(stage(x), empty_parity(x));
  }
  // What comes after the last of the key warp's tiles, of which it has issued that many.
  template <typename Bars>
  static __host__ __device__ __forceinline__ void after_keys(Bars &b, int tiles) {
    if (tiles == 1 && b.wait_full(0, 0u)) b.arrive_begun();
  }
};

}  // namespace bastion
