// ring.h -- a ring of barriers that copies complete on: which waits end all
// copies in flight.  (Host code too, so that it can be checked without a GPU.)
#pragma once

#ifdef __CUDACC__
#define DC_RING __host__ __device__ __forceinline__
#else
#define DC_RING inline
#endif

namespace dc {

// Use u of a ring of `slots` barriers is on barrier u % slots, in its phase u / slots.
// wait(barrier, parity) for the last uses of `used`, one a barrier at most: the
// ones before them have completed, or their barrier would not have been used again.
template <class Wait>
DC_RING void last_uses(int used, int slots, Wait wait) {
  for (int u = used > slots ? used - slots : 0; u < used; ++u) wait(u % slots, (u / slots) & 1);
}

// The copies of a block's units, begun for `units` of them: their Q (two
// buffers) and their rows' factors (kAheadUnits).
constexpr int kAheadUnits = 16;
template <class WaitQ, class WaitFactors>
DC_RING void unit_copies(int units, WaitQ wait_q, WaitFactors wait_factors) {
  last_uses(units, 2, wait_q);
  last_uses(units, kAheadUnits, wait_factors);
}

}  // namespace dc
