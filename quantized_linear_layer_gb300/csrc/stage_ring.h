// Filling a ring of shared-memory stages with asynchronous copies in a block
// whose roles go on when one of their waits runs out.
//
// A role that goes on without waiting still signals: a stage can be given free
// while the copies into it are under way, by a reader that did not see them
// arrive.  Filling it then would arm a barrier whose phase is not over and put a
// second copy over the first.  So every role whose wait runs out raises the
// block's flag before it signals anything, and the filling role reads the flag
// after its wait for the free stage and before it issues anything: a signal that
// should not have been given comes with the flag.  Before it ends, the filling
// role waits for the stages it filled last, so that no copy outlives the block.
//
// The operations on barriers, the flag and the warp are the caller's (Ops), so
// that a host program can run the same code:
//   bool wait_free(stage, parity), bool wait_full(stage, parity)
//                          false: the wait ran out
//   bool raised(), void raise()   the block's flag
//   bool any(bool)         of the threads that fill together
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define QLIN_RING_FN __host__ __device__ __forceinline__
#else
#define QLIN_RING_FN inline
#endif

namespace qlin {
namespace ring {

// Whether `takers` readers may take the fills of a ring in turn (reader w the fills w, w + takers, ...), each waiting on
// the full barrier of its fill alone, by parity.  A parity cannot tell a phase from the one two before it: a reader that
// waits for fill u has to know that fill u - stages, the one before it in the same stage, has arrived, or it takes the
// end of the phase before that for its own.  It has seen fill u - takers arrive; so fills must arrive in order (as a
// thread's asynchronous copies do: each arrival follows all its earlier copies), and stages >= takers.
constexpr bool turns_are_safe(int stages, int takers) { return stages >= takers; }

// The filling role: STAGES stages in turn.
template <int STAGES>
struct Filler {
  uint32_t filled = 0;   // stages filled so far
  bool stopped = false;  // nothing is filled any more

  QLIN_RING_FN uint32_t stage() const { return filled % STAGES; }

  // Waits until stage() is free; false: it must not be filled, nor any later one.
  template <class Ops>
  QLIN_RING_FN bool wait(Ops& ops) {
    if (stopped) return false;
    const bool out = filled >= STAGES && !ops.wait_free(stage(), (filled / STAGES - 1) & 1);
    stopped = ops.any(out || ops.raised());
    if (stopped) ops.raise();
    return !stopped;
  }

  // Waits for the copies into the stages filled last (those before them arrived, or their stage would not have been
  // filled again).
  template <class Ops>
  QLIN_RING_FN void drain(Ops& ops) const {
    for (uint32_t i = filled < STAGES ? 0 : filled - STAGES; i < filled; ++i) ops.wait_full(i % STAGES, (i / STAGES) & 1);
  }
};

// Any other role's wait: `ran_out` stays true once a wait ran out, and no further one is made.
template <class Ops, class Wait>
QLIN_RING_FN void wait_or_raise(Ops& ops, bool& ran_out, Wait wait) {
  if (!ran_out && !wait()) {
    ran_out = true;
    ops.raise();
  }
}

}  // namespace ring
}  // namespace qlin
