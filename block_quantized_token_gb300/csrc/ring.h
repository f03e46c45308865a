// A ring whose items two consumers take by turns (items 0, 2, 4, ... and 1, 3, 5, ...).  Each slot has a barrier that completes
// a phase when an item has landed there, and one when its consumer gives the slot back.  Plain C++ on the host too, where
// a test walks it (tests/test_pages_ring_cpu.py).
#pragma once

#ifdef __CUDACC__
#define ER_RING_FN __host__ __device__ __forceinline__
#else
#define ER_RING_FN inline
#endif

namespace er {

// SLOTS is odd, so a slot goes to the consumers by turns.
template <int SLOTS>
struct RingWalk {
    static_assert(SLOTS % 2 == 1 && SLOTS > 1, "by turns");
    int slot, par;  // where the consumer's next item lies, and the parity of that use of the slot
    ER_RING_FN explicit RingWalk(int first) : slot(first), par(0) {}  // first: 0 or 1
    ER_RING_FN void step() {
        slot += 2;
        if (slot >= SLOTS) {
            slot -= SLOTS;
            par ^= 1;
        }
    }
    // Whether the next item has landed; landed(slot, parity) and freed(slot, parity) wait as mbarriers do, for a phase of that
    // parity.  Such a wait cannot tell a phase from the one two before it: `landed` alone passes while the use BEFORE the one
    // meant, the other consumer's, is still on its way (copies land in any order).  Once that use is given back it has landed.  The
    // use two before, this consumer's own, must have been given back by all its warps: they may drift apart by less than
    // three items (three slots are two uses of each).
    template <class Freed, class Landed>
    ER_RING_FN bool ready(Freed freed, Landed landed) const {
        return freed(slot, par ^ 1) && landed(slot, par);
    }
};

}  // namespace er
