// Which copies a loader of the dense attention has issued and may still have on
// their way, so that it can wait for every one of them before its CTA ends. Plain
// bookkeeping, compiled for the host too.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define DSA_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define DSA_HOST_DEVICE inline
#endif

namespace dsa {

template <uint32_t RING>
struct DenseLoads {
  uint32_t mine = 0, phase = 0;    // slots this loader has filled, and the parity of their last use
  bool tail = false;               // copies that signal `tail` are on their way

  // The slot of entry e: true once released(slot, use) says that use `use`, the one
  // before, has been read. Else nothing may be issued, and the slot's books
  // stay those of the copy that may still be on its way.
  template <class Released>
  DSA_HOST_DEVICE bool claim(uint32_t e, uint32_t& slot, Released released) {
    slot = e % RING;
    const uint32_t use = e / RING;
    if (use > 0 && !released(slot, use - 1)) return false;
    mine |= 1u << slot;
    phase = (phase & ~(1u << slot)) | ((use & 1) << slot);
    return true;
  }
  // The copy into `slot` signals `tail`; the slot's own barrier completes this use
  // only when the loader itself arrives there, and its uses before have been read.
  DSA_HOST_DEVICE void by_tail(uint32_t slot) {
    mine &= ~(1u << slot);
    tail = true;
  }
  DSA_HOST_DEVICE void tail_landed() { tail = false; }
  // Waits by wait(slot, parity) for every slot with a copy of this loader, and by
  // wait_tail() for copies that signal `tail`.
  template <class Wait, class WaitTail>
  DSA_HOST_DEVICE void drain(Wait wait, WaitTail wait_tail) const {
    for (uint32_t s = 0; s < RING; ++s)
      if ((mine >> s) & 1u) wait(s, (phase >> s) & 1u);
    if (tail) wait_tail();
  }
};

}  // namespace dsa
