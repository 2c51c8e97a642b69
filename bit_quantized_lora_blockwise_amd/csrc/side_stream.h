// A second stream for work that fills CUs which a persistent product leaves idle in its
// last round (the adapter's gradients beside the dX product).
#pragma once

#include <hip/hip_runtime.h>

namespace qlabi {

struct SideStream {
  hipStream_t s = nullptr;
  hipEvent_t fork = nullptr, join = nullptr;
  int cus = 0;
  bool failed = false;
};

// The calling thread's second stream on the current device (default priority,
// created on first use and kept until the process ends), or nullptr when it
// cannot be had; the caller then keeps everything on its own stream.
SideStream* side_stream();

// Joins the second stream back into the caller's stream s, also after a failed
// launch `e` on it, so that what was enqueued there stays ordered before s's
// later work; returns the first error.
hipError_t join_side(SideStream& d, hipStream_t s, hipError_t e);

}  // namespace qlabi
