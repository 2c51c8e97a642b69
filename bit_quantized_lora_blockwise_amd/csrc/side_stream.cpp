#include "side_stream.h"

namespace qlabi {

constexpr int kMaxDevices = 64;

SideStream* side_stream() {
  thread_local SideStream per_dev[kMaxDevices];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
  SideStream& d = per_dev[dev];
  if (d.failed) return nullptr;
  if (!d.s) {
    int cus = 0;
    if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cus < 8 ||
        hipEventCreateWithFlags(&d.fork, hipEventDisableTiming) != hipSuccess ||
        hipEventCreateWithFlags(&d.join, hipEventDisableTiming) != hipSuccess ||
        hipStreamCreateWithFlags(&d.s, hipStreamNonBlocking) != hipSuccess) {
      d.failed = true;
      d.s = nullptr;
      return nullptr;
    }
    d.cus = cus;
  }
  return &d;
}

hipError_t join_side(SideStream& d, hipStream_t s, hipError_t e) {
  hipError_t j = hipEventRecord(d.join, d.s);
  if (j == hipSuccess) j = hipStreamWaitEvent(s, d.join, 0);
  return e != hipSuccess ? e : j;
}

}  // namespace qlabi
