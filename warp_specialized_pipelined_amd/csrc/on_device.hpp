// on_device.hpp -- kernel attributes belong to the device that is current when
// they are set, and a plan may be made while another one is.
#pragma once

#include <hip/hip_runtime.h>

namespace migemm {

// prepare() with `device` current; the caller's device is current again after it.
template <class Prepare>
bool prepare_on(int device, Prepare&& prepare) {
  int current = -1;
  if (hipGetDevice(&current) != hipSuccess) return false;
  if (current != device && hipSetDevice(device) != hipSuccess) return false;
  const bool done = prepare() == hipSuccess;
  return (current == device || hipSetDevice(current) == hipSuccess) && done;
}

}  // namespace migemm
