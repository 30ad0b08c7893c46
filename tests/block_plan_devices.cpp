// block_plan_devices.cpp -- plans of the int8 product, the block norm and the
// checkpoint (csrc/operators/block_api.cpp) for a device that is not the current
// one, on a machine of two devices that exists only here: the HIP calls that a
// plan's creation makes, and the kernels' preparation, are the ones below.  Each
// preparation sets attributes of the current device's kernels, so it must find
// the plan's device current, and leave the caller's current device as it was.
// Prints what went wrong.
#include <hip/hip_runtime.h>

#include <cstdio>
#include <cstring>
#include <vector>

#include "../include/migemm.h"
#include "../warp_specialized_pipelined_amd/csrc/operators/operators.h"

static int g_current = 0;
static bool g_refuse = false;  // hipSetDevice
static std::vector<int> g_prepared;
static hipError_t prepare() {
  g_prepared.push_back(g_current);
  return hipSuccess;
}

extern "C" {
hipError_t hipGetDeviceCount(int* n) { return *n = 2, hipSuccess; }
hipError_t hipGetDevice(int* d) { return *d = g_current, hipSuccess; }
hipError_t hipSetDevice(int d) {
  if (g_refuse) return hipErrorInvalidDevice;
  return g_current = d, hipSuccess;
}
hipError_t hipGetDevicePropertiesR0600(hipDeviceProp_tR0600* p, int) {
  std::memset(p, 0, sizeof(*p));
  std::strcpy(p->gcnArchName, "gfx950:sramecc+:xnack-");
  p->multiProcessorCount = 256;
  return hipSuccess;
}
}

namespace migemm {
hipError_t prepare_int8() { return prepare(); }
hipError_t prepare_block_norm() { return prepare(); }
hipError_t prepare_checkpoint() { return prepare(); }
ScaledChoice choose_int8(int64_t, int64_t, int64_t, int) { return {0, 1, 256, 0}; }
CheckpointChoice choose_checkpoint(int64_t, int64_t, int64_t, int, int) { return {0, 1, 0}; }
int64_t block_norm_partial_rows(int64_t, int64_t, int) { return 1; }
}  // namespace migemm

static int g_bad = 0;
static void check(bool ok, const char* what, int device) {
  if (!ok) std::printf("%s (device %d)\n", what, device), ++g_bad;
}

// Plans for `device` while the other is current: a first and a second one,
// where the first has to prepare the device and the second may.
template <class Create>
static void plans(const char* name, Create&& create) {
  for (int device : {1, 0}) {
    g_current = 1 - device;
    g_prepared.clear();
    g_refuse = true;
    check(create(device) == MIGEMM_ERR_DEVICE, name, device);
    g_refuse = false;
    check(g_prepared.empty() && g_current == 1 - device, name, device);
    check(create(device) == MIGEMM_OK, name, device);
    check(!g_prepared.empty(), name, device);
    check(create(device) == MIGEMM_OK, name, device);
    for (int d : g_prepared) check(d == device, name, device);
    check(g_current == 1 - device, name, device);
  }
}

int main() {
  plans("int8", [](int device) {
    const migemm_int8_desc d = {64, 64, 512, 512, 512, 64, device, 0};
    migemm_int8_plan* p;
    return gemm_int8_plan_create(&d, &p);
  });
  plans("block_norm", [](int device) {
    migemm_block_norm_desc d = {64, 64, 64, 64, 64, 64, 0, 64, 64, 64, 0, 0, 1e-5f, 1.0f, 1.0f, 1, MIGEMM_BF16, device};
    migemm_block_norm_plan* p;
    return gemm_block_norm_plan_create(&d, &p);
  });
  plans("checkpoint", [](int device) {
    const migemm_checkpoint_desc d = {64, 64, 64, 64, 64, 64, MIGEMM_BF16, 0, device, 0};
    migemm_checkpoint_plan* p;
    return gemm_checkpoint_plan_create(&d, &p);
  });
  // A plan of a device that is not current runs nothing.
  g_current = 0;
  const migemm_quantize_desc d = {4, 64, 64, 64, MIGEMM_INT8, 1, 0};
  migemm_quantize_plan* p = nullptr;
  check(gemm_quantize_plan_create(&d, &p) == MIGEMM_OK, "quantize", 1);
  alignas(16) static unsigned char m[1024];
  check(gemm_quantize_run(p, m, m, reinterpret_cast<float*>(m), nullptr) == MIGEMM_ERR_DEVICE, "quantize", 1);
  check(gemm_quantize_plan_destroy(p) == MIGEMM_OK, "quantize", 1);
  if (!g_bad) std::printf("block_plan_devices: OK\n");
  return g_bad != 0;
}
