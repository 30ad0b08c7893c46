// plan_devices.cpp -- the plan layers (csrc/api.cpp and
// csrc/operators/operators_api.cpp) on a machine of two devices that exists
// only here: the HIP calls that a plan's creation makes, and the kernels'
// preparation, are the ones below.  Each preparation sets attributes of the
// current device's kernels, so it must find the plan's device current, and
// leave the caller's current device as it was.  Prints what went wrong.
#include <hip/hip_runtime.h>

#include <cstdio>
#include <cstring>
#include <vector>

#include "../include/migemm.h"
#include "../warp_specialized_pipelined_amd/csrc/launch.h"
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
  p->sharedMemPerBlock = 160 * 1024;
  return hipSuccess;
}
}

namespace migemm {
hipError_t prepare_kernel(const KernelSelect&) { return prepare(); }
int kernel_lds_bytes(const KernelSelect&) { return 0; }
hipError_t prepare_scaled() { return prepare(); }
hipError_t prepare_loss() { return prepare(); }
ScaledChoice choose_scaled(int64_t, int64_t, int64_t, int) { return {0, 1, 256, 0}; }
LossChoice choose_loss(int64_t, int64_t, int64_t, int64_t, int) { return {0, 0, 0, 0, 1, 1}; }
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
  plans("scaled", [](int device) {
    const migemm_scaled_desc d = {64, 64, 512, 512, 512, 64, device, 0};
    migemm_scaled_plan* p;
    return gemm_scaled_plan_create(&d, &p);
  });
  plans("vocab_loss", [](int device) {
    const migemm_vocab_loss_desc d = {64, 640, 64, 64, 64, 64, 64, device, 0};
    migemm_vocab_loss_plan* p;
    return gemm_vocab_loss_plan_create(&d, &p);
  });
  plans("gemm", [](int device) {
    migemm_desc d = {};
    d.M = d.N = d.K = 512;
    d.a_type = d.b_type = d.c_type = d.d_type = MIGEMM_BF16;
    d.a_rs = d.b_rs = d.c_rs = d.d_rs = 512;
    d.a_cs = d.b_cs = d.c_cs = d.d_cs = 1;
    d.L = 1;
    d.device = device;
    migemm_plan* p;
    return gemm_plan_create(&d, &p);
  });
  if (!g_bad) std::printf("plan_devices: OK\n");
  return g_bad != 0;
}
