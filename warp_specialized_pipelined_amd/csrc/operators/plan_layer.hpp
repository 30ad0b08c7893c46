// plan_layer.hpp -- what the C ABI layers of the operators share: checks of
// descriptions and arguments, the device's query, and the plans alive.
#pragma once

#include <hip/hip_runtime.h>

#include <atomic>
#include <cstring>
#include <mutex>
#include <unordered_map>

#include "../../../include/migemm.h"
#include "../on_device.hpp"
#include "operators.h"

namespace migemm {

constexpr int64_t kMaxSpanBytes = (int64_t)1 << 47;

inline bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// A row-major rows x cols matrix with row stride rs: rs covers the columns
// (INVALID_ARG), starts every row on 16 bytes (MISALIGNED), and the matrix
// stays within 2^47 bytes (UNSUPPORTED), which keeps every later product of
// sizes and strides far from overflow.
inline int check_matrix(int64_t rows, int64_t cols, int64_t rs, int es) {
  if (rs < (cols > 1 ? cols : 1)) return MIGEMM_ERR_INVALID_ARG;
  if (rs % (16 / es) != 0) return MIGEMM_ERR_MISALIGNED;
  if (rows > kMaxSpanBytes || cols > kMaxSpanBytes || rs > kMaxSpanBytes) return MIGEMM_ERR_UNSUPPORTED;
  if ((__int128)rows * rs * es > kMaxSpanBytes) return MIGEMM_ERR_UNSUPPORTED;
  return MIGEMM_OK;
}

// What plans need of a device is found out once (the queries take longer than
// the rest of a plan): its compute units, or a negative status.  `prepare`
// is the operator's kernels' own preparation, done once a device too.
constexpr int kMaxDevices = 64;
inline int query_device(int32_t device) {
  hipDeviceProp_t prop;
  if (hipGetDeviceProperties(&prop, device) != hipSuccess) return MIGEMM_ERR_DEVICE;
  if (std::strncmp(prop.gcnArchName, "gfx950", 6) != 0) return MIGEMM_ERR_DEVICE;
  return prop.multiProcessorCount;
}
template <class Prepare>
int check_device(int32_t device, int* cu_count, std::atomic<bool>* prepared, Prepare&& prepare) {
  static std::atomic<int> found[kMaxDevices];  // 0: not asked yet
  int count = 0;
  if (hipGetDeviceCount(&count) != hipSuccess || count <= 0) return MIGEMM_ERR_DEVICE;
  if (device < 0 || device >= count) return MIGEMM_ERR_DEVICE;
  int cus = device < kMaxDevices ? found[device].load() : 0;
  if (cus == 0) {
    cus = query_device(device);
    if (cus <= 0) return MIGEMM_ERR_DEVICE;
    if (device < kMaxDevices) found[device].store(cus);
  }
  const bool known = device < kMaxDevices;
  if (!known || !prepared[device].load()) {
    if (!prepare_on(device, prepare)) return MIGEMM_ERR_DEVICE;
    if (known) prepared[device].store(true);
  }
  *cu_count = cus;
  return MIGEMM_OK;
}

inline bool current_device_is(int32_t device) {
  int cur = -1;
  return hipGetDevice(&cur) == hipSuccess && cur == device;
}

// The operators' plans alive in this process, by kind, so that a destroyed
// plan or any other pointer is refused unread.  (Never freed, so that plans
// destroyed while the process exits still find it.)
enum PlanKind { kNorm = 1, kScaled, kVocabLoss, kInt8, kQuantize, kBlockNorm, kCheckpoint };
inline std::mutex g_mu;
inline std::unordered_map<const void*, PlanKind>& live() {
  static auto* m = new std::unordered_map<const void*, PlanKind>();
  return *m;
}
inline bool is_live(const void* p, PlanKind kind) try {
  if (!p) return false;
  std::lock_guard<std::mutex> lock(g_mu);
  auto it = live().find(p);
  return it != live().end() && it->second == kind;
} catch (...) {
  return false;
}
template <class Plan>
int add_live(Plan* p, PlanKind kind, Plan** out) {
  try {
    std::lock_guard<std::mutex> lock(g_mu);
    live()[p] = kind;
  } catch (...) {  // no memory for the entry: no exception leaves a C entry point
    delete p;
    return MIGEMM_ERR_INVALID_ARG;
  }
  *out = p;
  return MIGEMM_OK;
}
template <class Plan>
int destroy(Plan* p, PlanKind kind) try {
  if (!p) return MIGEMM_OK;
  {
    std::lock_guard<std::mutex> lock(g_mu);
    auto it = live().find(p);
    if (it == live().end() || it->second != kind) return MIGEMM_ERR_INVALID_ARG;
    live().erase(it);
  }
  delete p;
  return MIGEMM_OK;
} catch (...) {
  return MIGEMM_ERR_INVALID_ARG;
}

inline int launched(hipError_t e) { return e == hipSuccess ? MIGEMM_OK : MIGEMM_ERR_LAUNCH; }

inline int check_workspace(size_t bytes, const void* workspace) {
  if (bytes == 0) return MIGEMM_OK;
  if (!workspace) return MIGEMM_ERR_INVALID_ARG;
  return aligned(workspace, 256) ? MIGEMM_OK : MIGEMM_ERR_MISALIGNED;
}

// The tile_m x 256 tiles of an M x N product and their order, as the GEMM's
// plan lays them out.
inline void set_tiles(KernelArgs& a, int tile_m = kTileM) {
  a.tiles_m = (int32_t)((a.M + tile_m - 1) / tile_m);
  a.tiles_n = (int32_t)((a.N + kTileN - 1) / kTileN);
  a.num_tiles = a.tiles_per_batch = a.tiles_m * a.tiles_n;
  a.group_m = a.tiles_m < 8 ? (a.tiles_m > 0 ? a.tiles_m : 1) : 8;
}

// The kernels reach 256 rows of an operand with 32-bit offsets.
constexpr int64_t kMaxBand = 0x7FFFFFF0 - 1024;
inline bool band_fits(int64_t rs, int es) { return (__int128)256 * rs * es <= kMaxBand; }

// Tile counts are 32-bit.
inline bool tiles_fit(int64_t rows, int64_t cols) {
  const __int128 t = ((__int128)rows / 16 + 1) * ((__int128)cols / 16 + 1);
  return rows / 256 < (1 << 20) && cols / 256 < (1 << 20) && t < 0x7FFFFFFF;
}

inline int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

}  // namespace migemm
