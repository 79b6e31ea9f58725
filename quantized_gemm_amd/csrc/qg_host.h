// What the files that implement the C ABI share: logging, alignment, the device's architecture, launch errors.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <mutex>

#include "qg.h"

namespace qg {

inline bool log_enabled() {
  static int v = -1;
  if (v < 0) {
    const char* e = getenv("QG_LOG");
    v = (e && e[0] == '1') ? 1 : 0;
  }
  return v == 1;
}

#define QG_LOG(...)                         \
  do {                                      \
    if (log_enabled()) {                    \
      fprintf(stderr, "[qg] " __VA_ARGS__); \
      fputc('\n', stderr);                  \
    }                                       \
  } while (0)

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
inline int64_t align256(int64_t x) { return (x + 255) / 256 * 256; }

// Architecture of the current device: 950 for gfx950, 0 if unknown, -1 on error.
inline int current_arch() {
  static std::mutex mu;
  static int cached[64];
  static bool init[64];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) return -1;
  std::lock_guard<std::mutex> lk(mu);
  if (dev < 64 && init[dev]) return cached[dev];
  hipDeviceProp_t prop;
  int arch = -1;
  if (hipGetDeviceProperties(&prop, dev) == hipSuccess) arch = strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 950 : 0;
  if (dev < 64) { cached[dev] = arch; init[dev] = true; }
  return arch;
}

inline qg_status check_arch() {
  const int a = current_arch();
  if (a < 0) return QG_ERR_HIP;
  if (a != 950) return QG_ERR_ARCH_MISMATCH;
  return QG_OK;
}

inline qg_status launched() {
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) {
    QG_LOG("launch failed: %s", hipGetErrorString(e));
    return QG_ERR_HIP;
  }
  return QG_OK;
}

}  // namespace qg
