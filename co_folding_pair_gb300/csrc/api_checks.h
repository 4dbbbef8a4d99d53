// api_checks.h -- what the C ABI's entry points around the layer share: the
// device of a call, and checks of arguments (internal).
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <cstddef>
#include <cstdint>

#include "api_status.h"
#include "trimul.h"

namespace trimul {

// Makes `device` current for a call, and the caller's device again after it.
class DeviceScope {
 public:
  trimul_status enter(int device) {
    TRY_CUDA(cudaGetDevice(&before_), "cudaGetDevice");
    if (before_ == device) return TRIMUL_OK;
    TRY_CUDA(cudaSetDevice(device), "cudaSetDevice");
    changed_ = true;
    return TRIMUL_OK;
  }
  ~DeviceScope() {
    if (changed_) cudaSetDevice(before_);
  }

 private:
  int before_ = 0;
  bool changed_ = false;
};

// Checks the device (compute capability 10.3) and gives its SM count; both are
// asked for once a device.
inline trimul_status device_sms(int device, int* sms) {
  constexpr int kMost = 64;
  static std::atomic<int> known[kMost];
  int ndev = 0;
  if (device >= 0 && device < kMost && (*sms = known[device].load()) > 0) return TRIMUL_OK;
  TRY_CUDA(cudaGetDeviceCount(&ndev), "cudaGetDeviceCount");
  if (device < 0 || device >= ndev) return fail(TRIMUL_ERR_INVALID_ARG, "device %d out of range (%d devices)", device, ndev);
  int major = 0, minor = 0;
  TRY_CUDA(cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, device), "cudaDeviceGetAttribute");
  TRY_CUDA(cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, device), "cudaDeviceGetAttribute");
  if (major != 10 || minor != 3)
    return fail(TRIMUL_ERR_UNSUPPORTED_ARCH, "TriMul kernels are built for sm_103 (GB300); got sm_%d%d", major, minor);
  TRY_CUDA(cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, device), "cudaDeviceGetAttribute");
  if (device < kMost) known[device].store(*sms);
  return TRIMUL_OK;
}

inline bool aligned(const void* p, size_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

inline bool overlap(const void* p, size_t pn, const void* q, size_t qn) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return p && q && a < b + qn && b < a + pn;
}

inline trimul_status check_flags(unsigned flags, unsigned known) {
  if (flags & ~known) return fail(TRIMUL_ERR_INVALID_ARG, "flags 0x%x are not taken by this entry point", flags & ~known);
  return TRIMUL_OK;
}

inline trimul_status check_workspace(const void* ws, size_t have, size_t need, size_t align) {
  if (have < need || !ws) return fail(TRIMUL_ERR_INVALID_ARG, "the workspace holds %zu bytes, %zu are needed", ws ? have : 0, need);
  if (!aligned(ws, align)) return fail(TRIMUL_ERR_INVALID_ARG, "the workspace must be %zu-byte aligned", align);
  return TRIMUL_OK;
}

inline trimul_status finish(cudaError_t launched, cudaStream_t s, unsigned flags, const char* what) {
  TRY_CUDA(launched, what);
  if (flags & TRIMUL_FLAG_CHECK) TRY_CUDA(cudaStreamSynchronize(s), "stream synchronize");
  return TRIMUL_OK;
}

#define TRY(expr)                            \
  do {                                       \
    const trimul_status s_ = (expr);         \
    if (s_ != TRIMUL_OK) return s_;          \
  } while (0)

struct Buffer {
  const void* p;
  size_t bytes;
  const char* name;
};

// Every output apart from every input and from the other outputs; output 0 may be input 0 itself.
inline trimul_status check_apart(const Buffer* in, int n_in, const Buffer* out, int n_out) {
  for (int i = 0; i < n_out; ++i) {
    for (int k = 0; k < n_in; ++k)
      if (overlap(out[i].p, out[i].bytes, in[k].p, in[k].bytes) && !(i == 0 && k == 0 && out[0].p == in[0].p))
        return fail(TRIMUL_ERR_INVALID_ARG, "%s overlaps %s", out[i].name, in[k].name);
    for (int k = 0; k < i; ++k)
      if (overlap(out[i].p, out[i].bytes, out[k].p, out[k].bytes))
        return fail(TRIMUL_ERR_INVALID_ARG, "%s overlaps %s", out[i].name, out[k].name);
  }
  return TRIMUL_OK;
}

inline size_t type_bytes(trimul_dtype t) { return t == TRIMUL_F32 ? 4 : 2; }

}  // namespace trimul
