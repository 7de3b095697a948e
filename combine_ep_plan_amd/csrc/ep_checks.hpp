// Host-side checks shared by the C ABI's translation units: the calling
// thread's last error, the stream's device, and device-buffer checks.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstring>
#include <string>

#include "ep.h"

namespace ep {

inline thread_local std::string g_last_error;

inline int fail(int code, const char* msg) {
  g_last_error = msg;
  return code;
}

inline int fail_hip(hipError_t e, const char* where) {
  g_last_error = std::string(where) + ": " + hipGetErrorString(e);
  return EP_ERR_HIP;
}

// Makes the stream's device current for the lifetime of the object.
class DeviceScope {
 public:
  explicit DeviceScope(hipStream_t s) {
    err_ = hipGetDevice(&prev_);
    if (err_ != hipSuccess) return;
    err_ = hipStreamGetDevice(s, &dev_);
    if (err_ != hipSuccess) return;
    if (dev_ != prev_) err_ = hipSetDevice(dev_);
  }
  ~DeviceScope() {
    if (err_ == hipSuccess && dev_ != prev_) (void)hipSetDevice(prev_);
  }
  hipError_t error() const { return err_; }
  int device() const { return dev_; }

 private:
  int prev_ = -1;
  int dev_ = -1;
  hipError_t err_ = hipSuccess;
};

// A non-empty buffer must be device (or managed) memory of the stream's GPU
// and, where the runtime reports the allocation's range, lie inside it for
// all `bytes`; an empty one (bytes == 0) is never touched and may be
// anything.
inline int check_ptr(const void* p, int dev, const char* name, int64_t bytes) {
  if (bytes == 0) return EP_OK;
  if (!p) return fail(EP_ERR_INVALID_ARG, (std::string("null pointer: ") + name).c_str());
  hipPointerAttribute_t a;
  std::memset(&a, 0, sizeof a);
  const hipError_t e = hipPointerGetAttributes(&a, p);
  if (e != hipSuccess) {
    (void)hipGetLastError();
    return fail(EP_ERR_INVALID_ARG, (std::string("not device memory: ") + name).c_str());
  }
  if (a.type != hipMemoryTypeDevice && a.type != hipMemoryTypeManaged)
    return fail(EP_ERR_INVALID_ARG, (std::string("not device memory: ") + name).c_str());
  if (a.type == hipMemoryTypeDevice && a.device != dev)
    return fail(EP_ERR_DEVICE_MISMATCH,
                (std::string("buffer on another device: ") + name).c_str());
  hipDeviceptr_t base = nullptr;
  size_t size = 0;
  if (hipMemGetAddressRange(&base, &size, (hipDeviceptr_t)p) == hipSuccess && base != nullptr) {
    const uintptr_t end = (uintptr_t)base + size;
    if ((uintptr_t)p < (uintptr_t)base || (uint64_t)bytes > end - (uintptr_t)p)
      return fail(EP_ERR_INVALID_ARG,
                  (std::string("buffer smaller than the call needs: ") + name).c_str());
  } else {
    (void)hipGetLastError();
  }
  return EP_OK;
}

// Row buffers are moved with 16-byte vector accesses: their base must be
// 16-byte aligned (every row then is, row sizes being multiples of 16 or
// moved 4 bytes at a time).
inline int check_aligned16(const void* p, const char* name) {
  if (((uintptr_t)p & 15) != 0)
    return fail(EP_ERR_INVALID_ARG, (std::string("not 16-byte aligned: ") + name).c_str());
  return EP_OK;
}

#define EP_CHECK(expr)            \
  do {                            \
    const int rc_ = (expr);       \
    if (rc_ != EP_OK) return rc_; \
  } while (0)

}  // namespace ep
