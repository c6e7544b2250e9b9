/*
 * mk_device.h -- what the handles of mk_append.cu and mk_rules.cu have in common: the device a
 * call runs on, and the first device error on its way to the host.
 */
#ifndef MK_DEVICE_H
#define MK_DEVICE_H

#include <cuda_runtime.h>

#include <cstdint>

#include "mk.h"

namespace mk_dev {

/* Makes `dev` current for a scope: a handle may be called with another device current. */
struct OnDevice {
  int was = 0;
  bool ok = true, changed = false;
  explicit OnDevice(int dev) {
    ok = cudaGetDevice(&was) == cudaSuccess;
    if (ok && was != dev) {
      ok = cudaSetDevice(dev) == cudaSuccess;
      changed = ok;
    }
  }
  ~OnDevice() {
    if (changed) cudaSetDevice(was);
  }
};

inline bool aligned(const void *p, unsigned n) { return ((uintptr_t)p & (n - 1)) == 0; }

/* Whether rows of wa bytes, sa apart, and rows of wb bytes, sb apart, n of each, share a byte.
 * With the same distance they may lie between one another; else their spans must not meet. */
inline bool rows_meet(const void *a, int64_t sa, int64_t wa, const void *b, int64_t sb, int64_t wb,
                      int64_t n) {
  const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
  if (a0 + (uint64_t)((n - 1) * sa + wa) <= b0 || b0 + (uint64_t)((n - 1) * sb + wb) <= a0) return false;
  if (n > 1 && sa != sb) return true;
  if (n == 1) return true;
  const int64_t ahead = (int64_t)(b0 - a0) % sa, d = ahead < 0 ? ahead + sa : ahead; /* b's row behind a's */
  return d < wa || d + wb > sa;
}

/* A device error: the first since the last sync is kept on the device and told to the host. */
struct Errors {
  int32_t *first; /* DEVICE */
  int32_t *host;  /* mapped */
};
#ifdef __CUDACC__
__device__ __forceinline__ void report(const Errors &e, int code) {
  if (atomicCAS(e.first, 0, code) == 0) *(volatile int32_t *)e.host = code;
}
#endif

/* Waits for the stream; the first error since the last call, which is cleared. */
inline mk_status take_error(int dev, cudaStream_t stream, const Errors &e, int32_t *host) {
  OnDevice on(dev);
  if (!on.ok) return MK_ERR_CUDA;
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(stream, &cap) != cudaSuccess) return MK_ERR_CUDA;
  if (cap != cudaStreamCaptureStatusNone) return MK_ERR_INVALID_ARG;
  if (cudaStreamSynchronize(stream) != cudaSuccess) return MK_ERR_CUDA;
  const int32_t code = *(volatile int32_t *)host;
  if (code == 0) return MK_OK;
  *(volatile int32_t *)host = 0;
  if (cudaMemsetAsync(e.first, 0, sizeof(int32_t), stream) != cudaSuccess) return MK_ERR_CUDA;
  return code;
}

/* The device that new handles are made for; false where it is no sm_103. */
inline bool this_device(int *dev, int *n_sm) {
  cudaDeviceProp prop;
  if (cudaGetDevice(dev) != cudaSuccess || cudaGetDeviceProperties(&prop, *dev) != cudaSuccess) return false;
  *n_sm = prop.multiProcessorCount;
  return prop.major == 10 && prop.minor == 3;
}

}  // namespace mk_dev

#endif /* MK_DEVICE_H */
