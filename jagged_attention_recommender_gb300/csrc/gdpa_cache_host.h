// gdpa_cache_host.h -- what the host sides of the cache's and the rotation's
// entry points share: argument checks, the current device, a kernel's settings.
#pragma once

#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <mutex>

#include "gdpa_cache.cuh"
#include "gdpa_internal.h"

namespace gdpa {

// gdpa_kernels.cu
int* device_status_word(int device);
unsigned long long bounded_wait_ns();

constexpr int kMaxDevices = 64;

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Whether an array of 32-bit words can be there: not null, and aligned.
inline bool words(const void* p) { return p && aligned(p, 4); }

struct Device {
  int id = 0, sms = 0;
  int* status = nullptr;
};

// The current device, its SM count and status word.  The first call on a
// device may load the module there, which a strictly captured thread must be
// allowed to do.
inline gdpa_status_t current_device(Device* d) {
  if (cudaGetDevice(&d->id) != cudaSuccess) return GDPA_ERR_CUDA;
  if (d->id < 0 || d->id >= kMaxDevices) return GDPA_ERR_UNSUPPORTED;
  cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
  if (cudaThreadExchangeStreamCaptureMode(&mode) != cudaSuccess) return GDPA_ERR_CUDA;
  d->status = device_status_word(d->id);
  const bool ok = cudaDeviceGetAttribute(&d->sms, cudaDevAttrMultiProcessorCount, d->id) == cudaSuccess && d->sms > 0;
  if (cudaThreadExchangeStreamCaptureMode(&mode) != cudaSuccess || !ok || !d->status) return GDPA_ERR_CUDA;
  return GDPA_OK;
}

inline gdpa_status_t check_cache(const gdpa_cache_t* c) {
  if (!c) return GDPA_ERR_INVALID_ARG;
  if (c->num_pages < 0 || c->H <= 0 || c->page_tokens <= 0 || c->rot_dim < 0) return GDPA_ERR_INVALID_ARG;
  if (c->rope_style != GDPA_ROPE_HALF && c->rope_style != GDPA_ROPE_INTERLEAVED) return GDPA_ERR_INVALID_ARG;
  if (c->D != 64 && c->D != 128) return GDPA_ERR_UNSUPPORTED;
  if (c->page_tokens < kCacheBlock || c->page_tokens > 1024 || (c->page_tokens & (c->page_tokens - 1)))
    return GDPA_ERR_UNSUPPORTED;
  if ((int64_t)c->H * c->D > (1 << 20)) return GDPA_ERR_UNSUPPORTED;
  if (c->rot_dim > c->D) return GDPA_ERR_INVALID_ARG;
  if (c->rot_dim % 16) return GDPA_ERR_UNSUPPORTED;
  if (c->rot_dim > 0) {
    if (!c->inv_freq) return GDPA_ERR_INVALID_ARG;
    for (int i = 0; i < c->rot_dim / 2; ++i)
      if (!std::isfinite(c->inv_freq[i])) return GDPA_ERR_INVALID_ARG;
  }
  if (c->num_pages > 0 && (!c->k_codes || !c->v_codes || !c->k_sf || !c->v_sf || !aligned(c->k_codes, 16) ||
                           !aligned(c->v_codes, 16) || !aligned(c->k_sf, 4) || !aligned(c->v_sf, 4)))
    return GDPA_ERR_INVALID_ARG;
  return GDPA_OK;
}

// Rows of H heads of D at a stride: both in elements.
inline gdpa_status_t check_rows(const void* p, int64_t stride, int64_t H, int64_t D) {
  if (!p || !aligned(p, 16) || stride < H * D) return GDPA_ERR_INVALID_ARG;
  return stride % 8 ? GDPA_ERR_UNSUPPORTED : GDPA_OK;
}

inline gdpa_status_t check_batch(const gdpa_cache_t* c, int64_t T, int B, int max_pages) {
  if (T < 0 || B < 0 || max_pages < 0) return GDPA_ERR_INVALID_ARG;
  // Rows and sequences are counted in 32 bits, up to a warp's or a block's stretch past the last one.
  if (T >= ((int64_t)1 << 31) - 256 || B >= INT32_MAX - 4096) return GDPA_ERR_UNSUPPORTED;
  if ((int64_t)max_pages * c->page_tokens >= (int64_t)1 << 31) return GDPA_ERR_UNSUPPORTED;
  return GDPA_OK;
}

inline CacheView view(const gdpa_cache_t* c) {
  int lp = 0;
  while ((1 << lp) < c->page_tokens) ++lp;
  return CacheView{static_cast<uint8_t*>(c->k_codes), static_cast<uint8_t*>(c->v_codes),
                   static_cast<uint8_t*>(c->k_sf),    static_cast<uint8_t*>(c->v_sf),
                   c->num_pages,                      lp,
                   c->H};
}

// Shared memory above 48 KB has to be asked for, once a device and kernel.
// `min_regs`: a kernel that trades registers between its warpgroups needs that
// many at launch, or its increase would wait for ever; such a build is refused.
template <typename Kernel>
gdpa_status_t allow_smem(Kernel kernel, int bytes, int min_regs, int device, std::mutex& mu, bool* done) {
  std::lock_guard<std::mutex> lock(mu);
  if (done[device]) return GDPA_OK;
  // (as in current_device: the first call may load the kernel while a stream is captured)
  cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
  if (cudaThreadExchangeStreamCaptureMode(&mode) != cudaSuccess) return GDPA_ERR_CUDA;
  cudaFuncAttributes fa;
  gdpa_status_t st = GDPA_OK;
  if (cudaFuncGetAttributes(&fa, kernel) != cudaSuccess)
    st = GDPA_ERR_CUDA;
  else if (fa.numRegs < min_regs)
    st = GDPA_ERR_UNSUPPORTED;
  else if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
    st = GDPA_ERR_CUDA;
  if (cudaThreadExchangeStreamCaptureMode(&mode) != cudaSuccess) st = GDPA_ERR_CUDA;
  done[device] = st == GDPA_OK;
  return st;
}

}  // namespace gdpa
