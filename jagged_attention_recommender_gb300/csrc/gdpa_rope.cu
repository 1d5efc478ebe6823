// gdpa_rope.cu -- the C ABI of the rotary positions (gdpa_rope_freqs,
// gdpa_rope; declared in include/gdpa.h): argument checks and the launch.
// Nothing here allocates, synchronises or reads device data.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "gdpa_cache_host.h"
#include "gdpa_rope.cuh"

using namespace gdpa;

extern "C" gdpa_status_t gdpa_rope_freqs(int rot_dim, double base, int scaling, double factor, int64_t trained,
                                         double fast, double slow, double* inv_freq, float* magnitude) {
  if (!inv_freq || !magnitude || rot_dim <= 0 || !(base > 1) || !std::isfinite(base)) return GDPA_ERR_INVALID_ARG;
  if (rot_dim % 16 || rot_dim > 128) return GDPA_ERR_UNSUPPORTED;
  if (scaling < GDPA_ROPE_SCALE_NONE || scaling > GDPA_ROPE_SCALE_RAMP) return GDPA_ERR_INVALID_ARG;
  if (scaling != GDPA_ROPE_SCALE_NONE && !(factor >= 1 && std::isfinite(factor))) return GDPA_ERR_INVALID_ARG;
  if (scaling == GDPA_ROPE_SCALE_RAMP && !(trained > 0 && slow > 0 && fast > slow && std::isfinite(fast)))
    return GDPA_ERR_INVALID_ARG;
  if (scaling == GDPA_ROPE_SCALE_BASE) base *= std::pow(factor, rot_dim / (rot_dim - 2.0));
  if (!std::isfinite(base)) return GDPA_ERR_UNSUPPORTED;
  *magnitude = 1.0f;
  for (int i = 0; i < rot_dim / 2; ++i) inv_freq[i] = std::pow(base, -2.0 * i / rot_dim);
  if (scaling == GDPA_ROPE_SCALE_LINEAR)
    for (int i = 0; i < rot_dim / 2; ++i) inv_freq[i] /= factor;
  if (scaling == GDPA_ROPE_SCALE_RAMP) {
    const double two_pi = 6.283185307179586;
    auto index = [&](double turns) { return rot_dim * std::log(trained / (two_pi * turns)) / (2 * std::log(base)); };
    const double lo = std::min(std::max(std::floor(index(fast)), 0.0), rot_dim - 1.0);
    const double hi = std::max(std::min(std::ceil(index(slow)), rot_dim - 1.0), 0.0);
    for (int i = 0; i < rot_dim / 2; ++i) {
      const double ramp = std::min(std::max((i - lo) / std::max(hi - lo, 1e-3), 0.0), 1.0);
      inv_freq[i] = inv_freq[i] / factor * ramp + inv_freq[i] * (1 - ramp);
    }
    *magnitude = static_cast<float>(0.1 * std::log(factor) + 1);
  }
  return GDPA_OK;
}

extern "C" gdpa_status_t gdpa_rope(const void* x, int64_t x_stride, const int32_t* offsets, const int32_t* first,
                                   int64_t T, int B, int H, int D, const double* inv_freq, int rot_dim, int rope_style,
                                   float magnitude, int inverse, void* y, int64_t y_stride, void* stream) {
  if (T < 0 || B < 0 || H <= 0 || rot_dim < 0 || rot_dim > D || (inverse != 0 && inverse != 1) ||
      (rope_style != GDPA_ROPE_HALF && rope_style != GDPA_ROPE_INTERLEAVED) || !std::isfinite(magnitude))
    return GDPA_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return GDPA_ERR_UNSUPPORTED;
  if (rot_dim % 16 || (int64_t)H * D > (1 << 20)) return GDPA_ERR_UNSUPPORTED;
  if (T >= ((int64_t)1 << 31) - 256 || B >= INT32_MAX - 4096) return GDPA_ERR_UNSUPPORTED;
  if (rot_dim > 0 && !inv_freq) return GDPA_ERR_INVALID_ARG;
  for (int i = 0; i < rot_dim / 2; ++i)
    if (!std::isfinite(inv_freq[i])) return GDPA_ERR_INVALID_ARG;
  if (T == 0 || B == 0) return GDPA_OK;
  gdpa_status_t st = check_rows(x, x_stride, H, D);
  if (st != GDPA_OK) return st;
  if ((st = check_rows(y, y_stride, H, D)) != GDPA_OK) return st;
  if (x == y && x_stride != y_stride) return GDPA_ERR_INVALID_ARG;
  if (x != y && rows_overlap((static_cast<const char*>(y) - static_cast<const char*>(x)) / 2, x_stride, y_stride, (int64_t)H * D, T))
    return GDPA_ERR_INVALID_ARG;
  if (!words(offsets) || !aligned(first, 4)) return GDPA_ERR_INVALID_ARG;
  Device dev;
  if ((st = current_device(&dev)) != GDPA_OK) return st;
  RopeParams p;
  p.x = static_cast<const __nv_bfloat16*>(x);
  p.y = static_cast<__nv_bfloat16*>(y);
  p.x_stride = x_stride;
  p.y_stride = y_stride;
  p.offsets = offsets;
  p.first = first;
  p.status = dev.status;
  p.T = static_cast<int>(T);
  p.B = B;
  p.H = H;
  p.rot = rot_dim;
  p.interleaved = rope_style == GDPA_ROPE_INTERLEAVED ? 1 : 0;
  p.magnitude = magnitude;
  p.sign = inverse ? -magnitude : magnitude;
  for (int i = 0; i < 64; ++i) p.freq[i] = i < rot_dim / 2 ? turn_fraction(inv_freq[i]) : 0;
  // A lane takes all heads of its row, or, where rows are too few for four CTAs an
  // SM, a part of them, four at least (each part computes the angles again).
  const int rows = kRopeThreads / (D / 16);
  const int64_t blocks = (T + rows - 1) / rows;
  const int parts = static_cast<int>(
      std::max<int64_t>(1, std::min<int64_t>((int64_t)dev.sms * 4 / blocks, (H + 3) / 4)));
  p.heads = (H + parts - 1) / parts;
  const dim3 grid(static_cast<unsigned>(blocks), (H + p.heads - 1) / p.heads);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (D == 128)
    gdpa_rope_kernel<128><<<grid, kRopeThreads, 0, s>>>(p);
  else
    gdpa_rope_kernel<64><<<grid, kRopeThreads, 0, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? GDPA_OK : GDPA_ERR_CUDA;
}
