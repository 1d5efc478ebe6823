// gdpa_cache_weights.cu -- the C ABI of the weight that stored keys receive
// (gdpa_cache_weights; declared in include/gdpa.h): argument checks and
// launches.  Nothing here allocates, synchronises or reads device data.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "gdpa_cache_host.h"
#include "gdpa_cache_weights.cuh"
#include "gdpa_cache_weights_tile.cuh"

namespace gdpa {

// gdpa_kernels.cu: a view [rows, H, D] of bf16 rows `stride` elements apart, boxes
// of 64 columns, box_heads heads and box_rows rows with the 128-byte swizzle.
gdpa_status_t encode_heads_3d(CUtensorMap* m, const void* base, int64_t rows, int H, int D, int64_t stride, int box_heads,
                              int box_rows);

namespace {

template <int D, int NT>
gdpa_status_t launch_split(const CacheWeightsParams& p, const Device& dev, cudaStream_t s) {
  using C = WeightCfg<D, NT>;
  static std::mutex mu;
  static bool done[kMaxDevices] = {};
  const gdpa_status_t st = allow_smem(gdpa_cache_weights_split_kernel<D, NT>, C::SMEM, 0, dev.id, mu, done);
  if (st != GDPA_OK) return st;
  const int64_t keys = (int64_t)p.batch.max_pages << p.cache.lp;
  const int64_t work = (int64_t)p.batch.B * p.cache.H * ((keys + C::SPAN - 1) / C::SPAN + C::START);
  const int ctas = static_cast<int>(std::min<int64_t>((work + C::WARPS - 1) / C::WARPS, (int64_t)dev.sms * C::CTAS));
  gdpa_cache_weights_split_kernel<D, NT><<<ctas, C::THREADS, C::SMEM, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? GDPA_OK : GDPA_ERR_CUDA;
}

template <int D>
gdpa_status_t launch_tile(const CacheWeightsParams& w, const Device& dev, cudaStream_t s) {
  using C = WeightTileCfg<D>;
  static std::mutex mu;
  static bool done[kMaxDevices] = {};
  gdpa_status_t st = allow_smem(gdpa_cache_weights_tile_kernel<D>, C::SMEM, 0, dev.id, mu, done);
  if (st != GDPA_OK) return st;
  WeightTileParams p;
  p.w = w;
  p.heads = std::min(w.G, C::COLS);
  p.tokens = C::COLS / p.heads;
  p.parts = (w.G + p.heads - 1) / p.heads;
  p.limit = bounded_wait_ns() * wait_stretch((int64_t)w.batch.T * w.G, w.batch.B);
  if ((st = encode_heads_3d(&p.tm_q, w.q, w.batch.T, w.Hq, D, w.q_stride, p.heads, p.tokens)) != GDPA_OK) return st;
  const int64_t keys = (int64_t)w.batch.max_pages << w.cache.lp, items = (keys + 255) / 256;
  const int ctas = static_cast<int>(std::min<int64_t>((int64_t)w.batch.B * w.cache.H * items, dev.sms));
  gdpa_cache_weights_tile_kernel<D><<<ctas, C::THREADS, C::SMEM, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? GDPA_OK : GDPA_ERR_CUDA;
}

// The kernel for so many rows of a key head.  Measured (us; 48 sequences of 500
// to 6001 keys, 4 key heads, D = 128; 128 sequences of 100 to 6000 keys, 8 key
// heads, D = 64 behind the stroke), with 8, 16, 32, 64 and 128 rows a warp and by
// the kernel for many:
//     8 rows      - / 47     - / 51     - / 52     - / 57     - / 73     - / 253
//    16 rows      -         22 / 58    25 / 59    26 / 63    39 / 80    68 / 253
//    32 rows      -          -         32 / 73    33 / 78    47 / 97    63 / 227
//    64 rows      -          -          -         49 / 113   66 / 144   65 / 226
//    96 rows      -          -          -          -         93 / 193   66 / 226
//   128 rows      -          -          -          -        115 / 239   67 / 226
// Causal rows of D = 64, 128 a warp and the kernel for many: 48 sequences of 500 to
// 6001 keys, 4 heads, 72 rows 42 / 62, 112 rows 55 / 65; 8 of 25 000 to 30 000, 8
// heads, 72 rows 86 / 152, 112 rows 115 / 157.
template <int D>
gdpa_status_t launch_weights(const CacheWeightsParams& p, int max_q, const Device& dev, cudaStream_t s) {
  const int64_t rows = (int64_t)max_q * p.G;
  if (rows <= 8) return launch_split<D, 1>(p, dev, s);
  if (rows <= 16) return launch_split<D, 2>(p, dev, s);
  if (rows <= 32) return launch_split<D, 4>(p, dev, s);
  if (rows <= 64) return launch_split<D, 8>(p, dev, s);
  if constexpr (D == 64)
    if (rows <= 112) return launch_split<D, 16>(p, dev, s);
  return launch_tile<D>(p, dev, s);
}

}  // namespace
}  // namespace gdpa

using namespace gdpa;

extern "C" gdpa_status_t gdpa_cache_weights(const gdpa_cache_t* cache, const void* q, int64_t q_stride,
                                            const float* lse, const int32_t* offsets, const int32_t* kv_lens,
                                            const int32_t* page_table, int64_t T, int B, int Hq, int max_pages,
                                            int max_q, int causal, int window_tokens, float scale, float decay,
                                            const float* weights_in, float* weights, void* stream) {
  gdpa_status_t st = check_cache(cache);
  if (st != GDPA_OK) return st;
  if ((st = check_batch(cache, T, B, max_pages)) != GDPA_OK) return st;
  if (Hq <= 0 || Hq % cache->H || max_q <= 0 || window_tokens < 0 || (causal != 0 && causal != 1) ||
      (window_tokens > 0 && !causal) || !std::isfinite(scale) || !std::isfinite(decay) || decay < 0)
    return GDPA_ERR_INVALID_ARG;
  if ((int64_t)Hq * cache->D > (1 << 20)) return GDPA_ERR_UNSUPPORTED;
  if (T * (Hq / cache->H) >= ((int64_t)1 << 31) - 256) return GDPA_ERR_UNSUPPORTED;  // query rows of a key head
  if (T == 0 || B == 0) return GDPA_OK;
  if ((st = check_rows(q, q_stride, Hq, cache->D)) != GDPA_OK) return st;
  if (!words(lse) || !words(offsets) || !words(kv_lens) || !words(page_table) || max_pages == 0)
    return GDPA_ERR_INVALID_ARG;
  if (!weights || !aligned(weights, 16) || !aligned(weights_in, 16)) return GDPA_ERR_INVALID_ARG;
  if (weights_in && weights_in != weights) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(weights_in), b = reinterpret_cast<uintptr_t>(weights);
    const uintptr_t n = (uintptr_t)cache->num_pages * cache->H * cache->page_tokens * sizeof(float);
    if (a < b + n && b < a + n) return GDPA_ERR_INVALID_ARG;
  }
  Device dev;
  if ((st = current_device(&dev)) != GDPA_OK) return st;
  CacheWeightsParams p;
  p.cache = view(cache);
  p.batch = CacheBatch{offsets, kv_lens, page_table, static_cast<int>(T), B, max_pages, dev.status};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_stride = q_stride;
  p.lse = lse;
  p.w_in = weights_in;
  p.w = weights;
  p.Hq = Hq;
  p.G = Hq / cache->H;
  p.causal = causal;
  p.window = window_tokens;
  p.scale2 = scale * kLog2e;
  p.decay = decay;
  p.keep = weights_in == weights && decay == 1.0f;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return cache->D == 128 ? launch_weights<128>(p, max_q, dev, s) : launch_weights<64>(p, max_q, dev, s);
}
