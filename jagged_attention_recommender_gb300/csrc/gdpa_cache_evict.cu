// gdpa_cache_evict.cu -- the C ABI of the cache's eviction (gdpa_cache_evict;
// declared in include/gdpa.h): argument checks and launches.  Nothing here
// allocates, synchronises or reads device data.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "gdpa_cache_evict.cuh"
#include "gdpa_cache_host.h"

namespace gdpa {
namespace {

constexpr int kMostCluster = 16;

// `ctas` CTAs a sequence and head, with up to `part` tokens each.
template <int THREADS>
gdpa_status_t launch_choose(const EvictParams& p, int ctas, int64_t part, const Device& dev, cudaStream_t s) {
  static std::mutex mu;
  static bool done[kMaxDevices] = {}, wide[kMaxDevices] = {};
  const gdpa_status_t st = allow_smem(gdpa_cache_choose_kernel<THREADS>, kMostKeys * 4, 0, dev.id, mu, done);
  if (st != GDPA_OK) return st;
  if (ctas > 8) {  // more CTAs a cluster than every device has room for
    std::lock_guard<std::mutex> lock(mu);
    if (!wide[dev.id]) {
      cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;  // (as in allow_smem)
      if (cudaThreadExchangeStreamCaptureMode(&mode) != cudaSuccess) return GDPA_ERR_CUDA;
      const bool ok = cudaFuncSetAttribute(gdpa_cache_choose_kernel<THREADS>,
                                           cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess;
      if (cudaThreadExchangeStreamCaptureMode(&mode) != cudaSuccess || !ok) return GDPA_ERR_CUDA;
      wide[dev.id] = true;
    }
  }
  const int slots = part <= kMostKeys ? static_cast<int>(part) : 0;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = ctas;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>((int64_t)p.B * p.cache.H, 1 << 20) * ctas));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = slots * 4;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, gdpa_cache_choose_kernel<THREADS>, p, slots) == cudaSuccess ? GDPA_OK : GDPA_ERR_CUDA;
}

}  // namespace
}  // namespace gdpa

using namespace gdpa;

extern "C" gdpa_status_t gdpa_cache_evict(const gdpa_cache_t* cache, float* weights, const int32_t* kv_lens,
                                          const int32_t* page_table, int B, int max_pages, int budget, int sink,
                                          int recent, const int32_t* new_table, int new_max_pages, int32_t* kept,
                                          int32_t* new_lens, void* stream) {
  gdpa_status_t st = check_cache(cache);
  if (st != GDPA_OK) return st;
  if ((st = check_batch(cache, 0, B, max_pages)) != GDPA_OK) return st;
  if (budget <= 0 || sink < 0 || recent < 0 || (int64_t)sink + recent > budget || new_max_pages < 0)
    return GDPA_ERR_INVALID_ARG;
  if (B == 0) return GDPA_OK;
  const int64_t most = (int64_t)max_pages * cache->page_tokens, room = (int64_t)new_max_pages * cache->page_tokens;
  if (max_pages == 0 || room < std::min<int64_t>(budget, most)) return GDPA_ERR_INVALID_ARG;
  if (!weights || !aligned(weights, 16) || !words(kv_lens) || !words(page_table) || !words(new_table) || !words(kept) ||
      !words(new_lens))
    return GDPA_ERR_INVALID_ARG;
  const uintptr_t a = reinterpret_cast<uintptr_t>(kv_lens), c = reinterpret_cast<uintptr_t>(new_lens), n = 4 * (uintptr_t)B;
  if (a < c + n && c < a + n) return GDPA_ERR_INVALID_ARG;
  Device dev;
  if ((st = current_device(&dev)) != GDPA_OK) return st;
  EvictParams p;
  p.cache = view(cache);
  p.weights = weights;
  p.kv_lens = kv_lens;
  p.table = page_table;
  p.new_table = new_table;
  p.kept = kept;
  p.new_lens = new_lens;
  p.B = B;
  p.max_pages = max_pages;
  p.new_max_pages = new_max_pages;
  p.budget = budget;
  p.most = static_cast<int>(std::min<int64_t>(budget, most));
  p.sink = sink;
  p.recent = recent;
  p.status = dev.status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t heads = (int64_t)B * cache->H;
  // CTAs of a sequence and head: one, or where those are few as many as fill the SMs with 2048 tokens each.
  int ctas = 1;
  while (ctas < kMostCluster && heads * ctas * 2 <= dev.sms && most / (ctas * 2) >= 2048) ctas *= 2;
  const int64_t part = ((most + ctas - 1) / ctas + 3) & ~(int64_t)3;
  st = part <= 4096 || heads >= 2 * dev.sms ? launch_choose<256>(p, ctas, part, dev, s) : launch_choose<1024>(p, ctas, part, dev, s);
  if (st != GDPA_OK) return st;
  cudaLaunchAttribute attr;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  // Its blocks are placed while the last of the first kernel's CTAs finish, and wait there.
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  constexpr int tokens = kMoveWarps * kMoveTokens;
  cfg.gridDim = dim3(static_cast<unsigned>(((int64_t)p.most + tokens - 1) / tokens), static_cast<unsigned>(std::min<int64_t>(heads, 65535)));
  cfg.blockDim = dim3(32 * kMoveWarps);
  const cudaError_t e = cache->D == 128 ? cudaLaunchKernelEx(&cfg, gdpa_cache_move_kernel<128>, p)
                                        : cudaLaunchKernelEx(&cfg, gdpa_cache_move_kernel<64>, p);
  return e == cudaSuccess ? GDPA_OK : GDPA_ERR_CUDA;
}
