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

// What a device has room for: whether a cluster of `cfg`, larger than every device
// places, fits it.  Asked once for a size of shared memory (a few us), since what fits
// with more fits with less.
template <int THREADS>
gdpa_status_t place_wide(const cudaLaunchConfig_t& cfg, const Device& dev, bool* fits) {
  static std::mutex mu;
  static int64_t most[kMaxDevices] = {}, least[kMaxDevices] = {};  // bytes that fit, that do not: 1 more, 0 unknown
  std::lock_guard<std::mutex> lock(mu);
  const int64_t bytes = static_cast<int64_t>(cfg.dynamicSmemBytes) + 1;
  *fits = bytes <= most[dev.id];
  if (*fits || (least[dev.id] && bytes >= least[dev.id])) return GDPA_OK;
  cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;  // (as in allow_smem)
  if (cudaThreadExchangeStreamCaptureMode(&mode) != cudaSuccess) return GDPA_ERR_CUDA;
  int n = 0;
  const bool ok = cudaFuncSetAttribute(gdpa_cache_choose_kernel<THREADS>, cudaFuncAttributeNonPortableClusterSizeAllowed,
                                       1) == cudaSuccess;
  *fits = ok && cudaOccupancyMaxActiveClusters(&n, gdpa_cache_choose_kernel<THREADS>, &cfg) == cudaSuccess && n > 0;
  if (!*fits) cudaGetLastError();  // (an error of these two says that no such cluster can be placed)
  if (cudaThreadExchangeStreamCaptureMode(&mode) != cudaSuccess) return GDPA_ERR_CUDA;
  (*fits ? most : least)[dev.id] = bytes;
  return GDPA_OK;
}

// `ctas` CTAs a sequence and head, with up to `part` tokens each.  Nothing is
// launched, and *placed is false, where the device has no room for such a cluster.
template <int THREADS>
gdpa_status_t launch_choose(const EvictParams& p, int ctas, int64_t part, const Device& dev, cudaStream_t s, bool* placed) {
  static std::mutex mu;
  static bool done[kMaxDevices] = {};
  *placed = true;
  const gdpa_status_t st = allow_smem(gdpa_cache_choose_kernel<THREADS>, kMostKeys * 4, 0, dev.id, mu, done);
  if (st != GDPA_OK) return st;
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
  if (ctas > kEveryCluster) {
    const gdpa_status_t wide = place_wide<THREADS>(cfg, dev, placed);
    if (wide != GDPA_OK || !*placed) return wide;
  }
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
  bool placed = false;
  for (int widest = kMostCluster; !placed; widest = kEveryCluster) {
    const ChooseShape c = choose_shape(heads, most, dev.sms, widest);
    st = c.threads == 256 ? launch_choose<256>(p, c.ctas, c.part, dev, s, &placed)
                          : launch_choose<1024>(p, c.ctas, c.part, dev, s, &placed);
    if (st != GDPA_OK) return st;
  }
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
