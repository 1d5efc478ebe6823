// gdpa_cache.cu -- the C ABI of the paged key/value cache (gdpa_cache_append,
// gdpa_cache_fwd; declared in include/gdpa.h): argument checks and launches.
// Nothing here allocates, synchronises or reads device data.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "gdpa_cache_append.cuh"
#include "gdpa_cache_fwd.cuh"
#include "gdpa_cache_tile.cuh"
#include "gdpa_internal.h"

namespace gdpa {

// gdpa_kernels.cu
int* device_status_word(int device);
unsigned long long bounded_wait_ns();

namespace {

constexpr int kMaxDevices = 64;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

struct Device {
  int id = 0, sms = 0;
  int* status = nullptr;
};

// The current device, its SM count and status word.  The first call on a
// device may load the module there, which a strictly captured thread must be
// allowed to do.
gdpa_status_t current_device(Device* d) {
  if (cudaGetDevice(&d->id) != cudaSuccess) return GDPA_ERR_CUDA;
  if (d->id < 0 || d->id >= kMaxDevices) return GDPA_ERR_UNSUPPORTED;
  cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
  if (cudaThreadExchangeStreamCaptureMode(&mode) != cudaSuccess) return GDPA_ERR_CUDA;
  d->status = device_status_word(d->id);
  const bool ok = cudaDeviceGetAttribute(&d->sms, cudaDevAttrMultiProcessorCount, d->id) == cudaSuccess && d->sms > 0;
  if (cudaThreadExchangeStreamCaptureMode(&mode) != cudaSuccess || !ok || !d->status) return GDPA_ERR_CUDA;
  return GDPA_OK;
}

gdpa_status_t check_cache(const gdpa_cache_t* c) {
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
gdpa_status_t check_rows(const void* p, int64_t stride, int64_t H, int64_t D) {
  if (!p || !aligned(p, 16) || stride < H * D) return GDPA_ERR_INVALID_ARG;
  return stride % 8 ? GDPA_ERR_UNSUPPORTED : GDPA_OK;
}

gdpa_status_t check_batch(const gdpa_cache_t* c, int64_t T, int B, int max_pages) {
  if (T < 0 || B < 0 || max_pages < 0) return GDPA_ERR_INVALID_ARG;
  // Rows and sequences are counted in 32 bits, up to a warp's or a block's stretch past the last one.
  if (T >= ((int64_t)1 << 31) - 256 || B >= INT32_MAX - 4096) return GDPA_ERR_UNSUPPORTED;
  if ((int64_t)max_pages * c->page_tokens >= (int64_t)1 << 31) return GDPA_ERR_UNSUPPORTED;
  return GDPA_OK;
}

CacheView view(const gdpa_cache_t* c) {
  int lp = 0;
  while ((1 << lp) < c->page_tokens) ++lp;
  return CacheView{static_cast<uint8_t*>(c->k_codes), static_cast<uint8_t*>(c->v_codes),
                   static_cast<uint8_t*>(c->k_sf),    static_cast<uint8_t*>(c->v_sf),
                   c->num_pages,                      lp,
                   c->H};
}

// Keys a segment can have, as far as the host knows.
int64_t most_keys(const CacheFwdParams& p, int max_q) {
  const int64_t keys = (int64_t)p.batch.max_pages << p.cache.lp;
  return p.window > 0 ? std::min<int64_t>(keys, (int64_t)p.window + max_q + kCacheBlock) : keys;
}

// Segments of so many rows, at most.
int64_t most_segments(const CacheFwdParams& p, int rows) {
  return ((int64_t)p.batch.T * p.G / rows + p.batch.B) * p.cache.H;
}

// The kernel for so many query rows of a key head: eights of rows in a tile of
// the one for few rows, or 0: the one for many.  Measured (us, 48 sequences of
// 500 to 6001 keys, 4 key heads, D = 128; D = 64 behind the stroke), in tiles
// of 16, 24, 32 rows and by the kernel for many:
//   24 rows  76 / 56   62 / 50   84 / 54   102 / 66
//   32 rows  78 / 57   92 / 69   87 / 58   101 / 66
//   48 rows 107 / 72   93 / 70  134 / 79   105 / 72
//   64 rows 135 / 90  127 / 95  136 / 80   107 / 72
// for 96 sequences of up to 1500 keys, in tiles of 16 and by the kernel for many,
//   64 rows  89 / 60   100 / 68       96 rows  123 / 82   103 / 70
// and of up to 700
//   96 rows  72 / 51    75 / 55      128 rows   91 / 62    76 / 55
// Tiles of 32 rows at D = 128 do not fit the registers; at D = 64 they take 172
// us for 32 candidates of 128 samples, where two of 16 take 202.
template <int D>
int split_columns(int64_t rows, int64_t keys) {
  if (rows <= 24) return rows <= 8 ? 1 : rows <= 16 ? 2 : 3;
  if (rows <= 32) return D == 64 ? 4 : 2;
  if (rows <= 48) return 3;
  return rows <= 96 && (rows + 15) / 16 * keys <= 6144 ? 2 : 0;
}

// Bytes of meta data and parts for so many workers.
int64_t part_bytes(int64_t workers, int rows, int D) {
  return workers * 2 * (8 * sizeof(int) + (int64_t)rows * (D + 2) * sizeof(float));
}

template <class C>
int64_t workspace_of(const Device& dev, int D) {
  return part_bytes((int64_t)dev.sms * C::CTAS * C::WORKERS, C::ROWS, D);
}

// ... whatever the number of keys
template <int D>
int64_t workspace_bytes(const Device& dev, int max_q, int G) {
  const int64_t rows = (int64_t)max_q * G;
  if (rows <= 8) return workspace_of<SplitCfg<D, 1>>(dev, D);
  int64_t most = std::max(workspace_of<SplitCfg<D, 2>>(dev, D), workspace_of<SplitCfg<D, 3>>(dev, D));
  if (D == 64) most = std::max(most, workspace_of<SplitCfg<64, 4>>(dev, D));
  return rows <= 48 ? most : std::max(most, workspace_of<TileCfg<D>>(dev, D));
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

template <int D>
gdpa_status_t launch_append(const AppendParams& p, int64_t groups, int share, int rows, int smem, const Device& dev,
                            cudaStream_t s) {
  static std::mutex mu;
  static bool done[kMaxDevices] = {};
  constexpr int most = (2 * kCacheBlock - 1) * (D / 2) * (int)sizeof(float2) + kAppendThreads / 32 * 4096;
  const gdpa_status_t st = allow_smem(gdpa_cache_append_kernel<D>, most, 0, dev.id, mu, done);
  if (st != GDPA_OK) return st;
  gdpa_cache_append_kernel<D><<<dim3(static_cast<unsigned>(groups), share), kAppendThreads, smem, s>>>(p, rows);
  return cudaGetLastError() == cudaSuccess ? GDPA_OK : GDPA_ERR_CUDA;
}

// Sets up a launch of configuration C: whether segments may be cut, the
// workspace, and how many CTAs have work at most.
template <class C>
int prepare_launch(CacheFwdParams& p, void* workspace, int max_q, const Device& dev) {
  const int64_t keys = most_keys(p, max_q), segments = most_segments(p, C::ROWS);
  // Whole segments need no second kernel (about 5 us): so few keys that one
  // worker is done with them before that had begun, or enough segments for all
  // workers (a warp takes 0.7 us for 32 keys).
  p.no_split = C::TEAM || keys <= 128 || (keys <= 512 && segments >= 2 * (int64_t)dev.sms * C::CTAS * C::WORKERS);
  const int64_t workers = p.no_split ? segments : segments * ((keys / C::SPAN + 1 + C::START) / C::RUN_STEPS + 1);
  const int ctas = static_cast<int>(
      std::min<int64_t>((workers + C::WORKERS - 1) / C::WORKERS, (int64_t)dev.sms * C::CTAS));
  p.meta = static_cast<int*>(workspace);
  p.part = reinterpret_cast<float*>(p.meta + (int64_t)ctas * C::WORKERS * 16);
  return ctas;
}

// The second kernel.  Its blocks are placed while the last of the first
// kernel's CTAs finish, and wait there.
template <int D, class C>
gdpa_status_t launch_join(const CacheFwdParams& p, int ctas, cudaStream_t s) {
  if (cudaGetLastError() != cudaSuccess) return GDPA_ERR_CUDA;
  if (p.no_split) return GDPA_OK;
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, std::max(1, C::ROWS * C::WORKERS / 32));
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.stream = s;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, gdpa_cache_join_kernel<D, C::ROWS, C::WORKERS>, p) == cudaSuccess ? GDPA_OK
                                                                                                    : GDPA_ERR_CUDA;
}

template <int D, int NT, bool TEAM>
gdpa_status_t launch_split_as(CacheFwdParams& p, void* workspace, int max_q, const Device& dev, cudaStream_t s) {
  using C = SplitCfg<D, NT, TEAM>;
  static std::mutex mu;
  static bool done[kMaxDevices] = {};
  const gdpa_status_t st = allow_smem(gdpa_cache_split_kernel<D, NT, TEAM>, C::SMEM, 0, dev.id, mu, done);
  if (st != GDPA_OK) return st;
  const int ctas = prepare_launch<C>(p, workspace, max_q, dev);
  gdpa_cache_split_kernel<D, NT, TEAM><<<ctas, C::THREADS, C::SMEM, s>>>(p);
  if constexpr (TEAM)
    return cudaGetLastError() == cudaSuccess ? GDPA_OK : GDPA_ERR_CUDA;
  else
    return launch_join<D, C>(p, ctas, s);
}

// A second kernel costs a call about 5 us: up to 2048 keys the eight warps of a
// CTA are done with a whole segment sooner, if every segment has an SM (one token
// over 201 keys, 50 calls in a graph: 6.3 us a call, cut into parts 13.7).
template <int D, int NT>
gdpa_status_t launch_split(CacheFwdParams& p, void* workspace, int max_q, const Device& dev, cudaStream_t s) {
  const bool team = most_keys(p, max_q) <= 2048 && most_segments(p, 8 * NT) <= dev.sms;
  return team ? launch_split_as<D, NT, true>(p, workspace, max_q, dev, s)
              : launch_split_as<D, NT, false>(p, workspace, max_q, dev, s);
}

template <int D>
gdpa_status_t launch_tile(CacheFwdParams& p, void* workspace, int max_q, const Device& dev, cudaStream_t s) {
  using C = TileCfg<D>;
  static std::mutex mu;
  static bool done[kMaxDevices] = {};
  const gdpa_status_t st = allow_smem(gdpa_cache_tile_kernel<D>, C::SMEM, C::LAUNCH_REGS, dev.id, mu, done);
  if (st != GDPA_OK) return st;
  const int ctas = prepare_launch<C>(p, workspace, max_q, dev);
  gdpa_cache_tile_kernel<D><<<ctas, C::THREADS, C::SMEM, s>>>(p, bounded_wait_ns());
  return launch_join<D, C>(p, ctas, s);
}

template <int D>
gdpa_status_t launch_fwd(CacheFwdParams& p, void* workspace, int max_q, const Device& dev, cudaStream_t s) {
  switch (split_columns<D>((int64_t)max_q * p.G, most_keys(p, max_q))) {
    case 1: return launch_split<D, 1>(p, workspace, max_q, dev, s);
    case 2: return launch_split<D, 2>(p, workspace, max_q, dev, s);
    case 3: return launch_split<D, 3>(p, workspace, max_q, dev, s);
    case 4:
      if constexpr (D == 64) return launch_split<D, 4>(p, workspace, max_q, dev, s);
      return GDPA_ERR_UNSUPPORTED;
    default: return launch_tile<D>(p, workspace, max_q, dev, s);
  }
}

}  // namespace
}  // namespace gdpa

using namespace gdpa;

extern "C" gdpa_status_t gdpa_cache_append(const gdpa_cache_t* cache, const void* q, int64_t q_stride, const void* k,
                                           int64_t k_stride, const void* v, int64_t v_stride, const int32_t* offsets,
                                           const int32_t* kv_lens, const int32_t* page_table, int64_t T, int B,
                                           int Hq, int max_pages, void* q_out, void* stream) {
  gdpa_status_t st = check_cache(cache);
  if (st != GDPA_OK) return st;
  if ((st = check_batch(cache, T, B, max_pages)) != GDPA_OK) return st;
  if (q && Hq <= 0) return GDPA_ERR_INVALID_ARG;
  if (q && (int64_t)Hq * cache->D > (1 << 20)) return GDPA_ERR_UNSUPPORTED;
  if (T == 0 || B == 0) return GDPA_OK;
  if ((st = check_rows(k, k_stride, cache->H, cache->D)) != GDPA_OK) return st;
  if ((st = check_rows(v, v_stride, cache->H, cache->D)) != GDPA_OK) return st;
  if (q) {
    if ((st = check_rows(q, q_stride, Hq, cache->D)) != GDPA_OK) return st;
    if ((st = check_rows(q_out, (int64_t)Hq * cache->D, Hq, cache->D)) != GDPA_OK) return st;
  }
  if (!offsets || !kv_lens || !page_table || max_pages == 0) return GDPA_ERR_INVALID_ARG;
  Device dev;
  if ((st = current_device(&dev)) != GDPA_OK) return st;
  AppendParams p;
  p.cache = view(cache);
  p.batch = CacheBatch{offsets, kv_lens, page_table, static_cast<int>(T), B, max_pages, dev.status};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.Hq = q ? Hq : 0;
  p.rot = cache->rot_dim;
  p.interleaved = cache->rope_style == GDPA_ROPE_INTERLEAVED ? 1 : 0;
  for (int i = 0; i < 64; ++i) p.freq[i] = i < p.rot / 2 ? turn_fraction(cache->inv_freq[i]) : 0;
  // Rows of a CTA: 16 where sequences bring several tokens (a scale block's
  // worth); for single tokens as few as keep its eight warps busy (256 tokens of
  // 32 query and 8 key heads of 128, 50 calls in a graph: 6.4 us a call, with 16
  // rows 13.8).
  const int items = cache->D / 16;
  const int64_t row_tasks = 2 * ((int64_t)cache->H * items + 127) / 128 + ((int64_t)p.Hq * items + 127) / 128;
  int rows = 16;
  while (T <= 4 * (int64_t)B && rows > 1 && rows * row_tasks > kAppendThreads / 32) rows >>= 1;
  const int64_t groups = (T + rows - 1) / rows;
  // Few groups: several CTAs share the tasks of one (each finds its rows and
  // angles again).  A piece of 64 tokens of such heads takes 9.8 us so and 24.6
  // without, one of 1000 13.1 and 25.0; from 4000 tokens on there is none to spare.
  const int64_t spare = (int64_t)dev.sms * 3 / groups, useful = (rows * row_tasks + 7) / 8;
  const int share = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(spare, useful)));
  const int smem = (rows + kCacheBlock - 1) * (p.rot / 2) * (int)sizeof(float2) + kAppendThreads / 32 * 4096;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return cache->D == 128 ? launch_append<128>(p, groups, share, rows, smem, dev, s)
                         : launch_append<64>(p, groups, share, rows, smem, dev, s);
}

extern "C" gdpa_status_t gdpa_cache_workspace_size(const gdpa_cache_t* cache, int Hq, int max_q, int64_t* bytes) {
  if (!bytes) return GDPA_ERR_INVALID_ARG;
  *bytes = 0;
  gdpa_status_t st = check_cache(cache);
  if (st != GDPA_OK) return st;
  if (Hq <= 0 || Hq % cache->H || max_q <= 0) return GDPA_ERR_INVALID_ARG;
  if ((int64_t)Hq * cache->D > (1 << 20)) return GDPA_ERR_UNSUPPORTED;
  Device dev;
  if ((st = current_device(&dev)) != GDPA_OK) return st;
  const int G = Hq / cache->H;
  *bytes = cache->D == 128 ? gdpa::workspace_bytes<128>(dev, max_q, G) : gdpa::workspace_bytes<64>(dev, max_q, G);
  return GDPA_OK;
}

extern "C" gdpa_status_t gdpa_cache_fwd(const gdpa_cache_t* cache, const void* q, int64_t q_stride,
                                        const int32_t* offsets, const int32_t* kv_lens, const int32_t* page_table,
                                        int64_t T, int B, int Hq, int max_pages, int max_q, int causal,
                                        int window_tokens, float scale, void* out, float* lse, void* workspace,
                                        int64_t workspace_bytes, void* stream) {
  gdpa_status_t st = check_cache(cache);
  if (st != GDPA_OK) return st;
  if ((st = check_batch(cache, T, B, max_pages)) != GDPA_OK) return st;
  if (Hq <= 0 || Hq % cache->H || max_q <= 0 || window_tokens < 0 || (causal != 0 && causal != 1) ||
      (window_tokens > 0 && !causal) || !std::isfinite(scale))
    return GDPA_ERR_INVALID_ARG;
  if ((int64_t)Hq * cache->D > (1 << 20)) return GDPA_ERR_UNSUPPORTED;
  if (T * (Hq / cache->H) >= ((int64_t)1 << 31) - 256) return GDPA_ERR_UNSUPPORTED;  // query rows of a key head
  if (T == 0 || B == 0) return GDPA_OK;
  if ((st = check_rows(q, q_stride, Hq, cache->D)) != GDPA_OK) return st;
  if ((st = check_rows(out, (int64_t)Hq * cache->D, Hq, cache->D)) != GDPA_OK) return st;
  if (!offsets || !kv_lens || !page_table || max_pages == 0 || !aligned(lse, 4)) return GDPA_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 16)) return GDPA_ERR_INVALID_ARG;
  int64_t need = 0;
  if ((st = gdpa_cache_workspace_size(cache, Hq, max_q, &need)) != GDPA_OK) return st;
  if (workspace_bytes < need) return GDPA_ERR_NO_MEMORY;
  Device dev;
  if ((st = current_device(&dev)) != GDPA_OK) return st;
  CacheFwdParams p;
  p.cache = view(cache);
  p.batch = CacheBatch{offsets, kv_lens, page_table, static_cast<int>(T), B, max_pages, dev.status};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_stride = q_stride;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.Hq = Hq;
  p.G = Hq / cache->H;
  p.inv_g = p.G == 1 ? 0 : static_cast<uint32_t>((((uint64_t)1 << 32) + p.G - 1) / p.G);
  p.causal = causal;
  p.window = window_tokens;
  p.scale2 = scale * 1.4426950408889634f;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return cache->D == 128 ? launch_fwd<128>(p, workspace, max_q, dev, s) : launch_fwd<64>(p, workspace, max_q, dev, s);
}
