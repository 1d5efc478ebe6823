// gdpa_cache.cuh -- the paged key/value cache as the kernels see it: layout,
// scale codes, and the lookup from a row of the new tokens to its sequence.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "gdpa_cache_index.h"
#include "gdpa_fwd_common.cuh"
#include "gdpa_internal.h"

namespace gdpa {

struct CacheView {
  uint8_t* k;
  uint8_t* v;
  uint8_t* k_sf;
  uint8_t* v_sf;
  int num_pages;
  int lp;  // log2(page_tokens)
  int H;   // key/value heads
};

// One batch of new tokens beside the cache.
struct CacheBatch {
  const int32_t* offsets;  // [B + 1]
  const int32_t* kv_lens;  // [B], after the append
  const int32_t* table;    // [B, max_pages]
  int T, B, max_pages;
  int* status;
};

// First row of codes of (page, head, slot), in tokens: 64 bits, since a cache
// of 280 GB holds more than 2^31 codes.
__device__ __forceinline__ int64_t cache_row(const CacheView& c, int page, int head, int slot) {
  return ((static_cast<int64_t>(page) * c.H + head) << c.lp) + slot;
}
// The scale of the block that holds it.
__device__ __forceinline__ int64_t cache_sf(const CacheView& c, int page, int head, int slot) {
  return ((static_cast<int64_t>(page) * c.H + head) << (c.lp - 4)) + (slot >> 4);
}

// 2^(code - 127); code 0 is the subnormal 2^-127, 255 is NaN (E8M0).
__device__ __forceinline__ float sf_value(int code) {
  return code == 255 ? __int_as_float(0x7fc00000) : code ? __int_as_float(code << 23) : __int_as_float(0x00400000);
}

__device__ __forceinline__ float e4m3_to_float(uint32_t byte) {
  float f;
  asm("{ .reg .b16 t, lo, hi; .reg .b32 h; cvt.u16.u32 t, %1; cvt.rn.f16x2.e4m3x2 h, t; mov.b32 {lo, hi}, h;"
      " cvt.f32.f16 %0, lo; }"
      : "=f"(f)
      : "r"(byte));
  return f;
}

// The sequence that holds row r of the new tokens, or B if none does: the
// first b with offsets[b + 1] > r.  Never reads outside offsets[1..B],
// whatever they hold.
__device__ __forceinline__ int find_sequence(const int32_t* __restrict__ offsets, int B, int r) {
  int lo = 0, hi = B;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(offsets + mid + 1) > r) hi = mid; else lo = mid + 1;
  }
  return lo;
}

// The same by all lanes of a warp, for the same row: 32 places a step.
__device__ __forceinline__ int find_sequence_warp(const int32_t* __restrict__ offsets, int B, int r) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = B;  // the answer is in lo..hi
  while (lo < hi) {
    const int step = (hi - lo + 31) >> 5, at = min(lo + step * (lane + 1), hi) - 1;
    // lanes whose place still lies in front of the answer
    const unsigned before = __ballot_sync(0xffffffffu, __ldg(offsets + at + 1) <= r);
    const int n = before == 0xffffffffu ? 32 : __ffs(~before) - 1;
    lo = min(lo + step * n, hi);
    if (n < 32) hi = min(lo + step - 1, hi);
  }
  return lo;
}

// Sequence b's rows and length (an invalid one flags the launch).
__device__ __forceinline__ CacheSeq load_sequence(const CacheBatch& c, int lp, int b) {
  const CacheSeq s = cache_sequence(__ldg(c.offsets + b), __ldg(c.offsets + b + 1), __ldg(c.kv_lens + b), c.T,
                                    static_cast<int64_t>(c.max_pages) << lp);
  if (!s.ok) atomicOr(c.status, kStatusBadPlan);
  return s;
}

// The page of position pos (a block start or any token), or -1 (flagged) when
// the table's entry is no page of the cache.
__device__ __forceinline__ int load_page(const CacheView& c, const CacheBatch& a, int b, int pos) {
  const int page = __ldg(a.table + static_cast<int64_t>(b) * a.max_pages + (pos >> c.lp));
  if (page >= 0 && page < c.num_pages) return page;
  atomicOr(a.status, kStatusBadPlan);
  return -1;
}

}  // namespace gdpa
