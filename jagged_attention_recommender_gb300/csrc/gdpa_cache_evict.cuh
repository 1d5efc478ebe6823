// gdpa_cache_evict.cuh -- cuts sequences of the cache to their most attended
// tokens: a kernel that chooses them, head by head, and one that moves them.
//
// Choosing.  A weight's bits, turned so that larger numbers have larger unsigned
// keys, are searched for the smallest key that is kept, eight bits a pass: a
// histogram of the keys that agree so far says which digit the k-th largest
// has.  A last pass over the tokens, in order, keeps what is above that key and
// the first of what equals it.
//
// Moving.  A warp makes one block of 16 new tokens of one head, for K and for V:
// their scales, the largest of them, and the codes, which are copied as they
// are where the scale is the same.
#pragma once

#include "gdpa_cache_append.cuh"

namespace gdpa {

struct EvictParams {
  CacheView cache;
  float* weights;
  const int32_t* kv_lens;
  const int32_t* table;      // [B, max_pages]
  const int32_t* new_table;  // [B, new_max_pages]
  int32_t* kept;             // [B, H, budget]
  int32_t* new_lens;
  int B, max_pages, new_max_pages;
  int budget, sink, recent;
  int most;  // tokens that any sequence keeps, as far as the host knows
  int* status;
};

// Larger weights have larger keys; NaN has the least; both zeros are the same.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (!(w == w)) return 0;
  const uint32_t u = __float_as_uint(w + 0.0f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// A sequence's length, -1 (flagged) where it does not fit the table.
__device__ __forceinline__ int evict_len(const EvictParams& p, int b) {
  const int len = __ldg(p.kv_lens + b);
  if (len >= 0 && len <= static_cast<int64_t>(p.max_pages) << p.cache.lp) return len;
  atomicOr(p.status, kStatusBadPlan);
  return -1;
}

// Token j's row of the cache, -1 on a page out of range (flagged).
__device__ __forceinline__ int64_t token_row(const EvictParams& p, const int32_t* table, int max_pages, int b, int h, int j) {
  const int page = __ldg(table + static_cast<int64_t>(b) * max_pages + (j >> p.cache.lp));
  if (page >= 0 && page < p.cache.num_pages) return cache_row(p.cache, page, h, j & ((1 << p.cache.lp) - 1));
  atomicOr(p.status, kStatusBadPlan);
  return -1;
}

constexpr int kChooseThreads = 512;

__global__ void __launch_bounds__(kChooseThreads) gdpa_cache_choose_kernel(const __grid_constant__ EvictParams p) {
  __shared__ int s_hist[256];
  __shared__ uint32_t s_digit;
  __shared__ int s_need;
  __shared__ int s_scan[2][kChooseThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t heads = static_cast<int64_t>(p.B) * p.cache.H;
  for (int64_t bh = blockIdx.x; bh < heads; bh += gridDim.x) {
    const int b = static_cast<int>(bh / p.cache.H), h = static_cast<int>(bh - static_cast<int64_t>(b) * p.cache.H);
    const int len = evict_len(p, b), keep = min(len, p.budget);
    if (h == 0 && tid == 0) p.new_lens[b] = max(keep, 0);
    if (keep <= 0) continue;
    int32_t* const kept = p.kept + bh * p.budget;
    if (keep == len) {
      for (int j = tid; j < keep; j += kChooseThreads) kept[j] = j;
      continue;
    }
    auto key = [&](int j) -> uint32_t {
      const int64_t row = token_row(p, p.table, p.max_pages, b, h, j);
      return row < 0 ? 0 : weight_key(p.weights[row]);
    };
    // sink + recent <= budget < len: the tokens between them compete
    const int lo = p.sink, hi = len - p.recent;
    int need = keep - p.sink - p.recent;  // 0: none of them stays
    uint32_t prefix = 0;
    if (need > 0) {
      for (int shift = 24; shift >= 0; shift -= 8) {
        for (int i = tid; i < 256; i += kChooseThreads) s_hist[i] = 0;
        __syncthreads();
        const uint32_t mask = shift == 24 ? 0 : 0xffffffffu << (shift + 8);
        for (int64_t j = lo + tid; j < hi; j += kChooseThreads) {
          const uint32_t k = key(static_cast<int>(j));
          if ((k & mask) == prefix) atomicAdd(&s_hist[k >> shift & 255], 1);
        }
        __syncthreads();
        if (tid == 0) {
          int d = 255, left = need;
          while (d > 0 && s_hist[d] < left) left -= s_hist[d--];
          s_digit = d;
          s_need = left;
        }
        __syncthreads();
        prefix |= s_digit << shift;
        need = s_need;  // how many of those that equal the key so far stay
        __syncthreads();
      }
    }
    int out = 0, equal = 0;  // kept so far; candidates so far that equal the key
    for (int64_t j0 = 0; j0 < len; j0 += kChooseThreads) {
      const int64_t j = j0 + tid;
      bool always = j < lo || (j >= hi && j < len), above = false, same = false;
      if (!always && j < len && keep - p.sink - p.recent > 0) {
        const uint32_t k = key(static_cast<int>(j));
        above = k > prefix;
        same = k == prefix;
      }
      const unsigned eq = __ballot_sync(0xffffffffu, same);
      if (lane == 0) s_scan[0][warp] = __popc(eq);
      __syncthreads();
      int e = equal;
      for (int w = 0; w < kChooseThreads / 32; ++w) {
        if (w < warp) e += s_scan[0][w];
        equal += s_scan[0][w];
      }
      const bool take = always || above || (same && e + __popc(eq & ((1u << lane) - 1)) < need);
      const unsigned all = __ballot_sync(0xffffffffu, take);
      if (lane == 0) s_scan[1][warp] = __popc(all);
      __syncthreads();
      int at = out + __popc(all & ((1u << lane) - 1));
      for (int w = 0; w < kChooseThreads / 32; ++w) {
        if (w < warp) at += s_scan[1][w];
        out += s_scan[1][w];
      }
      if (take && at < keep) kept[at] = static_cast<int>(j);
      __syncthreads();
    }
  }
}

// 16 codes from scale `from` to the larger scale `to`.
__device__ __forceinline__ uint4 rescale16(uint4 x, int from, int to) {
  if (from == to) return x;
  const float f = sf_value(127 - min(to - from, 126));
  return make_uint4(rescale4(x.x, f), rescale4(x.y, f), rescale4(x.z, f), rescale4(x.w, f));
}

template <int D>
__global__ void __launch_bounds__(256) gdpa_cache_move_kernel(const __grid_constant__ EvictParams p) {
  constexpr int LPT = D / 16, TPS = 32 / LPT;  // lanes of a token, tokens of a step
  const int lane = threadIdx.x & 31, H = p.cache.H;
  const int64_t blocks = (static_cast<int64_t>(p.most) + kCacheBlock - 1) / kCacheBlock;
  const int64_t tasks = blocks * p.B * H, step = gridDim.x * 8ll;
  for (int64_t task = blockIdx.x * 8ll + (threadIdx.x >> 5); task < tasks; task += step) {
    const int64_t bh = task / blocks;
    const int i0 = static_cast<int>(task - bh * blocks) * kCacheBlock;
    const int b = static_cast<int>(bh / H), h = static_cast<int>(bh - static_cast<int64_t>(b) * H);
    const int keep = min(evict_len(p, b), p.budget), cnt = min(keep - i0, kCacheBlock);
    if (cnt <= 0) continue;
    const int64_t to = token_row(p, p.new_table, p.new_max_pages, b, h, i0);
    if (to < 0) continue;
    // lanes 0..15 and 16..31 hold the tokens' old rows
    const int t = lane & 15;
    int64_t from = -1;
    if (t < cnt) from = token_row(p, p.table, p.max_pages, b, h, __ldg(p.kept + bh * p.budget + i0 + t));
    int sf = -1;  // of K in the lower lanes, of V in the upper ones
    if (from >= 0) sf = __ldg((lane < 16 ? p.cache.k_sf : p.cache.v_sf) + (from >> 4));
    if (lane < 16 && from >= 0) p.weights[to + t] = p.weights[from];
    int top = sf;
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
    if (t == 0 && top >= 0) (lane < 16 ? p.cache.k_sf : p.cache.v_sf)[to >> 4] = static_cast<uint8_t>(top);
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const uint8_t* const codes = which ? p.cache.v : p.cache.k;
      uint8_t* const dst = which ? p.cache.v : p.cache.k;
      const int most = __shfl_sync(0xffffffffu, top, 16 * which);
#pragma unroll
      for (int u = 0; u < kCacheBlock; u += TPS) {
        const int tok = u + lane / LPT;
        const int64_t src = __shfl_sync(0xffffffffu, from, tok);
        const int old = __shfl_sync(0xffffffffu, sf, 16 * which + tok);
        if (tok < cnt && src >= 0) {
          const uint4 x = *reinterpret_cast<const uint4*>(codes + src * D + lane % LPT * 16);
          *reinterpret_cast<uint4*>(dst + (to + tok) * D + lane % LPT * 16) = rescale16(x, old, most);
        }
      }
    }
  }
}

}  // namespace gdpa
