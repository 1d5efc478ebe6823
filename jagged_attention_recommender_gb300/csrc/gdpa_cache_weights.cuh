// gdpa_cache_weights.cuh -- the attention weight that each stored key receives
// from the rows of a call.
//
// Mathematics.  With the rows' logsumexp at hand the weight of a row for a key
// is exp(scale <q, k> - lse): no maximum, no second product, and a key's sum is
// its own, so keys are split over the GPU and nothing is joined.
#pragma once

#include "gdpa_cache.cuh"

namespace gdpa {

struct CacheWeightsParams {
  CacheView cache;
  CacheBatch batch;
  const __nv_bfloat16* q;
  int64_t q_stride;
  const float* lse;
  const float* w_in;  // may be null
  float* w;
  int Hq, G;
  int causal, window;
  float scale2, decay;  // scale log2(e)
};

// The rows [lo, hi) of a sequence that see key j.
struct RowSpan {
  int lo, hi;
};
__device__ __forceinline__ RowSpan rows_of_key(const CacheSeq& s, int j, int causal, int window) {
  RowSpan r = {0, s.n};
  if (!causal) return r;
  const int at = j - (s.len - s.n);  // the row whose own position is j
  r.lo = max(at, 0);
  if (window > 0) r.hi = static_cast<int>(min(static_cast<int64_t>(s.n), max(static_cast<int64_t>(at) + window, (int64_t)0)));
  return r;
}

template <int D>
__global__ void __launch_bounds__(128) gdpa_cache_weights_kernel(const __grid_constant__ CacheWeightsParams p) {
  const CacheBatch& bt = p.batch;
  const int64_t heads = static_cast<int64_t>(bt.B) * p.cache.H;
  for (int64_t bh = blockIdx.y; bh < heads; bh += gridDim.y) {
    const int b = static_cast<int>(bh / p.cache.H), h = static_cast<int>(bh - static_cast<int64_t>(b) * p.cache.H);
    const CacheSeq s = load_sequence(bt, p.cache.lp, b);
    if (!s.ok || s.n == 0) continue;
    for (int64_t j64 = blockIdx.x * 128ll + threadIdx.x; j64 < s.len; j64 += gridDim.x * 128ll) {
      const int j = static_cast<int>(j64);
      const int page = load_page(p.cache, bt, b, j);
      if (page < 0) continue;
      const int64_t row = cache_row(p.cache, page, h, j & ((1 << p.cache.lp) - 1));
      float k[D];
      const uint8_t* codes = p.cache.k + row * D;
      for (int d = 0; d < D; ++d) k[d] = e4m3_to_float(codes[d]);
      const float f = sf_value(p.cache.k_sf[row >> 4]) * p.scale2;
      float sum = p.w_in && j < s.len - s.n ? p.decay * p.w_in[row] : 0.0f;
      const RowSpan rows = rows_of_key(s, j, p.causal, p.window);
      for (int i = rows.lo; i < rows.hi; ++i) {
        for (int g = 0; g < p.G; ++g) {
          const int head = h * p.G + g;
          const float lse = __ldg(p.lse + static_cast<int64_t>(s.first + i) * p.Hq + head);
          const __nv_bfloat16* q = p.q + (s.first + i) * p.q_stride + head * D;
          float x = 0.0f;
          for (int d = 0; d < D; ++d) x = fmaf(__bfloat162float(q[d]), k[d], x);
          if (lse != -INFINITY) sum += ptx::ex2_approx(x * f - lse * 1.4426950408889634f);
        }
      }
      p.w[row] = sum;
    }
  }
}

}  // namespace gdpa
