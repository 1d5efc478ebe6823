// gdpa_cache_fwd.cuh -- attention of new tokens over the paged e4m3 cache.
#pragma once

#include "gdpa_cache.cuh"

namespace gdpa {

struct CacheFwdParams {
  CacheView cache;
  CacheBatch batch;
  const __nv_bfloat16* q;
  int64_t q_stride;
  __nv_bfloat16* out;
  float* lse;
  int Hq, G;       // query heads, query heads of a key/value head
  int causal, window;
  float scale2;    // scale * log2(e)
};

__device__ __forceinline__ float e4m3_to_float(uint32_t byte) {
  float f;
  asm("{ .reg .b16 t, lo, hi; .reg .b32 h; cvt.u16.u32 t, %1; cvt.rn.f16x2.e4m3x2 h, t; mov.b32 {lo, hi}, h;"
      " cvt.f32.f16 %0, lo; }"
      : "=f"(f)
      : "r"(byte));
  return f;
}

// One warp for each (row, query head): one pass over the row's keys with the
// running maximum and sum of the softmax, D / 32 coordinates a lane.
template <int D>
__global__ void __launch_bounds__(128) gdpa_cache_fwd_row_kernel(const CacheFwdParams p) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int r = static_cast<int>(id / p.Hq), hq = static_cast<int>(id % p.Hq);
  if (r >= p.batch.T) return;
  const int b = find_sequence(p.batch.offsets, p.batch.B, r);
  if (b >= p.batch.B) return;
  const CacheSeq s = load_sequence(p.batch, p.cache.lp, b);
  if (!s.ok || r < s.first) return;
  const int pos = s.len - s.n + (r - s.first), h = hq / p.G;
  const int end = p.causal ? min(s.len, pos + 1) : s.len;
  const int begin = p.window > 0 ? max(0, pos - p.window + 1) : 0;
  float q[E], o[E], m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = __bfloat162float(p.q[r * p.q_stride + hq * D + lane * E + e]);
    o[e] = 0.0f;
  }
  for (int j = begin; j < end; ++j) {
    const int page = load_page(p.cache, p.batch, b, j);
    if (page < 0) continue;
    const int slot = j & ((1 << p.cache.lp) - 1);
    const int64_t at = cache_row(p.cache, page, h, slot) * D + lane * E, sf = cache_sf(p.cache, page, h, slot);
    float x = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) x += q[e] * e4m3_to_float(p.cache.k[at + e]);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    x = x * sf_value(p.cache.k_sf[sf]) * p.scale2;
    const float top = fmaxf(m, x);
    const float keep = m == top ? 1.0f : exp2f(m - top), w = exp2f(x - top);
    const float vs = sf_value(p.cache.v_sf[sf]);
    l = l * keep + w;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * keep + w * (e4m3_to_float(p.cache.v[at + e]) * vs);
    m = top;
  }
  const int64_t at = (static_cast<int64_t>(r) * p.Hq + hq) * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) p.out[at + e] = __float2bfloat16_rn(l != 0.0f ? o[e] / l : 0.0f);
  if (p.lse && lane == 0) p.lse[static_cast<int64_t>(r) * p.Hq + hq] = l != 0.0f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

}  // namespace gdpa
