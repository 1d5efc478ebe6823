// gdpa_rope.cuh -- rotary positions of the rows of a jagged batch, and their
// gradient.
//
// Mathematics.  A pair (x, y) at position p turns by a = p f; a rotation's
// gradient is the rotation back, so one kernel does both with the sine's sign.
// The angle is the cache's (gdpa_cache_index.h): p times f as a 64-bit fraction
// of a turn, modulo 2^64, exact at every position.
//
// Bound: memory, 4 bytes an element in and out against about 2 flops.  Measured:
// queries and keys (8 heads of 128) of 267k rows of a training batch, strided in,
// 171 us (6.4 TB/s, 94 % of a copy's rate); their gradient, strided out, 170; pieces
// of 36k rows, 9 heads of 64, half rotated, interleaved, 15 us (5.4 TB/s); ten heads of
// four tokens 2.8 us on the device.
//
// Work split.  An item is 16 coordinates of a head, whole pairs of them in two
// 16-byte chunks (gdpa_cache_append.cuh: ItemAt).  A lane keeps one row and one
// item, computes its eight angles once, in registers, and walks the row's heads
// with them; the D / 16 lanes of a row read whole 128-byte lines.
#pragma once

#include "gdpa_cache_append.cuh"

namespace gdpa {

struct RopeParams {
  const __nv_bfloat16* x;
  __nv_bfloat16* y;
  int64_t x_stride, y_stride;
  const int32_t* offsets;  // [B + 1]
  const int32_t* first;    // [B], or null
  int* status;
  int T, B, H;
  int rot, interleaved;
  int heads;               // of a lane
  float magnitude, sign;   // sign: of the sine
  unsigned long long freq[64];  // fraction of a turn a position, times 2^64
};

constexpr int kRopeThreads = 256;

// The sequence of each lane's row r (the same for the lanes of a row; rows of
// a warp ascend from r0).
__device__ __forceinline__ int rope_sequence(const RopeParams& p, int r0, int r) {
  int b = find_sequence_warp(p.offsets, p.B, r0);
  if (b < p.B && r != r0 && __ldg(p.offsets + b + 1) <= r) b = find_sequence(p.offsets, p.B, r);
  return b;
}

template <int D>
__global__ void __launch_bounds__(kRopeThreads) gdpa_rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int IPR = D / 16, RPW = 32 / IPR;  // items of a row and head; rows of a warp
  constexpr int U = 4;                         // heads in flight
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, it = lane % IPR;
  const int r0 = (blockIdx.x * (kRopeThreads / 32) + warp) * RPW, r = r0 + lane / IPR;
  if (r0 >= p.T) return;
  const int b = rope_sequence(p, r0, r);
  if (r >= p.T || b >= p.B) return;
  const int begin = __ldg(p.offsets + b), end = __ldg(p.offsets + b + 1);
  if (begin < 0 || begin > r || end > p.T) {
    atomicOr(p.status, kStatusBadPlan);
    return;
  }
  const ItemAt at = item_at(it, p.rot, p.interleaved);
  if (at.pair < 0 && p.x == p.y) return;  // in place: what does not turn stays
  const int h0 = blockIdx.y * p.heads, h1 = min(p.H, h0 + p.heads);
  const __nv_bfloat16* src = p.x + r * p.x_stride;
  __nv_bfloat16* dst = p.y + r * p.y_stride;
  Angles t;
  if (at.pair >= 0) {
    const int64_t pos = (p.first ? static_cast<int64_t>(__ldg(p.first + b)) : 0) + (r - begin);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 u = rope_angle(p.freq[at.pair + 2 * i], pos), v = rope_angle(p.freq[at.pair + 2 * i + 1], pos);
      t.c[i] = ptx::f2_pack(u.x * p.magnitude, v.x * p.magnitude);
      t.s[i] = ptx::f2_pack(u.y * p.sign, v.y * p.sign);
    }
  }
  for (int h = h0; h < h1; h += U) {
    uint4 u[U], v[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (h + i >= h1) break;
      u[i] = *reinterpret_cast<const uint4*>(src + (h + i) * D + at.d0);
      v[i] = *reinterpret_cast<const uint4*>(src + (h + i) * D + at.d1);
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (h + i >= h1) break;
      if (at.pair >= 0) {
        uint64_t x[8];
        unpack8(u[i], x);
        unpack8(v[i], x + 4);
        rotate_item(p.interleaved, t, x);
        u[i] = pack8(x);
        v[i] = pack8(x + 4);
      }
      *reinterpret_cast<uint4*>(dst + (h + i) * D + at.d0) = u[i];
      *reinterpret_cast<uint4*>(dst + (h + i) * D + at.d1) = v[i];
    }
  }
}

}  // namespace gdpa
