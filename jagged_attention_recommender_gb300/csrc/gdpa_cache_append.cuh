// gdpa_cache_append.cuh -- stores new tokens in the paged e4m3 cache, with
// the position rotation of keys and queries on the way.
//
// Mathematics.  A pair (x, y) at position p turns by theta = p f.  With
// F = f / 2 pi as a 64-bit fraction of a turn, p F modulo 2^64 IS theta
// modulo one turn, with an error of p 2^-64 turns: one integer product, no
// argument reduction and no 64-bit floating point at any position.  The top 32
// bits, rounded to fp32's 24 (2^-26 turns at most), go to sincospif.  A block
// of 16 tokens of one head has one scale 2^e, e the smallest integer with
// amax <= 448 2^e, so from the bits of amax (exponent field E, mantissa M):
// e + 127 = E - 8 + (M > 0.75 2^23).
//
// Bound: memory.  Per new token Hq D 4 bytes (queries in and out) and
// H D (4 + 2) (keys and values in, codes out) against about 3 flops an element.
//
// Work split.  A scale block takes its new tokens from consecutive rows, so
// the row that is the first of them owns the block, and whoever finds the row
// needs no plan and no list: a CTA looks at a group of rows, keeps the owners,
// tabulates sine and cosine of their blocks' rows (shared by all heads), and
// its warps take tasks of up to 128 items of 16 elements: keys or values of a
// block and as many heads as that makes (one for 16 tokens, 16 for a single
// one of 128), or query items of a few rows.  A task's elements come to shared
// memory by the lanes' own asynchronous copies (4 KB a warp, 24 warps an SM)
// and are read from there twice, for the largest magnitude and for the codes:
// held in registers they left room for 16 warps and took 387 us for 68 423 tokens
// of 32 query and 8 key heads of 128, where this takes 284 (5.4 TB/s).
#pragma once

#include "gdpa_cache.cuh"

namespace gdpa {

struct AppendParams {
  CacheView cache;
  CacheBatch batch;
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  int64_t q_stride, k_stride, v_stride;
  __nv_bfloat16* q_out;
  int Hq;
  int rot;         // rotated coordinates
  int interleaved;
  unsigned long long freq[64];  // fraction of a turn a position, times 2^64
};

constexpr int kAppendThreads = 256;

// cos, sin of position pos times fraction F of a turn.
__device__ __forceinline__ float2 rope_angle(unsigned long long F, int64_t pos) {
  const int turn = static_cast<int>((static_cast<unsigned long long>(pos) * F) >> 32);  // [-1/2, 1/2) turns, 2^-32 units
  float s, c;
  sincospif(static_cast<float>(turn) * 4.656612873077393e-10f, &s, &c);  // 2^-31: half turns
  return make_float2(c, s);
}

// Eight bf16 as four pairs of fp32 (the arithmetic below is on packed pairs).
__device__ __forceinline__ void unpack8(const uint4& u, uint64_t* x) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = ptx::f2_pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}

__device__ __forceinline__ uint4 pack8(const uint64_t* x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    ptx::f2_unpack(x[i], lo, hi);
    w[i] = ptx::pack_bf16x2(lo, hi);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// An item: 16 coordinates of one head as two chunks of 8, at d0 and d1.
// Rotated items hold whole pairs: across the chunks (half) or inside them
// (interleaved).
struct ItemAt {
  int d0, d1, pair;  // pair: first rotated pair of the item, -1 if none
};
__device__ __forceinline__ ItemAt item_at(int it, int rot, int interleaved) {
  if (16 * it < rot && !interleaved) return ItemAt{8 * it, (rot >> 1) + 8 * it, 8 * it};
  return ItemAt{16 * it, 16 * it + 8, 16 * it < rot ? 8 * it : -1};
}

// Cosines and sines of an item's eight pairs, two in a word.
struct Angles {
  uint64_t c[4], s[4];
};
__device__ __forceinline__ Angles load_angles(const float* cos_at, const float* sin_at) {
  Angles t;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const ulonglong2 c = reinterpret_cast<const ulonglong2*>(cos_at)[i], s = reinterpret_cast<const ulonglong2*>(sin_at)[i];
    t.c[2 * i] = c.x, t.c[2 * i + 1] = c.y;
    t.s[2 * i] = s.x, t.s[2 * i + 1] = s.y;
  }
  return t;
}

// Rotates an item: x[0..3] its first chunk, x[4..7] its second.
__device__ __forceinline__ void rotate_item(int interleaved, const Angles& t, uint64_t (&x)[8]) {
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float a, b, c, s, c2, s2;
      ptx::f2_unpack(x[i], a, b);
      ptx::f2_unpack(t.c[i >> 1], c, c2);
      ptx::f2_unpack(t.s[i >> 1], s, s2);
      if (i & 1) c = c2, s = s2;
      x[i] = ptx::f2_pack(a * c - b * s, b * c + a * s);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t a = x[i], b = x[4 + i];
      x[i] = ptx::f2_fma(a, t.c[i], ptx::f2_mul(b, t.s[i] ^ 0x8000000080000000ull));
      x[4 + i] = ptx::f2_fma(b, t.c[i], ptx::f2_mul(a, t.s[i]));
    }
  }
}

// The largest magnitude of an item, NaN left out.
__device__ __forceinline__ float item_max(const uint64_t (&x)[8]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float a, b;
    ptx::f2_unpack(x[i], a, b);
    m = fmaxf(m, fmaxf(fabsf(a), fabsf(b)));
  }
  return m;
}
// The same of 16 values as loaded.
__device__ __forceinline__ float raw_max(const uint4& u, const uint4& v) {
  const uint32_t w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) asm("max.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w[i] & 0x7fff7fffu));
  return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
}

// Eight values times `inv` (a power of two) as e4m3 codes.  What is not finite
// becomes the NaN code: the conversion does that to NaN, but makes an infinity
// 448, so a task that holds one (`inf`, uniform) replaces it first.
__device__ __forceinline__ uint2 quantise8(const uint64_t* x, float inv, bool inf) {
  const uint64_t f = ptx::f2_splat(inv);
  float y[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) ptx::f2_unpack(ptx::f2_mul(x[i], f), y[2 * i], y[2 * i + 1]);
  if (inf) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a, b;
      ptx::f2_unpack(x[i], a, b);
      if (fabsf(a) == INFINITY) y[2 * i] = __int_as_float(0x7fffffff);
      if (fabsf(b) == INFINITY) y[2 * i + 1] = __int_as_float(0x7fffffff);
    }
  }
  return make_uint2(ptx::pack_e4m3x4(y[0], y[1], y[2], y[3]), ptx::pack_e4m3x4(y[4], y[5], y[6], y[7]));
}

__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t two) {
  uint32_t h;
  asm("{ .reg .b16 t; cvt.u16.u32 t, %1; cvt.rn.f16x2.e4m3x2 %0, t; }" : "=r"(h) : "r"(two));
  float2 f;
  asm("{ .reg .b16 lo, hi; mov.b32 {lo, hi}, %2; cvt.f32.f16 %0, lo; cvt.f32.f16 %1, hi; }"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}

// Four codes times f (a power of two), rounded to codes again.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float f) {
  const float2 a = e4m3x2_to_float2(w & 0xffffu), b = e4m3x2_to_float2(w >> 16);
  return ptx::pack_e4m3x4(a.x * f, a.y * f, b.x * f, b.y * f);
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// This thread's own copies have arrived.
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.commit_group;\n cp.async.wait_group 0;" ::: "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
  uint4 u;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "r"(addr));
  return u;
}

// The largest of each L lanes (a power of two).
__device__ __forceinline__ float head_max(float x, int L) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    const float y = __shfl_xor_sync(0xffffffffu, x, d);
    if (d < L) x = fmaxf(x, y);
  }
  return x;
}

// A scale block that this launch writes to: `cnt` new tokens from row `row`
// on, the first at position `pos`.
struct OwnedBlock {
  int row, cnt, pos, page, tab;  // tab: its first row in the angle table
};

template <int D>
__global__ void __launch_bounds__(kAppendThreads, 3) gdpa_cache_append_kernel(const __grid_constant__ AppendParams p,
                                                                           int rows_per_cta) {
  constexpr int IPR = D / 16;             // items of a row and head
  constexpr int HPW = 32 / IPR;           // heads (or rows of one head) whose items a warp holds once
  __shared__ OwnedBlock s_own[16];
  __shared__ int s_n;
  extern __shared__ __align__(16) float s_cos[];  // [rows][rot / 2], and the sines behind them
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const CacheBatch& bt = p.batch;
  const int g0 = blockIdx.x * rows_per_cta;

  if (warp == 0) {
    OwnedBlock o{0, 0, 0, -1, 0};
    const int r = g0 + lane;
    // the group's first sequence by all lanes, then each row's among the next 32
    const int b0 = find_sequence_warp(bt.offsets, bt.B, g0);
    const int end = b0 + lane < bt.B ? __ldg(bt.offsets + b0 + lane + 1) : 0x7fffffff;
    int b = b0;
#pragma unroll
    for (int i = 0; i < 32; ++i) b += __shfl_sync(0xffffffffu, end, i) <= r ? 1 : 0;
    if (lane < rows_per_cta && r < bt.T) {
      if (b == b0 + 32) b = find_sequence(bt.offsets, bt.B, r);  // many empty sequences
      if (b < bt.B) {
        const OwnedRows rows = owned_rows(load_sequence(bt, p.cache.lp, b), r);
        if (rows.bad) atomicOr(bt.status, kStatusBadPlan);
        if (rows.cnt > 0) {
          o.row = r;
          o.pos = rows.pos;
          o.cnt = rows.cnt;
          o.page = load_page(p.cache, bt, b, rows.pos);
        }
      }
    }
    int tab = o.cnt;  // running sum of the owners' row counts
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, tab, d);
      if (lane >= d) tab += t;
    }
    o.tab = tab - o.cnt;
    // Blocks of one group never overlap, so that their rows fit the table;
    // offsets that decrease can make them, and are caught here (no count is
    // negative, so a place in the table never is).
    if (o.cnt > 0 && tab > rows_per_cta + kCacheBlock - 1) {
      o.cnt = 0;
      atomicOr(bt.status, kStatusBadPlan);
    }
    const unsigned owners = __ballot_sync(0xffffffffu, o.cnt > 0);
    if (o.cnt > 0) s_own[__popc(owners & ((1u << lane) - 1))] = o;
    if (lane == 0) s_n = __popc(owners);
  }
  __syncthreads();
  const int n = s_n;
  if (n == 0) return;
  const int half = p.rot >> 1;
  float* const s_sin = s_cos + (rows_per_cta + kCacheBlock - 1) * half;
  if (half > 0) {
    for (int j = 0; j < n; ++j) {
      const OwnedBlock o = s_own[j];
      for (int i = tid; i < o.cnt * half; i += kAppendThreads) {
        const int t = i / half, f = i - t * half;
        const float2 cs = rope_angle(p.freq[f], o.pos + t);
        s_cos[(o.tab + t) * half + f] = cs.x;
        s_sin[(o.tab + t) * half + f] = cs.y;
      }
    }
    __syncthreads();
  }

  const int H = p.cache.H;
  const int workers = (kAppendThreads / 32) * gridDim.y;
  const int it = lane % IPR;  // a lane's items are the same one of several heads or rows
  const int groups = p.q ? (p.Hq + HPW - 1) / HPW : 0;  // a row's heads, in warps
  const int span = groups >= 3 ? 4 : max(groups, 1);    // groups of a row in a task ...
  const int trows = 4 / span;                           // ... and rows of a task
  const int per_row = (groups + 3) / 4;                 // tasks of a row where trows is 1
  // this lane's 16-byte pieces of a task: first chunks of its four items, then second ones
  const uint32_t stage = ptx::smem_u32(s_cos) + static_cast<uint32_t>((rows_per_cta + kCacheBlock - 1) * half) * 8 +
                         warp * 4096 + lane * 16;
  auto angles = [&](int row, const ItemAt& at) {
    const int i = row * half + at.pair;
    return load_angles(s_cos + i, s_sin + i);
  };
  int w = blockIdx.y * (kAppendThreads / 32) + warp;  // this warp's next task, counted over all blocks
  for (int j = 0; j < n; ++j) {
    const OwnedBlock o = s_own[j];
    // keys and values: tokens (to a power of two) times items of a head; the
    // heads of a task; lanes, and steps of 32 items, of a head
    const int ltok = o.cnt > 1 ? 32 - __clz(o.cnt - 1) : 0, lhead = ltok + (IPR == 8 ? 3 : 2);
    const int heads = 128 >> lhead, L = min(32, 1 << lhead), steps = max(1, (1 << lhead) >> 5);
    const int kv_tasks = (H + heads - 1) / heads;
    const int q_tasks = groups == 0 ? 0 : trows == 1 ? o.cnt * per_row : (o.cnt + trows - 1) / trows;
    const int tasks = 2 * kv_tasks + q_tasks;
#pragma unroll 1
    for (; w < tasks; w += workers) {
      if (w >= 2 * kv_tasks) {  // queries: rotate and store
        const int task = w - 2 * kv_tasks;
        const int t0 = trows == 1 ? task / per_row : task * trows;
        const int h0 = (trows == 1 ? task % per_row * 4 * HPW : 0) + lane / IPR;
        const ItemAt at = item_at(it, p.rot, p.interleaved);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int t = t0 + u / span, head = h0 + u % span * HPW;
          if (t < o.cnt && head < p.Hq) {
            const __nv_bfloat16* src = p.q + (o.row + t) * p.q_stride + head * D;
            copy16(stage + u * 512, src + at.d0);
            copy16(stage + 2048 + u * 512, src + at.d1);
          }
        }
        copies_wait();
        Angles cs;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int t = t0 + u / span, head = h0 + u % span * HPW;
          if (u % span == 0 && at.pair >= 0 && t < o.cnt) cs = angles(o.tab + t, at);
          if (t < o.cnt && head < p.Hq) {
            uint64_t x[8];
            unpack8(lds16(stage + u * 512), x);
            unpack8(lds16(stage + 2048 + u * 512), x + 4);
            if (at.pair >= 0) rotate_item(p.interleaved, cs, x);
            __nv_bfloat16* dst = p.q_out + (static_cast<int64_t>(o.row + t) * p.Hq + head) * D;
            *reinterpret_cast<uint4*>(dst + at.d0) = pack8(x);
            *reinterpret_cast<uint4*>(dst + at.d1) = pack8(x + 4);
          }
        }
        continue;
      }
      if (o.page < 0) continue;
      const int is_v = w >= kv_tasks, h0 = (is_v ? w - kv_tasks : w) * heads;
      const ItemAt at = item_at(it, is_v ? 0 : p.rot, p.interleaved);
      const int64_t stride = is_v ? p.v_stride : p.k_stride;
      const __nv_bfloat16* src = is_v ? p.v + o.row * p.v_stride : p.k + o.row * p.k_stride;
      const int slot = o.pos & ((1 << p.cache.lp) - 1);
      uint8_t* const codes = is_v ? p.cache.v : p.cache.k;
      uint8_t* const sfs = is_v ? p.cache.v_sf : p.cache.k_sf;
      const int held = o.pos & 15;  // earlier tokens of the block
      // item u of this lane: its head and token
      auto where = [&](int u, int& h, int& t) {
        const int idx = 32 * u + lane;
        h = h0 + (idx >> lhead);
        t = (idx & ((1 << lhead) - 1)) / IPR;
        return h < H && t < o.cnt;
      };
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        int h, t;
        if (where(u, h, t)) {
          copy16(stage + u * 512, src + t * stride + h * D + at.d0);
          copy16(stage + 2048 + u * 512, src + t * stride + h * D + at.d1);
        }
      }
      copies_wait();
      // largest magnitudes, a head at a time: `steps` steps of 32 items, or 32 / L heads a step
#pragma unroll 1
      for (int u0 = 0; u0 < 4; u0 += steps) {
        const int h = h0 + (32 * u0 + lane >> lhead);
        if (__all_sync(0xffffffffu, h >= H)) break;
        auto item = [&](int u, int t, uint64_t (&x)[8]) {
          unpack8(lds16(stage + u * 512), x);
          unpack8(lds16(stage + 2048 + u * 512), x + 4);
          if (at.pair >= 0) rotate_item(p.interleaved, angles(o.tab + t, at), x);
        };
        float amax = 0.0f;
#pragma unroll 1
        for (int u = u0; u < u0 + steps; ++u) {
          int hh, t;
          if (!where(u, hh, t)) continue;
          if (at.pair < 0) {
            amax = fmaxf(amax, raw_max(lds16(stage + u * 512), lds16(stage + 2048 + u * 512)));
          } else {
            uint64_t x[8];
            item(u, t, x);
            amax = fmaxf(amax, item_max(x));
          }
        }
        amax = head_max(amax, L);
        const bool inf = __any_sync(0xffffffffu, amax == INFINITY);
        if (inf) {  // again without what is not finite
          amax = 0.0f;
#pragma unroll 1
          for (int u = u0; u < u0 + steps; ++u) {
            int hh, t;
            if (!where(u, hh, t)) continue;
            uint64_t x[8];
            item(u, t, x);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float a, b;
              ptx::f2_unpack(x[i], a, b);
              if (fabsf(a) < INFINITY) amax = fmaxf(amax, fabsf(a));
              if (fabsf(b) < INFINITY) amax = fmaxf(amax, fabsf(b));
            }
          }
          amax = head_max(amax, L);
        }
        const uint32_t bits = __float_as_uint(amax);
        int code = max(0, static_cast<int>(bits >> 23) - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0));
        const int64_t row = cache_row(p.cache, o.page, min(h, H - 1), slot);
        uint8_t* const sf = sfs + (row >> 4);
        if (held > 0) {
          const int before = *sf;
          // where the scale grows the earlier tokens follow it, head by head
          uint32_t grow = __ballot_sync(0xffffffffu, h < H && before < code && lane % L == 0);
          const float f = sf_value(127 - min(max(code - before, 0), 126));
          while (grow) {
            const int from = __ffs(grow) - 1;
            grow &= grow - 1;
            const float ff = __shfl_sync(0xffffffffu, f, from);
            uint8_t* const old = codes + (__shfl_sync(0xffffffffu, row, from) - held) * D;
            for (int i = lane; i < held * IPR; i += 32) {
              uint4 x = *reinterpret_cast<uint4*>(old + 16 * i);
              x = make_uint4(rescale4(x.x, ff), rescale4(x.y, ff), rescale4(x.z, ff), rescale4(x.w, ff));
              *reinterpret_cast<uint4*>(old + 16 * i) = x;
            }
          }
          code = max(code, before);
          __syncwarp();  // every lane has read the scale
        }
        if (h < H && lane % L == 0) *sf = static_cast<uint8_t>(code);
        const float inv = sf_value(max(254 - code, 0));  // code <= 247 for what this kernel stored (amax < 2^128)
#pragma unroll 1
        for (int u = u0; u < u0 + steps; ++u) {
          int hh, t;
          if (!where(u, hh, t)) continue;
          uint64_t x[8];
          item(u, t, x);
          uint8_t* const to = codes + (row + t) * D;
          *reinterpret_cast<uint2*>(to + at.d0) = quantise8(x, inv, inf);
          *reinterpret_cast<uint2*>(to + at.d1) = quantise8(x + 4, inv, inf);
        }
      }
    }
    w -= tasks;
  }
}

}  // namespace gdpa
