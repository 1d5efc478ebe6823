// gdpa_cache_tile.cuh -- attention of many new rows over the paged e4m3 cache
// (pieces of prompts, candidates, many drafted tokens): 128 query rows of a
// key head at a time on the 5th-generation tensor cores.
//
// Mathematics.  Both products take fp16 operands.  e4m3 codes are fp16
// exactly, and a query row is divided by a power of two (as in the kernel for
// few rows).  K stays as codes: the scales of the 16-key blocks multiply the
// scores.  V is multiplied by its block's scale over 2^E, E the largest scale's
// exponent so far (raised when a block exceeds it by 7, the output following):
// exact while a block is less than 2^15 below it, and a block of other than
// zeros further below sends its segment to the plain form.  Weights are 2^(x - r)
// with a reference r 7 below the running maximum, moved when a score exceeds it
// by 15, and rounded to fp16, as in the kernel for few rows.  Sums stay in fp32;
// the row sum takes the weights before their rounding.
//
// Bound: the instruction issue (softmax and conversions), the tensor core and
// the special-function unit (512 cycles each of a 128 x 64 tile at D = 128)
// close behind.
//
// Work split.  Segments (sequence, 128 rows, key head) and runs as in the
// kernel for few rows, a CTA being the worker and 64 keys a step; a cut
// segment's parts are joined by the same second kernel.  Two CTAs an SM, each
// with 256 of the 512 TMEM columns, fill each other's gaps.  Roles:
//   warps 0-3  softmax, a query row a thread: load Q of the segment into
//              shared memory, then for every tile S -> P (over S in TMEM), and
//              the output;
//   warps 4-7  copy codes to shared memory a tile ahead, convert and store K
//              and V tiles (128-byte swizzle) in two stages;
//   warp 8     issues the MMAs, S one tile ahead of P V (warps 9-11 only give
//              their registers to the softmax).
//
// A value that is NaN must not reach rows that do not see its token, and 0
// times NaN is NaN: a segment with a NaN value in a tile that some row sees
// only in part takes the plain form too (row by row, after the other).
#pragma once

#include "gdpa_cache_fwd.cuh"

namespace gdpa {

template <int D_>
struct TileCfg {
  static constexpr int D = D_;
  static constexpr int THREADS = 384, WORKERS = 1;  // three warpgroups
  static constexpr int START = 3, RUN_STEPS = 8;
  static constexpr int ROWS = 128, SPAN = 64;
  static constexpr int CTAS = 2;
  static constexpr int CHUNKS = D / 64;              // 128-byte column chunks
  static constexpr int Q_CHUNK = ROWS * 128, KV_CHUNK = SPAN * 128;
  static constexpr int Q_BYTES = CHUNKS * Q_CHUNK, KV_BYTES = CHUNKS * KV_CHUNK;
  static constexpr int OFF_K = Q_BYTES, OFF_V = OFF_K + 2 * KV_BYTES;
  static constexpr int OFF_RAW = OFF_V + 2 * KV_BYTES;   // codes of the next tile, K then V
  static constexpr int RAW = SPAN * D;
  // the barrier block behind it; two CTAs an SM and no more, for the TMEM's sake
  static constexpr int USED = OFF_RAW + 2 * RAW + 1024;
  static constexpr int SMEM = USED > 98 * 1024 ? USED : 98 * 1024;
  // registers a thread after the warpgroups have traded them: together what
  // the launch allocates, three times LAUNCH_REGS
  static constexpr int LAUNCH_REGS = 80, REGS_SOFTMAX = 128, REGS_CONVERT = 72, REGS_MMA = 40;
  static_assert(REGS_SOFTMAX + REGS_CONVERT + REGS_MMA <= 3 * LAUNCH_REGS, "registers");
  static constexpr uint32_t TM_S = 0, TM_O = 128, TM_COLS = 256;  // two S buffers of 64 columns, O
  static_assert(2 * (SMEM + 1024) <= 228 * 1024, "two CTAs an SM");
};

namespace tile {

struct Bars {
  uint64_t q_full, k_full[2], k_free[2], v_full[2], v_free[2], s_full[2], p_full[2];
  uint64_t pv_done;  // after every P V
  uint64_t o_full;   // after a segment's last
  uint64_t drain;
  uint32_t tmem;
  int abort;
};

// What the converting warps tell the softmax of tile i, in a ring of four: the
// refill of an entry waits for S(i + 2), which waits for P(i).
struct Notes {
  float k_scale[4][4];  // of the tile's blocks; -1: no page, hidden from all rows
  int plain[4][4];      // a warp found what only the plain form takes
  int exponent[4];      // E
};

// One row of a segment over keys [j0, j1), one warp, D / 32 coordinates a lane:
// the plain form, for segments that the tensor core cannot take.
template <int D>
__device__ __noinline__ void attend_row(const CacheFwdParams& p, int b, int h, int64_t q_at, int j0, int j1,
                                        float& top, float& total, float* o) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  float q[E], m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = __bfloat162float(p.q[q_at + lane * E + e]);
    o[e] = 0.0f;
  }
#pragma unroll 1
  for (int j = j0; j < j1; ++j) {
    const int page = load_page(p.cache, p.batch, b, j);
    if (page < 0) continue;
    const int slot = j & ((1 << p.cache.lp) - 1);
    const int64_t row = cache_row(p.cache, page, h, slot), at = row * D + lane * E;
    float x = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) x += q[e] * e4m3_to_float(p.cache.k[at + e]);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    x = x * sf_value(p.cache.k_sf[row >> 4]) * p.scale2;
    const float up = fmaxf(m, x), zero = up == -INFINITY ? 0.0f : up;
    const float keep = ptx::ex2_approx(m - zero), w = ptx::ex2_approx(x - zero);
    const float sv = sf_value(p.cache.v_sf[row >> 4]);
    l = l * keep + w;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * keep + w * (e4m3_to_float(p.cache.v[at + e]) * sv);
    m = up;
  }
  top = m;
  total = l;
}

// Where a segment's results go: `out`, or the worker's part of it.
struct Target {
  int pieces;
  float* part;
};
template <class C>
__device__ __forceinline__ Target target(const CacheFwdParams& p, const split::Walk<C>& w, int64_t chunk, int worker) {
  Target r;
  const int64_t unit0 = w.start + C::START;
  const int first = static_cast<int>(unit0 / chunk);
  r.pieces = p.no_split ? 1 : static_cast<int>((unit0 + w.w.steps - 1) / chunk) - first + 1;
  const int slot = first == worker ? 1 : 0;
  r.part = p.part + (static_cast<int64_t>(worker) * 2 + slot) * C::ROWS * (C::D + 2);
  if (r.pieces > 1 && threadIdx.x == 0) {
    int* m = p.meta + worker * 16 + slot * 8;
    m[0] = first, m[1] = r.pieces, m[2] = w.w.s.first, m[3] = w.w.s.n, m[4] = w.tile, m[5] = w.h;
  }
  return r;
}

// ------------------------------------------------------------------ softmax
template <int D>
__device__ void run_softmax(const CacheFwdParams& p, uint8_t* sm, Bars& B, const Notes& notes, uint32_t tmem,
                            const split::Schedule<TileCfg<D>>& sh, int64_t at, int64_t stop, int64_t chunk,
                            unsigned long long limit) {
  using C = TileCfg<D>;
  const int lane = threadIdx.x & 31, quarter = threadIdx.x >> 5, r = threadIdx.x;
  const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
  const uint32_t o_addr = tmem + lane_off + C::TM_O;
  volatile int* abort = &B.abort;
  split::Walk<C> w;
  w.begin(p, sh.seq[0], sh.base[0], at);
  uint32_t gi = 0, seg = 0;  // tiles, and segments with tiles, so far
  bool ok = true;
#pragma unroll 1
  for (; ok && w.more(p, stop); w.next(p)) {
    if (!w.enter(p, at, stop)) continue;
    const CacheSeq s = w.w.s;
    const Target to = target<C>(p, w, chunk, blockIdx.x);
    const int64_t rr = w.row0 + r;
    const bool valid = r < w.rows;
    const int head = w.h * p.G + static_cast<int>(rr % p.G);
    const int64_t q_at = (s.first + rr / p.G) * p.q_stride + static_cast<int64_t>(head) * D;
    const int64_t out_row = (s.first + rr / p.G) * p.Hq + head;
    const int pos = s.len - s.n + static_cast<int>(rr / p.G);
    // keys this row sees: [lo, hi)
    const int lo = p.window > 0 ? max(0, pos - p.window + 1) : 0;
    const int hi = valid ? max(0, p.causal ? min(s.len, pos + 1) : s.len) : 0;
    const int steps = w.u1 - w.u0;
    float m = -INFINITY, l = 0.0f;
    bool dirty = false;
    int exponent = 0;
    if (steps > 0) {
      // ---- this row of Q, divided by its largest power of two, as fp16
      // (read twice: registers are short, the row is in L1)
      const uint4* src = reinterpret_cast<const uint4*>(p.q + q_at);
      float amax = 0.0f;
#pragma unroll 4
      for (int i = 0; i < D / 8; ++i) {
        const uint4 u = valid ? src[i] : make_uint4(0, 0, 0, 0);
        const uint32_t x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          amax = fmaxf(amax, fabsf(__uint_as_float(x[e] << 16)));
          amax = fmaxf(amax, fabsf(__uint_as_float(x[e] & 0xffff0000u)));
        }
      }
      const int e2 = amax > 0.0f ? min(max(static_cast<int>(__float_as_uint(amax) >> 23) - 127, -126), 127) : 0;
      const float inv = sf_value(127 - e2), fac = sf_value(127 + e2) * p.scale2;
      const uint32_t q_smem = ptx::smem_u32(sm);
#pragma unroll 4
      for (int i = 0; i < D / 8; ++i) {
        const uint4 u = valid ? src[i] : make_uint4(0, 0, 0, 0);
        const uint32_t x[4] = {u.x, u.y, u.z, u.w};
        uint32_t y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          y[e] = split::pack_f16x2(__uint_as_float(x[e] << 16) * inv, __uint_as_float(x[e] & 0xffff0000u) * inv);
        ptx::st_shared_v4(q_smem + (i >> 3) * C::Q_CHUNK + r * 128 + (((i & 7) ^ (r & 7)) << 4), y[0], y[1], y[2], y[3]);
      }
      ptx::fence_proxy_async_smem();
      ptx::mbar_arrive(&B.q_full);

      const bool live = quarter * 32 < w.rows;  // a warp without rows keeps the barriers' protocol
      const bool fold = p.scale2 > 0.0f;
#pragma unroll 1
      for (int i = 0; i < steps; ++i, ++gi) {
        const int sb = gi & 1;
        ok = ptx::mbar_wait(&B.s_full[sb], (gi >> 1) & 1, limit, abort);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        ptx::tc_fence_after();
        if (live) {
          const int kb = w.w.kbase + (w.u0 + i) * C::SPAN;
          const uint32_t s_addr = tmem + lane_off + C::TM_S + sb * 64;
          uint32_t sr[64];
          ptx::tmem_ld32(s_addr, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
          ptx::tmem_ld32(s_addr + 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[32]));
          float f[4];
          uint32_t gone = 0;  // blocks on no page
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float sk = *const_cast<volatile const float*>(&notes.k_scale[gi & 3][j]);
            gone |= sk < 0.0f ? 1u << j : 0u;
            f[j] = fac * sk;
            dirty |= *const_cast<volatile const int*>(&notes.plain[gi & 3][j]) != 0;
          }
          const int e_now = *const_cast<volatile const int*>(&notes.exponent[gi & 3]);
          ptx::tmem_wait_ld_r64(sr);
          float mx = -INFINITY;
          const bool edge = kb < w.lo_max || kb > w.hi_min - C::SPAN || gone != 0 || !fold;
          if (!edge) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              float a = __uint_as_float(sr[16 * j]), c = __uint_as_float(sr[16 * j + 1]);
#pragma unroll
              for (int u = 2; u < 16; u += 4) {
                a = ptx::max3(a, __uint_as_float(sr[16 * j + u]), __uint_as_float(sr[16 * j + u + 1]));
                if (u + 3 < 16) c = ptx::max3(c, __uint_as_float(sr[16 * j + u + 2]), __uint_as_float(sr[16 * j + u + 3]));
              }
              mx = fmaxf(mx, fmaxf(a, c) * f[j]);
            }
          } else {
#pragma unroll
            for (int u = 0; u < 64; ++u) {
              float x = __uint_as_float(sr[u]) * f[u >> 4];
              const int key = kb + u;
              if (key < lo || key >= hi || (gone >> (u >> 4) & 1)) x = -INFINITY;
              sr[u] = __float_as_uint(x);
              mx = fmaxf(mx, x);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) f[j] = 1.0f;
          }
          // the reference moves when a score exceeds it by 15, to 7 below it;
          // the output follows, once P V of the last tile is in (where nothing
          // was added yet there is nothing to follow)
          float alpha = 1.0f;
          bool follow = false;
          if (mx > m + 15.0f || m == -INFINITY) {
            const float up = fmaxf(m, mx - 7.0f);
            alpha = m == -INFINITY ? 0.0f : ptx::ex2_approx(m - up);
            follow = i > 0 && l != 0.0f;
            l *= alpha;
            m = up;
          }
          if (i > 0 && e_now != exponent) {  // so it does V's exponent
            alpha *= exponent - e_now < -126 ? 0.0f : sf_value(127 + exponent - e_now);
            follow = l != 0.0f || follow;
          }
          exponent = e_now;
          if (__any_sync(0xffffffffu, follow)) {
            // S of this tile came after P V of the tile before the last, so
            // that pv_done is in the phase waited for, or has left it
            ok = ptx::mbar_wait(&B.pv_done, (gi - 1) & 1, limit, abort);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            ptx::tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              uint32_t o[16];
              ptx::tmem_ld16(o_addr + c, o);
              ptx::tmem_wait_ld();
#pragma unroll
              for (int u = 0; u < 16; ++u)
                if (follow) o[u] = __float_as_uint(__uint_as_float(o[u]) * alpha);
              ptx::tmem_st16(o_addr + c, o);
            }
          }
          const float neg = m == -INFINITY ? 0.0f : -m;
          uint64_t add[2] = {0, 0};
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t pk[16];
#pragma unroll
            for (int u = 0; u < 16; ++u) {
              const int v = 16 * half + u;
              const float a = ptx::ex2_approx(fmaf(__uint_as_float(sr[2 * v]), f[v >> 3], neg));
              const float c = ptx::ex2_approx(fmaf(__uint_as_float(sr[2 * v + 1]), f[v >> 3], neg));
              add[u & 1] = ptx::f2_add(add[u & 1], ptx::f2_pack(a, c));
              pk[u] = split::pack_f16x2(a, c);
            }
            ptx::tmem_st16(s_addr + 16 * half, pk);
          }
          float x, y;
          ptx::f2_unpack(ptx::f2_add(add[0], add[1]), x, y);
          l += x + y;
          ptx::tmem_wait_st();
        }
        ptx::tc_fence_before();
        ptx::mbar_arrive(&B.p_full[sb]);
      }
      if (!ok) break;
      ok = ptx::mbar_wait(&B.o_full, seg++ & 1, limit, abort);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      ptx::tc_fence_after();
    }
    // ---- the result
    if (quarter * 32 >= w.rows) continue;
    if (__any_sync(0xffffffffu, dirty)) {
      const int k0 = w.w.kbase + w.u0 * C::SPAN, k1 = w.w.kbase + w.u1 * C::SPAN;
#pragma unroll 1
      for (int row = 0; row < 32 && quarter * 32 + row < w.rows; ++row) {
        constexpr int E = D / 32;
        float top, total, o[E];
        const int64_t row_q = __shfl_sync(0xffffffffu, q_at, row), row_o = __shfl_sync(0xffffffffu, out_row, row);
        attend_row<D>(p, w.b, w.h, row_q, max(k0, __shfl_sync(0xffffffffu, lo, row)),
                      min(k1, __shfl_sync(0xffffffffu, hi, row)), top, total, o);
        const float inv = total == 0.0f ? 0.0f : 1.0f / total;
        const int at_row = quarter * 32 + row;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          if (to.pieces == 1)
            p.out[row_o * D + lane * E + e] = __float2bfloat16_rn(o[e] * inv);
          else
            to.part[2 * C::ROWS + at_row * D + lane * E + e] = o[e];
        }
        if (lane == 0) {
          if (to.pieces > 1)
            to.part[2 * at_row] = top, to.part[2 * at_row + 1] = total;
          else if (p.lse)
            p.lse[row_o] = total == 0.0f ? -INFINITY : (top + log2f(total)) * 0.6931471805599453f;
        }
      }
      continue;
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l, unit = sf_value(min(max(127 + exponent, 0), 254));
#pragma unroll 1
    for (int c = 0; c < D; c += 32) {
      uint32_t o[32];
      if (steps > 0) {
        ptx::tmem_ld32(o_addr + c, o);
        ptx::tmem_wait_ld_r32(o);
      }
      if (steps == 0 || l == 0.0f) {  // nothing was seen
#pragma unroll
        for (int u = 0; u < 32; ++u) o[u] = 0;
      }
      if (!valid) continue;
      if (to.pieces == 1) {
        uint4* dst = reinterpret_cast<uint4*>(p.out + out_row * D + c);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          uint32_t y[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            y[e] = ptx::pack_bf16x2(__uint_as_float(o[8 * u + 2 * e]) * inv * unit,
                                    __uint_as_float(o[8 * u + 2 * e + 1]) * inv * unit);
          dst[u] = make_uint4(y[0], y[1], y[2], y[3]);
        }
      } else {
        uint4* dst = reinterpret_cast<uint4*>(to.part + 2 * C::ROWS + r * D + c);
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          uint32_t y[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) y[e] = __float_as_uint(__uint_as_float(o[4 * u + e]) * unit);
          dst[u] = make_uint4(y[0], y[1], y[2], y[3]);
        }
      }
    }
    if (valid) {
      if (to.pieces > 1)
        to.part[2 * r] = m, to.part[2 * r + 1] = l;
      else if (p.lse)
        p.lse[out_row] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
    }
    ptx::tc_fence_before();  // O has been read when the next segment's P allows its first product
  }
  if (!ok && lane == 0) {
    *abort = 1;
    atomicOr(p.batch.status, kStatusActivation);
  }
}

// ------------------------------------------------------------------ conversion
template <int D>
__device__ void run_convert(const CacheFwdParams& p, uint8_t* sm, Bars& B, Notes& notes,
                            const split::Schedule<TileCfg<D>>& sh, int64_t at, int64_t stop,
                            unsigned long long limit) {
  using C = TileCfg<D>;
  constexpr int CPR = D / 16;               // 16-code chunks of a row
  constexpr int RPI = 128 / CPR;            // rows that 128 threads read at once
  constexpr int NI = C::SPAN / RPI;         // ... and how often for a tile
  const int tid = threadIdx.x - 128, lane = tid & 31, warp = tid >> 5;
  const int c = tid % CPR, r0 = tid / CPR;
  volatile int* abort = &B.abort;
  const int pmask = (1 << p.cache.lp) - 1;
  split::Walk<C> w;
  w.begin(p, sh.seq[0], sh.base[0], at);
  bool entered = false, more = true, first = true;  // first: of its segment
  int u = 0;  // the tile that is being read
  auto advance = [&]() {
    ++u;
    first = false;
    while (!entered || u >= w.u1) {
      if (entered) w.next(p);
      entered = false;
      while (w.more(p, stop) && !w.enter(p, at, stop)) w.next(p);
      if (!w.more(p, stop)) {
        more = false;
        return;
      }
      entered = true;
      first = true;
      u = w.u0;
    }
  };
  // Starts the copies of this thread's chunks of the tile's codes (tokens that
  // no row sees may hold anything: zeros), and reads its blocks' scale codes
  // (K's in the low byte, V's in the next; -1: no page).
  const uint32_t raw = ptx::smem_u32(sm + C::OFF_RAW) + tid * 16;
  int sf[4];
  auto fetch = [&]() {
    if (more) {
      const int kb = w.w.kbase + u * C::SPAN;
      const int32_t* table = p.batch.table + static_cast<int64_t>(w.b) * p.batch.max_pages;
      int64_t row[4];
      int page = -1;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int block = kb + kCacheBlock * j;
        sf[j] = -1;
        row[j] = -1;
        if (block < w.hi_max && block + kCacheBlock > w.lo_min) {
          if (page < 0 || (block & pmask) == 0) page = __ldg(table + (block >> p.cache.lp));
          if (page >= 0 && page < p.cache.num_pages) {
            row[j] = cache_row(p.cache, page, w.h, block & pmask);
            sf[j] = p.cache.k_sf[row[j] >> 4] | p.cache.v_sf[row[j] >> 4] << 8;
          } else {
            page = -1;
            if (tid == 0) atomicOr(p.batch.status, kStatusBadPlan);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < NI; ++j) {
        const int in = r0 + RPI * j, key = kb + in;  // RPI is 16 or 32: in >> 4 is j, or 2 j + (r0 >> 4)
        const int64_t block = RPI == 16 ? row[j & 3] : r0 >= 16 ? row[(2 * j + 1) & 3] : row[(2 * j) & 3];
        const bool there = block >= 0 && key < w.hi_max && key >= w.lo_min;
        const int64_t off = ((block >= 0 ? block : 0) + (in & 15)) * D + 16 * c;
        split::cp_async16(raw + j * 2048, p.cache.k + off, there ? 16 : 0);
        split::cp_async16(raw + C::RAW + j * 2048, p.cache.v + off, there ? 16 : 0);
      }
    }
    split::cp_commit();
  };
  // 16 codes of row r as two 16-byte pieces of the swizzled tile, in an order
  // that keeps the eight lanes of a row on different banks
  auto put = [&](uint32_t base, int r, const uint32_t (&x)[8]) {
    const uint32_t row = base + (c >> 2) * C::KV_CHUNK + r * 128;
    const int swap = c >> 2 & 1;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int e = h ^ swap;
      const uint32_t dst = row + (((2 * (c & 3) + e) ^ (r & 7)) << 4);
      if (e == 0)
        ptx::st_shared_v4(dst, x[0], x[1], x[2], x[3]);
      else
        ptx::st_shared_v4(dst, x[4], x[5], x[6], x[7]);
    }
  };
  uint32_t gi = 0;
  bool ok = true;
  int exponent = 0;
  advance();
  fetch();
#pragma unroll 1
  for (; ok && more; ++gi) {
    const int st = gi & 1;
    const uint32_t par = ((gi >> 1) & 1) ^ 1;
    ok = ptx::mbar_wait(&B.k_free[st], par, limit, abort);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) break;
    split::cp_wait<0>();  // this thread's own copies
    uint4 kr[NI], vr[NI];
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      uint32_t x[4];
      split::lds128(raw + j * 2048, x);
      kr[j] = make_uint4(x[0], x[1], x[2], x[3]);
      split::lds128(raw + C::RAW + j * 2048, x);
      vr[j] = make_uint4(x[0], x[1], x[2], x[3]);
    }
    // V's exponent E
    int top = -1000;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (sf[j] >= 0) top = max(top, (sf[j] >> 8) - 127);
    if (top > -1000 && (first || exponent == -1000 || top > exponent + 7)) exponent = top;
    else if (first) exponent = -1000;  // nothing is there yet
    const int kb = w.w.kbase + u * C::SPAN;
    const bool edge = kb < w.lo_max || kb > w.hi_min - C::SPAN;
    bool plain = false;
    const uint32_t k_at = ptx::smem_u32(sm + C::OFF_K + st * C::KV_BYTES);
    uint32_t sv[NI];  // V's scale over 2^E, twice in fp16
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      const uint32_t x[4] = {kr[j].x, kr[j].y, kr[j].z, kr[j].w};
      uint32_t y[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) y[2 * e] = split::codes_lo(x[e]), y[2 * e + 1] = split::codes_hi(x[e]);
      put(k_at, r0 + RPI * j, y);
      const int f = RPI == 16 ? sf[j & 3] : r0 >= 16 ? sf[(2 * j + 1) & 3] : sf[(2 * j) & 3];
      const int up = f < 0 ? 0 : (f >> 8) - 127 - exponent;  // at most 7
      sv[j] = up < -14 ? 0x00010001u << max(up + 24, 0) : static_cast<uint32_t>(up + 15) * 0x04000400u;
      // one thread of each block notes its scale
      if (c == 0 && ((r0 + RPI * j) & (kCacheBlock - 1)) == 0)
        notes.k_scale[gi & 3][(r0 + RPI * j) >> 4] = f < 0 ? -1.0f : sf_value(f & 0xff);
      const uint32_t z[4] = {vr[j].x, vr[j].y, vr[j].z, vr[j].w};
      plain |= static_cast<bool>((up < -15) & (((z[0] | z[1] | z[2] | z[3]) & 0x7f7f7f7fu) != 0));
      if (edge) {
#pragma unroll
        for (int e = 0; e < 4; ++e) plain |= split::has_nan_code(z[e]);
      }
    }
    plain = __any_sync(0xffffffffu, plain);
    if (lane == 0) notes.plain[gi & 3][warp] = plain;
    if (tid == 0) notes.exponent[gi & 3] = exponent;
    ptx::fence_proxy_async_smem();
    ptx::mbar_arrive(&B.k_full[st]);
    advance();
    fetch();
    ok = ptx::mbar_wait(&B.v_free[st], par, limit, abort);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) break;
    const uint32_t v_at = ptx::smem_u32(sm + C::OFF_V + st * C::KV_BYTES);
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      const uint32_t x[4] = {vr[j].x, vr[j].y, vr[j].z, vr[j].w};
      uint32_t y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t h2 = e & 1 ? split::codes_hi(x[e >> 1]) : split::codes_lo(x[e >> 1]);
        asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(y[e]) : "r"(h2), "r"(sv[j]));
      }
      put(v_at, r0 + RPI * j, y);
    }
    ptx::fence_proxy_async_smem();
    ptx::mbar_arrive(&B.v_full[st]);
  }
  split::cp_wait<0>();
  if (!ok && lane == 0) {
    *abort = 1;
    atomicOr(p.batch.status, kStatusProducer);
  }
}

// ------------------------------------------------------------------ MMA
template <int D>
__device__ __forceinline__ bool issue_pv(Bars& B, uint8_t* sm, uint32_t tmem, uint32_t gi, bool first,
                                         unsigned long long limit) {
  using C = TileCfg<D>;
  const int st = gi & 1;
  const uint32_t par = (gi >> 1) & 1;
  volatile int* abort = &B.abort;
  if (!ptx::mbar_wait(&B.p_full[st], par, limit, abort)) return false;
  if (!ptx::mbar_wait(&B.v_full[st], par, limit, abort)) return false;
  ptx::tc_fence_after();
  const uint32_t v_base = ptx::smem_u32(sm + C::OFF_V + st * C::KV_BYTES);
  constexpr uint32_t idesc = ptx::idesc_f16(128, D, 1);
#pragma unroll
  for (int kk = 0; kk < C::SPAN / 16; ++kk)
    // V is MN-major: 16 keys = two 8-row groups 1024 B apart; 64-column chunks KV_CHUNK apart
    ptx::mma_ts_elect(tmem + C::TM_O, tmem + C::TM_S + st * 64 + 8 * kk,
                      ptx::sdesc_sw128(v_base + kk * 2048, C::KV_CHUNK, 1024), idesc, first && kk == 0 ? 0u : 1u);
  ptx::mma_commit_elect(&B.v_free[st]);
  ptx::mma_commit_elect(&B.pv_done);
  return true;
}

template <int D>
__device__ void run_mma(const CacheFwdParams& p, uint8_t* sm, Bars& B, uint32_t tmem,
                        const split::Schedule<TileCfg<D>>& sh, int64_t at, int64_t stop, unsigned long long limit) {
  using C = TileCfg<D>;
  volatile int* abort = &B.abort;
  split::Walk<C> w;
  w.begin(p, sh.seq[0], sh.base[0], at);
  uint32_t gi = 0, seg = 0;
  bool ok = true;
  const uint32_t q_base = ptx::smem_u32(sm);
  constexpr uint32_t idesc = ptx::idesc_f16(128, C::SPAN, 0);
#pragma unroll 1
  for (; ok && w.more(p, stop); w.next(p)) {
    if (!w.enter(p, at, stop) || w.u1 <= w.u0) continue;
    ok = ptx::mbar_wait(&B.q_full, seg++ & 1, limit, abort);
    const int steps = w.u1 - w.u0;
#pragma unroll 1
    for (int i = 0; ok && i < steps; ++i, ++gi) {
      const int st = gi & 1;
      ok = ptx::mbar_wait(&B.k_full[st], (gi >> 1) & 1, limit, abort);
      if (!ok) break;
      ptx::tc_fence_after();
      const uint32_t k_base = ptx::smem_u32(sm + C::OFF_K + st * C::KV_BYTES);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        ptx::mma_ss_elect(tmem + C::TM_S + st * 64,
                          ptx::sdesc_sw128(q_base + (kk >> 2) * C::Q_CHUNK + (kk & 3) * 32, 16, 1024),
                          ptx::sdesc_sw128(k_base + (kk >> 2) * C::KV_CHUNK + (kk & 3) * 32, 16, 1024), idesc,
                          kk > 0 ? 1u : 0u);
      ptx::mma_commit_elect(&B.s_full[st]);
      ptx::mma_commit_elect(&B.k_free[st]);
      if (i > 0) ok = issue_pv<D>(B, sm, tmem, gi - 1, i == 1, limit);
    }
    if (ok) ok = issue_pv<D>(B, sm, tmem, gi - 1, steps == 1, limit);
    ptx::mma_commit_elect(&B.o_full);
  }
  if (!ok && (threadIdx.x & 31) == 0) {
    *abort = 1;
    atomicOr(p.batch.status, kStatusMma);
  }
  // every MMA this warp issued is complete once this commit lands
  ptx::mma_commit_elect(&B.drain);
  const int never = 0;
  ptx::mbar_wait(&B.drain, 0, 100000000ull, &never);
}

}  // namespace tile

template <int D>
__global__ void __launch_bounds__(384, 2) gdpa_cache_tile_kernel(const CacheFwdParams p, unsigned long long limit) {
  using C = TileCfg<D>;
  // All of it dynamic: two CTAs take the SM's last byte.  Nothing static in
  // front of it, so that it begins on the 1024 bytes that the swizzle wants.
  extern __shared__ __align__(1024) uint8_t sm[];
  struct Block {
    tile::Bars bars;
    tile::Notes notes;
    split::Schedule<C> schedule;
  };
  static_assert(sizeof(Block) <= 1024, "barrier block");
  Block& block = *reinterpret_cast<Block*>(sm + C::OFF_RAW + 2 * C::RAW);
  tile::Bars& B = block.bars;
  tile::Notes& notes = block.notes;
  split::Schedule<C>& sh = block.schedule;
  if (ptx::smem_u32(sm) & 1023u) {
    if (threadIdx.x == 0) atomicOr(p.batch.status, kStatusProducer);
    return;
  }
  const int tid = threadIdx.x, warp = tid >> 5;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid == 0 && !p.no_split) p.meta[blockIdx.x * 16 + 1] = p.meta[blockIdx.x * 16 + 9] = 0;  // no parts yet
  if (tid == 0) {
    ptx::mbar_init(&B.q_full, 128);
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&B.k_full[i], 128);
      ptx::mbar_init(&B.k_free[i], 1);
      ptx::mbar_init(&B.v_full[i], 128);
      ptx::mbar_init(&B.v_free[i], 1);
      ptx::mbar_init(&B.s_full[i], 1);
      ptx::mbar_init(&B.p_full[i], 128);
    }
    ptx::mbar_init(&B.pv_done, 1);
    ptx::mbar_init(&B.o_full, 1);
    ptx::mbar_init(&B.drain, 1);
    B.abort = 0;
    ptx::fence_mbar_init();
  }
  int64_t total, chunk;
  split::schedule<C>(p, sh, total, chunk);  // synchronises: the barriers are there
  const int64_t at = chunk * blockIdx.x, stop = min(total, at + chunk);
  if (at >= stop) return;
  if (warp == 8) {
    ptx::tmem_alloc(&B.tmem, C::TM_COLS);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = B.tmem;
  if (warp < 4) {
    ptx::regs_inc<C::REGS_SOFTMAX>();
    tile::run_softmax<D>(p, sm, B, notes, tmem, sh, at, stop, chunk, limit);
  } else if (warp < 8) {
    ptx::regs_dec<C::REGS_CONVERT>();
    tile::run_convert<D>(p, sm, B, notes, sh, at, stop, limit);
  } else {
    ptx::regs_dec<C::REGS_MMA>();
    if (warp == 8) tile::run_mma<D>(p, sm, B, tmem, sh, at, stop, limit);
  }
  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == 8) ptx::tmem_dealloc(tmem, C::TM_COLS);
}

}  // namespace gdpa
