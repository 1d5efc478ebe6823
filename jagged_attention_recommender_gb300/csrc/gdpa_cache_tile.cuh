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
// zeros further below sends its segment to the plain form: row by row, a warp
// each, 1400 times as slow (2321 prompt rows with one such block: 360 ms).
// Weights are 2^(x - r) with a reference r 7 below the running maximum, moved when
// a score exceeds it by 15, and rounded to fp16, as in the kernel for few rows.
// Sums stay in fp32; the row sum takes the weights before their rounding.
//
// Bound: the chain of hand-overs between the roles.  The tensor core and the
// special-function unit each need about 1050 cycles for 256 rows and 64 keys at
// D = 128 and a step takes about 2000: 258 to 277 us on different boards (746 to
// 695 TFLOP/s) for 2321 rows of prompts behind 2100 to 8192 keys, 32 query and 8
// key heads of 128.  With a
// softmax that only hands over 194 us are left, with an eighth of S's and a
// quarter of P V's MMAs as well 157.
//
// Work split.  Segments (sequence, 256 rows, key head) and runs as in the
// kernel for few rows, a CTA being the worker and 64 keys a step; a cut
// segment's parts are joined by the same second kernel.  A CTA works on two
// halves of 128 rows.  Where a segment has more than 128 rows they are its
// first and second 128, and every converted tile serves both; where it has
// fewer, both hold the same rows and take every other tile, and the second half
// hands its result to the first through shared memory.  Roles:
//   warps 0-3, 4-7    softmax of a half, a query row a thread: load Q, then for
//                     every tile S -> P (over S in TMEM), and the output;
//   warps 8-11        convert K tiles (128-byte swizzle, two stages);
//   warps 12-15       convert V tiles;
//   warp 16           issues the MMAs of S;
//   warp 18           issues those of P V (one warp for both was the longest
//                     of all chains: 297 us);
//   warp 17           finds pages and scales, and brings codes to shared memory
//                     by bulk copies, RAWS tiles ahead.
// (Conversion by the warps that also looked up pages and copied, one tile ahead
// and two CTAs of 128 rows an SM, took 435 us.  Results written by way of shared
// memory, whole lines at a time, took 8 us more than a row a thread.)
//
// A value that is NaN must not reach rows that do not see its token, and 0
// times NaN is NaN: a segment with a NaN value in a tile that some row sees
// only in part takes the plain form too (row by row, after the other).
#pragma once

#include "gdpa_cache_fwd.cuh"

namespace gdpa {

namespace ptx {

// Announces bytes without arriving.
__device__ __forceinline__ void mbar_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}

// Untiled bulk copy global -> shared (both 16-byte aligned, whole 16 bytes),
// completion counted in bytes on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t smem_dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_dst),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// Instruction descriptor, kind::f16: fp16 A and B, fp32 accumulator.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, int b_mn_major) {
  return (1u << 4) | (static_cast<uint32_t>(b_mn_major) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

}  // namespace ptx

template <int D_>
struct TileCfg {
  static constexpr int D = D_;
  static constexpr bool TEAM = false;
  static constexpr int THREADS = 640, WORKERS = 1;  // five warpgroups
  // What a segment's start and end cost, in steps (48 sequences of 500 to 6001
  // keys, 128 rows: 111 us with 16 at D = 128, 120 with 8; 76 with 8 at D = 64, 82
  // with 16), and the fewest that are worth a part.
  static constexpr int START = D == 128 ? 16 : 8, RUN_STEPS = START + 4;
  static constexpr int HALF = 128, ROWS = 2 * HALF, SPAN = 64;
  static constexpr int CTAS = 1;
  static constexpr int Q_CHUNK = HALF * 128, KV_CHUNK = SPAN * 128;  // 64 columns of a tile
  static constexpr int Q_BYTES = D / 64 * Q_CHUNK, KV_BYTES = D / 64 * KV_CHUNK;
  static constexpr int RAW = SPAN * D;      // codes of a tile of K or V
  static constexpr int RAWS = D == 64 ? 8 : 5;
  static constexpr int OFF_K = 2 * Q_BYTES, OFF_V = OFF_K + 2 * KV_BYTES, OFF_RAW = OFF_V + 2 * KV_BYTES;
  static constexpr int OFF_BLOCK = OFF_RAW + RAWS * 2 * RAW;  // barriers and notes
  static constexpr int USED = OFF_BLOCK + 3072;
  // one CTA an SM (all of its TMEM)
  static constexpr int SMEM = USED > 120 * 1024 ? USED : 120 * 1024;
  static constexpr uint32_t TM_S = 0, TM_O = 256, TM_COLS = 512;  // S: half, buffer, 64 columns; O: half, 128
  // registers a thread after the warpgroups have traded them: together what
  // the launch allocates, five times LAUNCH_REGS
  static constexpr int LAUNCH_REGS = 96, REGS_SOFTMAX = 144, REGS_CONVERT = 64, REGS_ISSUE = 64;
  static_assert(2 * REGS_SOFTMAX + 2 * REGS_CONVERT + REGS_ISSUE <= 5 * LAUNCH_REGS, "registers");
  static_assert(SMEM <= 227 * 1024, "shared memory");
  static_assert(2 * Q_BYTES >= HALF * D * 4, "a half's output fits Q's room");
};

namespace tile {

// What the roles of a CTA tell one another while they wait.
struct Watch {
  int abort;  // a wait has given up
  int turns;  // steps of the plain form that warps have taken
};

struct Bars {
  uint64_t raw_full[8], raw_free[8];
  uint64_t q_full, k_full[2], k_free[2], v_full[2], v_free[2];
  uint64_t s_full[2][2], p_full[2][2], pv_done[2][2];  // of a half and S buffer
  uint64_t o_full;                                  // after a segment's last P V
  uint64_t x_full, x_free;                          // the second half's result is there, is read
  uint64_t drain[2];
  uint32_t tmem;
  Watch watch;
};

// ptx::mbar_wait for the roles of a CTA.  A segment in the plain form takes
// hundreds of times as long as its tiles, and every role may wait for it: the
// limit is on the time in which no warp gets on with it.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, uint64_t limit_ns, const volatile Watch* watch) {
  if (ptx::mbar_test_wait(bar, parity)) return true;
  if (ptx::mbar_try_wait(bar, parity)) return true;
  uint64_t t0 = ptx::global_timer_ns();
  int turns = watch->turns;
  while (true) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    if (watch->abort) return false;
    const uint64_t now = ptx::global_timer_ns();
    const int at = watch->turns;
    if (at != turns) {
      turns = at;
      t0 = now;
    } else if (now - t0 > limit_ns) {
      return false;
    }
  }
}

// Beside the codes of a tile, in their ring.
struct __align__(16) RawNote {
  float k_scale[4];   // of its blocks; -1: no page, or nobody sees it
  uint32_t v_mul[4];  // V's scale over 2^E, twice in fp16; 0: none
  uint32_t state;     // bit 0 it exists, 1 the first of its segment, 2 some row sees only part of it,
                      // 3 all of V's codes and scales are plain to use
  int exponent;       // E
  int kb, lo, hi;     // its first key; keys that any row sees
  uint32_t low;       // bit j: block j's scale is too far below 2^E for that
};

struct Notes {
  RawNote raw[8];
  // For the softmax of tile i, in a ring of eight: the refill of an entry waits
  // for S(i + 6), which waits for P V of tile i + 2 of this half at least.
  float4 k_scale[8];
  int exponent[8];
  // Segments of this CTA, in a ring: some tile takes the plain form.  Entries
  // are cleared four segments before their use.
  int plain[8];
  float x_ref[128], x_sum[128];  // the second half's references and sums
};

// One row of a segment over keys [j0, j1), one warp, D / 32 coordinates a lane:
// the plain form, for segments that the tensor core cannot take.  o: the mean;
// turns: where it shows that it gets on (every 64 keys).
template <int D>
__device__ __noinline__ void attend_row(const CacheFwdParams& p, int b, int h, int64_t q_at, int j0, int j1,
                                        float& top, float& total, float* o, int* turns) {
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
    if (((j - j0) & 63) == 0 && lane == 0) atomicAdd(turns, 1);
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
    const float all = l * keep + w, inv = all == 0.0f ? 0.0f : 1.0f / all;
    const float stay = l * keep * inv, add = w * inv;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * stay + add * (e4m3_to_float(p.cache.v[at + e]) * sv);
    l = all;
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
  const int first = p.no_split ? 0 : static_cast<int>(split::quotient(unit0, chunk));
  r.pieces = p.no_split ? 1 : static_cast<int>(split::quotient(unit0 + w.w.steps - 1, chunk)) - first + 1;
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
__device__ void run_softmax(const CacheFwdParams& p, uint8_t* sm, Bars& B, Notes& notes, uint32_t tmem,
                            const split::Schedule<TileCfg<D>>& sh, int64_t at, int64_t stop, int64_t chunk,
                            unsigned long long limit) {
  using C = TileCfg<D>;
  const int lane = threadIdx.x & 31, half = threadIdx.x >> 7, r = threadIdx.x & 127, quarter = r >> 5;
  const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
  const uint32_t o_addr = tmem + lane_off + C::TM_O + half * 128;
  volatile Watch* watch = &B.watch;
  split::Walk<C> w;
  w.begin(p, sh.seq[0], sh.base[0], at);
  uint32_t gi = 0, ti = 0, seg = 0, xs = 0;  // tiles of the CTA, of this half; segments with tiles; exchanges
  bool ok = true, exchanged = false;
#pragma unroll 1
  for (; ok && w.more(p, stop); w.next(p)) {
    if (!w.enter(p, at, stop)) continue;
    const CacheSeq s = w.w.s;
    const Target to = target<C>(p, w, chunk, blockIdx.x);
    const bool pair = w.rows > C::HALF;  // the halves hold different rows
    const int ri = pair ? half * C::HALF + r : r;
    const bool valid = ri < w.rows;
    const int in_seq = w.map.token(p, ri), head = w.h * p.G + w.map.head(p, ri, in_seq);
    const int64_t tok = s.first + in_seq;
    const int64_t q_at = tok * p.q_stride + static_cast<int64_t>(head) * D;
    const int64_t out_row = tok * p.Hq + head;
    const int pos = s.len - s.n + in_seq;
    // keys this row sees: [lo, hi)
    const int lo = first_key(pos, p.window);
    const int hi = valid ? max(0, p.causal ? min(s.len, pos + 1) : s.len) : 0;
    const int steps = w.u1 - w.u0;
    const bool live = (ri & ~31) < w.rows;  // a warp without rows keeps the barriers' protocol
    float m = -INFINITY, l = 0.0f;
    int exponent = 0, mine = 0;  // V's exponent; tiles of this half in this segment
    bool plain = false;
    if (steps > 0) {
      if (exchanged) {  // Q's room held the last segment's exchange
        ok = wait(&B.x_free, (xs - 1) & 1, limit, watch);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        exchanged = false;
      }
      // ---- this row of Q, divided by its largest power of two, as fp16
      const uint4* src = reinterpret_cast<const uint4*>(p.q + q_at);
      uint4 raw[D / 8];
      float amax = 0.0f;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) raw[i] = valid ? src[i] : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        const uint32_t x[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          amax = fmaxf(amax, fabsf(__uint_as_float(x[e] << 16)));
          amax = fmaxf(amax, fabsf(__uint_as_float(x[e] & 0xffff0000u)));
        }
      }
      const int e2 = amax > 0.0f ? min(max(static_cast<int>(__float_as_uint(amax) >> 23) - 127, -126), 127) : 0;
      const float inv = sf_value(127 - e2), fac = sf_value(127 + e2) * p.scale2;
      const uint32_t q_smem = ptx::smem_u32(sm) + half * C::Q_BYTES;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        const uint32_t x[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
        uint32_t y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          y[e] = split::pack_f16x2(__uint_as_float(x[e] << 16) * inv, __uint_as_float(x[e] & 0xffff0000u) * inv);
        ptx::st_shared_v4(q_smem + (i >> 3) * C::Q_CHUNK + r * 128 + (((i & 7) ^ (r & 7)) << 4), y[0], y[1], y[2], y[3]);
      }
      ptx::fence_proxy_async_smem();
      ptx::mbar_arrive(&B.q_full);

      const bool fold = p.scale2 > 0.0f;
#pragma unroll 1
      for (int i = 0; i < steps; ++i, ++gi) {
        if (!pair && (i & 1) != half) continue;
        const int sb = ti & 1;
        ok = wait(&B.s_full[half][sb], (ti >> 1) & 1, limit, watch);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        ptx::tc_fence_after();
        if (live) {
          const int kb = w.w.kbase + (w.u0 + i) * C::SPAN;
          const uint32_t s_addr = tmem + lane_off + C::TM_S + half * 128 + sb * 64;
          const float4 sk = *reinterpret_cast<const float4*>(&notes.k_scale[gi & 7]);
          const int e_now = notes.exponent[gi & 7];
          float f[4] = {fac * sk.x, fac * sk.y, fac * sk.z, fac * sk.w};
          const uint32_t gone = (sk.x < 0.0f) | (sk.y < 0.0f) << 1 | (sk.z < 0.0f) << 2 | (sk.w < 0.0f) << 3;  // blocks on no page
          const bool edge = kb < w.lo_max || kb > w.hi_min - C::SPAN || gone != 0 || !fold;
          // Weights against the present reference, in one pass: nearly always
          // no score exceeds it by 15 and nothing else has to move.
          bool redo = edge || m == -INFINITY || (mine > 0 && e_now != exponent);
          if (!__all_sync(0xffffffffu, redo)) {
            uint32_t sr[64], pk[32];
            ptx::tmem_ld32(s_addr, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
            ptx::tmem_ld32(s_addr + 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[32]));
            ptx::tmem_wait_ld_r64(sr);
            const float neg = -m;
            float mx[2] = {-INFINITY, -INFINITY};
            uint64_t add[2] = {0, 0};
#pragma unroll
            for (int u = 0; u < 32; ++u) {
              const float a = fmaf(__uint_as_float(sr[2 * u]), f[u >> 3], neg);
              const float c = fmaf(__uint_as_float(sr[2 * u + 1]), f[u >> 3], neg);
              mx[u & 1] = ptx::max3(mx[u & 1], a, c);
              const float x = ptx::ex2_approx(a), y = ptx::ex2_approx(c);
              add[u & 1] = ptx::f2_add(add[u & 1], ptx::f2_pack(x, y));
              pk[u] = split::pack_f16x2(x, y);
            }
            redo |= fmaxf(mx[0], mx[1]) > 15.0f;
            if (!__any_sync(0xffffffffu, redo)) {
              float x, y;
              ptx::f2_unpack(ptx::f2_add(add[0], add[1]), x, y);
              l += x + y;
              ptx::tmem_st32(s_addr, pk);
            }
          }
          if (__any_sync(0xffffffffu, redo)) {  // the largest score first (S is still there)
            uint32_t sr[64];
            ptx::tmem_ld32(s_addr, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
            ptx::tmem_ld32(s_addr + 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[32]));
            ptx::tmem_wait_ld_r64(sr);
            float mx = -INFINITY;
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
              follow = mine > 0 && l != 0.0f;
              l *= alpha;
              m = up;
            }
            if (mine > 0 && e_now != exponent) {  // so it does V's exponent
              alpha *= exponent - e_now < -126 ? 0.0f : sf_value(127 + exponent - e_now);
              follow = l != 0.0f || follow;
            }
            exponent = e_now;
            if (__any_sync(0xffffffffu, follow)) {
              ok = wait(&B.pv_done[half][(ti - 1) & 1], ((ti - 1) >> 1) & 1, limit, watch);
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
            for (int part = 0; part < 2; ++part) {
              uint32_t pk[16];
#pragma unroll
              for (int u = 0; u < 16; ++u) {
                const int v = 16 * part + u;
                const float a = ptx::ex2_approx(fmaf(__uint_as_float(sr[2 * v]), f[v >> 3], neg));
                const float c = ptx::ex2_approx(fmaf(__uint_as_float(sr[2 * v + 1]), f[v >> 3], neg));
                add[u & 1] = ptx::f2_add(add[u & 1], ptx::f2_pack(a, c));
                pk[u] = split::pack_f16x2(a, c);
              }
              ptx::tmem_st16(s_addr + 16 * part, pk);
            }
            float x, y;
            ptx::f2_unpack(ptx::f2_add(add[0], add[1]), x, y);
            l += x + y;
          }
          ptx::tmem_wait_st();
        }
        ptx::tc_fence_before();
        ptx::mbar_arrive(&B.p_full[half][sb]);
        ++ti;
        ++mine;
      }
      if (!ok) break;
      ok = wait(&B.o_full, seg & 1, limit, watch);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      ptx::tc_fence_after();
      plain = *const_cast<volatile int*>(&notes.plain[seg & 7]) != 0;
      if (threadIdx.x == 0) notes.plain[(seg + 4) & 7] = 0;
      ++seg;
    }
    // ---- the result
    if (plain) {
      if (!live || (!pair && half == 1)) continue;
      const int k0 = w.w.kbase + w.u0 * C::SPAN, k1 = w.w.kbase + w.u1 * C::SPAN;
#pragma unroll 1
      for (int row = 0; row < 32 && (ri & ~31) + row < w.rows; ++row) {
        constexpr int E = D / 32;
        float top, total, o[E];
        const int64_t row_q = __shfl_sync(0xffffffffu, q_at, row), row_o = __shfl_sync(0xffffffffu, out_row, row);
        attend_row<D>(p, w.b, w.h, row_q, max(k0, __shfl_sync(0xffffffffu, lo, row)),
                      min(k1, __shfl_sync(0xffffffffu, hi, row)), top, total, o, &B.watch.turns);
        const int at_row = (ri & ~31) + row;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          if (to.pieces == 1)
            p.out[row_o * D + lane * E + e] = __float2bfloat16_rn(o[e]);
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
    // this half's output is in units of 2^exponent; its weight makes it a mean
    // (as large as values: their sums may not be held)
    const float unit = sf_value(min(max(127 + exponent, 0), 254));
    float own = l == 0.0f ? 0.0f : 1.0f / l;
    float other = 0.0f;  // weight of the second half's mean
    const uint32_t x_row = ptx::smem_u32(sm) + r * D * 4;
    if (!pair && steps > 0) {
      if (half == 1) {  // hand over: reference, sum, output
        if (live) {
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            ptx::tmem_ld32(o_addr + c, o);
            ptx::tmem_wait_ld_r32(o);
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              uint32_t y[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                y[e] = l == 0.0f ? 0 : __float_as_uint(__uint_as_float(o[4 * u + e]) * own * unit);
              ptx::st_shared_v4(x_row + (((c / 4 + u) ^ (r & 7)) << 4), y[0], y[1], y[2], y[3]);
            }
          }
          notes.x_ref[r] = m;
          notes.x_sum[r] = l;
        }
        ptx::tc_fence_before();
        ptx::mbar_arrive(&B.x_full);
        exchanged = true;
        ++xs;
        continue;
      }
      ok = wait(&B.x_full, xs & 1, limit, watch);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      if (live) {
        const float m2 = *const_cast<volatile float*>(&notes.x_ref[r]), l2 = *const_cast<volatile float*>(&notes.x_sum[r]);
        const float top = fmaxf(m, m2), zero = top == -INFINITY ? 0.0f : top;
        const float f1 = ptx::ex2_approx(m - zero), f2 = l2 == 0.0f ? 0.0f : ptx::ex2_approx(m2 - zero);
        const float all = l * f1 + l2 * f2, inv = all == 0.0f ? 0.0f : 1.0f / all;
        own = l == 0.0f ? 0.0f : f1 * inv;
        other = l2 * f2 * inv;
        l = all;
        m = top;
      }
    }
    if (live) {
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t o[32];
        if (mine > 0) {
          ptx::tmem_ld32(o_addr + c, o);
          ptx::tmem_wait_ld_r32(o);
        }
#pragma unroll
        for (int u = 0; u < 32; ++u)  // (where this half saw nothing its output may be anything)
          o[u] = mine == 0 || own == 0.0f ? 0 : __float_as_uint(__uint_as_float(o[u]) * own * unit);
        if (other != 0.0f) {
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            uint32_t y[4];
            split::lds128(x_row + (((c / 4 + u) ^ (r & 7)) << 4), y);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              o[4 * u + e] = __float_as_uint(fmaf(__uint_as_float(y[e]), other, __uint_as_float(o[4 * u + e])));
          }
        }
        if (!valid) continue;
        if (to.pieces == 1) {
          uint4* dst = reinterpret_cast<uint4*>(p.out + out_row * D + c);
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            uint32_t y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              y[e] = ptx::pack_bf16x2(__uint_as_float(o[8 * u + 2 * e]), __uint_as_float(o[8 * u + 2 * e + 1]));
            dst[u] = make_uint4(y[0], y[1], y[2], y[3]);
          }
        } else {
          uint4* dst = reinterpret_cast<uint4*>(to.part + 2 * C::ROWS + ri * D + c);
#pragma unroll
          for (int u = 0; u < 8; ++u) dst[u] = make_uint4(o[4 * u], o[4 * u + 1], o[4 * u + 2], o[4 * u + 3]);
        }
      }
      if (valid) {
        if (to.pieces > 1)
          to.part[2 * ri] = m, to.part[2 * ri + 1] = l;
        else if (p.lse)
          p.lse[out_row] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
      }
    }
    if (!pair && steps > 0) {
      ptx::mbar_arrive(&B.x_free);
      exchanged = true;
      ++xs;
    }
    ptx::tc_fence_before();  // O has been read when the next segment's P allows its first product
  }
  if (!ok && lane == 0) {
    watch->abort = 1;
    atomicOr(p.batch.status, kStatusActivation);
  }
}

// ------------------------------------------------------------------ codes
template <int D>
__device__ void run_copies(const CacheFwdParams& p, uint8_t* sm, Bars& B, Notes& notes,
                           const split::Schedule<TileCfg<D>>& sh, int64_t at, int64_t stop,
                           unsigned long long limit) {
  using C = TileCfg<D>;
  // Eight tiles at a time: a lane looks after one block of one of them, so that
  // the latency of page and scales is met once for all.
  const int lane = threadIdx.x & 31, mine = lane >> 2, j = lane & 3;
  volatile Watch* watch = &B.watch;
  const int pmask = (1 << p.cache.lp) - 1;
  const uint32_t raw = ptx::smem_u32(sm + C::OFF_RAW) + j * kCacheBlock * D;
  split::Walk<C> w;
  w.begin(p, sh.seq[0], sh.base[0], at);
  bool ok = true;
  int exponent = 0;
  uint32_t gi = 0;
#pragma unroll 1
  for (; ok && w.more(p, stop); w.next(p)) {
    if (!w.enter(p, at, stop)) continue;
    const int32_t* table = p.batch.table + static_cast<int64_t>(w.b) * p.batch.max_pages;
#pragma unroll 1
    for (int u = w.u0; ok && u < w.u1; u += 8) {
      const int cnt = min(8, w.u1 - u);
      const int block = w.w.kbase + (u + mine) * C::SPAN + kCacheBlock * j;
      bool there = mine < cnt && block < w.hi_max && block + kCacheBlock > w.lo_min;
      int64_t row = 0;
      int sk = 127, sv = 127;
      if (there) {
        const int page = __ldg(table + (block >> p.cache.lp));
        if (page >= 0 && page < p.cache.num_pages) {
          row = cache_row(p.cache, page, w.h, block & pmask);
          sk = p.cache.k_sf[row >> 4];
          sv = p.cache.v_sf[row >> 4];
        } else {
          there = false;
          atomicOr(p.batch.status, kStatusBadPlan);
        }
      }
      const uint32_t blocks = __ballot_sync(0xffffffffu, there);
      // blocks that lie one behind the other in memory travel together
      const int64_t before = __shfl_up_sync(0xffffffffu, row, 1);
      const bool joins = there && j > 0 && (blocks >> (lane - 1) & 1) && row == before + kCacheBlock;
      const uint32_t run = __ballot_sync(0xffffffffu, joins) >> (lane & 28) >> j >> 1;  // bit i: block j + 1 + i joins
      const uint32_t bytes = there && !joins ? (1 + __ffs(~run) - 1) * kCacheBlock * D : 0;
      const int ev = there ? sv - 127 : -1000;
      int top = max(ev, __shfl_xor_sync(0xffffffffu, ev, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
#pragma unroll 1
      for (int t = 0; t < cnt; ++t) {
        const int slot = gi % C::RAWS;
        ok = wait(&B.raw_free[slot], ((gi / C::RAWS) & 1) ^ 1, limit, watch);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        ++gi;
        const uint32_t have = blocks >> (4 * t) & 15;
        if (lane == 0 && have) ptx::mbar_expect_tx(&B.raw_full[slot], __popc(have) * 2 * kCacheBlock * D);
        __syncwarp();
        if (bytes && mine == t) {
          const uint32_t dst = raw + slot * 2 * C::RAW;
          ptx::bulk_load(dst, p.cache.k + row * D, bytes, &B.raw_full[slot]);
          ptx::bulk_load(dst + C::RAW, p.cache.v + row * D, bytes, &B.raw_full[slot]);
        }
        const bool first = t == 0 && u == w.u0;
        const int tile_top = __shfl_sync(0xffffffffu, top, 4 * t);
        const int kb = w.w.kbase + (u + t) * C::SPAN;
        const bool edge = kb < w.lo_max || kb > w.hi_min - C::SPAN;
        // At an edge a row may see nothing of a block far above the units, and
        // what it has summed must not vanish in that block's (five such tiles at
        // most lie behind a row's last key): the plain form.
        const bool above = edge && !first && exponent > -1000 && tile_top > exponent + 24;
        if (first || tile_top > exponent + 7) exponent = tile_top;  // -1000: nothing is there yet
        const int up = ev - exponent;  // at most 7
        const uint32_t low = above ? have : __ballot_sync(0xffffffffu, there && up < -15) >> (4 * t) & 15;
        RawNote& n = notes.raw[slot];
        if (mine == t) {
          n.k_scale[j] = there ? sf_value(sk) : -1.0f;
          n.v_mul[j] = !there ? 0 : up < -14 ? 0x00010001u << max(up + 24, 0) : static_cast<uint32_t>(up + 15) * 0x04000400u;
        }
        if (lane == 0) {
          n.state = 1 | (first ? 2 : 0) | (edge ? 4 : 0) | (!edge && have == 15 && low == 0 ? 8 : 0);
          n.exponent = exponent;
          n.kb = kb, n.lo = w.lo_min, n.hi = w.hi_max;
          n.low = low;
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&B.raw_full[slot]);
      }
    }
  }
  if (ok) {  // the last entry: no tile
    const int slot = gi % C::RAWS;
    ok = wait(&B.raw_free[slot], ((gi / C::RAWS) & 1) ^ 1, limit, watch);
    ok = __all_sync(0xffffffffu, ok);
    if (ok) {
      ++gi;
      if (lane == 0) {
        notes.raw[slot].state = 0;
        ptx::mbar_arrive(&B.raw_full[slot]);
      }
    }
  }
  if (!ok && lane == 0) {
    watch->abort = 1;
    atomicOr(p.batch.status, kStatusProducer);
  }
  // no copy may land after the CTA has ended
  const int never = 0;
  for (uint32_t g = gi > C::RAWS ? gi - C::RAWS : 0; g < gi; ++g)
    ptx::mbar_wait(&B.raw_full[g % C::RAWS], (g / C::RAWS) & 1, 100000000ull, &never);
}

// ------------------------------------------------------------------ conversion
// Warps of one warpgroup convert K, of another V.
template <int D, bool V>
__device__ void run_convert(const CacheFwdParams& p, uint8_t* sm, Bars& B, Notes& notes, unsigned long long limit) {
  using C = TileCfg<D>;
  constexpr int CPR = D / 16;               // 16-code chunks of a row
  constexpr int RPI = 128 / CPR;            // rows that 128 threads convert at once
  constexpr int NI = C::SPAN / RPI;         // ... and how often for a tile
  const int tid = threadIdx.x & 127, lane = tid & 31;
  const int c = tid % CPR, r0 = tid / CPR;
  volatile Watch* watch = &B.watch;
  const int swap = c >> 2 & 1;
  uint32_t seg = 0xffffffffu;  // the segment's number
  bool ok = true;
#pragma unroll 1
  for (uint32_t gi = 0;; ++gi) {
    const int slot = gi % C::RAWS, st = gi & 1;
    ok = wait(&B.raw_full[slot], (gi / C::RAWS) & 1, limit, watch);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) break;
    const RawNote& n = notes.raw[slot];
    const uint32_t state = *const_cast<volatile const uint32_t*>(&n.state);
    if (!(state & 1)) break;
    seg += state >> 1 & 1;
    ok = wait(V ? &B.v_free[st] : &B.k_free[st], ((gi >> 1) & 1) ^ 1, limit, watch);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) break;
    const uint32_t from = ptx::smem_u32(sm + C::OFF_RAW) + slot * 2 * C::RAW + (V ? C::RAW : 0) + tid * 16;
    const uint32_t to = ptx::smem_u32(sm + (V ? C::OFF_V : C::OFF_K)) + st * C::KV_BYTES + (c >> 2) * C::KV_CHUNK;
    uint32_t x[NI][4];
#pragma unroll
    for (int j = 0; j < NI; ++j) split::lds128(from + j * 2048, x[j]);
    uint32_t mul[4];
    if (V) {
      const uint4 u = *reinterpret_cast<const uint4*>(n.v_mul);
      mul[0] = u.x, mul[1] = u.y, mul[2] = u.z, mul[3] = u.w;
      if (!(state & 8)) {
        bool plain = false;
#pragma unroll
        for (int j = 0; j < NI; ++j) {
          const int r = r0 + RPI * j, key = n.kb + r;
          // tokens that no row sees (and blocks on no page) may hold anything: zeros
          if (n.v_mul[r >> 4] == 0 || key < n.lo || key >= n.hi) x[j][0] = x[j][1] = x[j][2] = x[j][3] = 0;
          if (state & 4) {
#pragma unroll
            for (int e = 0; e < 4; ++e) plain |= split::has_nan_code(x[j][e]);
          }
          if (n.low >> (r >> 4) & 1) plain |= ((x[j][0] | x[j][1] | x[j][2] | x[j][3]) & 0x7f7f7f7fu) != 0;
        }
        if (__any_sync(0xffffffffu, plain) && lane == 0) *const_cast<volatile int*>(&notes.plain[seg & 7]) = 1;
      }
    }
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      const int r = r0 + RPI * j;  // in block j (16 rows at once), or 2 j and 2 j + 1
      const uint32_t f = !V ? 0 : RPI == 16 ? mul[j & 3] : r0 >= 16 ? mul[(2 * j + 1) & 3] : mul[(2 * j) & 3];
      uint32_t y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        y[e] = e & 1 ? split::codes_hi(x[j][e >> 1]) : split::codes_lo(x[j][e >> 1]);
        if (V) asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(y[e]) : "r"(y[e]), "r"(f));
      }
      // two 16-byte pieces of the swizzled row, in an order that keeps the
      // eight lanes of a row on different banks
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t dst = to + r * 128 + (((2 * (c & 3) + (h ^ swap)) ^ (r & 7)) << 4);
        const bool second = h ^ swap;
        ptx::st_shared_v4(dst, second ? y[4] : y[0], second ? y[5] : y[1], second ? y[6] : y[2], second ? y[7] : y[3]);
      }
    }
    if (!V && tid == 0) {
      notes.k_scale[gi & 7] = *reinterpret_cast<const float4*>(n.k_scale);
      notes.exponent[gi & 7] = n.exponent;
    }
    ptx::fence_proxy_async_smem();
    ptx::mbar_arrive(V ? &B.v_full[st] : &B.k_full[st]);
    ptx::mbar_arrive(&B.raw_free[slot]);
  }
  if (!ok && lane == 0) {
    watch->abort = 1;
    atomicOr(p.batch.status, kStatusProducer);
  }
}

// ------------------------------------------------------------------ MMA
// S = Q K^T of every tile, up to two tiles of a half ahead of its softmax.  A
// buffer of S holds P of the tile that used it last, until P V of that one is
// done.
template <int D>
__device__ void run_scores(const CacheFwdParams& p, uint8_t* sm, Bars& B, uint32_t tmem,
                           const split::Schedule<TileCfg<D>>& sh, int64_t at, int64_t stop, unsigned long long limit) {
  using C = TileCfg<D>;
  volatile Watch* watch = &B.watch;
  split::Walk<C> w;
  w.begin(p, sh.seq[0], sh.base[0], at);
  uint32_t gi = 0, seg = 0, ti[2] = {0, 0};
  bool ok = true;
  // Descriptors of the first tiles: all others are a constant further on (the
  // address field counts 16 bytes and has room).
  const uint64_t q_desc = ptx::sdesc_sw128(ptx::smem_u32(sm), 16, 1024);
  const uint64_t k_desc = ptx::sdesc_sw128(ptx::smem_u32(sm + C::OFF_K), 16, 1024);
  constexpr uint32_t idesc = ptx::idesc_f16(128, C::SPAN, 0);
#pragma unroll 1
  for (; ok && w.more(p, stop); w.next(p)) {
    if (!w.enter(p, at, stop) || w.u1 <= w.u0) continue;
    ok = wait(&B.q_full, seg++ & 1, limit, watch);
    const int steps = w.u1 - w.u0;
    const bool pair = w.rows > C::HALF;
#pragma unroll 1
    for (int i = 0; ok && i < steps; ++i, ++gi) {
      const int ks = gi & 1;
      ok = wait(&B.k_full[ks], (gi >> 1) & 1, limit, watch);
      if (!ok) break;
      const uint64_t k = k_desc + ks * (C::KV_BYTES >> 4);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (!pair && (i & 1) != h) continue;
        const uint32_t sb = ti[h] & 1;
        ok = ok && wait(&B.pv_done[h][sb], ((ti[h] >> 1) & 1) ^ 1, limit, watch);
        if (!ok) break;
        ptx::tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          ptx::mma_ss_elect(tmem + C::TM_S + h * 128 + sb * 64,
                            q_desc + ((h * C::Q_BYTES + (kk >> 2) * C::Q_CHUNK + (kk & 3) * 32) >> 4),
                            k + (((kk >> 2) * C::KV_CHUNK + (kk & 3) * 32) >> 4), idesc, kk > 0 ? 1u : 0u);
        ptx::mma_commit_elect(&B.s_full[h][sb]);
        ++ti[h];
      }
      ptx::mma_commit_elect(&B.k_free[ks]);
    }
  }
  if (!ok && (threadIdx.x & 31) == 0) {
    watch->abort = 1;
    atomicOr(p.batch.status, kStatusMma);
  }
  // every MMA this warp issued is complete once this commit lands
  ptx::mma_commit_elect(&B.drain[0]);
  const int never = 0;
  ptx::mbar_wait(&B.drain[0], 0, 100000000ull, &never);
}

// O += P V of every tile.
template <int D>
__device__ void run_values(const CacheFwdParams& p, uint8_t* sm, Bars& B, uint32_t tmem,
                           const split::Schedule<TileCfg<D>>& sh, int64_t at, int64_t stop, unsigned long long limit) {
  using C = TileCfg<D>;
  volatile Watch* watch = &B.watch;
  split::Walk<C> w;
  w.begin(p, sh.seq[0], sh.base[0], at);
  uint32_t gi = 0, ti[2] = {0, 0};
  bool ok = true;
  const uint64_t v_desc = ptx::sdesc_sw128(ptx::smem_u32(sm + C::OFF_V), C::KV_CHUNK, 1024);
  constexpr uint32_t idesc = ptx::idesc_f16(128, D, 1);
#pragma unroll 1
  for (; ok && w.more(p, stop); w.next(p)) {
    if (!w.enter(p, at, stop) || w.u1 <= w.u0) continue;
    const int steps = w.u1 - w.u0;
    const bool pair = w.rows > C::HALF;
#pragma unroll 1
    for (int i = 0; ok && i < steps; ++i, ++gi) {
      const int vs = gi & 1;
      ok = wait(&B.v_full[vs], (gi >> 1) & 1, limit, watch);
      if (!ok) break;
      const uint64_t v = v_desc + vs * (C::KV_BYTES >> 4);
      const bool first = i < (pair ? 1 : 2);  // a half's first in this segment
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (!pair && (i & 1) != h) continue;
        const uint32_t sb = ti[h] & 1;
        ok = ok && wait(&B.p_full[h][sb], (ti[h] >> 1) & 1, limit, watch);
        if (!ok) break;
        ptx::tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < C::SPAN / 16; ++kk)
          // V is MN-major: 16 keys = two 8-row groups 1024 B apart; 64-column chunks KV_CHUNK apart
          ptx::mma_ts_elect(tmem + C::TM_O + h * 128, tmem + C::TM_S + h * 128 + sb * 64 + 8 * kk,
                            v + (kk * 2048 >> 4), idesc, kk > 0 ? 1u : first ? 0u : 1u);
        ptx::mma_commit_elect(&B.pv_done[h][sb]);
        ++ti[h];
      }
      ptx::mma_commit_elect(&B.v_free[vs]);
    }
    ptx::mma_commit_elect(&B.o_full);
  }
  if (!ok && (threadIdx.x & 31) == 0) {
    watch->abort = 1;
    atomicOr(p.batch.status, kStatusMma);
  }
  ptx::mma_commit_elect(&B.drain[1]);
  const int never = 0;
  ptx::mbar_wait(&B.drain[1], 0, 100000000ull, &never);
}

}  // namespace tile

template <int D>
__global__ void __launch_bounds__(640, 1) gdpa_cache_tile_kernel(const CacheFwdParams p, unsigned long long limit) {
  using C = TileCfg<D>;
  // All of it dynamic: nothing static in front of it, so that it begins on the
  // 1024 bytes that the swizzle wants.
  extern __shared__ __align__(1024) uint8_t sm[];
  struct Block {
    tile::Bars bars;
    tile::Notes notes;
    split::Schedule<C> schedule;
  };
  static_assert(sizeof(Block) <= 3072, "barrier block");
  Block& block = *reinterpret_cast<Block*>(sm + C::OFF_BLOCK);
  tile::Bars& B = block.bars;
  tile::Notes& notes = block.notes;
  split::Schedule<C>& sh = block.schedule;
  const int tid = threadIdx.x, warp = tid >> 5;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid == 0 && !p.no_split) p.meta[blockIdx.x * 16 + 1] = p.meta[blockIdx.x * 16 + 9] = 0;  // no parts yet
  if (ptx::smem_u32(sm) & 1023u) {
    if (tid == 0) atomicOr(p.batch.status, kStatusProducer);
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < C::RAWS; ++i) {
      ptx::mbar_init(&B.raw_full[i], 1);
      ptx::mbar_init(&B.raw_free[i], 256);
    }
    ptx::mbar_init(&B.q_full, 256);
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&B.k_full[i], 128);
      ptx::mbar_init(&B.k_free[i], 1);
      ptx::mbar_init(&B.v_full[i], 128);
      ptx::mbar_init(&B.v_free[i], 1);
      for (int h = 0; h < 2; ++h) {
        ptx::mbar_init(&B.s_full[h][i], 1);
        ptx::mbar_init(&B.p_full[h][i], 128);
        ptx::mbar_init(&B.pv_done[h][i], 1);
      }
      ptx::mbar_init(&B.drain[i], 1);
    }
    ptx::mbar_init(&B.o_full, 1);
    ptx::mbar_init(&B.x_full, 128);
    ptx::mbar_init(&B.x_free, 128);
    B.watch.abort = B.watch.turns = 0;
    ptx::fence_mbar_init();
  }
  if (tid < 8) notes.plain[tid] = 0;
  int64_t total, chunk;
  split::schedule<C>(p, sh, total, chunk);  // synchronises: the barriers are there
  const int64_t at = chunk * blockIdx.x, stop = min(total, at + chunk);
  if (at >= stop) return;
  if (warp == 16) {
    ptx::tmem_alloc(&B.tmem, C::TM_COLS);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = B.tmem;
  if (warp < 8) {
    ptx::regs_inc<C::REGS_SOFTMAX>();
    tile::run_softmax<D>(p, sm, B, notes, tmem, sh, at, stop, chunk, limit);
  } else if (warp < 16) {
    ptx::regs_dec<C::REGS_CONVERT>();
    if (warp < 12)
      tile::run_convert<D, false>(p, sm, B, notes, limit);
    else
      tile::run_convert<D, true>(p, sm, B, notes, limit);
  } else {
    ptx::regs_dec<C::REGS_ISSUE>();
    if (warp == 16) tile::run_scores<D>(p, sm, B, tmem, sh, at, stop, limit);
    if (warp == 18) tile::run_values<D>(p, sm, B, tmem, sh, at, stop, limit);
    if (warp == 17) tile::run_copies<D>(p, sm, B, notes, sh, at, stop, limit);
  }
  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == 16) ptx::tmem_dealloc(tmem, C::TM_COLS);
}

}  // namespace gdpa
