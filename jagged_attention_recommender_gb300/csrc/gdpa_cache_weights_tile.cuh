// gdpa_cache_weights_tile.cuh -- the weight that stored keys receive from many
// rows (pieces of prompts, many candidates): 128 keys at a time on the
// 5th-generation tensor cores.
//
// Mathematics.  S^T = K Q^T with keys on the 128 lanes of TMEM, so a thread owns
// a key: its score's factor (the block's scale) is one register, its weight one
// sum, and what changes along its row of S^T, the queries' logsumexp, is read
// from shared memory by all lanes at once: a fused multiply-add, an exponential
// and an addition for each score.  Both operands are bf16: queries as they are,
// codes exactly.
//
// Work split.  An item is 256 keys of a sequence and head, converted once and kept
// in shared memory while all rows that see any of them pass in chunks of 128
// columns (tokens times heads of the group); sequences whose rows fit one
// chunk keep the chunk instead and pass p.group items.  CTAs take every
// gridDim.x-th group of items.  Roles:
//   warps 0-3, 4-7  the sums of the item's first and second 128 keys, a key a thread
//   warps 8-11      convert K (128-byte swizzle, four tiles)
//   warp 12         issues the MMAs
//   warp 13         brings the queries by TMA, their logsumexp and last keys
#pragma once

#include "gdpa_cache_append.cuh"
#include "gdpa_cache_tile.cuh"
#include "gdpa_cache_weights.cuh"

namespace gdpa {

namespace ptx {

// 3-D tiled bulk tensor load global -> shared, completion counted in bytes on `bar`.
__device__ __forceinline__ void tma_load_3d(uint32_t smem_dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
          smem_dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

}  // namespace ptx

struct WeightTileParams {
  CUtensorMap tm_q;  // [T, Hq, D] bf16, boxes of 64 x heads x tokens, 128-byte swizzle
  CacheWeightsParams w;
  int heads, tokens;  // of a chunk: heads * tokens <= 128 (heads: G, or 128 of more)
  int parts;          // chunks that the heads of a group make
  int group;          // items of a group
  unsigned long long limit;
};

template <int D_>
struct WeightTileCfg {
  static constexpr int D = D_, THREADS = 448, KEYS = 128, COLS = 128;
  static constexpr int SUB = 128 * 128;            // 64 columns of a tile: 128 rows of 128 bytes
  static constexpr int TILE = D / 64 * SUB;
  static constexpr int KS = 4, QS = 2;             // stages of K and of Q
  static constexpr int OFF_Q = KS * TILE, OFF_NOTES = OFF_Q + QS * TILE;
  static constexpr int USED = OFF_NOTES + KS * 512 + QS * 1024;
  static constexpr int SMEM = (USED > 120 * 1024 ? USED : 120 * 1024) + 1024;  // one CTA an SM (all of its TMEM)
  static constexpr uint32_t TM_COLS = 512;         // S of two tiles, two buffers each
  static_assert(SMEM <= 226 * 1024, "shared memory");
};

namespace wtile {

struct Bars {
  uint64_t k_full[4], k_free[4], q_full[2], q_free[2], s_full[2][2], s_free[2][2], drain;
  uint32_t tmem;
  int abort;  // a wait has given up
};

struct Notes {
  float* factor;  // [KS][128]: of each key's scores, in units of log2
  float* lse;     // [QS][128]: minus each column's logsumexp, in units of log2
  int* last;      // [QS][128]: the last key that each column sees, -1 for none
};

// Groups of items of one CTA, in order.
struct Walk {
  CacheSeq s;
  int64_t idx;  // among the sequence's groups
  int b, h, kbase, pairs, groups;
  int pair, pair_end;
  bool single;  // its rows fit one chunk

  __device__ __forceinline__ void load(const WeightTileParams& p) {
    const CacheWeightsParams& w = p.w;
    s = load_sequence(w.batch, w.cache.lp, b);
    pairs = groups = kbase = 0;
    single = false;
    if (!s.ok || s.n == 0 || s.len == 0) return;
    if (w.keep) kbase = min(first_key(s.len - s.n, w.window), s.len) & ~255;
    pairs = static_cast<int>((static_cast<unsigned>(s.len - kbase) + 255) >> 8);
    groups = (pairs + p.group - 1) / p.group;
    single = p.parts == 1 && s.n <= p.tokens;
  }
  __device__ __forceinline__ bool settle(const WeightTileParams& p) {
    while (true) {
      const int64_t all = static_cast<int64_t>(groups) * p.w.cache.H;
      if (idx < all) break;
      idx -= all;
      if (++b >= p.w.batch.B) return false;
      load(p);
    }
    h = static_cast<int>(idx / groups);
    pair = static_cast<int>(idx - static_cast<int64_t>(h) * groups) * p.group;
    pair_end = min(pairs, pair + p.group);
    return true;
  }
  __device__ __forceinline__ bool begin(const WeightTileParams& p) {
    b = 0;
    idx = blockIdx.x;
    load(p);
    return settle(p);
  }
  __device__ __forceinline__ bool next(const WeightTileParams& p) {
    idx += gridDim.x;
    return settle(p);
  }
};

// An item: its first key, its tiles, and the tokens [lo, hi) whose rows see any of it, in chunks.
struct Item {
  int k0, tiles, lo, hi, chunks;
};
__device__ __forceinline__ Item item_of(const WeightTileParams& p, const Walk& w, int pair) {
  Item it;
  it.k0 = w.kbase + (pair << 8);
  it.tiles = w.s.len - it.k0 > 128 ? 2 : 1;
  const int last = it.k0 + min(255, w.s.len - 1 - it.k0);
  it.lo = rows_of_key(w.s, it.k0, p.w.causal, p.w.window).lo;
  it.hi = rows_of_key(w.s, last, p.w.causal, p.w.window).hi;
  it.chunks = 0;
  if (it.hi <= it.lo) return it;
  if (w.single) it.lo = 0, it.hi = w.s.n;
  it.chunks = (it.hi - it.lo + p.tokens - 1) / p.tokens * p.parts;
  return it;
}
// Columns of chunk c, to the last one that is a row.
__device__ __forceinline__ int chunk_columns(const WeightTileParams& p, const Item& it, int c) {
  const int part = p.parts == 1 ? 0 : c % p.parts, tok = it.lo + (p.parts == 1 ? c : c / p.parts) * p.tokens;
  return (min(p.tokens, it.hi - tok) - 1) * p.heads + min(p.heads, p.w.G - part * p.heads);
}

template <int D>
__device__ void run_sums(const WeightTileParams& p, Bars& B, const Notes& notes, uint32_t tmem) {
  using C = WeightTileCfg<D>;
  const CacheWeightsParams& w = p.w;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, m = warp >> 2;  // m: this warpgroup's tile of an item
  const int key_in = (warp & 3) * 32 + lane;
  const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + m * 256;
  const volatile int* abort = &B.abort;
  const int pmask = (1 << w.cache.lp) - 1;
  uint32_t ki = 0, qi = 0, si = 0;  // tiles of K, chunks and tiles of S so far
  bool ok = true;
  Walk walk;
  for (bool more = walk.begin(p); more && ok; more = walk.next(p)) {
    const CacheSeq& s = walk.s;
    bool held = false;  // this group's only chunk is there
#pragma unroll 1
    for (int pair = walk.pair; pair < walk.pair_end && ok; ++pair) {
      const Item it = item_of(p, walk, pair);
      const bool mine = m < it.tiles;
      const int k0 = it.k0 + m * 128;
      const bool stored = mine && s.len - k0 > key_in;
      const int key = k0 + key_in;
      // where the key's weight is, and what it was
      int64_t row = -1;
      float old = 0.0f;
      if (stored) {
        const int page = load_page(w.cache, w.batch, walk.b, key);
        if (page >= 0) {
          row = cache_row(w.cache, page, walk.h, key & pmask);
          if (w.w_in && key < s.len - s.n) old = w.decay * w.w_in[row];
        }
      }
      __syncwarp();
      float factor = 0.0f;
      if (it.chunks > 0 && mine) {
        const uint32_t k = ki + m;
        ok = ptx::mbar_wait(&B.k_full[k % C::KS], k / C::KS & 1, p.limit, abort);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        factor = notes.factor[k % C::KS * 128 + key_in];
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&B.k_free[k % C::KS]);
      }
      if (it.chunks > 0) ki += it.tiles;
      const uint64_t f2 = ptx::f2_splat(factor);
      uint64_t sum[2] = {0, 0};
      float edge_sum = 0.0f;
      const int k_last = k0 + min(127, s.len - 1 - k0);
#pragma unroll 1
      for (int c = 0; c < it.chunks; ++c) {
        const uint32_t qs = qi % C::QS;
        if (!held) ok = ptx::mbar_wait(&B.q_full[qs], qi / C::QS & 1, p.limit, abort);
        held = walk.single;
        if (ok && mine) ok = ptx::mbar_wait(&B.s_full[m][si & 1], si >> 1 & 1, p.limit, abort);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (mine) {
          ptx::tc_fence_after();
          const int n = (chunk_columns(p, it, c) + 31) >> 5;
          const float* lse = notes.lse + qs * 128;
          const int* last = notes.last + qs * 128;
#pragma unroll 1
          for (int q = 0; q < n; ++q) {
            uint32_t r[32];
            ptx::tmem_ld32(lanes + (si & 1) * 128 + q * 32, r);
            ptx::tmem_wait_ld_r32(r);
            if (q == n - 1) {  // the buffer is read
              ptx::tc_fence_before();
              __syncwarp();
              if (lane == 0) ptx::mbar_arrive(&B.s_free[m][si & 1]);
              __syncwarp();
            }
            const int end0 = last[q * 32], end1 = last[q * 32 + 31];  // tokens, and so last keys, ascend
            if (end0 >= k_last && end1 >= end0 && (w.window == 0 || end1 - w.window < k0)) {
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const ulonglong2 l = reinterpret_cast<const ulonglong2*>(lse + q * 32)[i];
                const uint64_t x = ptx::f2_pack(__uint_as_float(r[4 * i]), __uint_as_float(r[4 * i + 1]));
                const uint64_t y = ptx::f2_pack(__uint_as_float(r[4 * i + 2]), __uint_as_float(r[4 * i + 3]));
                float a, b, e, d;
                ptx::f2_unpack(ptx::f2_fma(x, f2, l.x), a, b);
                ptx::f2_unpack(ptx::f2_fma(y, f2, l.y), e, d);
                sum[0] = ptx::f2_add(sum[0], ptx::f2_pack(ptx::ex2_approx(a), ptx::ex2_approx(b)));
                sum[1] = ptx::f2_add(sum[1], ptx::f2_pack(ptx::ex2_approx(e), ptx::ex2_approx(d)));
              }
            } else {
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const int end = last[q * 32 + i];
                const float e = ptx::ex2_approx(fmaf(__uint_as_float(r[i]), factor, lse[q * 32 + i]));
                if (key <= end && (w.window == 0 || key > end - w.window)) edge_sum += e;
              }
            }
            __syncwarp();
          }
          ++si;
        }
        if (!walk.single) {
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&B.q_free[qs]);
          ++qi;
        }
      }
      if (!ok) break;
      if (row >= 0) {
        float a, b, c, d;
        ptx::f2_unpack(sum[0], a, b);
        ptx::f2_unpack(sum[1], c, d);
        w.w[row] = old + (((a + b) + (c + d)) + edge_sum);
      }
      __syncwarp();
    }
    if (!ok) break;
    if (walk.single) {
      if (!held) {  // (its keys saw no row: the chunk came all the same)
        ok = ptx::mbar_wait(&B.q_full[qi % C::QS], qi / C::QS & 1, p.limit, abort);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&B.q_free[qi % C::QS]);
      ++qi;
    }
  }
  if (!ok && lane == 0) {
    B.abort = 1;
    atomicOr(w.batch.status, kStatusActivation);
  }
}

// Four codes as bf16.
__device__ __forceinline__ void codes_bf16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const float2 a = e4m3x2_to_float2(w & 0xffffu), b = e4m3x2_to_float2(w >> 16);
  lo = ptx::pack_bf16x2(a.x, a.y);
  hi = ptx::pack_bf16x2(b.x, b.y);
}

template <int D>
__device__ void run_convert(const WeightTileParams& p, uint8_t* sm, Bars& B, const Notes& notes) {
  using C = WeightTileCfg<D>;
  constexpr int CPR = D / 16, ROWS = 128 / CPR, N = 128 / ROWS;  // chunks of a key; keys of a pass; passes
  const CacheWeightsParams& w = p.w;
  const int tid = threadIdx.x - 256, lane = tid & 31;
  const volatile int* abort = &B.abort;
  const int pmask = (1 << w.cache.lp) - 1;
  const int r0 = tid / CPR, c = tid % CPR;  // its row in a pass, and 16 coordinates
  // 16-byte chunks 2c and 2c + 1 of a row, 64 columns a sub-tile
  const uint32_t base = ptx::smem_u32(sm) + (c >> 2) * C::SUB;
  uint32_t ki = 0;
  bool ok = true;
  Walk walk;
  for (bool more = walk.begin(p); more && ok; more = walk.next(p)) {
#pragma unroll 1
    for (int pair = walk.pair; pair < walk.pair_end && ok; ++pair) {
      const Item it = item_of(p, walk, pair);
      if (it.chunks == 0) continue;
#pragma unroll 1
      for (int m = 0; m < it.tiles; ++m, ++ki) {
        const int k0 = it.k0 + m * 128;
        int page = -1;  // lane i: of the tile's i-th block of 16
        if (lane < 8 && walk.s.len - k0 > lane * 16) page = load_page(w.cache, w.batch, walk.b, k0 + lane * 16);
        __syncwarp();
        uint4 x[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int r = r0 + i * ROWS, pg = __shfl_sync(0xffffffffu, page, r >> 4);
          x[i] = make_uint4(0, 0, 0, 0);
          if (pg >= 0)
            x[i] = __ldg(reinterpret_cast<const uint4*>(
                w.cache.k + cache_row(w.cache, pg, walk.h, (k0 + r) & pmask) * D + c * 16));
        }
        const int pg = __shfl_sync(0xffffffffu, page, tid >> 4);
        const float f =
            pg >= 0 ? sf_value(__ldg(w.cache.k_sf + cache_sf(w.cache, pg, walk.h, (k0 + tid) & pmask))) * w.scale2 : 0.0f;
        const uint32_t ks = ki % C::KS;
        ok = ptx::mbar_wait(&B.k_free[ks], (ki / C::KS & 1) ^ 1, p.limit, abort);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        notes.factor[ks * 128 + tid] = f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int r = r0 + i * ROWS;
          const uint32_t at = base + ks * C::TILE + r * 128, j = 2 * c & 7;
          uint32_t a[8];
          codes_bf16(x[i].x, a[0], a[1]);
          codes_bf16(x[i].y, a[2], a[3]);
          codes_bf16(x[i].z, a[4], a[5]);
          codes_bf16(x[i].w, a[6], a[7]);
          ptx::st_shared_v4(at + ((j ^ (r & 7)) << 4), a[0], a[1], a[2], a[3]);
          ptx::st_shared_v4(at + (((j + 1) ^ (r & 7)) << 4), a[4], a[5], a[6], a[7]);
        }
        ptx::fence_proxy_async_smem();
        ptx::mbar_arrive(&B.k_full[ks]);
      }
    }
  }
  if (!ok && lane == 0) {
    B.abort = 1;
    atomicOr(w.batch.status, kStatusProducer);
  }
}

template <int D>
__device__ void run_queries(const WeightTileParams& p, uint8_t* sm, Bars& B, const Notes& notes) {
  using C = WeightTileCfg<D>;
  const CacheWeightsParams& w = p.w;
  const int lane = threadIdx.x & 31;
  const volatile int* abort = &B.abort;
  const uint32_t bytes = static_cast<uint32_t>(p.heads) * p.tokens * D * 2;
  int tok_of[4], head_of[4];  // of this lane's four columns in a chunk
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    tok_of[i] = (lane * 4 + i) / p.heads;
    head_of[i] = lane * 4 + i - tok_of[i] * p.heads;
  }
  uint32_t qi = 0;
  bool ok = true;
  auto bring = [&](const Walk& walk, const Item& it, int c) {
    const CacheSeq& s = walk.s;
    const int part = p.parts == 1 ? 0 : c % p.parts, tok0 = it.lo + (p.parts == 1 ? c : c / p.parts) * p.tokens;
    float lse[4];
    int last[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int tok = tok0 + tok_of[i], head = part * p.heads + head_of[i];
      lse[i] = INFINITY;
      last[i] = -1;
      if (tok_of[i] < p.tokens && tok < it.hi && head < w.G) {
        const float x = __ldg(w.lse + static_cast<int64_t>(s.first + tok) * w.Hq + walk.h * w.G + head);
        lse[i] = x == -INFINITY ? INFINITY : x * kLog2e;
        last[i] = w.causal ? s.len - s.n + tok : s.len - 1;
      }
    }
    const uint32_t qs = qi % C::QS;
    ok = ptx::mbar_wait(&B.q_free[qs], (qi / C::QS & 1) ^ 1, p.limit, abort);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) return;
    if (lane == 0) {
      ptx::mbar_arrive_expect_tx(&B.q_full[qs], bytes);
#pragma unroll
      for (int d = 0; d < D / 64; ++d)
        ptx::tma_load_3d(ptx::smem_u32(sm) + C::OFF_Q + qs * C::TILE + d * C::SUB, &p.tm_q, &B.q_full[qs], d * 64,
                         walk.h * w.G + part * p.heads, s.first + tok0);
    }
    __syncwarp();
    reinterpret_cast<float4*>(notes.lse + qs * 128)[lane] = make_float4(-lse[0], -lse[1], -lse[2], -lse[3]);
    reinterpret_cast<int4*>(notes.last + qs * 128)[lane] = make_int4(last[0], last[1], last[2], last[3]);
    ptx::mbar_arrive(&B.q_full[qs]);
    ++qi;
  };
  Walk walk;
  for (bool more = walk.begin(p); more && ok; more = walk.next(p)) {
    if (walk.single) {
      const Item it = {0, 0, 0, walk.s.n, 1};
      bring(walk, it, 0);
      continue;
    }
    for (int pair = walk.pair; pair < walk.pair_end && ok; ++pair) {
      const Item it = item_of(p, walk, pair);
#pragma unroll 1
      for (int c = 0; c < it.chunks && ok; ++c) bring(walk, it, c);
    }
  }
  if (!ok && lane == 0) {
    B.abort = 1;
    atomicOr(w.batch.status, kStatusProducer);
  }
  // no copy may land behind the CTA's end
  for (uint32_t i = qi > C::QS ? qi - C::QS : 0; i < qi; ++i) {
    const int never = 0;
    ptx::mbar_wait(&B.q_full[i % C::QS], i / C::QS & 1, 100000000ull, &never);
  }
}

template <int D>
__device__ void run_mma(const WeightTileParams& p, uint8_t* sm, Bars& B, uint32_t tmem) {
  using C = WeightTileCfg<D>;
  const volatile int* abort = &B.abort;
  const uint64_t k_desc = ptx::sdesc_sw128(ptx::smem_u32(sm), 16, 1024);
  const uint64_t q_desc = ptx::sdesc_sw128(ptx::smem_u32(sm) + C::OFF_Q, 16, 1024);
  uint32_t ki = 0, qi = 0, si[2] = {0, 0};
  bool ok = true;
  Walk walk;
  for (bool more = walk.begin(p); more && ok; more = walk.next(p)) {
    bool held = false;
#pragma unroll 1
    for (int pair = walk.pair; pair < walk.pair_end && ok; ++pair) {
      const Item it = item_of(p, walk, pair);
#pragma unroll 1
      for (int c = 0; c < it.chunks && ok; ++c) {
        const uint32_t qs = qi % C::QS;
        if (!held) ok = ptx::mbar_wait(&B.q_full[qs], qi / C::QS & 1, p.limit, abort);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        held = walk.single;
        const uint32_t idesc = ptx::idesc_bf16(128, (chunk_columns(p, it, c) + 15) & ~15, 0);
        const uint64_t q = q_desc + qs * (C::TILE >> 4);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          if (m >= it.tiles || !ok) break;
          const uint32_t k = ki + m, ks = k % C::KS, sb = si[m] & 1;
          if (c == 0) ok = ptx::mbar_wait(&B.k_full[ks], k / C::KS & 1, p.limit, abort);
          ok = ok && ptx::mbar_wait(&B.s_free[m][sb], (si[m] >> 1 & 1) ^ 1, p.limit, abort);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          ptx::tc_fence_after();
          const uint64_t a = k_desc + ks * (C::TILE >> 4);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = ((kk >> 2) * C::SUB + (kk & 3) * 32) >> 4;
            ptx::mma_ss_elect(tmem + m * 256 + sb * 128, a + off, q + off, idesc, kk > 0 ? 1u : 0u);
          }
          ptx::mma_commit_elect(&B.s_full[m][sb]);
          ++si[m];
        }
        if (!ok) break;
        if (!walk.single) {
          ptx::mma_commit_elect(&B.q_free[qs]);
          ++qi;
        }
      }
      if (it.chunks > 0 && ok) {
        for (int m = 0; m < it.tiles; ++m) ptx::mma_commit_elect(&B.k_free[(ki + m) % C::KS]);
        ki += it.tiles;
      }
    }
    if (walk.single && ok) {
      if (!held) ok = ptx::mbar_wait(&B.q_full[qi % C::QS], qi / C::QS & 1, p.limit, abort);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      ptx::mma_commit_elect(&B.q_free[qi % C::QS]);
      ++qi;
    }
  }
  if (!ok && (threadIdx.x & 31) == 0) {
    B.abort = 1;
    atomicOr(p.w.batch.status, kStatusMma);
  }
  __syncwarp();
  // every MMA this warp issued is complete once this commit lands
  ptx::mma_commit_elect(&B.drain);
  const int never = 0;
  ptx::mbar_wait(&B.drain, 0, 100000000ull, &never);
}

}  // namespace wtile

template <int D>
__global__ void __launch_bounds__(WeightTileCfg<D>::THREADS, 1)
    gdpa_cache_weights_tile_kernel(const __grid_constant__ WeightTileParams p) {
  using C = WeightTileCfg<D>;
  extern __shared__ uint8_t raw[];
  __shared__ wtile::Bars B;
  uint8_t* const sm = raw + ((1024 - (ptx::smem_u32(raw) & 1023)) & 1023);
  wtile::Notes notes;
  notes.factor = reinterpret_cast<float*>(sm + C::OFF_NOTES);
  notes.lse = notes.factor + C::KS * 128;
  notes.last = reinterpret_cast<int*>(notes.lse + C::QS * 128);
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::KS; ++i) ptx::mbar_init(&B.k_full[i], 128), ptx::mbar_init(&B.k_free[i], 1 + 4);
    for (int i = 0; i < C::QS; ++i) ptx::mbar_init(&B.q_full[i], 1 + 32), ptx::mbar_init(&B.q_free[i], 1 + 8);
    for (int m = 0; m < 2; ++m)
      for (int i = 0; i < 2; ++i) ptx::mbar_init(&B.s_full[m][i], 1), ptx::mbar_init(&B.s_free[m][i], 4);
    ptx::mbar_init(&B.drain, 1);
    B.abort = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 12) {
    ptx::tmem_alloc(&B.tmem, C::TM_COLS);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = B.tmem;
  if (warp < 8)
    wtile::run_sums<D>(p, B, notes, tmem);
  else if (warp < 12)
    wtile::run_convert<D>(p, sm, B, notes);
  else if (warp == 12)
    wtile::run_mma<D>(p, sm, B, tmem);
  else
    wtile::run_queries<D>(p, sm, B, notes);
  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == 12) ptx::tmem_dealloc(tmem, C::TM_COLS);
}

}  // namespace gdpa
