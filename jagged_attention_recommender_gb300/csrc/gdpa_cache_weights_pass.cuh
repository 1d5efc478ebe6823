// gdpa_cache_weights_pass.cuh -- the weight that stored keys receive from few
// rows (single tokens, drafted ones, candidates): the queries of a sequence and
// key head stay in shared memory, and its keys pass them, 128 at a time, on the
// 5th-generation tensor cores.
//
// Mathematics.  As in gdpa_cache_weights.cuh: S^T = K Q^T with keys on the 128
// lanes of TMEM, a key a thread.  Both operands are fp16: codes exactly, queries
// divided by their largest element's power of two as in gdpa_cache_fwd, which
// multiplies the column again.
//
// Bound: memory, D bytes a key and head, and 8 of its weight.
//
// Work split.  The tiles of 128 keys of all sequences and heads are counted from
// the lengths on the device, and every CTA takes an equal run of them; a group is
// the part of a run in one sequence and head.  Nothing waits for a load: codes
// come by bulk copies RAWS tiles ahead, scales and earlier weights by
// asynchronous copies, the next group's queries while the present one's are
// used.  Roles:
//   warps 0-15   the sums, a key a thread, a warpgroup every fourth tile
//   warps 16-19  convert K (128-byte swizzle)
//   warps 20-23  the queries: to fp16, with what goes with each column
//   warp 24      finds pages and issues the copies
//   warp 25      issues the MMAs
// Sequences with more rows than fit 128 columns are passed chunk by chunk, the
// queries converted anew for every tile.
#pragma once

#include "gdpa_cache_weights_mma.cuh"

namespace gdpa {

struct WeightPassParams {
  CacheWeightsParams w;
  int heads, tokens;  // of a chunk: heads * tokens <= 128 (heads: G, or 128 of more)
  int parts;          // chunks that the heads of a group make
  unsigned long long limit;
};

template <int D_>
struct WeightPassCfg {
  static constexpr int D = D_, THREADS = 832, COLS = 128;
  static constexpr int SUB = 128 * 128;  // 64 columns of a tile: 128 rows of 128 bytes
  static constexpr int TILE = D / 64 * SUB;
  static constexpr int RAW = 128 * D, RAWS = D == 128 ? 5 : 8;  // codes of a tile, on their way
  static constexpr int KS = D == 128 ? 2 : 3, QS = 2, NS = 8;   // stages of K, of Q, of keys' notes
  static constexpr int OFF_Q = KS * TILE, OFF_RAW = OFF_Q + QS * TILE, OFF_NOTES = OFF_RAW + RAWS * RAW;
  static constexpr int KEY_NOTES = 640, COLUMN_NOTES = 1536;
  static constexpr int USED = OFF_NOTES + NS * KEY_NOTES + QS * COLUMN_NOTES;
  static constexpr int SMEM = (USED > 120 * 1024 ? USED : 120 * 1024) + 1024;  // one CTA an SM (all of its TMEM)
  static constexpr uint32_t TM_COLS = 512;  // S of four tiles
  static_assert(SMEM <= 226 * 1024, "shared memory");
};

namespace wpass {

struct Bars {
  uint64_t raw_full[8], raw_free[8], k_full[3], k_free[3], q_full[2], q_free[2], n_full[8], n_free[8], s_full[4], s_free[4];
  uint64_t drain;
  uint32_t tmem;
  int abort;  // a wait has given up
};

// What goes with a column: its factor and minus its logsumexp, both in units
// of log2, and the last key that it sees.
struct ColumnNotes {
  float factor[128], lse[128];
  int last[128];
};

// First key that any row of a sequence sees, and its tiles.
__device__ __forceinline__ int see(const WeightPassParams& p, const CacheSeq& q) {
  return min(first_key(q.len - q.n, p.w.window), q.len);
}
__device__ __forceinline__ int tiles_of(const WeightPassParams& p, const CacheSeq& q) {
  if (!q.ok || q.n == 0 || q.len == 0) return 0;
  const int from = p.w.keep ? see(p, q) & ~127 : 0;
  return static_cast<int>((static_cast<unsigned>(q.len - from) + 127) >> 7);
}

// A CTA's run of the tiles: [at, stop), counted from sequence `seq`'s first.
struct Run {
  int64_t scan[32];
  int64_t at, stop;
  int seq;
};
template <int THREADS>
__device__ __forceinline__ void find_run(const WeightPassParams& p, Run& run) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, B = p.w.batch.B;
  const int per = (B + THREADS - 1) / THREADS, b_lo = min(B, tid * per), b_hi = min(B, b_lo + per);
  auto tiles = [&](int b) {
    return static_cast<int64_t>(tiles_of(p, load_sequence(p.w.batch, p.w.cache.lp, b))) * p.w.cache.H;
  };
  int64_t mine = 0;
  for (int b = b_lo; b < b_hi; ++b) mine += tiles(b);
  int64_t incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += x;
  }
  if (lane == 31) run.scan[warp] = incl;
  if (tid == 0) run.seq = 0, run.at = run.stop = 0;
  __syncthreads();
  int64_t total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) incl += run.scan[w];
    total += run.scan[w];
  }
  const int64_t chunk = split::quotient(total + gridDim.x - 1, gridDim.x);
  const int64_t from = chunk * blockIdx.x, to = min(total, from + chunk);
  if (from < total && from >= incl - mine && from < incl) {
    int64_t before = incl - mine;
    int b = b_lo;
    for (; b < b_hi; ++b) {
      const int64_t n = tiles(b);
      if (from < before + n) break;
      before += n;
    }
    run.seq = b;
    run.at = from - before;
    run.stop = to - before;
  }
  __syncthreads();
}

// The groups of a run, in order, by a whole warp: its lanes hold 32 sequences, so
// that the next group is found without a load.
struct Walk {
  int64_t upto;      // tiles of the sequences up to this lane's
  CacheSeq lane_s;   // this lane's sequence
  int64_t at, stop;  // the rest of the run, counted from the first lane's sequence
  int base;          // that sequence
  // the present group
  CacheSeq s;
  int b, h, kbase, tile, tile_end;
  int seen;    // its first tile that a row sees
  int chunks;  // of the sequence's rows

  __device__ __forceinline__ void load(const WeightPassParams& p) {
    const int lane = threadIdx.x & 31;
    lane_s = CacheSeq{0, 0, 0, 0};
    if (base + lane < p.w.batch.B) lane_s = load_sequence(p.w.batch, p.w.cache.lp, base + lane);
    upto = static_cast<int64_t>(tiles_of(p, lane_s)) * p.w.cache.H;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += x;
    }
  }
  __device__ __forceinline__ bool settle(const WeightPassParams& p) {
    if (at >= stop) return false;
    while (true) {
      const int64_t all = __shfl_sync(0xffffffffu, upto, 31);
      if (at < all) break;
      at -= all;
      stop -= all;
      if (p.w.batch.B - base <= 32) return false;
      base += 32;
      load(p);
    }
    const int i = __popc(__ballot_sync(0xffffffffu, upto <= at));
    const int64_t before = __shfl_sync(0xffffffffu, upto, max(i - 1, 0));
    s.first = __shfl_sync(0xffffffffu, lane_s.first, i);
    s.n = __shfl_sync(0xffffffffu, lane_s.n, i);
    s.len = __shfl_sync(0xffffffffu, lane_s.len, i);
    s.ok = 1;
    b = base + i;
    const int64_t rest = at - (i > 0 ? before : 0);
    const int tiles = tiles_of(p, s), from = see(p, s);
    h = static_cast<int>(split::quotient(rest, tiles));
    tile = static_cast<int>(rest - static_cast<int64_t>(h) * tiles);
    tile_end = static_cast<int>(min(static_cast<int64_t>(tiles), tile + (stop - at)));
    kbase = p.w.keep ? from & ~127 : 0;
    seen = max(tile, (from - kbase) >> 7);
    chunks = p.parts == 1 && s.n <= p.tokens ? 1 : (s.n + p.tokens - 1) / p.tokens * p.parts;
    return true;
  }
  __device__ __forceinline__ bool begin(const WeightPassParams& p, const Run& run) {
    base = run.seq;
    at = run.at;
    stop = run.stop;
    if (at >= stop) return false;
    load(p);
    return settle(p);
  }
  __device__ __forceinline__ bool next(const WeightPassParams& p) {
    at += tile_end - tile;
    return settle(p);
  }
};

// Chunk c of a sequence's rows: its first token, the part of its tokens' heads,
// and its columns, to the last one that is a row.
struct Chunk {
  int tok, part, tokens, columns;
};
__device__ __forceinline__ Chunk chunk_of(const WeightPassParams& p, const Walk& w, int c) {
  Chunk k;
  k.part = p.parts == 1 ? 0 : c % p.parts;
  k.tok = (p.parts == 1 ? c : c / p.parts) * p.tokens;
  k.tokens = min(p.tokens, w.s.n - k.tok);
  k.columns = (k.tokens - 1) * p.heads + min(p.heads, p.w.G - k.part * p.heads);
  return k;
}

template <int D>
__device__ void run_sums(const WeightPassParams& p, const Run& run, Bars& B, const KeyNotes* keys, const ColumnNotes* columns, uint32_t tmem) {
  using C = WeightPassCfg<D>;
  const CacheWeightsParams& w = p.w;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t mine = warp >> 2;  // this warpgroup's tiles, of every four, and its buffer of S
  const int key_in = (warp & 3) * 32 + lane;
  const uint32_t from = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + mine * 128;
  const volatile int* abort = &B.abort;
  StageRing n, q;         // of this warpgroup's notes (two of the eight stages), of chunks
  uint32_t count = 0, s_turn = 0;
  bool ok = true;
  Walk walk;
  for (bool more = walk.begin(p, run); more && ok; more = walk.next(p)) {
    const CacheSeq& s = walk.s;
    const bool single = walk.chunks == 1;
    bool held = false;  // this group's only chunk is there
#pragma unroll 1
    for (int tile = walk.tile; tile < walk.tile_end; ++tile, ++count) {
      const bool due = (count & 3) == mine, seen = tile >= walk.seen;
      if (!due && (single || !seen)) continue;
      const int k0 = walk.kbase + (tile << 7), key = k0 + key_in;
      int64_t row = -1;
      float old = 0.0f, factor = 0.0f;
      if (due) {
        const uint32_t stage = n.at * 4 + mine;
        ok = ptx::mbar_wait(&B.n_full[stage], n.turn, p.limit, abort);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const KeyNotes& note = keys[stage];
        row = note.row[key_in >> 4];
        factor = note.scale(key_in);
        if (w.w_in && s.len - s.n - k0 > key_in) old = w.decay * note.old[key_in];
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&B.n_free[stage]);
        n.next(2);
      }
      const uint64_t f2 = ptx::f2_splat(factor);
      uint64_t sum[2] = {0, 0};
      const int k_last = k0 + min(127, s.len - 1 - k0);
#pragma unroll 1
      for (int c = 0; c < (seen ? walk.chunks : 0); ++c) {
        if (!held) ok = ptx::mbar_wait(&B.q_full[q.at], q.turn, p.limit, abort);
        held = single;
        if (ok && due) ok = ptx::mbar_wait(&B.s_full[mine], s_turn, p.limit, abort);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (due) {
          s_turn ^= 1;
          ptx::tc_fence_after();
          const Chunk k = chunk_of(p, walk, c);
          const int first = w.causal ? s.len - s.n + k.tok : s.len - 1;  // the last key that the first row sees
          const int end = w.causal ? first + k.tokens - 1 : first;       // ... and the last one
          const bool all = first >= k_last && (w.window == 0 || end - w.window < k0);
          const ColumnNotes& col = columns[q.at];
          const int blocks = (k.columns + 15) >> 4;
#pragma unroll 1
          for (int i = 0; i < blocks; ++i) {
            uint32_t r[16];
            ptx::tmem_read16(from + i * 16, r);
            if (i == blocks - 1) {  // the buffer is read
              ptx::tc_fence_before();
              __syncwarp();
              if (lane == 0) ptx::mbar_arrive(&B.s_free[mine]);
              __syncwarp();
            }
            const ulonglong2* fac = reinterpret_cast<const ulonglong2*>(col.factor + i * 16);
            const ulonglong2* lse = reinterpret_cast<const ulonglong2*>(col.lse + i * 16);
            const int4* last = reinterpret_cast<const int4*>(col.last + i * 16);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const ulonglong2 f = fac[j], l = lse[j];
              const uint64_t x = ptx::f2_pack(__uint_as_float(r[4 * j]), __uint_as_float(r[4 * j + 1]));
              const uint64_t y = ptx::f2_pack(__uint_as_float(r[4 * j + 2]), __uint_as_float(r[4 * j + 3]));
              float a, b, d, e;
              ptx::f2_unpack(ptx::f2_fma(x, ptx::f2_mul(f.x, f2), l.x), a, b);
              ptx::f2_unpack(ptx::f2_fma(y, ptx::f2_mul(f.y, f2), l.y), d, e);
              a = ptx::ex2_approx(a), b = ptx::ex2_approx(b), d = ptx::ex2_approx(d), e = ptx::ex2_approx(e);
              if (!all) {
                const int4 t = last[j];
                const int w1 = w.window > 0 ? w.window : 0x7fffffff;  // (key > last - window; none: always)
                if (key > t.x || key <= t.x - w1) a = 0.0f;
                if (key > t.y || key <= t.y - w1) b = 0.0f;
                if (key > t.z || key <= t.z - w1) d = 0.0f;
                if (key > t.w || key <= t.w - w1) e = 0.0f;
              }
              sum[0] = ptx::f2_add(sum[0], ptx::f2_pack(a, b));
              sum[1] = ptx::f2_add(sum[1], ptx::f2_pack(d, e));
            }
          }
        }
        if (!single) {
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&B.q_free[q.at]);
          q.next(C::QS);
        }
      }
      if (!ok) break;
      if (due && row >= 0 && s.len - k0 > key_in) {
        float a, b, d, e;
        ptx::f2_unpack(sum[0], a, b);
        ptx::f2_unpack(sum[1], d, e);
        w.w[row + (key_in & 15)] = old + ((a + b) + (d + e));
      }
      __syncwarp();
    }
    if (!ok) break;
    if (single) {
      if (!held) {  // (every warp sees every chunk arrive: one that skipped some could take a later turn for its own)
        ok = ptx::mbar_wait(&B.q_full[q.at], q.turn, p.limit, abort);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&B.q_free[q.at]);
      q.next(C::QS);
    }
  }
  if (!ok && lane == 0) {
    B.abort = 1;
    atomicOr(w.batch.status, kStatusActivation);
  }
}

template <int D>
__device__ void run_convert(const WeightPassParams& p, const Run& run, uint8_t* sm, Bars& B) {
  using C = WeightPassCfg<D>;
  constexpr int CPR = D / 16, ROWS = 128 / CPR, N = 128 / ROWS;  // chunks of a key; keys of a pass; passes
  const int tid = threadIdx.x - 512, lane = tid & 31;
  const volatile int* abort = &B.abort;
  const int r0 = tid / CPR, c = tid % CPR;  // its row in a pass, and 16 coordinates
  const uint32_t raw = ptx::smem_u32(sm) + C::OFF_RAW + tid * 16;
  // 16-byte chunks 2c and 2c + 1 of a row, 64 columns a sub-tile (a pass's rows are 8 or 16 or 32: r & 7 is r0's)
  const uint32_t j = 2 * c & 7, base = ptx::smem_u32(sm) + (c >> 2) * C::SUB + r0 * 128;
  const uint32_t to0 = base + ((j ^ (r0 & 7)) << 4), to1 = base + (((j + 1) ^ (r0 & 7)) << 4);
  StageRing in, k;
  bool ok = true;
  Walk walk;
  for (bool more = walk.begin(p, run); more && ok; more = walk.next(p)) {
#pragma unroll 1
    for (int tile = walk.seen; tile < walk.tile_end; ++tile) {
      ok = ptx::mbar_wait(&B.raw_full[in.at], in.turn, p.limit, abort);
      uint32_t x[N][4];
      if (ok) {
#pragma unroll
        for (int i = 0; i < N; ++i) split::lds128(raw + in.at * C::RAW + i * 2048, x[i]);
        ok = ptx::mbar_wait(&B.k_free[k.at], k.turn ^ 1, p.limit, abort);
      }
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const uint32_t at = k.at * C::TILE + i * ROWS * 128;
        ptx::st_shared_v4(to0 + at, split::codes_lo(x[i][0]), split::codes_hi(x[i][0]), split::codes_lo(x[i][1]),
                          split::codes_hi(x[i][1]));
        ptx::st_shared_v4(to1 + at, split::codes_lo(x[i][2]), split::codes_hi(x[i][2]), split::codes_lo(x[i][3]),
                          split::codes_hi(x[i][3]));
      }
      ptx::fence_proxy_async_smem();
      ptx::mbar_arrive(&B.k_full[k.at]);
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&B.raw_free[in.at]);
      in.next(C::RAWS);
      k.next(C::KS);
    }
  }
  if (!ok && lane == 0) {
    B.abort = 1;
    atomicOr(p.w.batch.status, kStatusProducer);
  }
}

template <int D>
__device__ void run_queries(const WeightPassParams& p, const Run& run, uint8_t* sm, Bars& B, ColumnNotes* columns) {
  using C = WeightPassCfg<D>;
  constexpr int LPR = D / 8, ROWS = 128 / LPR;  // lanes of a row; rows of a pass of the four warps
  const CacheWeightsParams& w = p.w;
  const int tid = threadIdx.x - 640, lane = tid & 31;
  const volatile int* abort = &B.abort;
  const int r0 = tid / LPR, c = tid % LPR;
  const uint32_t base = ptx::smem_u32(sm) + C::OFF_Q + (c >> 3) * C::SUB;
  StageRing q;
  bool ok = true;
  auto bring = [&](const Walk& walk, int chunk) {
    const CacheSeq& s = walk.s;
    const Chunk k = chunk_of(p, walk, chunk);
    ok = ptx::mbar_wait_idle(&B.q_free[q.at], q.turn ^ 1, p.limit, abort);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) return;
    ColumnNotes& col = columns[q.at];
    const int rows = (k.columns + 15) & ~15;
#pragma unroll 2
    for (int r1 = 0; r1 < rows; r1 += ROWS) {  // (rows past `rows` are written too: there are 128)
      const int r = r1 + r0, t = r / p.heads, head = k.part * p.heads + r - t * p.heads;
      const bool row = t < k.tokens && head < w.G;
      uint4 u = make_uint4(0, 0, 0, 0);
      float lse = -INFINITY;
      if (row) {
        u = __ldg(reinterpret_cast<const uint4*>(w.q + (s.first + k.tok + t) * w.q_stride + (walk.h * w.G + head) * D + c * 8));
        lse = __ldg(w.lse + static_cast<int64_t>(s.first + k.tok + t) * w.Hq + walk.h * w.G + head);
      }
      const uint32_t x[4] = {u.x, u.y, u.z, u.w};
      float v[8], amax = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(x[i] << 16);
        v[2 * i + 1] = __uint_as_float(x[i] & 0xffff0000u);
        amax = fmaxf(amax, fmaxf(fabsf(v[2 * i]), fabsf(v[2 * i + 1])));
      }
#pragma unroll
      for (int d = LPR / 2; d > 0; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, d));
      // 2^e: the largest element's power of two (1 for an all-zero row)
      const int e = amax > 0.0f ? min(max(static_cast<int>(__float_as_uint(amax) >> 23) - 127, -126), 127) : 0;
      const float inv = sf_value(127 - e);
      ptx::st_shared_v4(base + q.at * C::TILE + r * 128 + (((c & 7) ^ (r & 7)) << 4),
                        split::pack_f16x2(v[0] * inv, v[1] * inv), split::pack_f16x2(v[2] * inv, v[3] * inv),
                        split::pack_f16x2(v[4] * inv, v[5] * inv), split::pack_f16x2(v[6] * inv, v[7] * inv));
      if (c == 0) {
        col.factor[r] = row ? sf_value(127 + e) * w.scale2 : 0.0f;
        col.lse[r] = lse == -INFINITY ? -INFINITY : -lse * kLog2e;  // (a row that saw nothing gives nothing)
        col.last[r] = w.causal ? s.len - s.n + k.tok + t : s.len - 1;
      }
    }
    ptx::fence_proxy_async_smem();
    ptx::mbar_arrive(&B.q_full[q.at]);
    q.next(C::QS);
  };
  Walk walk;
  for (bool more = walk.begin(p, run); more && ok; more = walk.next(p)) {
    if (walk.chunks == 1) {
      bring(walk, 0);
      continue;
    }
    for (int tile = walk.seen; tile < walk.tile_end && ok; ++tile)
#pragma unroll 1
      for (int chunk = 0; chunk < walk.chunks && ok; ++chunk) bring(walk, chunk);
  }
  if (!ok && lane == 0) {
    B.abort = 1;
    atomicOr(w.batch.status, kStatusProducer);
  }
}

template <int D>
__device__ void run_copies(const WeightPassParams& p, const Run& run, uint8_t* sm, Bars& B, KeyNotes* keys) {
  using C = WeightPassCfg<D>;
  const CacheWeightsParams& w = p.w;
  const int lane = threadIdx.x & 31;
  const volatile int* abort = &B.abort;
  const int pmask = (1 << w.cache.lp) - 1;
  const uint32_t raw = ptx::smem_u32(sm) + C::OFF_RAW;
  StageRing in, n;
  uint32_t count = 0;
  bool ok = true;
  Walk walk;
  bool more = walk.begin(p, run);
  int tile = more ? walk.tile : 0;
  // lane i: the page of the tile's i-th block of 16 keys
  auto page_of = [&]() {
    const int k0 = walk.kbase + (tile << 7);
    if (lane >= 8 || walk.s.len - k0 <= lane * 16) return -1;
    return load_page(w.cache, w.batch, walk.b, k0 + lane * 16);
  };
  int page = more ? page_of() : -1;  // (looked up a tile ahead)
  __syncwarp();
  while (more) {
    const int k0 = walk.kbase + (tile << 7);
    const bool seen = tile >= walk.seen;
    const int64_t row = page >= 0 ? cache_row(w.cache, page, walk.h, (k0 + lane * 16) & pmask) : -1;
    if (++tile == walk.tile_end) {
      more = walk.next(p);
      tile = walk.tile;
    }
    page = more ? page_of() : -1;
    __syncwarp();
    ok = ptx::mbar_wait(&B.n_free[n.at], n.turn ^ 1, p.limit, abort);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) break;
    bring_notes(w, keys[n.at], &B.n_full[n.at], row);
    n.next(C::NS);
    if (!seen) continue;
    ok = ptx::mbar_wait(&B.raw_free[in.at], in.turn ^ 1, p.limit, abort);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) break;
    bring_codes<D>(w, raw + in.at * C::RAW, &B.raw_full[in.at], row);
    in.next(C::RAWS);
    ++count;
  }
  if (!ok && lane == 0) {
    B.abort = 1;
    atomicOr(w.batch.status, kStatusProducer);
  }
  // no copy may land behind the CTA's end: this thread's own, and the last turn of every stage
  split::cp_commit();
  split::cp_wait<0>();
  drain_stages(B.raw_full, in, C::RAWS, count);
}

template <int D>
__device__ void run_mma(const WeightPassParams& p, const Run& run, uint8_t* sm, Bars& B, uint32_t tmem) {
  using C = WeightPassCfg<D>;
  const volatile int* abort = &B.abort;
  const uint64_t k_desc = ptx::sdesc_sw128(ptx::smem_u32(sm), 16, 1024);
  const uint64_t q_desc = ptx::sdesc_sw128(ptx::smem_u32(sm) + C::OFF_Q, 16, 1024);
  StageRing k, q;
  uint32_t count = 0, s_turns = 0;  // s_turns: a bit for each buffer
  bool ok = true;
  Walk walk;
  for (bool more = walk.begin(p, run); more && ok; more = walk.next(p)) {
    const bool single = walk.chunks == 1;
    bool held = false;
    count += walk.seen - walk.tile;
#pragma unroll 1
    for (int tile = walk.seen; tile < walk.tile_end && ok; ++tile, ++count) {
      const uint32_t sb = count & 3;
#pragma unroll 1
      for (int c = 0; c < walk.chunks; ++c) {
        if (!held) ok = ptx::mbar_wait(&B.q_full[q.at], q.turn, p.limit, abort);
        held = single;
        if (ok && c == 0) ok = ptx::mbar_wait(&B.k_full[k.at], k.turn, p.limit, abort);
        if (ok) ok = ptx::mbar_wait(&B.s_free[sb], (s_turns >> sb & 1) ^ 1, p.limit, abort);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        s_turns ^= 1u << sb;
        ptx::tc_fence_after();
        const uint32_t idesc = ptx::idesc_f16(128, (chunk_of(p, walk, c).columns + 15) & ~15, 0);
        const uint64_t a = k_desc + k.at * (C::TILE >> 4), b = q_desc + q.at * (C::TILE >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * C::SUB + (kk & 3) * 32) >> 4;
          ptx::mma_ss_elect(tmem + sb * 128, a + off, b + off, idesc, kk > 0 ? 1u : 0u);
        }
        ptx::mma_commit_elect(&B.s_full[sb]);
        if (c == walk.chunks - 1) ptx::mma_commit_elect(&B.k_free[k.at]);
        if (!single) {
          ptx::mma_commit_elect(&B.q_free[q.at]);
          q.next(C::QS);
        }
      }
      k.next(C::KS);
    }
    if (walk.seen > walk.tile_end) count -= walk.seen - walk.tile_end;
    if (single && ok) {
      if (!held) ok = ptx::mbar_wait(&B.q_full[q.at], q.turn, p.limit, abort);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      ptx::mma_commit_elect(&B.q_free[q.at]);
      q.next(C::QS);
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

}  // namespace wpass

template <int D>
__global__ void __launch_bounds__(WeightPassCfg<D>::THREADS, 1)
    gdpa_cache_weights_pass_kernel(const __grid_constant__ WeightPassParams p) {
  using C = WeightPassCfg<D>;
  extern __shared__ uint8_t raw[];
  __shared__ wpass::Bars B;
  uint8_t* const sm = raw + ((1024 - (ptx::smem_u32(raw) & 1023)) & 1023);
  static_assert(sizeof(KeyNotes) <= C::KEY_NOTES && sizeof(wpass::ColumnNotes) == C::COLUMN_NOTES, "notes");
  KeyNotes* const keys = reinterpret_cast<KeyNotes*>(sm + C::OFF_NOTES);
  wpass::ColumnNotes* const columns = reinterpret_cast<wpass::ColumnNotes*>(sm + C::OFF_NOTES + C::NS * C::KEY_NOTES);
  __shared__ wpass::Run run;
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::RAWS; ++i) ptx::mbar_init(&B.raw_full[i], 1), ptx::mbar_init(&B.raw_free[i], 4);
    for (int i = 0; i < C::KS; ++i) ptx::mbar_init(&B.k_full[i], 128), ptx::mbar_init(&B.k_free[i], 1);
    for (int i = 0; i < C::QS; ++i) ptx::mbar_init(&B.q_full[i], 128), ptx::mbar_init(&B.q_free[i], 1 + 16);
    for (int i = 0; i < C::NS; ++i) ptx::mbar_init(&B.n_full[i], 1 + 32), ptx::mbar_init(&B.n_free[i], 4);
    for (int i = 0; i < 4; ++i) ptx::mbar_init(&B.s_full[i], 1), ptx::mbar_init(&B.s_free[i], 4);
    ptx::mbar_init(&B.drain, 1);
    B.abort = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 25) {
    ptx::tmem_alloc(&B.tmem, C::TM_COLS);
    ptx::tmem_relinquish();
  }
  wpass::find_run<C::THREADS>(p, run);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = B.tmem;
  if (warp < 16)
    wpass::run_sums<D>(p, run, B, keys, columns, tmem);
  else if (warp < 20)
    wpass::run_convert<D>(p, run, sm, B);
  else if (warp < 24)
    wpass::run_queries<D>(p, run, sm, B, columns);
  else if (warp == 24)
    wpass::run_copies<D>(p, run, sm, B, keys);
  else
    wpass::run_mma<D>(p, run, sm, B, tmem);
  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == 25) ptx::tmem_dealloc(tmem, C::TM_COLS);
}

}  // namespace gdpa
