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
// Bound: the chain of hand-overs around the special-function unit, which takes four
// cycles for a warp's 32 exponentials (measured), 512 for 128 keys and 128 rows, as
// long as their products at D = 128 do.  Measured: 2321 prompt rows behind 2100 to
// 8192 keys, 32 query and 8 key heads of 128, 108 to 111 us (865 to 890 TFLOP/s; the tensor
// core's floor is 50); a warp is at its columns for half of that, the rest is waiting and
// the work around a chunk and an item.  Eight roles share the instruction caches, so
// their code is kept short: loops that are not unrolled, one copy of the waits' loop
// (128 rows of 48 sequences 67 us instead of 93).  25 warps leave 72 registers: 40 bytes
// of a thread's stack are spilled to (56 stored, 88 loaded).  Through windows, keys that no row sees cost their items' round of the roles:
// 100 rows of 64 sequences of 6000 keys, 8 heads of 128, a window of 512, fading, 108 us.
//
// Work split.  An item is 256 keys of a sequence and head, converted once and kept
// in shared memory while all rows that see any of them pass in chunks of 128
// columns (tokens times heads of the group).  CTAs take items there and back over
// the grid.  Roles:
//   warps 0-15   the sums, a key a thread: warpgroups 0 and 2 those of the item's
//                first 128 keys, 1 and 3 of its second, each every other chunk
//   warps 16-19  convert K (128-byte swizzle)
//   warp 20      issues the MMAs
//   warp 21      brings the queries by TMA
//   warp 22      notes their logsumexp and the last keys they see
//   warp 23      finds pages and brings codes, scales and earlier weights
//   warp 24      finds the items, and notes them for the others (each of which
//                took 4600 cycles an item to find them itself)
#pragma once

#include "gdpa_cache_append.cuh"
#include "gdpa_cache_order.h"
#include "gdpa_cache_weights_mma.cuh"

namespace gdpa {

struct WeightTileParams {
  CUtensorMap tm_q;  // [T, Hq, D] bf16, boxes of 64 x heads x tokens, 128-byte swizzle
  CacheWeightsParams w;
  int heads, tokens;  // of a chunk: heads * tokens <= 128 (heads: G, or 128 of more)
  int parts;          // chunks that the heads of a group make
  unsigned long long limit;
};

template <int D_>
struct WeightTileCfg {
  static constexpr int D = D_, THREADS = 800, COLS = 128;
  static constexpr int SUB = 128 * 128;            // 64 columns of a tile: 128 rows of 128 bytes
  static constexpr int TILE = D / 64 * SUB;
  // stages of K, of Q (a chunk's way from L2 is longer than its products), of notes
  // (a third of K, and two of Q at D = 128 for its room: 2321 prompt rows 110.0 us for 110.1,
  // 200 rows of 128 samples at D = 64 330 for 320)
  static constexpr int KS = 2, QS = 3, NS = 4;
  static constexpr int RAW = 128 * D, RAWS = D == 128 ? 3 : 6;  // codes of a tile, on their way
  static constexpr int OFF_Q = KS * TILE, OFF_RAW = OFF_Q + QS * TILE, OFF_NOTES = OFF_RAW + RAWS * RAW;
  static constexpr int USED = OFF_NOTES + NS * 640 + NS * 1024 + 1024 + NS * 16 + NS * 48;
  static constexpr int SMEM = (USED > 120 * 1024 ? USED : 120 * 1024) + 1024;  // one CTA an SM (all of its TMEM)
  static constexpr uint32_t TM_COLS = 512;         // S of two tiles, two buffers each
  static_assert(SMEM <= 226 * 1024, "shared memory");
};

namespace wtile {

struct Bars {
  uint64_t item_full[4], item_free[4];                          // items
  uint64_t raw_full[6], raw_free[6], k_full[2], k_free[2];      // tiles' codes, and converted
  uint64_t key_full[4], key_free[4];                            // tiles' notes
  uint64_t q_full[3], q_free[3], n_full[4], n_free[4];          // chunks' queries, and notes
  uint64_t s_full[2][2], s_free[2][2], x_full[2], x_free[2], drain;  // of a tile of an item and buffer; sums' halves
  uint32_t tmem;
  int abort;  // a wait has given up
};

struct Notes {
  int4* item;     // [NS][3]: items: first key, tiles, first and last token; chunks (-1: no more), sequence, head; its rows
  KeyNotes* key;  // [NS]: of tiles of keys
  float* lse;     // [NS][128]: minus each column's logsumexp, in units of log2
  int* last;      // [NS][128]: the last key that each column sees, -1 for none
  float* half;    // [2][128]: sums on their way from one warpgroup to the other
  int4* chunk;    // [NS]: its columns' blocks of 32, how many of them hold rows alone, the last keys of its first and last row
};

// An item: its first key, its tiles, and the tokens [lo, hi) whose rows see any of
// it, in chunks.
struct Item {
  int k0, tiles, lo, hi, chunks;
};

// The items of one CTA, in order, by a whole warp: its lanes hold 32 sequences, so
// that the next item is found without a load.
struct Finder {
  int64_t upto;     // items of the sequences up to this lane's
  CacheSeq lane_s;  // this lane's sequence
  int64_t idx;      // the present item, counted from the first lane's sequence
  int base;         // that sequence
  bool back;
  // the present item
  CacheSeq s;
  int b, h;
  Item it;

  __device__ __forceinline__ int first_stored(const WeightTileParams& p, const CacheSeq& q) const {
    return p.w.keep ? min(first_key(q.len - q.n, p.w.window), q.len) & ~255 : 0;
  }
  __device__ __forceinline__ int items_of(const WeightTileParams& p, const CacheSeq& q) const {
    return static_cast<int>((static_cast<unsigned>(q.len - first_stored(p, q)) + 255) >> 8);
  }
  __device__ __forceinline__ void load(const WeightTileParams& p) {
    const int lane = threadIdx.x & 31;
    lane_s = CacheSeq{0, 0, 0, 0};
    if (base + lane < p.w.batch.B) lane_s = load_sequence(p.w.batch, p.w.cache.lp, base + lane);
    upto = 0;
    if (lane_s.ok && lane_s.n > 0 && lane_s.len > 0) upto = static_cast<int64_t>(items_of(p, lane_s)) * p.w.cache.H;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += x;
    }
  }
  __device__ __forceinline__ bool settle(const WeightTileParams& p) {
    while (true) {
      const int64_t all = __shfl_sync(0xffffffffu, upto, 31);
      if (idx < all) break;
      idx -= all;
      if (p.w.batch.B - base <= 32) return false;
      base += 32;
      load(p);
    }
    const int at = __popc(__ballot_sync(0xffffffffu, upto <= idx));
    const int64_t before = __shfl_sync(0xffffffffu, upto, max(at - 1, 0));
    s.first = __shfl_sync(0xffffffffu, lane_s.first, at);
    s.n = __shfl_sync(0xffffffffu, lane_s.n, at);
    s.len = __shfl_sync(0xffffffffu, lane_s.len, at);
    s.ok = 1;
    b = base + at;
    const int64_t i = idx - (at > 0 ? before : 0);
    const int items = items_of(p, s);
    h = static_cast<int>(split::quotient(i, items));
    it.k0 = first_stored(p, s) + (static_cast<int>(i - static_cast<int64_t>(h) * items) << 8);
    it.tiles = s.len - it.k0 > 128 ? 2 : 1;
    const int last = it.k0 + min(255, s.len - 1 - it.k0);
    it.lo = rows_of_key(s, it.k0, p.w.causal, p.w.window).lo;
    it.hi = rows_of_key(s, last, p.w.causal, p.w.window).hi;
    it.chunks = it.hi > it.lo ? (it.hi - it.lo + p.tokens - 1) / p.tokens * p.parts : 0;
    return true;
  }
  __device__ __forceinline__ bool begin(const WeightTileParams& p) {
    base = 0;
    back = false;
    idx = blockIdx.x;
    load(p);
    return settle(p);
  }
  __device__ __forceinline__ bool next(const WeightTileParams& p) {
    back = !back;  // there and back: neighbours' costs are alike
    idx += 2 * static_cast<int64_t>(back ? gridDim.x - 1 - blockIdx.x : blockIdx.x) + 1;
    return settle(p);
  }
};

__device__ void run_items(const WeightTileParams& p, Bars& B, const Notes& notes) {
  const int lane = threadIdx.x & 31;
  const volatile int* abort = &B.abort;
  StageRing ring;
  Finder find;
  bool more = find.begin(p), ok = true;
  while (true) {
    ok = ptx::mbar_wait_idle(&B.item_free[ring.at], ring.turn ^ 1, p.limit, abort);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) break;
    if (lane == 0) {
      int4* const to = notes.item + ring.at * 3;
      to[0] = make_int4(find.it.k0, find.it.tiles, find.it.lo, find.it.hi);
      to[1] = make_int4(more ? find.it.chunks : -1, find.b, find.h, 0);
      to[2] = make_int4(find.s.first, find.s.n, find.s.len, find.s.ok);
      ptx::mbar_arrive(&B.item_full[ring.at]);
    }
    __syncwarp();
    ring.next(4);
    if (!more) break;
    more = find.next(p);
  }
  if (!ok && lane == 0) {
    B.abort = 1;
    atomicOr(p.w.batch.status, kStatusProducer);
  }
}

// The items as the other warps read them, every one of them.
struct Walk {
  StageRing ring;
  CacheSeq s;
  Item it;
  int b, h;
  bool ok = true;  // false: a wait has given up
  __device__ __forceinline__ bool next(const WeightTileParams& p, Bars& B, const Notes& notes) {
    ok = ptx::mbar_wait_near(&B.item_full[ring.at], ring.turn, p.limit, &B.abort);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) return false;
    const int4 x = notes.item[ring.at * 3], y = notes.item[ring.at * 3 + 1], z = notes.item[ring.at * 3 + 2];
    __syncwarp();
    if ((threadIdx.x & 31) == 0) ptx::mbar_arrive(&B.item_free[ring.at]);
    ring.next(4);
    it.k0 = x.x, it.tiles = x.y, it.lo = x.z, it.hi = x.w;
    it.chunks = y.x, b = y.y, h = y.z;
    s.first = z.x, s.n = z.y, s.len = z.z, s.ok = z.w;
    return it.chunks >= 0;
  }
  // To the next item that any row sees.
  __device__ __forceinline__ bool next_seen(const WeightTileParams& p, Bars& B, const Notes& notes) {
    do
      if (!next(p, B, notes)) return false;
    while (it.chunks == 0);
    return true;
  }
};

// Columns of chunk c, to the last one that is a row.
__device__ __forceinline__ int chunk_columns(const WeightTileParams& p, const Item& it, int c) {
  const int part = p.parts == 1 ? 0 : c % p.parts, tok = it.lo + (p.parts == 1 ? c : c / p.parts) * p.tokens;
  return (min(p.tokens, it.hi - tok) - 1) * p.heads + min(p.heads, p.w.G - part * p.heads);
}

template <int D>
__device__ void run_sums(const WeightTileParams& p, Bars& B, const Notes& notes, uint32_t tmem) {
  using C = WeightTileCfg<D>;
  const CacheWeightsParams& w = p.w;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int m = warp >> 2 & 1;        // this warpgroup's tile of an item ...
  const uint32_t turn = warp >> 3;    // ... and its chunks, of every two: their notes and buffer of S
  const int key_in = (warp & 3) * 32 + lane;
  const uint32_t from = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + m * 256 + turn * 128;
  const volatile int* abort = &B.abort;
  const int pmask = (1 << w.cache.lp) - 1;
  StageRing k, n;                      // of tiles' notes, of this warpgroup's notes (two of the four stages)
  uint32_t ci = 0, s_turn = 0, xi = 0;  // chunks, turns of S's buffer, and sums in two halves, so far
  bool ok = true;
  Walk walk;
  while (ok && walk.next(p, B, notes)) {
    const CacheSeq& s = walk.s;
    const Item it = walk.it;
    const bool mine = m < it.tiles;
    const int k0 = it.k0 + m * 128, key = k0 + key_in;
    if (it.chunks == 0) {  // no row sees these keys: earlier weights alone
      if (mine && turn == 0 && s.len - k0 > key_in) {
        const int page = load_page(w.cache, w.batch, walk.b, key);
        if (page >= 0) {
          const int64_t row = cache_row(w.cache, page, walk.h, key & pmask);
          w.w[row] = w.w_in && key < s.len - s.n ? w.decay * w.w_in[row] : 0.0f;
        }
      }
      __syncwarp();
      continue;
    }
    // (every warp sees every tile's notes arrive: one that skipped some could
    // take a later turn of a stage for the one it waits for)
    int64_t row = -1;
    float old = 0.0f, factor = 0.0f;
#pragma unroll 1
    for (int j = 0; j < it.tiles; ++j) {
      ok = ptx::mbar_wait_near(&B.key_full[k.at], k.turn, p.limit, abort);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      if (j == m) {
        const KeyNotes& note = notes.key[k.at];
        row = note.row[key_in >> 4];
        factor = note.scale(key_in) * w.scale2;
        if (w.w_in && s.len - s.n - k0 > key_in) old = w.decay * note.old[key_in];
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&B.key_free[k.at]);
      k.next(C::NS);
    }
    if (!ok) break;
    const uint64_t f2 = ptx::f2_splat(factor);
    uint64_t sum[2] = {0, 0};
    const int k_last = k0 + min(127, s.len - 1 - k0);
#pragma unroll 1
    for (int c = (ci ^ turn) & 1; c < it.chunks; c += 2) {
      const uint32_t stage = n.at * 2 + turn;
      ok = ptx::mbar_wait(&B.n_full[stage], n.turn, p.limit, abort);
      if (ok && mine) ok = ptx::mbar_wait(&B.s_full[m][turn], s_turn, p.limit, abort);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      if (mine) {
        s_turn ^= 1;
        ptx::tc_fence_after();
        const int4 chunk = notes.chunk[stage];
        const int blocks = chunk.x;
        const float* lse = notes.lse + stage * 128;
        const int* last = notes.last + stage * 128;
        // blocks whose columns are all rows that see all of these keys (tokens, and so last keys, ascend)
        const int whole = chunk.z >= k_last && (w.window == 0 || chunk.w - w.window < k0) ? chunk.y : 0;
        auto tile = [&](auto all_tag, int i0, int i1) {
#pragma unroll 1
          for (int i = i0; i < i1; ++i) {
            uint32_t r[32];
            ptx::tmem_read32(from + i * 32, r);
            if (i == blocks - 1) {  // the buffer is read
              ptx::tc_fence_before();
              __syncwarp();
              if (lane == 0) ptx::mbar_arrive(&B.s_free[m][turn]);
              __syncwarp();
            }
            const ulonglong2* l4 = reinterpret_cast<const ulonglong2*>(lse + i * 32);
            const int4* e4 = reinterpret_cast<const int4*>(last + i * 32);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const ulonglong2 l = l4[j];
              const uint64_t x = ptx::f2_pack(__uint_as_float(r[4 * j]), __uint_as_float(r[4 * j + 1]));
              const uint64_t y = ptx::f2_pack(__uint_as_float(r[4 * j + 2]), __uint_as_float(r[4 * j + 3]));
              float a, b, d, e;
              ptx::f2_unpack(ptx::f2_fma(x, f2, l.x), a, b);
              ptx::f2_unpack(ptx::f2_fma(y, f2, l.y), d, e);
              a = ptx::ex2_approx(a), b = ptx::ex2_approx(b), d = ptx::ex2_approx(d), e = ptx::ex2_approx(e);
              if (!decltype(all_tag)::value) {
                const int4 end = e4[j];
                const int width = w.window > 0 ? w.window : 0x7fffffff;  // (end - key < window; none: always)
                if (key > end.x || end.x - key >= width) a = 0.0f;
                if (key > end.y || end.y - key >= width) b = 0.0f;
                if (key > end.z || end.z - key >= width) d = 0.0f;
                if (key > end.w || end.w - key >= width) e = 0.0f;
              }
              sum[0] = ptx::f2_add(sum[0], ptx::f2_pack(a, b));
              sum[1] = ptx::f2_add(sum[1], ptx::f2_pack(d, e));
            }
          }
        };
        tile(std::true_type{}, 0, whole);
        tile(std::false_type{}, whole, blocks);
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&B.n_free[stage]);
      n.next(2);
    }
    if (!ok) break;
    const bool writes = it.chunks == 1 ? (ci & 1) == turn : turn == 0;
    ci += it.chunks;
    if (!mine) continue;
    float a, b, c, d;
    ptx::f2_unpack(sum[0], a, b);
    ptx::f2_unpack(sum[1], c, d);
    float total = (a + b) + (c + d);
    if (it.chunks > 1) {  // both warpgroups have a part
      if (turn == 1) {
        ok = ptx::mbar_wait_near(&B.x_free[m], (xi & 1) ^ 1, p.limit, abort);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        notes.half[m * 128 + key_in] = total;
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&B.x_full[m]);
      } else {
        ok = ptx::mbar_wait_near(&B.x_full[m], xi & 1, p.limit, abort);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        total += notes.half[m * 128 + key_in];
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&B.x_free[m]);
      }
      ++xi;
    }
    if (writes && row >= 0 && s.len - k0 > key_in) w.w[row + (key_in & 15)] = old + total;
    __syncwarp();
  }
  ok = ok && walk.ok;
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

// The tiles of K that a CTA needs, in order.
struct TileWalk {
  Walk walk;
  int m;
  // To the next tile, or the first.
  __device__ __forceinline__ bool begin(const WeightTileParams& p, Bars& B, const Notes& notes) {
    m = 0;
    return walk.next_seen(p, B, notes);
  }
  __device__ __forceinline__ bool next(const WeightTileParams& p, Bars& B, const Notes& notes) {
    return ++m < walk.it.tiles || begin(p, B, notes);
  }
};

template <int D>
__device__ void run_copies(const WeightTileParams& p, uint8_t* sm, Bars& B, const Notes& notes) {
  using C = WeightTileCfg<D>;
  const CacheWeightsParams& w = p.w;
  const int lane = threadIdx.x & 31;
  const volatile int* abort = &B.abort;
  const int pmask = (1 << w.cache.lp) - 1;
  const uint32_t raw = ptx::smem_u32(sm) + C::OFF_RAW;
  const int second = lane >> 3 & 1;  // lanes 0-7: the blocks of an item's first tile; 8-15: of its second
  StageRing in, n;
  uint32_t count = 0, notes_count = 0;
  Walk walk;
  // The page of this lane's block as the table has it; -1 behind the keys.  (Looked
  // up an item ahead, and not looked at until then.)
  int page = -1;
  // the item whose copies are to be issued: its tiles, and the row of this lane's block
  int tiles = 0;
  int64_t row = -1;
  const bool ok = bring_in_order(
      [&]() { return walk.next(p, B, notes); }, [&]() { return walk.it.chunks > 0; },
      [&]() {
        page = lane >= 16 || walk.s.len - walk.it.k0 <= lane * 16
                   ? -1
                   : __ldg(w.batch.table + static_cast<int64_t>(walk.b) * w.batch.max_pages +
                           ((walk.it.k0 + lane * 16) >> w.cache.lp));
      },
      [&]() {
        tiles = walk.it.tiles;
        row = -1;
        if (page >= 0 && page < w.cache.num_pages)
          row = cache_row(w.cache, page, walk.h, (walk.it.k0 + lane * 16) & pmask);
        else if (lane < 16 && walk.s.len - walk.it.k0 > lane * 16)
          atomicOr(w.batch.status, kStatusBadPlan);
        __syncwarp();
      },
      [&]() {
        StageRing n2 = n, in2 = in;
        n2.next(C::NS);
        in2.next(C::RAWS);
        bool there = ptx::mbar_wait_idle(&B.key_free[n.at], n.turn ^ 1, p.limit, abort);
        if (tiles == 2) there = there && ptx::mbar_wait_idle(&B.key_free[n2.at], n2.turn ^ 1, p.limit, abort);
        if (!__all_sync(0xffffffffu, there)) return false;
        const uint32_t n_at = second ? n2.at : n.at, in_at = second ? in2.at : in.at;
        bring_notes(w, notes.key[n_at], &B.key_full[n_at], row, tiles);
        notes_count += tiles;
        n = n2;
        if (tiles == 2) n.next(C::NS);
        there = ptx::mbar_wait_idle(&B.raw_free[in.at], in.turn ^ 1, p.limit, abort);
        if (tiles == 2) there = there && ptx::mbar_wait_idle(&B.raw_free[in2.at], in2.turn ^ 1, p.limit, abort);
        if (!__all_sync(0xffffffffu, there)) return false;
        bring_codes<D>(w, raw + in_at * C::RAW, &B.raw_full[in_at], row, tiles);
        count += tiles;
        in = in2;
        if (tiles == 2) in.next(C::RAWS);
        return true;
      }) && walk.ok;
  if (!ok && lane == 0) {
    B.abort = 1;
    atomicOr(w.batch.status, kStatusProducer);
  }
  // no copy may land behind the CTA's end: this thread's own, and the last turn of every stage
  split::cp_commit();
  split::cp_wait<0>();
  drain_stages(B.key_full, n, C::NS, notes_count);
  drain_stages(B.raw_full, in, C::RAWS, count);
}

template <int D>
__device__ void run_convert(const WeightTileParams& p, uint8_t* sm, Bars& B, const Notes& notes) {
  using C = WeightTileCfg<D>;
  constexpr int CPR = D / 16, ROWS = 128 / CPR, N = 128 / ROWS;  // chunks of a key; keys of a pass; passes
  const int tid = threadIdx.x - 512, lane = tid & 31;
  const volatile int* abort = &B.abort;
  const int r0 = tid / CPR, c = tid % CPR;  // its row in a pass, and 16 coordinates
  const uint32_t raw = ptx::smem_u32(sm) + C::OFF_RAW + tid * 16;
  // 16-byte chunks 2c and 2c + 1 of a row, 64 columns a sub-tile (the rows of a thread agree modulo 8)
  const uint32_t j = 2 * c & 7, base = ptx::smem_u32(sm) + (c >> 2) * C::SUB + r0 * 128;
  const uint32_t to0 = base + ((j ^ (r0 & 7)) << 4), to1 = base + (((j + 1) ^ (r0 & 7)) << 4);
  StageRing in, k;
  bool ok = true;
  TileWalk tiles;
  for (bool more = tiles.begin(p, B, notes); more; more = tiles.next(p, B, notes)) {
    ok = ptx::mbar_wait_near(&B.raw_full[in.at], in.turn, p.limit, abort);
    ok = ok && ptx::mbar_wait_near(&B.k_free[k.at], k.turn ^ 1, p.limit, abort);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) break;
#pragma unroll 1  // (unrolled it alone drives the other roles out of the instruction caches)
    for (int i = 0; i < N; ++i) {
      const uint32_t at = k.at * C::TILE + i * ROWS * 128;
      uint32_t x[4], a[8];
      split::lds128(raw + in.at * C::RAW + i * 2048, x);
      codes_bf16(x[0], a[0], a[1]);
      codes_bf16(x[1], a[2], a[3]);
      codes_bf16(x[2], a[4], a[5]);
      codes_bf16(x[3], a[6], a[7]);
      ptx::st_shared_v4(to0 + at, a[0], a[1], a[2], a[3]);
      ptx::st_shared_v4(to1 + at, a[4], a[5], a[6], a[7]);
    }
    ptx::fence_proxy_async_smem();
    ptx::mbar_arrive(&B.k_full[k.at]);
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(&B.raw_free[in.at]);
    in.next(C::RAWS);
    k.next(C::KS);
  }
  ok = ok && tiles.walk.ok;
  if (!ok && lane == 0) {
    B.abort = 1;
    atomicOr(p.w.batch.status, kStatusProducer);
  }
}

// f(walk, chunk) for every chunk of this CTA, in order, until it returns false.
template <class F>
__device__ __forceinline__ bool each_chunk(const WeightTileParams& p, Bars& B, const Notes& notes, const F& f) {
  Walk walk;
  while (walk.next(p, B, notes)) {
#pragma unroll 1
    for (int c = 0; c < walk.it.chunks; ++c)
      if (!f(walk, c)) return false;
  }
  return walk.ok;
}

// A chunk's first token, and which part of its tokens' heads it is.
__device__ __forceinline__ void chunk_at(const WeightTileParams& p, const Item& it, int c, int& tok, int& part) {
  part = p.parts == 1 ? 0 : c % p.parts;
  tok = it.lo + (p.parts == 1 ? c : c / p.parts) * p.tokens;
}

template <int D>
__device__ void run_queries(const WeightTileParams& p, uint8_t* sm, Bars& B, const Notes& notes) {
  using C = WeightTileCfg<D>;
  const int lane = threadIdx.x & 31;
  const volatile int* abort = &B.abort;
  const uint32_t bytes = static_cast<uint32_t>(p.heads) * p.tokens * D * 2;
  const uint32_t to = ptx::smem_u32(sm) + C::OFF_Q;
  StageRing q;
  uint32_t count = 0;
  const bool ok = each_chunk(p, B, notes, [&](const Walk& walk, int c) {
    int tok, part;
    chunk_at(p, walk.it, c, tok, part);
    const bool fine = ptx::mbar_wait_idle(&B.q_free[q.at], q.turn ^ 1, p.limit, abort);
    if (!__all_sync(0xffffffffu, fine)) return false;
    if (lane == 0) {
      ptx::mbar_arrive_expect_tx(&B.q_full[q.at], bytes);
#pragma unroll
      for (int d = 0; d < D / 64; ++d)
        ptx::tma_load_3d(to + q.at * C::TILE + d * C::SUB, &p.tm_q, &B.q_full[q.at], d * 64,
                         walk.h * p.w.G + part * p.heads, walk.s.first + tok);
    }
    __syncwarp();
    q.next(C::QS);
    ++count;
    return true;
  });
  if (!ok && lane == 0) {
    B.abort = 1;
    atomicOr(p.w.batch.status, kStatusProducer);
  }
  drain_stages(B.q_full, q, C::QS, count);
}

template <int D>
__device__ void run_notes(const WeightTileParams& p, Bars& B, const Notes& notes) {
  using C = WeightTileCfg<D>;
  const CacheWeightsParams& w = p.w;
  const int lane = threadIdx.x & 31;
  const volatile int* abort = &B.abort;
  int tok_of[4], head_of[4];  // of this lane's four columns in a chunk
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    tok_of[i] = (lane * 4 + i) / p.heads;
    head_of[i] = lane * 4 + i - tok_of[i] * p.heads;
  }
  StageRing n;
  const bool ok = each_chunk(p, B, notes, [&](const Walk& walk, int c) {
    int tok0, part;
    chunk_at(p, walk.it, c, tok0, part);
    float lse[4];
    int last[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int tok = tok0 + tok_of[i], head = part * p.heads + head_of[i];
      lse[i] = INFINITY;
      last[i] = -1;
      if (tok_of[i] < p.tokens && tok < walk.it.hi && head < w.G) {
        const float x = __ldg(w.lse + static_cast<int64_t>(walk.s.first + tok) * w.Hq + walk.h * w.G + head);
        lse[i] = x == -INFINITY ? INFINITY : x * kLog2e;
        last[i] = w.causal ? walk.s.len - walk.s.n + tok : walk.s.len - 1;
      }
    }
    const bool fine = ptx::mbar_wait_idle(&B.n_free[n.at], n.turn ^ 1, p.limit, abort);
    if (!__all_sync(0xffffffffu, fine)) return false;
    reinterpret_cast<float4*>(notes.lse + n.at * 128)[lane] = make_float4(-lse[0], -lse[1], -lse[2], -lse[3]);
    reinterpret_cast<int4*>(notes.last + n.at * 128)[lane] = make_int4(last[0], last[1], last[2], last[3]);
    if (lane == 0) {
      const int columns = chunk_columns(p, walk.it, c), first = w.causal ? walk.s.len - walk.s.n + tok0 : walk.s.len - 1;
      notes.chunk[n.at] = make_int4((columns + 31) >> 5, columns == p.heads * p.tokens ? (columns + 31) >> 5 : columns >> 5, first,
                                    w.causal ? first + min(p.tokens, walk.it.hi - tok0) - 1 : first);
    }
    ptx::mbar_arrive(&B.n_full[n.at]);
    n.next(C::NS);
    return true;
  });
  if (!ok && lane == 0) {
    B.abort = 1;
    atomicOr(w.batch.status, kStatusProducer);
  }
}

template <int D>
__device__ void run_mma(const WeightTileParams& p, uint8_t* sm, Bars& B, const Notes& notes, uint32_t tmem) {
  using C = WeightTileCfg<D>;
  const volatile int* abort = &B.abort;
  // Short code for short items (200 rows of 128 samples, D = 64, 320 us instead of 344; 2321
  // prompt rows 97 either way), quick issues where the products set the pace (those
  // rows at D = 128: 107 us instead of 112; 192 rows of 48 sequences 94 instead of 88).
  constexpr int M = D == 64 ? 1 : 2;
  const uint64_t k_desc = ptx::sdesc_sw128(ptx::smem_u32(sm), 16, 1024);
  const uint64_t q_desc = ptx::sdesc_sw128(ptx::smem_u32(sm) + C::OFF_Q, 16, 1024);
  StageRing k, q;
  uint32_t ci = 0, s_turns = 0;  // chunks so far; a bit for each buffer of S
  bool ok = true;
  Walk walk;
  while (ok && walk.next(p, B, notes)) {
    const Item it = walk.it;
    if (it.chunks == 0) continue;
    StageRing second = k;
    second.next(C::KS);
#pragma unroll 1
    for (int c = 0; c < it.chunks; ++c, ++ci) {
      ok = ptx::mbar_wait(&B.q_full[q.at], q.turn, p.limit, abort);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const uint32_t idesc = ptx::idesc_bf16(128, (chunk_columns(p, it, c) + 31) & ~31, 0), sb = ci & 1;
      const uint64_t b = q_desc + q.at * (C::TILE >> 4);
#pragma unroll M
      for (int m = 0; m < 2; ++m) {
        if (m >= it.tiles) break;
        const StageRing at = m ? second : k;
        const uint32_t bit = 1u << (2 * m + sb);
        if (c == 0) ok = ptx::mbar_wait(&B.k_full[at.at], at.turn, p.limit, abort);
        ok = ok && ptx::mbar_wait(&B.s_free[m][sb], (s_turns & bit) ? 0 : 1, p.limit, abort);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        s_turns ^= bit;
        ptx::tc_fence_after();
        const uint64_t a = k_desc + at.at * (C::TILE >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * C::SUB + (kk & 3) * 32) >> 4;
          ptx::mma_ss_elect(tmem + m * 256 + sb * 128, a + off, b + off, idesc, kk > 0 ? 1u : 0u);
        }
        ptx::mma_commit_elect(&B.s_full[m][sb]);
        if (c == it.chunks - 1) ptx::mma_commit_elect(&B.k_free[at.at]);
      }
      if (!ok) break;
      ptx::mma_commit_elect(&B.q_free[q.at]);
      q.next(C::QS);
    }
    k.next(C::KS);
    if (it.tiles == 2) k.next(C::KS);
  }
  ok = ok && walk.ok;
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
  static_assert(sizeof(KeyNotes) <= 640, "notes");
  notes.key = reinterpret_cast<KeyNotes*>(sm + C::OFF_NOTES);
  notes.lse = reinterpret_cast<float*>(sm + C::OFF_NOTES + C::NS * 640);
  notes.last = reinterpret_cast<int*>(notes.lse + C::NS * 128);
  notes.half = reinterpret_cast<float*>(notes.last + C::NS * 128);
  notes.chunk = reinterpret_cast<int4*>(notes.half + 256);
  notes.item = notes.chunk + C::NS;
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::KS; ++i) ptx::mbar_init(&B.k_full[i], 128), ptx::mbar_init(&B.k_free[i], 1);
    for (int i = 0; i < C::RAWS; ++i) ptx::mbar_init(&B.raw_full[i], 1), ptx::mbar_init(&B.raw_free[i], 4);
    for (int i = 0; i < C::NS; ++i) ptx::mbar_init(&B.key_full[i], 1 + 8), ptx::mbar_init(&B.key_free[i], 16);
    for (int i = 0; i < 4; ++i) ptx::mbar_init(&B.item_full[i], 1), ptx::mbar_init(&B.item_free[i], 24);
    for (int i = 0; i < C::QS; ++i) ptx::mbar_init(&B.q_full[i], 1), ptx::mbar_init(&B.q_free[i], 1);
    for (int i = 0; i < C::NS; ++i) ptx::mbar_init(&B.n_full[i], 32), ptx::mbar_init(&B.n_free[i], 8);
    for (int m = 0; m < 2; ++m) {
      for (int i = 0; i < 2; ++i) ptx::mbar_init(&B.s_full[m][i], 1), ptx::mbar_init(&B.s_free[m][i], 4);
      ptx::mbar_init(&B.x_full[m], 4), ptx::mbar_init(&B.x_free[m], 4);
    }
    ptx::mbar_init(&B.drain, 1);
    B.abort = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 20) {
    ptx::tmem_alloc(&B.tmem, C::TM_COLS);
    ptx::tmem_relinquish();
  }
  // rows behind a chunk's box are never copied to: their columns' weights are 2^-inf
  for (int i = threadIdx.x; i < C::QS * (D / 64) * 128 * 8; i += C::THREADS)
    if ((i >> 3) % 128 >= p.heads * p.tokens) ptx::st_shared_v4(ptx::smem_u32(sm) + C::OFF_Q + i * 16, 0, 0, 0, 0);
  ptx::fence_proxy_async_smem();
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = B.tmem;
  if (warp < 16)
    wtile::run_sums<D>(p, B, notes, tmem);
  else if (warp < 20)
    wtile::run_convert<D>(p, sm, B, notes);
  else if (warp == 20)
    wtile::run_mma<D>(p, sm, B, notes, tmem);
  else if (warp == 21)
    wtile::run_queries<D>(p, sm, B, notes);
  else if (warp == 22)
    wtile::run_notes<D>(p, B, notes);
  else if (warp == 23)
    wtile::run_copies<D>(p, sm, B, notes);
  else
    wtile::run_items(p, B, notes);
  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == 20) ptx::tmem_dealloc(tmem, C::TM_COLS);
}

}  // namespace gdpa
