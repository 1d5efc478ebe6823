// gdpa_cache_weights.cuh -- the attention weight that each stored key receives
// from the rows of a call: the kernel for few rows.
//
// Mathematics.  With the rows' logsumexp at hand the weight of a row for a key
// is exp(scale <q, k> - lse): no maximum, no second product, and a key's sum is
// its own, so keys are split over the GPU and nothing is joined.  The product
// runs as S^T = K Q^T, so that the 16-row side of the tensor-core instruction
// (mma m16n8k16) is filled with keys, which are many, and its 8-column side with
// query rows, which are few, and a key's sum over the rows is a sum over one
// lane's columns and two shuffles.  Codes become fp16 exactly, queries fp16 as in
// gdpa_cache_fwd.cuh (divided by their largest element's power of two), and the
// scale of a block of 16 tokens that of a whole tile.
//
// Bound: memory, D bytes a key and head, and 8 of its weight, with a warp's own
// latencies (conversions, fragments, the exponentials' chain) close behind: what
// hides them is warps, so stages are two and registers few.  Measured: one token of
// 64 histories of 100 to 8192 keys, 32 query and 8 key heads of 128, 53 us (5.6
// TB/s, 82 % of a copy's rate); of two histories of 130k keys, 16 and 2 heads, 16 us
// (4.5 TB/s; 4 us are the start); 32 rows of 128 samples of 100 to 6000 keys, 8 and 8 heads of
// 64, 73 us (3.1 TB/s, bound by the rows' own work: 47 us with 8 rows).
//
// Work split.  A step is 4 KB of codes (32 or 64 keys) of one sequence and head.  The steps of all
// sequences are counted from the lengths on the device, and every warp takes an
// equal run of them, so a batch of any raggedness or one long history loads all
// SMs alike.  A warp's own asynchronous copies bring codes, scales and
// earlier weights STAGES - 1 steps ahead, across the ends of heads and sequences.
#pragma once

#include <type_traits>

#include "gdpa_cache_fwd.cuh"

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
  int keep;  // earlier weights stay in place as they are: keys that no row sees need nothing
};

constexpr float kLog2e = 1.4426950408889634f;

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

// NT: row tiles of 8 whose fragments a warp keeps (sequences with more rows make
// them anew at every step).
template <int D, int NT_>
struct WeightCfg {
  static constexpr int NT = NT_, WARPS = 4, THREADS = 32 * WARPS;
  static constexpr int SPAN = 4096 / D, TILES = SPAN / kCacheBlock;
  static constexpr int START = 2;  // what a sequence and head's start costs, in steps
  static constexpr int KSTEPS = D / 16;
  // (two stages and more CTAs: 32 candidates of 128 samples 74 us so, 94 with three stages and two CTAs an SM)
  static constexpr int STAGES = 2;
  static constexpr int TILE = kCacheBlock * D;
  // of a stage: codes, earlier weights, words with scales, pages
  static constexpr int W_AT = 4096, SF_AT = W_AT + SPAN * 4, PAGE_AT = SF_AT + 16, STAGE = PAGE_AT + 16;
  static constexpr int QFRAG = NT * KSTEPS * 32 * 8;  // a warp's query fragments ...
  static constexpr int ROWS_AT = QFRAG;               // ... and what it knows of their rows
  static constexpr int WARP = STAGES * STAGE + QFRAG + NT * 8 * 16;
  static constexpr int SMEM = WARPS * WARP;
  // (as registers and shared memory allow; four at D = 128 leave 128 registers: one token of 64 histories 142 us)
  static constexpr int CTAS = D == 64 ? (NT <= 4 ? 4 : NT == 8 ? 3 : 2) : NT <= 2 ? 3 : 2;
  static_assert(STAGE % 16 == 0 && WARP % 16 == 0, "16-byte copies");
};

// A sequence's share of the work.
struct WeightSeq {
  CacheSeq s;
  int kbase;  // first key of its steps
  int steps;  // of a head
  int see;    // first key that any row sees
};
template <class C>
__device__ __forceinline__ WeightSeq weight_seq(const CacheWeightsParams& p, int b) {
  WeightSeq w;
  w.s = load_sequence(p.batch, p.cache.lp, b);
  w.kbase = w.steps = w.see = 0;
  if (!w.s.ok || w.s.n == 0 || w.s.len == 0) return w;
  w.see = min(first_key(w.s.len - w.s.n, p.window), w.s.len);
  if (p.keep) w.kbase = w.see & ~(C::SPAN - 1);
  w.steps = static_cast<int>((static_cast<unsigned>(w.s.len - w.kbase) + C::SPAN - 1) / C::SPAN);
  return w;
}
template <class C>
__device__ __forceinline__ int64_t weight_cost(const CacheWeightsParams& p, const WeightSeq& w) {
  return w.steps == 0 ? 0 : static_cast<int64_t>(w.steps + C::START) * p.cache.H;
}

// Where each warp's run begins.  All threads take part.
template <class C>
struct WeightSchedule {
  int64_t scan[C::WARPS];
  int64_t base[C::WARPS];  // the work in front of the sequence in which the run begins
  int seq[C::WARPS];
};
template <class C>
__device__ __forceinline__ void weight_schedule(const CacheWeightsParams& p, WeightSchedule<C>& sh, int64_t& total,
                                                int64_t& chunk) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, B = p.batch.B;
  const int per = (B + C::THREADS - 1) / C::THREADS;
  const int b_lo = min(B, tid * per), b_hi = min(B, b_lo + per);
  int64_t mine = 0;
#pragma unroll 4
  for (int b = b_lo; b < b_hi; ++b) mine += weight_cost<C>(p, weight_seq<C>(p, b));
  int64_t incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += x;
  }
  if (lane == 31) sh.scan[warp] = incl;
  __syncthreads();
  total = 0;
#pragma unroll
  for (int w = 0; w < C::WARPS; ++w) {
    if (w < warp) incl += sh.scan[w];
    total += sh.scan[w];
  }
  const int64_t workers = static_cast<int64_t>(gridDim.x) * C::WARPS;
  chunk = max(split::quotient(total + workers - 1, workers), (int64_t)1);
#pragma unroll 1
  for (int w = 0; w < C::WARPS; ++w) {
    const int64_t from = chunk * (static_cast<int64_t>(blockIdx.x) * C::WARPS + w);
    if (from < total && from >= incl - mine && from < incl) {
      int64_t base = incl - mine;
      int b = b_lo;
      for (; b < b_hi; ++b) {
        const int64_t n = weight_cost<C>(p, weight_seq<C>(p, b));
        if (from < base + n) break;
        base += n;
      }
      sh.seq[w] = b;
      sh.base[w] = base;
    }
  }
  __syncthreads();
}

// Walks the steps of a warp's run [at, stop) of the work.
template <class C>
struct WeightWalk {
  WeightSeq w;
  int64_t start;  // of the present head
  int b, h;
  int u, u1;      // the present step, and one past the last of this head in the run

  // The first step at or behind the present head's start, if the run has one.
  __device__ __forceinline__ bool settle(const CacheWeightsParams& p, int64_t at, int64_t stop) {
    while (start < stop) {
      u = static_cast<int>(max(at - start - C::START, (int64_t)0));
      u1 = static_cast<int>(min(max(stop - start - C::START, (int64_t)0), (int64_t)w.steps));
      if (u < u1) return true;
      if (!next_head(p)) return false;
    }
    return false;
  }
  __device__ __forceinline__ bool next_head(const CacheWeightsParams& p) {
    start += w.steps + C::START;
    if (++h < p.cache.H) return true;
    h = 0;
    do {
      if (++b >= p.batch.B) return false;
      w = weight_seq<C>(p, b);
    } while (w.steps == 0);
    return true;
  }
  __device__ __forceinline__ bool begin(const CacheWeightsParams& p, int seq, int64_t base, int64_t at, int64_t stop) {
    b = seq;
    w = weight_seq<C>(p, b);
    const int64_t cost = w.steps + C::START, seg = split::quotient(at - base, cost);
    h = static_cast<int>(seg);
    start = base + seg * cost;
    return settle(p, at, stop);
  }
  __device__ __forceinline__ bool next(const CacheWeightsParams& p, int64_t at, int64_t stop) {
    if (++u < u1) return true;
    return next_head(p) && settle(p, at, stop);
  }
};

// What a warp knows of a query row: the factor of its scores, its logsumexp
// (both in units of log2), and the keys it sees.
struct WeightRow {
  float fac, lse;
  int lo, hi;
};

template <int D, int NT>
__global__ void __launch_bounds__((WeightCfg<D, NT>::THREADS), (WeightCfg<D, NT>::CTAS))
    gdpa_cache_weights_split_kernel(const __grid_constant__ CacheWeightsParams p) {
  using namespace split;
  using C = WeightCfg<D, NT>;
  constexpr int KS = C::KSTEPS, SPAN = C::SPAN;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ WeightSchedule<C> sh;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const CacheBatch& bt = p.batch;
  int64_t total, chunk;
  weight_schedule<C>(p, sh, total, chunk);
  const int64_t at = chunk * (static_cast<int64_t>(blockIdx.x) * C::WARPS + warp), stop = min(total, at + chunk);
  if (at >= stop) return;
  uint8_t* const mine = smem + warp * C::WARP;
  const uint32_t ring = ptx::smem_u32(mine);
  uint2* const qfrag = reinterpret_cast<uint2*>(mine + C::STAGES * C::STAGE);
  WeightRow* const row_of = reinterpret_cast<WeightRow*>(mine + C::STAGES * C::STAGE + C::ROWS_AT);
  const int pmask = (1 << p.cache.lp) - 1;
  const bool one = (1 << p.cache.lp) >= SPAN;  // a step lies in one page
  const int64_t sf_bytes = static_cast<int64_t>(p.cache.num_pages) * p.cache.H << (p.cache.lp - 4);

  WeightWalk<C> ahead, now;
  bool more = ahead.begin(p, sh.seq[warp], sh.base[warp], at, stop);  // of the copies' walk
  now = ahead;
  bool left = more;

  // The page of a step's tile (lanes from 0 on), or of all of it; -1 where there is none (flagged if there should be).
  auto page_of = [&](const WeightWalk<C>& k) {
    const int key = k.w.kbase + k.u * SPAN, off = one ? 0 : lane * kCacheBlock;
    if (off >= SPAN || k.w.s.len - key <= off) return -1;
    const int x = __ldg(bt.table + static_cast<int64_t>(k.b) * bt.max_pages + ((key + off) >> p.cache.lp));
    if (x >= 0 && x < p.cache.num_pages) return x;
    atomicOr(bt.status, kStatusBadPlan);
    return -1;
  };
  // A step's copies: what a row may see, scales, earlier weights.
  int page_next = -1;
  const uint32_t chunk_to = tile_at<D>(lane / (D / 16), lane % (D / 16));  // of this lane's first 16 bytes of a tile
  auto issue = [&](int stage) {
    if (more) {
      const int key = ahead.w.kbase + ahead.u * SPAN;
      const uint32_t dst = ring + stage * C::STAGE;
      if (lane < 4) asm volatile("st.shared.b32 [%0], %1;" ::"r"(dst + C::PAGE_AT + lane * 4), "r"(page_next) : "memory");
      if (one) {
        if (page_next >= 0) {
          const int64_t row = cache_row(p.cache, page_next, ahead.h, key & pmask);
          if (key > ahead.w.see - SPAN) {
            const uint8_t* src = p.cache.k + row * D + lane * 16;
#pragma unroll
            for (int j = 0; j < 8; ++j)
              // 32 chunks further on: as many rows, and the same permutation (or another one, a constant too)
              cp_async16(dst + (D == 128 ? (chunk_to ^ (j & 1) * 64) : chunk_to) + j * 512, src + 512 * j, 16);
            const int64_t word = (row >> 4) & ~(int64_t)3;
            if (lane == 0)
              cp_async4(dst + C::SF_AT, p.cache.k_sf + word, static_cast<int>(min((int64_t)4, sf_bytes - word)));
          }
          if (p.w_in && lane < SPAN / 4) cp_async16(dst + C::W_AT + lane * 16, p.w_in + row + lane * 4, 16);
        }
      } else {
#pragma unroll 1
        for (int n = 0; n < C::TILES; ++n) {
          const int k0 = key + n * kCacheBlock, page = __shfl_sync(0xffffffffu, page_next, n);
          if (page < 0) continue;
          const int64_t row = cache_row(p.cache, page, ahead.h, k0 & pmask);
          if (k0 > ahead.w.see - kCacheBlock) {
            const uint8_t* src = p.cache.k + row * D + lane * 16;
#pragma unroll
            for (int j = 0; j < D / 32; ++j) {
              const int idx = lane + 32 * j;
              cp_async16(dst + n * C::TILE + tile_at<D>(idx / (D / 16), idx % (D / 16)), src + 512 * j, 16);
            }
            const int64_t word = (row >> 4) & ~(int64_t)3;
            if (lane == 0)
              cp_async4(dst + C::SF_AT + n * 4, p.cache.k_sf + word, static_cast<int>(min((int64_t)4, sf_bytes - word)));
          }
          if (p.w_in && lane < 4) cp_async16(dst + C::W_AT + n * 64 + lane * 16, p.w_in + row + lane * 4, 16);
        }
      }
      more = ahead.next(p, at, stop);
      if (more) page_next = page_of(ahead);
    }
    cp_commit();
  };
  if (more) page_next = page_of(ahead);
#pragma unroll 1
  for (int i = 0; i < C::STAGES - 1; ++i) issue(i);

  // Fragments of NT tiles of rows from row0 on of the present head, and their rows.
  auto load_rows = [&](int row0) {
    const CacheSeq& s = now.w.s;
    const int rows = min(s.n * p.G - row0, 8 * NT);
    __syncwarp();
#pragma unroll 1
    for (int nt = 0; nt * 8 < rows; ++nt) {
      const int r = nt * 8 + g, x = row0 + r;
      const int tok = p.G == 1 ? x : x / p.G, head = now.h * p.G + x - tok * p.G;
      uint4 u[D / 32];
      WeightRow wr = {0.0f, INFINITY, 0, 0};
#pragma unroll
      for (int i = 0; i < D / 32; ++i) u[i] = make_uint4(0, 0, 0, 0);
      if (r < rows) {
        const __nv_bfloat16* src = p.q + (s.first + tok) * p.q_stride + head * D + t * (D / 4);
        const float lse = __ldg(p.lse + static_cast<int64_t>(s.first + tok) * p.Hq + head);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) u[i] = *reinterpret_cast<const uint4*>(src + 8 * i);
        const int pos = s.len - s.n + tok;
        wr.lse = lse == -INFINITY ? INFINITY : lse * kLog2e;
        wr.lo = first_key(pos, p.window);
        wr.hi = p.causal ? min(s.len, pos + 1) : s.len;
      }
      float v[D / 4], amax = 0.0f;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[8 * i + 2 * e] = __uint_as_float(w[e] << 16);
          v[8 * i + 2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
        }
      }
#pragma unroll
      for (int i = 0; i < D / 4; ++i) amax = fmaxf(amax, fabsf(v[i]));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      // 2^e: the largest element's power of two (1 for an all-zero row)
      const int e = amax > 0.0f ? min(max(static_cast<int>(__float_as_uint(amax) >> 23) - 127, -126), 127) : 0;
      const float inv = sf_value(127 - e);
      wr.fac = r < rows ? sf_value(127 + e) * p.scale2 : 0.0f;
#pragma unroll
      for (int k = 0; k < KS; ++k)
        qfrag[(nt * KS + k) * 32 + lane] = make_uint2(pack_f16x2(v[4 * k] * inv, v[4 * k + 1] * inv),
                                                      pack_f16x2(v[4 * k + 2] * inv, v[4 * k + 3] * inv));
      if (t == 0) row_of[r] = wr;
    }
    __syncwarp();
    return rows;
  };

  int stage = 0, at_b = -1, at_h = -1, rows = 0, lo_max = 0, hi_min = 0;
#pragma unroll 1
  while (left) {
    const CacheSeq& s = now.w.s;
    const int key0 = now.w.kbase + now.u * SPAN;
    const bool many = static_cast<int64_t>(s.n) * p.G > 8 * NT;
    if (now.b != at_b || now.h != at_h) {
      at_b = now.b, at_h = now.h;
      if (!many) rows = load_rows(0);
      lo_max = first_key(s.len - 1, p.window);  // keys that all rows see: [lo_max, hi_min)
      hi_min = p.causal ? max(0, s.len - s.n + 1) : s.len;
    }
    issue(stage == 0 ? C::STAGES - 1 : stage - 1);
    cp_wait<C::STAGES - 1>();
    __syncwarp();
    const uint32_t st = ring + stage * C::STAGE;
    int page[4];
    uint32_t sf_word[4];
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(page[0]), "=r"(page[1]), "=r"(page[2]), "=r"(page[3])
                 : "r"(st + C::PAGE_AT));
    lds128(st + C::SF_AT, sf_word);
    const bool seen = key0 > now.w.see - SPAN;  // (a length may be as large as 2^31 - 16)
    const bool edge = key0 < lo_max || key0 > hi_min - SPAN;

#pragma unroll
    for (int half = 0; half < C::TILES / 2; ++half) {
      const int k0 = key0 + half * 2 * kCacheBlock;
      float sum[2][2] = {};
      if (seen) {
        float sk[2];  // the tiles' scales
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          // the scale's place in its word: the low bits of its index
          const int tile = 2 * half + n, pg = one ? page[0] : page[tile], key = k0 + n * kCacheBlock;
          const uint32_t block = ((static_cast<uint32_t>(pg) * p.cache.H + now.h) << (p.cache.lp - 4)) + ((key & pmask) >> 4);
          sk[n] = sf_value((one ? sf_word[0] : sf_word[tile]) >> (block & 3) * 8 & 0xff);
        }
        // 16-byte chunk j of this lane's two keys of tile n, as the fragments of four k-steps
        auto keys_of = [&](int n, int j, uint32_t (&a)[4][4]) {
          uint32_t ka[4], kc[4];
          const int c = D == 128 ? 2 * t + j : t;
          lds128(st + (2 * half + n) * C::TILE + tile_at<D>(g, c), ka);
          lds128(st + (2 * half + n) * C::TILE + tile_at<D>(g + 8, c), kc);
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            a[w][0] = codes_lo(ka[w]), a[w][2] = codes_hi(ka[w]);
            a[w][1] = codes_lo(kc[w]), a[w][3] = codes_hi(kc[w]);
          }
        };
        // (a single row tile takes the fragments as they are made; several keep them)
        uint32_t a[NT == 1 ? 1 : 2][NT == 1 ? 1 : D / 64][4][4];
        if constexpr (NT > 1) {
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int j = 0; j < D / 64; ++j) keys_of(n, j, a[n][j]);
        }
        auto tile = [&](auto edge_tag, int nt) {
          constexpr bool EDGE = decltype(edge_tag)::value;
          float x[2][4];
#pragma unroll
          for (int j = 0; j < D / 64; ++j)
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              uint32_t (&f)[4][4] = a[NT == 1 ? 0 : n][NT == 1 ? 0 : j];
              if constexpr (NT == 1) keys_of(n, j, f);
#pragma unroll
              for (int w = 0; w < 4; ++w) {
                const uint2 q = qfrag[(nt * KS + 4 * j + w) * 32 + lane];
                if (j == 0 && w == 0)
                  mma_f16_new(x[n], f[w][0], f[w][1], f[w][2], f[w][3], q.x, q.y);
                else
                  mma_f16(x[n], f[w][0], f[w][1], f[w][2], f[w][3], q.x, q.y);
              }
            }
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const WeightRow wr = row_of[nt * 8 + 2 * t + c];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              const float f = wr.fac * sk[n];
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                float e = ptx::ex2_approx(fmaf(x[n][2 * i + c], f, -wr.lse));
                if (EDGE) {
                  const int key = k0 + n * kCacheBlock + 8 * i + g;
                  if (key < wr.lo || key >= wr.hi) e = 0.0f;
                }
                sum[n][i] += e;
              }
            }
          }
        };
        auto tiles = [&](int count) {
          if (edge) {
#pragma unroll 1
            for (int nt = 0; nt * 8 < count; ++nt) tile(std::true_type{}, nt);
          } else {
#pragma unroll 2
            for (int nt = 0; nt * 8 < count; ++nt) tile(std::false_type{}, nt);
          }
        };
        if (!many) {
          tiles(rows);
        } else {
#pragma unroll 1
          for (int64_t r = 0; r < static_cast<int64_t>(s.n) * p.G; r += 8 * NT) tiles(load_rows(static_cast<int>(r)));
        }
        // a quad's lanes hold the same two rows of each tile: one key a lane
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            sum[n][i] += __shfl_xor_sync(0xffffffffu, sum[n][i], 1);
            sum[n][i] += __shfl_xor_sync(0xffffffffu, sum[n][i], 2);
          }
      }
      const int off = (t >> 1) * kCacheBlock + (t & 1) * 8 + g, key = k0 + off;
      float w = t == 0 ? sum[0][0] : t == 1 ? sum[0][1] : t == 2 ? sum[1][0] : sum[1][1];
      const int pg = one ? page[0] : t < 2 ? page[2 * half] : page[2 * half + 1];
      if (pg >= 0 && s.len - k0 > off) {
        if (p.w_in && key < s.len - s.n) {
          float old;
          asm volatile("ld.shared.f32 %0, [%1];" : "=f"(old) : "r"(st + C::W_AT + (half * 32 + off) * 4));
          w = fmaf(p.decay, old, w);
        }
        p.w[cache_row(p.cache, pg, now.h, key & pmask)] = w;
      }
    }
    __syncwarp();
    left = now.next(p, at, stop);
    stage = stage == C::STAGES - 1 ? 0 : stage + 1;
  }
  cp_wait<0>();
}

}  // namespace gdpa
