// gdpa_cache_fwd.cuh -- attention of a few new tokens over the paged e4m3
// cache: the kernel for single tokens, drafted tokens and small groups of
// rows, and the kernel that joins its parts.
//
// Mathematics.  One pass over the keys with the running maximum and sum of the
// softmax.  Both products run transposed, S^T = K Q^T and O^T = V^T P^T, so
// that the 16-row side of the tensor-core instruction (mma m16n8k16) is filled
// with keys and coordinates, which are many, and its 8-column side with query
// rows, which are few.  e4m3 codes become fp16 exactly; a query row is divided
// by a power of two into [-2, 2) and becomes fp16 (exact down to 2^-17 of its
// largest element, below that off by 2^-25 of it); products are summed in fp32.
// The scale of a block of 16 tokens is the scale of a whole 16-key tile: K's
// multiplies the tile's scores.  The output is in units of 2^E, E one above the
// largest scale of V so far; a scale up to 2^6 below goes into the weights (in
// fp32, before their rounding to fp16) and the tile's product is summed in place,
// one further below multiplies the tile's product in fp32: no block's precision
// depends on another's within fp32's range.  Weights are
// 2^(x - r) with a reference r 7 below the running maximum when it was last
// moved, and r only moves when a score exceeds it by 15: weights stay below
// 2^15 (fp16 holds 65504), those down to 2^-21 of the maximum (2^-15 with a
// scale 2^6 below) keep 11 bits, and nothing above 2^-31 (2^-25) of it is lost.
// The row sum takes the weights before their rounding to fp16.
//
// Bound: memory, 2 D bytes a key and head, with the latency of a warp's own
// instructions close behind (conversions, byte shuffles, products).  Measured:
// one token of 64 histories of 100 to 8192 keys, 32 query and 8 key heads of 128,
// 98 us (5.6 TB/s); of 512 histories of up to 1023 keys, 8 and 8 heads of 64, 75 us
// (3.6 TB/s; the start and the join are 12 us of it); 32 rows of 128 samples, 8
// and 8 heads of 64, 172 us.
//
// Work split.  A segment is (sequence, up to 8 NT query rows of one key head);
// a step is SPAN keys of it.  The steps of all segments are counted from the
// lengths on the device, and every warp takes an equal run of them (a segment's
// start is counted as START steps more), so a batch of any raggedness, or one
// very long sequence, loads all SMs alike and nothing is planned on the host.
// Warps never wait for one another (but where the eight warps of a CTA share one
// short segment: TEAM).  Each owns a ring of stages in shared
// memory that its own asynchronous copies fill, STAGES - 1 steps ahead and
// across the ends of segments (rows that are not stored are zero-filled).  A
// segment that lies in several warps' runs leaves its parts (reference, sum,
// mean) in the workspace and the second kernel joins them in the order of the
// keys: results do not depend on timing.
#pragma once

#include <type_traits>

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
  uint32_t inv_g;  // 2^32 / G rounded up (0 for G = 1)
  int causal, window;
  float scale2;    // scale * log2(e)
  int no_split;    // segments are never cut: `part` is not used
  int* meta;       // [workers][2][8]: the segments a warp left a part of
  float* part;     // [workers][2][rows (D + 2)]
};

// Query rows of a segment by token and head.  The division by G is a product
// with 2^32 / G rounded up, which is exact below 2^32 / G, so the row of the
// segment's start is divided once and only rows behind it take it.
struct RowMap {
  int tok0, rem0;  // the first row's token and head of the group
  __device__ __forceinline__ void begin(const CacheFwdParams& p, int row0) {
    tok0 = row0 / p.G;
    rem0 = row0 - tok0 * p.G;
  }
  // Row r of the segment: its token of the sequence, and its head of the group.
  __device__ __forceinline__ int token(const CacheFwdParams& p, int r) const {
    const uint32_t x = rem0 + r;
    return tok0 + static_cast<int>(p.inv_g ? __umulhi(x, p.inv_g) : x);
  }
  __device__ __forceinline__ int head(const CacheFwdParams& p, int r, int tok) const {
    return rem0 + r - (tok - tok0) * p.G;
  }
};

// Parts of a cut segment: worker `first` holds the first in its slot 1, the
// `pieces - 1` workers behind it the next ones in their slots 0.  Beside each
// part stand {first, pieces, first row of the sequence, its rows, row tile, head}.

// TEAM: a CTA has one whole segment at most, and its warps take the steps in turn:
// one token over 201 keys takes 6.3 us on the device so and 13.7 as cut parts.
template <int D, int NT, bool TEAM_ = false>
struct SplitCfg {
  static constexpr bool TEAM = TEAM_;
  static constexpr int WARPS = TEAM ? 8 : 4, THREADS = 32 * WARPS;
  static constexpr int WORKERS = TEAM ? 1 : WARPS;  // of a CTA: its warps, or itself
  // What a segment's start and end cost, in steps: about 16 000 cycles of 1 600
  // with 32 rows, 5 000 of 2 200 with 8.  (2 for all left warps with many short
  // segments working when others were done: 232 us for 32 rows of 128 samples,
  // 190 so; 7 took 200 and 20 took 197.)
  static constexpr int START = NT == 1 ? 2 : NT == 2 ? 5 : NT == 3 ? 8 : 10;
  static constexpr int RUN_STEPS = START + 4;  // the fewest steps (starts included) that are worth a part
  static constexpr int ROWS = 8 * NT;
  static constexpr int TILE = 16 * D;  // bytes of a tile of K or of V
  static constexpr int NB = NT == 1 ? 2 : 1;  // 16-key tiles of a step
  static constexpr int SPAN = NB * kCacheBlock;
  // CTAs an SM, and ring stages: enough tiles in flight to cover the memory's
  // latency (an SM's share of 6.8 TB/s is 45 KB a microsecond) at the
  // registers that the accumulators leave.  Two tiles a step: 64 histories take
  // 98 us so, 114 with one (512 short ones 75 and 86).  D = 64 with 8 rows: 75 us
  // on three CTAs, 96 on two, 80 on four of three stages.  With 16 rows at D = 128:
  // 53 us on two CTAs, 63 on three (registers); at D = 64 42 on three, 43 on two.
  static constexpr int CTAS = TEAM ? 1 : NT == 1 ? (D == 64 ? 3 : 2) : NT == 2 && D == 64 ? 3 : 2;
  static constexpr int STAGES = D == 64 ? (NT == 1 ? 4 : 6) : NT >= 2 ? 4 : 3;
  static_assert(STAGES * NB <= 8, "a nibble of state for each tile of the ring");
  static constexpr int STAGE = NB * 2 * TILE;
  static constexpr int RING = STAGES * STAGE;      // of a warp
  static constexpr int KSTEPS = D / 16;
  static constexpr int QFRAG = NT > 1 ? KSTEPS * NT * 32 * 8 : 0;  // a warp's query fragments
  static constexpr int SMEM = WARPS * (RING + QFRAG);
};

namespace split {

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void lds128(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void lds64(uint32_t addr, uint32_t& a, uint32_t& b) {
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(a), "=r"(b) : "r"(addr));
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same with nothing added to the product.
__device__ __forceinline__ void mma_f16_new(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, "
      "%10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// Two codes (the low or the high half of w) as two fp16 values.
__device__ __forceinline__ uint32_t codes_lo(uint32_t w) {
  uint32_t h;
  asm("{ .reg .b16 lo, hi; mov.b32 {lo, hi}, %1; cvt.rn.f16x2.e4m3x2 %0, lo; }" : "=r"(h) : "r"(w));
  return h;
}
__device__ __forceinline__ uint32_t codes_hi(uint32_t w) {
  uint32_t h;
  asm("{ .reg .b16 lo, hi; mov.b32 {lo, hi}, %1; cvt.rn.f16x2.e4m3x2 %0, hi; }" : "=r"(h) : "r"(w));
  return h;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// The transpose of an 8x8 matrix of fp16 held as a fragment.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// Whether one of four codes is NaN (0x7f or 0xff).
__device__ __forceinline__ bool has_nan_code(uint32_t w) {
  return (((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0;
}

// Byte offset of 16-byte chunk c of row r in a tile: the chunks are permuted
// so that the 8 lanes of a 16-byte (16 of an 8-byte) shared-memory access of
// either fragment's reads fall on different banks.
template <int D>
__device__ __forceinline__ uint32_t tile_at(int r, int c) {
  if (D == 128) return r * 128 + ((c ^ (r & 7)) << 4);
  return (r >> 1) * 128 + (((r ^ (r >> 1)) & 1) << 6) + ((c ^ ((r >> 1) & 2)) << 4);
}

// a / b of numbers that are nearly always below 2^32 (a 64-bit division takes
// several times as long, and the first tile waits for some of these).
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// A sequence's share of the work.
struct SeqWork {
  CacheSeq s;
  int kbase;  // first key any of its rows sees, rounded down to SPAN keys
  int steps;  // of one segment
  int tiles;  // row tiles: segments of a key head
};
template <class C>
__device__ __forceinline__ SeqWork seq_work(const CacheFwdParams& p, int b) {
  SeqWork w;
  w.s = load_sequence(p.batch, p.cache.lp, b);
  w.kbase = 0;
  w.steps = 0;
  w.tiles = 0;
  if (!w.s.ok || w.s.n == 0) return w;
  w.kbase = first_key(w.s.len - w.s.n, p.window) & ~(C::SPAN - 1);
  // (a length may be as large as 2^31 - 16)
  w.steps = static_cast<int>((static_cast<unsigned>(max(w.s.len - w.kbase, 1)) + C::SPAN - 1) / C::SPAN);
  w.tiles = static_cast<int>((static_cast<unsigned>(w.s.n) * p.G + C::ROWS - 1) / C::ROWS);  // T G is below 2^31
  return w;
}
template <class C>
__device__ __forceinline__ int64_t seq_cost(const CacheFwdParams& p, const SeqWork& w) {
  return static_cast<int64_t>(w.tiles) * p.cache.H * (C::TEAM ? 1 : w.steps + C::START);
}

// The runs of a CTA's workers: where each begins.  All threads take part.
template <class C>
struct Schedule {
  int64_t scan[C::THREADS / 32];
  int64_t base[C::WORKERS];  // the work in front of the sequence in which the worker's run begins
  int seq[C::WORKERS];
};
template <class C>
__device__ __forceinline__ void schedule(const CacheFwdParams& p, Schedule<C>& sh, int64_t& total, int64_t& chunk) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, B = p.batch.B;
  int64_t mine = 0;
  const int per = (B + C::THREADS - 1) / C::THREADS;
  const int b_lo = min(B, tid * per), b_hi = min(B, b_lo + per);
  for (int b = b_lo; b < b_hi; ++b) mine += seq_cost<C>(p, seq_work<C>(p, b));
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
  for (int w = 0; w < C::THREADS / 32; ++w) {
    if (w < warp) incl += sh.scan[w];
    total += sh.scan[w];
  }
  const int64_t workers = static_cast<int64_t>(gridDim.x) * C::WORKERS;
  chunk = max(quotient(total + workers - 1, workers), p.no_split ? (int64_t)1 : (int64_t)C::RUN_STEPS);
#pragma unroll 1
  for (int w = 0; w < C::WORKERS; ++w) {
    const int64_t from = chunk * (static_cast<int64_t>(blockIdx.x) * C::WORKERS + w);
    if (from < total && from >= incl - mine && from < incl) {
      int64_t base = incl - mine;
      int b = b_lo;
      for (; b < b_hi; ++b) {
        const int64_t n = seq_cost<C>(p, seq_work<C>(p, b));
        if (from < base + n) break;
        base += n;
      }
      sh.seq[w] = b;
      sh.base[w] = base;
    }
  }
  __syncthreads();
}

// Walks the segments of a worker's run [at, stop) of the work.
template <class C>
struct Walk {
  SeqWork w;
  int64_t start;  // of the present segment
  int b, h, tile;
  int row0;       // its first query row (of the sequence and key head)
  RowMap map;
  int rows;
  int u0, u1;     // its steps that are in the run and hold visible keys
  int lo_min, hi_max;  // keys any of its rows sees: [lo_min, hi_max)
  int lo_max, hi_min;  // keys all of them see: [lo_max, hi_min)

  __device__ __forceinline__ void begin(const CacheFwdParams& p, int seq, int64_t base, int64_t at) {
    b = seq;
    w = seq_work<C>(p, b);
    const int64_t cost = C::TEAM ? 1 : w.steps + C::START, seg = quotient(at - base, cost);
    start = base + seg * cost;
    tile = static_cast<int>(quotient(seg, p.cache.H));
    h = static_cast<int>(seg - static_cast<int64_t>(tile) * p.cache.H);
  }
  __device__ __forceinline__ void next(const CacheFwdParams& p) {
    start += C::TEAM ? 1 : w.steps + C::START;
    if (++h < p.cache.H) return;
    h = 0;
    if (++tile < w.tiles) return;
    tile = 0;
    do {
      if (++b >= p.batch.B) return;
      w = seq_work<C>(p, b);
    } while (w.tiles == 0);
  }
  __device__ __forceinline__ bool more(const CacheFwdParams& p, int64_t stop) const {
    return b < p.batch.B && start < stop;
  }
  // The present segment's rows and steps; false if none of it is this run's.
  __device__ __forceinline__ bool enter(const CacheFwdParams& p, int64_t at, int64_t stop) {
    const CacheSeq& s = w.s;
    if (p.no_split) {  // a segment belongs to the run it starts in
      if (start < at) return false;
      u0 = 0;
      u1 = w.steps;
    } else {
      u0 = static_cast<int>(max(at - start - C::START, (int64_t)0));
      u1 = static_cast<int>(min(stop - start - C::START, (int64_t)w.steps));
      if (u1 <= u0) return false;
    }
    row0 = tile * C::ROWS;
    rows = min(C::ROWS, s.n * p.G - row0);
    map.begin(p, row0);
    const int pos0 = s.len - s.n + map.tok0;
    const int pos1 = s.len - s.n + map.token(p, rows - 1);
    lo_min = first_key(pos0, p.window);
    hi_max = max(0, p.causal ? min(s.len, pos1 + 1) : s.len);
    lo_max = first_key(pos1, p.window);
    hi_min = max(0, p.causal ? min(s.len, pos0 + 1) : s.len);
    u0 = max(u0, (lo_min - w.kbase) / C::SPAN);
    u1 = hi_max > w.kbase ? min(u1, (hi_max - 1 - w.kbase) / C::SPAN + 1) : u0;
    return true;
  }
};

}  // namespace split

// A segment that the CTA's warps shared: their references, sums and
// outputs meet in shared memory, and each thread joins pieces of rows.
template <int D, int NT, class C>
__device__ __forceinline__ void team_join(const CacheFwdParams& p, uint8_t* smem,
                                          float (&s_team)[C::WARPS][C::ROWS][2],
                                          const float (&acc)[D / 16][NT][4], float unit, const float (&ref)[NT][2],
                                          const float (&room)[NT][2], const float (&sum)[NT][2], const CacheSeq& s,
                                          int h, const RowMap& map, int rows) {
  static_assert(C::WARPS * C::ROWS * D * 4 <= C::WARPS * C::RING, "the rings hold the outputs");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  split::cp_wait<0>();
  __syncthreads();  // every warp is done with its ring
  float* merge = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float l = sum[nt][c];
      l += __shfl_xor_sync(0xffffffffu, l, 4);
      l += __shfl_xor_sync(0xffffffffu, l, 8);
      l += __shfl_xor_sync(0xffffffffu, l, 16);
      const int r = nt * 8 + 2 * t + c;
      if (g == 0) s_team[warp][r][0] = room[nt][c] == -INFINITY ? -INFINITY : ref[nt][c], s_team[warp][r][1] = l;
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;  // means: they are as large as values, sums may not be held
      float4* dst = reinterpret_cast<float4*>(merge + (warp * C::ROWS + r) * D + g * (D / 8));
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
        dst[i] = make_float4(acc[2 * i][nt][c] * inv * unit, acc[2 * i][nt][c + 2] * inv * unit,
                             acc[2 * i + 1][nt][c] * inv * unit, acc[2 * i + 1][nt][c + 2] * inv * unit);
    }
  __syncthreads();
  for (int i = tid; i < rows * (D / 8); i += C::THREADS) {
    const int r = i / (D / 8), d = i % (D / 8) * 8;
    float top = -INFINITY, l = 0.0f, o[8] = {};
#pragma unroll
    for (int w = 0; w < C::WARPS; ++w) top = fmaxf(top, s_team[w][r][0]);
#pragma unroll
    for (int w = 0; w < C::WARPS; ++w)
      l += s_team[w][r][1] * ptx::ex2_approx(s_team[w][r][0] - (top == -INFINITY ? 0.0f : top));
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
    for (int w = 0; w < C::WARPS; ++w) {
      const float f = s_team[w][r][1] * ptx::ex2_approx(s_team[w][r][0] - (top == -INFINITY ? 0.0f : top)) * inv;
      const float4* src = reinterpret_cast<const float4*>(merge + (w * C::ROWS + r) * D + d);
      const float4 x = src[0], y = src[1];
      o[0] += x.x * f, o[1] += x.y * f, o[2] += x.z * f, o[3] += x.w * f;
      o[4] += y.x * f, o[5] += y.y * f, o[6] += y.z * f, o[7] += y.w * f;
    }
    const int tok = map.token(p, r);
    const int64_t at_row = static_cast<int64_t>(s.first + tok) * p.Hq + h * p.G + map.head(p, r, tok);
    *reinterpret_cast<uint4*>(p.out + at_row * D + d) =
        make_uint4(ptx::pack_bf16x2(o[0], o[1]), ptx::pack_bf16x2(o[2], o[3]), ptx::pack_bf16x2(o[4], o[5]),
                   ptx::pack_bf16x2(o[6], o[7]));
    if (p.lse && d == 0) p.lse[at_row] = l == 0.0f ? -INFINITY : (top + log2f(l)) * 0.6931471805599453f;
  }
}

template <int D, int NT, bool TEAM>
__global__ void __launch_bounds__((SplitCfg<D, NT, TEAM>::THREADS), (SplitCfg<D, NT, TEAM>::CTAS))
    gdpa_cache_split_kernel(const CacheFwdParams p) {
  using namespace split;
  using C = SplitCfg<D, NT, TEAM>;
  constexpr int KS = C::KSTEPS, ND = D / 16;  // k-steps of S^T; 16-row tiles of O^T
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Schedule<C> sh;
  __shared__ float s_team[C::TEAM ? C::WARPS : 1][C::TEAM ? C::ROWS : 1][2];
  __shared__ __align__(8) uint32_t s_sf[C::WARPS][C::STAGES][2 * C::NB];  // words that hold the scale codes
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  const CacheBatch& bt = p.batch;
  const int worker = C::TEAM ? blockIdx.x : blockIdx.x * C::WARPS + warp;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join may be set up beside this

  if (lane == 0 && !p.no_split) p.meta[worker * 16 + 1] = p.meta[worker * 16 + 9] = 0;  // no parts yet
  int64_t total, chunk;
  schedule<C>(p, sh, total, chunk);
  const int64_t at = chunk * worker, stop = min(total, at + chunk);
  if (at >= stop) return;

  const uint32_t ring = ptx::smem_u32(smem) + warp * C::RING;
  uint2* qfrag = reinterpret_cast<uint2*>(smem + C::WARPS * C::RING + warp * C::QFRAG);
  const uint32_t sf_at = ptx::smem_u32(&s_sf[warp][0][0]);
  const int pmask = (1 << p.cache.lp) - 1;
  const int64_t sf_bytes = static_cast<int64_t>(p.cache.num_pages) * p.cache.H << (p.cache.lp - 4);

  constexpr int stride = C::TEAM ? C::WARPS : 1;
  const int skip = C::TEAM ? warp : 0, self = C::TEAM ? 0 : warp;

  // ---- the copies: a walk that runs ahead of the one that computes
  Walk<C> ahead;
  ahead.begin(p, sh.seq[self], sh.base[self], at);
  Walk<C> now = ahead;
  int ahead_u = 0;
  bool ahead_more = false;
  // its next step: page of each tile, -1: nothing to read
  int page_next[C::NB];
  bool whole = false;  // all of the step is there, and in one page
  auto look = [&]() {
    while (!ahead_more || ahead_u >= ahead.u1) {
      if (ahead_more) ahead.next(p);
      ahead_more = true;
      if (!ahead.more(p, stop)) {
        ahead_u = ahead.u1 = -1;  // done
        ahead_more = false;
        return;
      }
      if (!ahead.enter(p, at, stop)) {
        ahead_u = ahead.u1 = 0;
        continue;
      }
      ahead_u = ahead.u0 + skip;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)  // its queries come while its first tiles do
        if (nt * 8 + g < ahead.rows) {
          const int r = nt * 8 + g, tok = ahead.map.token(p, r);
          const __nv_bfloat16* src = p.q + (ahead.w.s.first + tok) * p.q_stride +
                                     (ahead.h * p.G + ahead.map.head(p, r, tok)) * D + t * (D / 4);
          asm volatile("prefetch.global.L1 [%0];" ::"l"(src));
        }
    }
    const int kb = ahead.w.kbase + ahead_u * C::SPAN;
    const int32_t* table = bt.table + static_cast<int64_t>(ahead.b) * bt.max_pages;
    whole = kb >= ahead.lo_min && kb <= ahead.hi_max - C::SPAN && (C::NB == 1 || p.cache.lp > 4);
    if (whole) {
      page_next[0] = __ldg(table + (kb >> p.cache.lp));
      whole = static_cast<unsigned>(page_next[0]) < static_cast<unsigned>(p.cache.num_pages);
      if (whole) return;
    }
#pragma unroll
    for (int n = 0; n < C::NB; ++n) {
      const int k = kb + n * kCacheBlock;
      page_next[n] = -1;
      if (k < ahead.hi_max && k + kCacheBlock > ahead.lo_min) {
        page_next[n] = __ldg(table + (k >> p.cache.lp));
        if (page_next[n] < 0 || page_next[n] >= p.cache.num_pages) {
          if (lane == 0) atomicOr(bt.status, kStatusBadPlan);
          page_next[n] = -1;
        }
      }
    }
  };
  // A nibble for each tile of the ring: bit 0 the tile is there, bits 1-2
  // which byte of its words the scale codes are.
  uint32_t state = 0;
  const uint32_t chunk_at = tile_at<D>(lane / (D / 16), lane % (D / 16));  // of this lane's first 16 bytes of a tile
  auto issue = [&](int stage) {
    constexpr uint32_t nibbles = C::NB == 2 ? 0x11u : 1u;
    state &= ~(15u * nibbles << (stage * 4 * C::NB));
    if (ahead_more) {
      const int kb = ahead.w.kbase + ahead_u * C::SPAN;
      const uint32_t dst = ring + stage * C::STAGE;
      if (whole) {
        const int64_t row = cache_row(p.cache, page_next[0], ahead.h, kb & pmask);
        const uint8_t* ks = p.cache.k + row * D + lane * 16;
        const uint8_t* vs = p.cache.v + row * D + lane * 16;
#pragma unroll
        for (int n = 0; n < C::NB; ++n)
#pragma unroll
          for (int j = 0; j < D / 32; ++j) {
            // 32 chunks further on: as many rows, and the same permutation
            // (or another one, which is a constant too)
            const uint32_t to = dst + n * 2 * C::TILE + (D == 128 ? (chunk_at ^ (j & 1) * 64) : chunk_at) + j * 512;
            cp_async16(to, ks + (n * kCacheBlock * D + 512 * j), 16);
            cp_async16(to + C::TILE, vs + (n * kCacheBlock * D + 512 * j), 16);
          }
        const int64_t block = row >> 4, word = block & ~(int64_t)3;
        // (a step's second block is in the same word: its first one is even)
        state |= (nibbles + (nibbles * (static_cast<uint32_t>(block & 3) << 1)) + (C::NB == 2 ? 0x20u : 0u))
                 << (stage * C::NB * 4);
        if (lane < 2 * C::NB)
          cp_async4(sf_at + (stage * 2 * C::NB + lane) * 4, ((lane & 1) ? p.cache.v_sf : p.cache.k_sf) + word,
                    static_cast<int>(min((int64_t)4, sf_bytes - word)));
      } else {
#pragma unroll 1
        for (int n = 0; n < C::NB; ++n) {
          const int page = n == 0 ? page_next[0] : page_next[C::NB - 1], slot = (kb + n * kCacheBlock) & pmask;
          const int valid = ahead.w.s.len - (kb + n * kCacheBlock);
          const int64_t row = cache_row(p.cache, max(page, 0), ahead.h, slot);
          const uint8_t* ks = p.cache.k + row * D + lane * 16;
          const uint8_t* vs = p.cache.v + row * D + lane * 16;
          const uint32_t kd = dst + n * 2 * C::TILE, vd = kd + C::TILE;
#pragma unroll
          for (int j = 0; j < D / 32; ++j) {  // rows that are not stored: zeros
            const int idx = lane + 32 * j, r = idx / (D / 16), c = idx % (D / 16);
            const uint32_t to = tile_at<D>(r, c);
            if (page < 0) {  // (no address stands for them: a cache may have no page at all)
              ptx::st_shared_v4(kd + to, 0, 0, 0, 0);
              ptx::st_shared_v4(vd + to, 0, 0, 0, 0);
              continue;
            }
            const int bytes = r < valid ? 16 : 0;
            cp_async16(kd + to, ks + 512 * j, bytes);
            cp_async16(vd + to, vs + 512 * j, bytes);
          }
          if (page >= 0) {
            const int64_t block = row >> 4, word = block & ~(int64_t)3;
            state |= (1u | static_cast<uint32_t>(block & 3) << 1) << ((stage * C::NB + n) * 4);
            if (lane >> 1 == n)  // lanes 2n and 2n + 1: K's word and V's
              cp_async4(sf_at + (stage * 2 * C::NB + lane) * 4, ((lane & 1) ? p.cache.v_sf : p.cache.k_sf) + word,
                        static_cast<int>(min((int64_t)4, sf_bytes - word)));
          }
        }
      }
      ahead_u += stride;
      look();
    }
    cp_commit();
  };
  look();
#pragma unroll 1
  for (int i = 0; i < C::STAGES - 1; ++i) issue(i);
  int stage = 0;

#pragma unroll 1
  for (; now.more(p, stop); now.next(p)) {
    if (!now.enter(p, at, stop)) continue;
    const CacheSeq s = now.w.s;
    const int h = now.h, rows = now.rows;

    // ---- query fragments, and what each column (query row) sees
    uint32_t qf[NT == 1 ? KS : 1][2];
    float fac[NT][2];
    int lo[NT][2], hi[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = nt * 8 + g;
      float x[D / 4];
      float amax = 0.0f;
      if (r < rows) {
        const int tok = now.map.token(p, r);
        const __nv_bfloat16* src =
            p.q + (s.first + tok) * p.q_stride + (h * p.G + now.map.head(p, r, tok)) * D + t * (D / 4);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          const uint4 u = *reinterpret_cast<const uint4*>(src + 8 * i);
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            x[8 * i + 2 * e] = __uint_as_float(w[e] << 16);
            x[8 * i + 2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < D / 4; ++i) x[i] = 0.0f;
      }
#pragma unroll
      for (int i = 0; i < D / 4; ++i) amax = fmaxf(amax, fabsf(x[i]));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      // 2^e: the largest element's power of two (1 for an all-zero row)
      const int e = amax > 0.0f ? min(max(static_cast<int>(__float_as_uint(amax) >> 23) - 127, -126), 127) : 0;
      const float inv = sf_value(127 - e);
      const float f = sf_value(127 + e) * p.scale2;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const uint32_t b0 = pack_f16x2(x[4 * k] * inv, x[4 * k + 1] * inv);
        const uint32_t b1 = pack_f16x2(x[4 * k + 2] * inv, x[4 * k + 3] * inv);
        if (NT == 1) {
          qf[NT == 1 ? k : 0][0] = b0;
          qf[NT == 1 ? k : 0][1] = b1;
        } else {
          qfrag[(k * NT + nt) * 32 + lane] = make_uint2(b0, b1);
        }
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int col = nt * 8 + 2 * t + c;
        fac[nt][c] = __shfl_sync(0xffffffffu, f, 8 * t + 4 * c);
        const int pos = s.len - s.n + now.map.token(p, col);
        lo[nt][c] = first_key(pos, p.window);
        hi[nt][c] = col < rows ? (p.causal ? min(s.len, pos + 1) : s.len) : 0;
      }
    }
    const int lo_min = now.lo_min, hi_max = now.hi_max, lo_max = now.lo_max, hi_min = now.hi_min;
    if (NT > 1) __syncwarp();

    float acc[ND][NT][4];
    // the softmax's reference of each column, and by how much a score may
    // exceed it (not at all while there is none)
    float ref[NT][2], room[NT][2], sum[NT][2];
    int vexp = -1;  // the output is in units of 2^(vexp - 127)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int c = 0; c < 2; ++c) ref[nt][c] = 0.0f, room[nt][c] = -INFINITY, sum[nt][c] = 0.0f;
#pragma unroll
      for (int i = 0; i < ND; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[i][nt][c] = 0.0f;
    }

    // One step's products and softmax; EDGE: some of its keys are hidden from
    // some of the rows, or a tile is not there.
    auto compute = [&](auto edge_tag, const uint32_t kt, const int cur, const uint32_t there, const int kb) {
      constexpr bool EDGE = decltype(edge_tag)::value;
      // S^T = K Q^T: rows g and g + 8 are keys, columns 2t and 2t + 1 queries
      float st[C::NB][NT][4];
#pragma unroll
      for (int j = 0; j < D / 64; ++j)
#pragma unroll
        for (int n = 0; n < C::NB; ++n) {
          uint32_t ka[4], kc[4];
          const int c = D == 128 ? 2 * t + j : t;
          lds128(kt + n * 2 * C::TILE + tile_at<D>(g, c), ka);
          lds128(kt + n * 2 * C::TILE + tile_at<D>(g + 8, c), kc);
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const int k = 4 * j + w;
            const uint32_t a0 = codes_lo(ka[w]), a2 = codes_hi(ka[w]), a1 = codes_lo(kc[w]), a3 = codes_hi(kc[w]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              uint32_t q0, q1;
              if (NT == 1) {
                q0 = qf[NT == 1 ? k : 0][0], q1 = qf[NT == 1 ? k : 0][1];
              } else {
                const uint2 qq = qfrag[(k * NT + nt) * 32 + lane];
                q0 = qq.x, q1 = qq.y;
              }
              if (k == 0)
                mma_f16_new(st[n][nt], a0, a1, a2, a3, q0, q1);
              else
                mma_f16(st[n][nt], a0, a1, a2, a3, q0, q1);
            }
          }
        }

      // scores in units of log2, less the reference; hidden keys -inf; does
      // one leave the range, or a scale of V the output's units?
      int sv[C::NB];
      bool over = false;
#pragma unroll
      for (int n = 0; n < C::NB; ++n) {
        uint32_t kw, vw;
        lds64(sf_at + (cur * C::NB + n) * 8, kw, vw);
        const bool here = !EDGE || (there >> (4 * n) & 1);
        const int byte = (there >> (4 * n) & 6) * 4;
        const float sk = sf_value(here ? kw >> byte & 0xff : 127);
        sv[n] = here ? vw >> byte & 0xff : max(vexp, 0);
        over |= sv[n] > vexp;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float x = fmaf(st[n][nt][c], fac[nt][c & 1] * sk, -ref[nt][c & 1]);
            if (EDGE) {
              const int key = kb + n * kCacheBlock + g + (c & 2) * 4;
              if (key < lo[nt][c & 1] || key >= hi[nt][c & 1] || !here) x = -INFINITY;
            }
            st[n][nt][c] = x;
            over |= x > room[nt][c & 1];
          }
      }
      if (__any_sync(0xffffffffu, over)) {
        // V's units: one above the largest scale, so that they seldom move.  At
        // an edge a row may see nothing of a block that lies far above: what it
        // has summed, or will sum, must not vanish in that block's units.  There
        // they stay up to 2^90 behind (edges are three steps at most, at either
        // end of a row's keys, so that the sums stay finite).
        int top_sv = sv[0];
        if (C::NB == 2) top_sv = max(top_sv, sv[C::NB - 1]);
        float turn = 1.0f;
        if (top_sv > vexp) {
          int up = min(top_sv + 1, 254);
          if (EDGE && (up > 140 || (vexp >= 0 && top_sv - vexp > 40))) up = max(vexp < 0 ? 100 : vexp, top_sv - 90);
          turn = vexp < 0 ? 0.0f : up - vexp > 126 ? 0.0f : sf_value(127 - (up - vexp));
          vexp = up;
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float top = fmaxf(st[0][nt][c], st[0][nt][c + 2]);
#pragma unroll
            for (int n = 1; n < C::NB; ++n) top = fmaxf(top, fmaxf(st[n][nt][c], st[n][nt][c + 2]));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
            // (the column's reference stays unless a score of it has left the range)
            const bool none = room[nt][c] == -INFINITY, move = top > room[nt][c];
            const float up = !move ? 0.0f : none ? top - 7.0f : fmaxf(top - 7.0f, 0.0f);
            const float keep = none ? 0.0f : ptx::ex2_approx(-up);
            if (move) room[nt][c] = 15.0f;
            ref[nt][c] += up;
            sum[nt][c] *= keep;
            const float keep_o = keep * turn;
#pragma unroll
            for (int n = 0; n < C::NB; ++n) st[n][nt][c] -= up, st[n][nt][c + 2] -= up;
#pragma unroll
            for (int i2 = 0; i2 < ND; ++i2) {
              acc[i2][nt][c] *= keep_o;
              acc[i2][nt][c + 2] *= keep_o;
            }
          }
      }
#pragma unroll
      for (int n = 0; n < C::NB; ++n) {
        // a scale up to 2^6 below the units goes into the weights
        const int below = vexp - sv[n];
        const bool near = below >= 0 && below <= 6;
        const float unit = sf_value(127 - (near ? below : 0));
        uint32_t pb[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float p0 = ptx::ex2_approx(st[n][nt][0]), p1 = ptx::ex2_approx(st[n][nt][1]);
          const float p2 = ptx::ex2_approx(st[n][nt][2]), p3 = ptx::ex2_approx(st[n][nt][3]);
          sum[nt][0] += p0 + p2;
          sum[nt][1] += p1 + p3;
          pb[nt][0] = transpose8x8(pack_f16x2(p0 * unit, p1 * unit));
          pb[nt][1] = transpose8x8(pack_f16x2(p2 * unit, p3 * unit));
        }

        // O^T += V^T P^T: lane (g, t) holds D/8 coordinates of tokens 2t, 2t+1, 2t+8, 2t+9
        const uint32_t vt = kt + n * 2 * C::TILE + C::TILE;
        uint32_t v[4][D / 32];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = 2 * t + (j & 1) + (j & 2) * 4;
          if (D == 128) {
            uint32_t x[4];
            lds128(vt + tile_at<D>(r, g), x);
#pragma unroll
            for (int w = 0; w < D / 32; ++w) v[j][w] = x[w];
          } else {
            lds64(vt + tile_at<D>(r, g >> 1) + (g & 1) * 8, v[j][0], v[j][1]);
          }
        }
        // At an edge a token may be hidden from some rows only, and 0 times a
        // NaN value is NaN: such a tile is added token by token to the rows
        // that see it.  Tokens hidden from all rows are cleared.
        bool apart = !near;
        int tokens = 1;  // products that a tile apart takes
        if (EDGE) {
          bool nan = false;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int key = kb + n * kCacheBlock + 2 * t + (j & 1) + (j & 2) * 4;
#pragma unroll
            for (int w = 0; w < D / 32; ++w) {
              if (key < lo_min || key >= hi_max) v[j][w] = 0;
              nan |= has_nan_code(v[j][w]);
            }
          }
          if (__any_sync(0xffffffffu, nan)) apart = true, tokens = kCacheBlock;
        }
        if (!apart) {
#pragma unroll
          for (int w = 0; w < D / 32; ++w)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const uint32_t x01 = __byte_perm(v[0][w], v[1][w], half ? 0x7362 : 0x5140);
              const uint32_t x23 = __byte_perm(v[2][w], v[3][w], half ? 0x7362 : 0x5140);
              const uint32_t a0 = codes_lo(x01), a1 = codes_hi(x01), a2 = codes_lo(x23), a3 = codes_hi(x23);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma_f16(acc[2 * w + half][nt], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
            }
        } else {
          // what the weights do not hold of the scale, as a factor of the product
          const float rest = near        ? 1.0f
                             : below < 0 ? sf_value(127 - below)
                                         : sf_value(127 - (below >> 1)) * sf_value(127 - (below - (below >> 1)));
#pragma unroll 1
          for (int k = 0; k < tokens; ++k) {
            const int key = kb + n * kCacheBlock + k;
            const bool one = tokens > 1;
#pragma unroll
            for (int w = 0; w < D / 32; ++w)
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                uint32_t y[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) y[j] = !one || 2 * t + (j & 1) + (j & 2) * 4 == k ? v[j][w] : 0;
                const uint32_t x01 = __byte_perm(y[0], y[1], half ? 0x7362 : 0x5140);
                const uint32_t x23 = __byte_perm(y[2], y[3], half ? 0x7362 : 0x5140);
                const uint32_t a0 = codes_lo(x01), a1 = codes_hi(x01), a2 = codes_lo(x23), a3 = codes_hi(x23);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  float o[4];
                  mma_f16_new(o, a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
#pragma unroll
                  for (int c = 0; c < 4; ++c)
                    if (!one || (key >= lo[nt][c & 1] && key < hi[nt][c & 1]))
                      acc[2 * w + half][nt][c] = fmaf(o[c], rest, acc[2 * w + half][nt][c]);
                }
              }
          }
        }
      }
    };

#pragma unroll 1
    for (int u = now.u0 + skip; u < now.u1; u += stride) {
      cp_wait<C::STAGES - 2>();
      __syncwarp();
      issue(stage == 0 ? C::STAGES - 1 : stage - 1);
      const uint32_t kt = ring + stage * C::STAGE;
      const int cur = stage;
      const uint32_t there = state >> (cur * 4 * C::NB);
      stage = stage + 1 == C::STAGES ? 0 : stage + 1;
      constexpr uint32_t all = C::NB == 2 ? 0x11u : 1u;
      const int kb = now.w.kbase + u * C::SPAN;
      if (kb >= lo_max && kb <= hi_min - C::SPAN && (there & all) == all)
        compute(std::false_type(), kt, cur, there, kb);
      else if ((there & all) != 0)
        compute(std::true_type(), kt, cur, there, kb);
    }
    // the output in its own units
    const float unit = vexp < 0 ? 0.0f : sf_value(vexp);
    if constexpr (C::TEAM) {  // the warps' results meet in the rings' room
      team_join<D, NT, C>(p, smem, s_team, acc, unit, ref, room, sum, s, h, now.map, rows);
      return;  // the CTA's only one
    }

    // ---- the segment's result, or this run's part of it
    const int64_t unit0 = now.start + C::START;
    const int first = p.no_split ? 0 : static_cast<int>(quotient(unit0, chunk));
    const int pieces = p.no_split ? 1 : static_cast<int>(quotient(unit0 + now.w.steps - 1, chunk)) - first + 1;
    const int slot = first == worker ? 1 : 0;
    float* part = p.part + (static_cast<int64_t>(worker) * 2 + slot) * C::ROWS * (D + 2);
    if (pieces > 1 && lane == 0) {
      int* m = p.meta + worker * 16 + slot * 8;
      m[0] = first, m[1] = pieces, m[2] = s.first, m[3] = s.n, m[4] = now.tile, m[5] = h;
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float l = sum[nt][c];
        l += __shfl_xor_sync(0xffffffffu, l, 4);
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        const int r = nt * 8 + 2 * t + c;
        const float m = room[nt][c] == -INFINITY ? -INFINITY : ref[nt][c];
        if (r >= rows) continue;
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        if (pieces == 1) {
          const int tok = now.map.token(p, r);
          const int64_t at_row = static_cast<int64_t>(s.first + tok) * p.Hq + h * p.G + now.map.head(p, r, tok);
          uint32_t o[ND];
#pragma unroll
          for (int i = 0; i < ND; ++i)
            o[i] = ptx::pack_bf16x2(acc[i][nt][c] * inv * unit, acc[i][nt][c + 2] * inv * unit);
          uint4* dst = reinterpret_cast<uint4*>(p.out + at_row * D + g * (D / 8));
#pragma unroll
          for (int i = 0; i < ND / 4; ++i) dst[i] = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
          if (p.lse && g == 0) p.lse[at_row] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
        } else {
          if (g == 0) part[2 * r] = m, part[2 * r + 1] = l;
          float4* dst = reinterpret_cast<float4*>(part + 2 * C::ROWS + r * D + g * (D / 8));
#pragma unroll
          for (int i = 0; i < ND / 2; ++i)  // means, as large as values: their sums may not be held
            dst[i] = make_float4(acc[2 * i][nt][c] * inv * unit, acc[2 * i][nt][c + 2] * inv * unit,
                                 acc[2 * i + 1][nt][c] * inv * unit, acc[2 * i + 1][nt][c + 2] * inv * unit);
        }
      }
  }
}

// Joins the parts of cut segments.  A worker is a member of up to two of them
// (the segment that its run begins inside, slot 0, and the one it ends inside,
// slot 1), and the members of a segment share its rows evenly; a block stands
// for the WORKERS workers of a CTA and its slots are shared out to its warps, a
// row to D / 4 lanes.  A segment of more than kJoinFew parts: the block's warps
// take a row together, each a run of the parts.  All that is read of up to 8
// parts is under way at once: what this kernel takes is the latency of two
// dependent reads.  (With all warps going through all slots, a warp a row, the
// slots' own arithmetic was most of it: 27 us after 32 candidates of 128
// samples, which takes 12 so.)
constexpr int kJoinWarps = 8, kJoinFew = 8;

template <int D, int ROWS, int WORKERS>
__global__ void __launch_bounds__(32 * kJoinWarps, 3) gdpa_cache_join_kernel(const CacheFwdParams p) {
  constexpr int LANES = D / 4, SUBS = 32 / LANES;  // lanes of a row, rows of a warp
  constexpr int SLOTS = 2 * WORKERS, SHARE = kJoinWarps / SLOTS;
  __shared__ float s_part[kJoinWarps * SUBS][D + 4];
  __shared__ int s_meta[SLOTS][8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane / LANES, li = lane % LANES;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the parts are there
  if (threadIdx.x < 8 * SLOTS)
    s_meta[threadIdx.x >> 3][threadIdx.x & 7] = p.meta[blockIdx.x * 8 * SLOTS + threadIdx.x];
  __syncthreads();

  // Adds parts [j, j + cnt), cnt up to 8, of a row: four coordinates a lane.  A
  // part is a reference, a sum and the mean of the values; so is the result.
  auto add = [&](int first, int j, int cnt, int r, float& ref, float& l, float4& o) {
    constexpr int step = 2 * ROWS * (D + 2);
    const float* part = p.part + static_cast<int64_t>(first + j) * step;
    const int skip = j == 0 ? ROWS * (D + 2) : 0;  // slot 1 for the first part, 0 for the others
    const int i8 = li & 7;
    float2 own = make_float2(-INFINITY, 0.0f);
    if (i8 < cnt) own = *reinterpret_cast<const float2*>(part + i8 * step + (i8 == 0 ? skip : 0) + 2 * r);
    const float* src = part + 2 * ROWS + r * D + li * 4;
    float4 x[kJoinFew];
#pragma unroll
    for (int i = 0; i < kJoinFew; ++i) {
      x[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (i < cnt) x[i] = *reinterpret_cast<const float4*>(src + i * step + (i == 0 ? skip : 0));
    }
    float top = fmaxf(ref, own.x);
#pragma unroll
    for (int d = 4; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    const float zero = top == -INFINITY ? 0.0f : top;
    const float keep = ptx::ex2_approx(ref - zero), f = ptx::ex2_approx(own.x - zero);
    float more = own.y * f;
#pragma unroll
    for (int d = 4; d > 0; d >>= 1) more += __shfl_xor_sync(0xffffffffu, more, d);
    ref = top;
    const float all = l * keep + more, inv = all == 0.0f ? 0.0f : 1.0f / all, stay = l * keep * inv;
    const float share = own.y * f * inv;
    l = all;
    o.x *= stay, o.y *= stay, o.z *= stay, o.w *= stay;
#pragma unroll
    for (int i = 0; i < kJoinFew; ++i) {
      const float w = __shfl_sync(0xffffffffu, share, i, 8);  // (0 times 0 behind the last part)
      o.x = fmaf(x[i].x, w, o.x), o.y = fmaf(x[i].y, w, o.y), o.z = fmaf(x[i].z, w, o.z), o.w = fmaf(x[i].w, w, o.w);
    }
  };
  auto store = [&](const RowMap& map, const int* m, int r, float ref, float l, const float4& o) {
    const int tok = map.token(p, r);
    const int64_t at_row = static_cast<int64_t>(m[2] + tok) * p.Hq + m[5] * p.G + map.head(p, r, tok);
    *reinterpret_cast<uint2*>(p.out + at_row * D + li * 4) =
        make_uint2(ptx::pack_bf16x2(o.x, o.y), ptx::pack_bf16x2(o.z, o.w));
    if (p.lse && li == 0) p.lse[at_row] = l == 0.0f ? -INFINITY : (ref + log2f(l)) * 0.6931471805599453f;
  };
  // m: {first worker, pieces, first row of the sequence, its rows, row tile, head}
  auto share_of = [&](const int* m, int slot, RowMap& map, int& r0, int& r1) {
    const int pieces = m[1], member = blockIdx.x * WORKERS + (slot >> 1) - m[0];
    const int row0 = m[4] * ROWS, rows = min(ROWS, m[3] * p.G - row0);
    map.begin(p, row0);
    r0 = (member * rows + pieces - 1) / pieces;  // rows r with r pieces / rows == member
    r1 = ((member + 1) * rows + pieces - 1) / pieces;
  };

  {
    const int slot = warp % SLOTS;
    const int* m = s_meta[slot];
    if (m[1] > 0 && m[1] <= kJoinFew) {
      RowMap map;
      int r0, r1;
      share_of(m, slot, map, r0, r1);
      const int unit = blockIdx.y * SHARE + warp / SLOTS, units = gridDim.y * SHARE;
#pragma unroll 1
      for (int rb = r0 + unit * SUBS; rb < r1; rb += units * SUBS) {
        const int r = min(rb + sub, r1 - 1);
        float ref = -INFINITY, l = 0.0f;
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        add(m[0], 0, m[1], r, ref, l, o);
        if (rb + sub < r1) store(map, m, r, ref, l, o);
      }
    }
  }
#pragma unroll 1
  for (int slot = 0; slot < SLOTS; ++slot) {
    const int* m = s_meta[slot];
    const int pieces = m[1];
    if (pieces <= kJoinFew) continue;
    RowMap map;
    int r0, r1;
    share_of(m, slot, map, r0, r1);
    constexpr int RUNS = kJoinWarps * SUBS;
    const int run = warp * SUBS + sub;
    const int j0 = static_cast<int>(static_cast<int64_t>(pieces) * run / RUNS);
    const int j1 = static_cast<int>(static_cast<int64_t>(pieces) * (run + 1) / RUNS);
    const int turns = (pieces + RUNS * kJoinFew - 1) / (RUNS * kJoinFew);  // all lanes take as many
#pragma unroll 1
    for (int r = r0 + blockIdx.y; r < r1; r += gridDim.y) {
      float ref = -INFINITY, l = 0.0f;
      float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
      for (int i = 0; i < turns; ++i) {
        const int j = j0 + i * kJoinFew;
        add(m[0], j, min(max(j1 - j, 0), kJoinFew), r, ref, l, o);
      }
      __syncthreads();
      *reinterpret_cast<float4*>(&s_part[run][li * 4]) = o;
      if (li == 0) s_part[run][D] = ref, s_part[run][D + 1] = l;
      __syncthreads();
      if (warp != 0 || sub != 0) continue;
      ref = -INFINITY;
#pragma unroll
      for (int w = 0; w < RUNS; ++w) ref = fmaxf(ref, s_part[w][D]);
      l = 0.0f;
      o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < RUNS; ++w) l += s_part[w][D + 1] * ptx::ex2_approx(s_part[w][D] - (ref == -INFINITY ? 0.0f : ref));
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
      for (int w = 0; w < RUNS; ++w) {
        const float f = s_part[w][D + 1] * ptx::ex2_approx(s_part[w][D] - (ref == -INFINITY ? 0.0f : ref)) * inv;
        const float4 x = *reinterpret_cast<const float4*>(&s_part[w][li * 4]);
        o.x = fmaf(x.x, f, o.x), o.y = fmaf(x.y, f, o.y), o.z = fmaf(x.z, f, o.z), o.w = fmaf(x.w, f, o.w);
      }
      store(map, m, r, ref, l, o);
    }
  }
}

}  // namespace gdpa
