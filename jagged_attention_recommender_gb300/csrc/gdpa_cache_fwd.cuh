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
// multiplies the tile's scores, V's the tile's product as it is added to the
// output, in fp32, so no block's precision depends on another's.  Weights are
// 2^(x - r) with a reference r 7 below the running maximum when it was last
// moved, and r only moves when a score exceeds it by 15: weights stay below
// 2^15 (fp16 holds 65504), those down to 2^-21 of the maximum keep 11 bits,
// and nothing above 2^-31 of it is lost.  The row sum takes the weights before
// their rounding to fp16.
//
// Bound: memory, 2 D bytes a key and head.  A warp owns a ring of 16-key tiles
// in shared memory that its own asynchronous copies fill (rows behind the
// sequence's end are zero-filled), so warps never wait for one another until
// the keys of their segment are done.
//
// Work split.  A segment is (sequence, up to 8 NT query rows of one key head);
// a unit is 64 keys of it, one tile for each of the CTA's four warps.  The
// units of all segments are counted from the lengths on the device by every
// CTA, and each takes an equal run of them, so a batch of any raggedness, or
// one very long sequence, loads every SM alike and nothing is planned on the
// host.  A segment that lies in several CTAs' runs leaves its parts (maximum,
// sum, output) in the workspace and the second kernel joins them in the order
// of the keys: results do not depend on timing.
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
  int no_split;    // one segment is never cut: `part` is not used
  int* meta;       // [CTAs][2][8]: the segment a CTA left a part of (see SplitMeta)
  float* part;     // [CTAs][2][rows (D + 2)]
};

constexpr int kUnitKeys = 64;

// Parts of a cut segment: CTA `first` holds the first in its slot 1, the
// `pieces - 1` CTAs behind it the next ones in their slots 0.
struct SplitMeta {
  int first, pieces, row0, n, tile, head;
};

template <int D, int NT>
struct SplitCfg {
  static constexpr int THREADS = 128, WARPS = 4;
  static constexpr int ROWS = 8 * NT;
  static constexpr int TILE = 16 * D;  // bytes of a tile of K or of V
  // CTAs an SM, and ring stages: enough tiles in flight to cover the memory's
  // latency (an SM's share of 6.8 TB/s is 45 KB a microsecond) at the
  // registers that the accumulators leave
  static constexpr int CTAS = NT == 1 ? 4 : NT == 2 ? 3 : 2;
  static constexpr int STAGES = (NT == 1 ? 3 : NT == 2 ? 4 : 5) * (D == 64 ? 2 : 1) - (D == 64 ? 1 : 0);
  static constexpr int RING = WARPS * STAGES * 2 * TILE;
  static constexpr int MERGE = WARPS * ROWS * D * 4;  // takes the ring's place when the keys are done
  static constexpr int AREA = RING > MERGE ? RING : MERGE;
  static constexpr int KSTEPS = D / 16;
  static constexpr int QFRAG = NT > 1 ? KSTEPS * NT * 32 * 8 : 0;  // query fragments, shared by the warps
  static constexpr int SMEM = AREA + QFRAG;
};

namespace split {

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
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

// Units of so many keys (a length may be as large as 2^31 - 16).
__device__ __forceinline__ int key_units(int keys) {
  return static_cast<int>((static_cast<unsigned>(max(keys, 0)) + kUnitKeys - 1) / kUnitKeys);
}

// A sequence's share of the work.
struct SeqWork {
  CacheSeq s;
  int kbase;      // first key any of its rows sees, rounded down to a block
  int units;      // of one segment
  int64_t total;  // of all its segments
};
template <int ROWS>
__device__ __forceinline__ SeqWork seq_work(const CacheFwdParams& p, int b) {
  SeqWork w;
  w.s = load_sequence(p.batch, p.cache.lp, b);
  w.kbase = 0;
  w.units = 1;
  w.total = 0;
  if (!w.s.ok || w.s.n == 0) return w;
  if (p.window > 0) w.kbase = max(0, w.s.len - w.s.n - p.window + 1) & ~(kCacheBlock - 1);
  if (!p.no_split) w.units = max(1, key_units(w.s.len - w.kbase));
  const int64_t tiles = (static_cast<int64_t>(w.s.n) * p.G + ROWS - 1) / ROWS;
  w.total = tiles * p.cache.H * w.units;
  return w;
}

}  // namespace split

template <int D, int NT>
__global__ void __launch_bounds__(128, (SplitCfg<D, NT>::CTAS)) gdpa_cache_split_kernel(const CacheFwdParams p) {
  using namespace split;
  using C = SplitCfg<D, NT>;
  constexpr int KS = C::KSTEPS, ND = D / 16;  // k-steps of S^T; 16-row tiles of O^T
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t s_scan[4];
  __shared__ int64_t s_start;
  __shared__ int s_seq;
  __shared__ float s_ml[C::WARPS][C::ROWS][2];
  __shared__ uint8_t s_sf[C::WARPS][C::STAGES][2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  const CacheBatch& bt = p.batch;

  // ---- this CTA's run of units, and the sequence it begins in
  int64_t mine = 0;
  const int per = (bt.B + C::THREADS - 1) / C::THREADS;
  const int b_lo = min(bt.B, tid * per), b_hi = min(bt.B, b_lo + per);
  for (int b = b_lo; b < b_hi; ++b) mine += seq_work<C::ROWS>(p, b).total;
  int64_t incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += x;
  }
  if (lane == 31) s_scan[warp] = incl;
  if (tid < 2 && !p.no_split) p.meta[(blockIdx.x * 2 + tid) * 8 + 1] = 0;  // no parts yet
  __syncthreads();
  int64_t total = 0;
#pragma unroll
  for (int w = 0; w < C::WARPS; ++w) {
    if (w < warp) incl += s_scan[w];
    total += s_scan[w];
  }
  // a run is at least four units of one segment, or one segment
  const int64_t even = (total + gridDim.x - 1) / gridDim.x;
  const int64_t chunk = p.no_split ? max(even, (int64_t)1) : max(even, (int64_t)4);
  int64_t at = chunk * blockIdx.x;
  const int64_t stop = min(total, at + chunk);
  if (at >= stop) return;
  if (at >= incl - mine && at < incl) {
    int64_t base = incl - mine;
    int b = b_lo;
    for (; b < b_hi; ++b) {
      const int64_t n = seq_work<C::ROWS>(p, b).total;
      if (at < base + n) break;
      base += n;
    }
    s_seq = b;
    s_start = base;
  }
  __syncthreads();
  int b = s_seq;
  int64_t base = s_start;

  const uint32_t ring = ptx::smem_u32(smem) + warp * C::STAGES * 2 * C::TILE;
  uint2* qfrag = reinterpret_cast<uint2*>(smem + C::AREA);
  SeqWork sw = seq_work<C::ROWS>(p, b);

  while (at < stop) {
    if (at >= base + sw.total) {
      base += sw.total;
      sw = seq_work<C::ROWS>(p, ++b);
      continue;
    }
    const CacheSeq s = sw.s;
    const int64_t seg = (at - base) / sw.units;
    const int u0 = static_cast<int>((at - base) - seg * sw.units);
    const int u1 = static_cast<int>(min(static_cast<int64_t>(sw.units), u0 + (stop - at)));
    const int h = static_cast<int>(seg % p.cache.H), tile = static_cast<int>(seg / p.cache.H);
    const int64_t row0 = static_cast<int64_t>(tile) * C::ROWS;
    const int rows = static_cast<int>(min(static_cast<int64_t>(C::ROWS), static_cast<int64_t>(s.n) * p.G - row0));

    // ---- query fragments, and what each column (query row) sees
    uint32_t qf[NT == 1 ? KS : 1][2];
    float fac[NT][2];
    int lo[NT][2], hi[NT][2];
    int lo_max = 0, hi_min = s.len, lo_min = 0x7fffffff, hi_max = 0;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = nt * 8 + g;
      float x[D / 4];
      float amax = 0.0f;
      if (r < rows) {
        const int64_t rr = row0 + r;
        const __nv_bfloat16* src =
            p.q + (s.first + rr / p.G) * p.q_stride + (h * p.G + static_cast<int>(rr % p.G)) * D + t * (D / 4);
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
        } else if (warp == nt % C::WARPS) {
          qfrag[(k * NT + nt) * 32 + lane] = make_uint2(b0, b1);
        }
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int col = nt * 8 + 2 * t + c;
        fac[nt][c] = __shfl_sync(0xffffffffu, f, 8 * t + 4 * c);
        const int pos = s.len - s.n + static_cast<int>((row0 + col) / p.G);
        lo[nt][c] = p.window > 0 ? max(0, pos - p.window + 1) : 0;
        hi[nt][c] = col < rows ? (p.causal ? min(s.len, pos + 1) : s.len) : 0;
      }
    }
    {  // over the valid rows: they are in the order of their positions
      const int pos0 = s.len - s.n + static_cast<int>(row0 / p.G);
      const int pos1 = s.len - s.n + static_cast<int>((row0 + rows - 1) / p.G);
      lo_min = p.window > 0 ? max(0, pos0 - p.window + 1) : 0;
      lo_max = p.window > 0 ? max(0, pos1 - p.window + 1) : 0;
      hi_min = p.causal ? min(s.len, pos0 + 1) : s.len;
      hi_max = p.causal ? min(s.len, pos1 + 1) : s.len;
    }
    if (NT > 1) __syncthreads();

    // ---- this warp's tiles: kb(i) = kbase + 64 (u0 + i) + 16 warp
    const int first_kb = sw.kbase + u0 * kUnitKeys + warp * kCacheBlock;
    const int n_it = p.no_split ? key_units(s.len - sw.kbase) : u1 - u0;
    const int pmask = (1 << p.cache.lp) - 1;
    const int32_t* table = bt.table + static_cast<int64_t>(b) * bt.max_pages;
    auto live = [&](int kb) { return kb < hi_max && kb + kCacheBlock > lo_min; };
    auto page_of = [&](int i) {  // -1: nothing to read
      const int kb = first_kb + i * kUnitKeys;
      if (i >= n_it || !live(kb)) return -1;
      const int page = __ldg(table + (kb >> p.cache.lp));
      if (page >= 0 && page < p.cache.num_pages) return page;
      if (lane == 0) atomicOr(bt.status, kStatusBadPlan);
      return -1;
    };
    uint32_t filled = 0;   // bit s: stage s holds a tile
    int page_next = page_of(0);
    // Starts the copies of tile i; lanes 0 and 1 load its scale codes (K's,
    // V's) into `sf`, to be put beside the stage when they have arrived.
    auto issue = [&](int i, int stage, uint32_t& sf) {
      const int kb = first_kb + i * kUnitKeys, page = page_next;
      page_next = page_of(i + 1);
      if (page >= 0) {
        filled |= 1u << stage;
        const int slot = kb & pmask, valid = s.len - kb;  // rows from `valid` on are not stored yet: zeros
        const int64_t row = cache_row(p.cache, page, h, slot);
        const uint8_t* ks = p.cache.k + row * D + lane * 16;
        const uint8_t* vs = p.cache.v + row * D + lane * 16;
        const uint32_t dst = ring + stage * 2 * C::TILE;
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
          const int idx = lane + 32 * j, r = idx / (D / 16), c = idx % (D / 16);
          const int bytes = r < valid ? 16 : 0;
          cp_async16(dst + tile_at<D>(r, c), ks + 512 * j, bytes);
          cp_async16(dst + C::TILE + tile_at<D>(r, c), vs + 512 * j, bytes);
        }
        if (lane < 2) sf = (lane ? p.cache.v_sf : p.cache.k_sf)[cache_sf(p.cache, page, h, slot)];
      } else {
        filled &= ~(1u << stage);
      }
      cp_commit();
    };
    auto keep_sf = [&](int stage, uint32_t sf) {
      if (lane < 2) s_sf[warp][stage][lane] = static_cast<uint8_t>(sf);
    };

    float acc[ND][NT][4];
    float mref[NT][2], sum[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int c = 0; c < 2; ++c) mref[nt][c] = -INFINITY, sum[nt][c] = 0.0f;
#pragma unroll
      for (int i = 0; i < ND; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[i][nt][c] = 0.0f;
    }

    uint32_t sf[C::STAGES - 1];
#pragma unroll
    for (int i = 0; i < C::STAGES - 1; ++i) sf[i] = 0, issue(i, i, sf[i]);
#pragma unroll
    for (int i = 0; i < C::STAGES - 1; ++i) keep_sf(i, sf[i]);
    int stage = 0;
    uint32_t sf_next = sf[C::STAGES - 2];
#pragma unroll 1
    for (int i = 0; i < n_it; ++i) {
      const int behind = stage == 0 ? C::STAGES - 1 : stage - 1;  // the stage this iteration refills
      keep_sf(behind == 0 ? C::STAGES - 1 : behind - 1, sf_next);  // ... and the one the last iteration did
      cp_wait<C::STAGES - 2>();
      __syncwarp();
      issue(i + C::STAGES - 1, behind, sf_next);
      const uint32_t kt = ring + stage * 2 * C::TILE, vt = kt + C::TILE;
      const int cur = stage;
      stage = stage + 1 == C::STAGES ? 0 : stage + 1;
      if (!(filled >> cur & 1)) continue;
      const int kb = first_kb + i * kUnitKeys;
      const float sk = sf_value(s_sf[warp][cur][0]), sv = sf_value(s_sf[warp][cur][1]);

      // S^T = K Q^T: rows g and g + 8 are keys, columns 2t and 2t + 1 queries
      float st[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 4; ++c) st[nt][c] = 0.0f;
#pragma unroll
      for (int j = 0; j < D / 64; ++j) {
        uint32_t ka[4], kc[4];
        const int c = D == 128 ? 2 * t + j : t;
        lds128(kt + tile_at<D>(g, c), ka);
        lds128(kt + tile_at<D>(g + 8, c), kc);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const int k = 4 * j + w;
          const uint32_t a0 = codes_lo(ka[w]), a2 = codes_hi(ka[w]), a1 = codes_lo(kc[w]), a3 = codes_hi(kc[w]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if (NT == 1) {
              mma_f16(st[nt], a0, a1, a2, a3, qf[NT == 1 ? k : 0][0], qf[NT == 1 ? k : 0][1]);
            } else {
              const uint2 qq = qfrag[(k * NT + nt) * 32 + lane];
              mma_f16(st[nt], a0, a1, a2, a3, qq.x, qq.y);
            }
          }
        }
      }

      // scores in units of log2, hidden keys -inf; does one leave the range?
      const bool edge = kb < lo_max || kb + kCacheBlock > hi_min;
      bool over = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float x = st[nt][c] * (fac[nt][c & 1] * sk);
          if (edge) {
            const int key = kb + g + (c & 2) * 4;
            if (key < lo[nt][c & 1] || key >= hi[nt][c & 1]) x = -INFINITY;
          }
          st[nt][c] = x;
          over |= x > mref[nt][c & 1] + 15.0f;
        }
      if (__any_sync(0xffffffffu, over)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float top = fmaxf(st[nt][c], st[nt][c + 2]);
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
            const float ref = fmaxf(mref[nt][c], top - 7.0f);
            const float keep = ptx::ex2_approx(mref[nt][c] - (ref == -INFINITY ? 0.0f : ref));
            mref[nt][c] = ref;
            sum[nt][c] *= keep;
#pragma unroll
            for (int i2 = 0; i2 < ND; ++i2) {
              acc[i2][nt][c] *= keep;
              acc[i2][nt][c + 2] *= keep;
            }
          }
      }
      uint32_t pb[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float r0 = mref[nt][0] == -INFINITY ? 0.0f : mref[nt][0];
        const float r1 = mref[nt][1] == -INFINITY ? 0.0f : mref[nt][1];
        const float p0 = ptx::ex2_approx(st[nt][0] - r0), p1 = ptx::ex2_approx(st[nt][1] - r1);
        const float p2 = ptx::ex2_approx(st[nt][2] - r0), p3 = ptx::ex2_approx(st[nt][3] - r1);
        sum[nt][0] += p0 + p2;
        sum[nt][1] += p1 + p3;
        pb[nt][0] = transpose8x8(pack_f16x2(p0, p1));
        pb[nt][1] = transpose8x8(pack_f16x2(p2, p3));
      }

      // O^T += V^T P^T: lane (g, t) holds D/8 coordinates of tokens 2t, 2t+1, 2t+8, 2t+9
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
      bool by_token = false;
      if (edge) {
        bool nan = false;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int key = kb + 2 * t + (j & 1) + (j & 2) * 4;
#pragma unroll
          for (int w = 0; w < D / 32; ++w) {
            if (key < lo_min || key >= hi_max) v[j][w] = 0;
            nan |= has_nan_code(v[j][w]);
          }
        }
        by_token = __any_sync(0xffffffffu, nan);
      }
      if (!by_token) {
#pragma unroll
        for (int w = 0; w < D / 32; ++w)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint32_t x01 = __byte_perm(v[0][w], v[1][w], half ? 0x7362 : 0x5140);
            const uint32_t x23 = __byte_perm(v[2][w], v[3][w], half ? 0x7362 : 0x5140);
            const uint32_t a0 = codes_lo(x01), a1 = codes_hi(x01), a2 = codes_lo(x23), a3 = codes_hi(x23);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
              mma_f16(o, a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
#pragma unroll
              for (int c = 0; c < 4; ++c) acc[2 * w + half][nt][c] = fmaf(o[c], sv, acc[2 * w + half][nt][c]);
            }
          }
      } else {
#pragma unroll 1
        for (int k = 0; k < kCacheBlock; ++k) {
          const int key = kb + k;
#pragma unroll
          for (int w = 0; w < D / 32; ++w)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              uint32_t y[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) y[j] = 2 * t + (j & 1) + (j & 2) * 4 == k ? v[j][w] : 0;
              const uint32_t x01 = __byte_perm(y[0], y[1], half ? 0x7362 : 0x5140);
              const uint32_t x23 = __byte_perm(y[2], y[3], half ? 0x7362 : 0x5140);
              const uint32_t a0 = codes_lo(x01), a1 = codes_hi(x01), a2 = codes_lo(x23), a3 = codes_hi(x23);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                float o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                mma_f16(o, a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
#pragma unroll
                for (int c = 0; c < 4; ++c)
                  if (key >= lo[nt][c & 1] && key < hi[nt][c & 1])
                    acc[2 * w + half][nt][c] = fmaf(o[c], sv, acc[2 * w + half][nt][c]);
              }
            }
        }
      }
    }
    cp_wait<0>();

    // ---- the four warps' results, joined in shared memory
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float x = sum[nt][c];
        x += __shfl_xor_sync(0xffffffffu, x, 4);
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        x += __shfl_xor_sync(0xffffffffu, x, 16);
        if (g == 0) {
          s_ml[warp][nt * 8 + 2 * t + c][0] = mref[nt][c];
          s_ml[warp][nt * 8 + 2 * t + c][1] = x;
        }
      }
    __syncthreads();  // every warp is done with its ring
    float* merge = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float* dst = merge + (static_cast<int64_t>(warp) * C::ROWS + nt * 8 + 2 * t + c) * D + g * (D / 8);
#pragma unroll
        for (int i = 0; i < ND; i += 2)
          *reinterpret_cast<float4*>(dst + 2 * i) =
              make_float4(acc[i][nt][c], acc[i][nt][c + 2], acc[i + 1][nt][c], acc[i + 1][nt][c + 2]);
      }
    __syncthreads();
    const int64_t seg_start = base + seg * sw.units;
    const int first = static_cast<int>(seg_start / chunk);
    const int pieces = p.no_split ? 1 : static_cast<int>((seg_start + sw.units - 1) / chunk) - first + 1;
    const int slot = first == static_cast<int>(blockIdx.x) ? 1 : 0;
    float* part = p.part + (static_cast<int64_t>(blockIdx.x) * 2 + slot) * C::ROWS * (D + 2);
    for (int i = tid; i < rows * (D / 8); i += C::THREADS) {
      const int r = i / (D / 8), d = (i % (D / 8)) * 8;
      float ref = -INFINITY;
#pragma unroll
      for (int w = 0; w < C::WARPS; ++w) ref = fmaxf(ref, s_ml[w][r][0]);
      float l = 0.0f, o[8] = {};
#pragma unroll
      for (int w = 0; w < C::WARPS; ++w) {
        const float f = ptx::ex2_approx(s_ml[w][r][0] - (ref == -INFINITY ? 0.0f : ref));
        l += s_ml[w][r][1] * f;
        const float* src = merge + (static_cast<int64_t>(w) * C::ROWS + r) * D + d;
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] += src[e] * f;
      }
      if (pieces == 1) {
        const int64_t rr = row0 + r;
        const int64_t at_row = (s.first + rr / p.G) * p.Hq + h * p.G + rr % p.G;
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        uint4 u;
        u.x = ptx::pack_bf16x2(o[0] * inv, o[1] * inv);
        u.y = ptx::pack_bf16x2(o[2] * inv, o[3] * inv);
        u.z = ptx::pack_bf16x2(o[4] * inv, o[5] * inv);
        u.w = ptx::pack_bf16x2(o[6] * inv, o[7] * inv);
        *reinterpret_cast<uint4*>(p.out + at_row * D + d) = u;
        if (p.lse && d == 0) p.lse[at_row] = l == 0.0f ? -INFINITY : (ref + log2f(l)) * 0.6931471805599453f;
      } else {
        if (d == 0) part[2 * r] = ref, part[2 * r + 1] = l;
        float4* dst = reinterpret_cast<float4*>(part + 2 * C::ROWS + r * D + d);
        dst[0] = make_float4(o[0], o[1], o[2], o[3]);
        dst[1] = make_float4(o[4], o[5], o[6], o[7]);
      }
    }
    if (pieces > 1 && tid == 0) {
      int* m = p.meta + (blockIdx.x * 2 + slot) * 8;
      m[0] = first, m[1] = pieces, m[2] = s.first, m[3] = s.n, m[4] = tile, m[5] = h;
    }
    __syncthreads();  // the merge area is a ring again
    at += u1 - u0;
  }
}

// Joins the parts of cut segments.  Block c is a member of up to two of them
// (the segment that its CTA's run begins inside, slot 0, and the one it ends
// inside, slot 1); the members of a segment share its rows.  Up to 16 parts: a
// warp takes a row.  More: the 16 warps take a row together, each a run of the
// parts.
template <int D, int ROWS>
__global__ void __launch_bounds__(512) gdpa_cache_join_kernel(const CacheFwdParams p) {
  constexpr int E = D / 32;
  __shared__ float s_part[16][D + 2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int slot = 0; slot < 2; ++slot) {
    const int* m = p.meta + (blockIdx.x * 2 + slot) * 8;
    const int pieces = m[1];
    if (pieces == 0) continue;
    const int first = m[0], row_first = m[2], n = m[3], tile = m[4], h = m[5];
    const int member = blockIdx.x - first;
    const int64_t row0 = static_cast<int64_t>(tile) * ROWS;
    const int rows = static_cast<int>(min(static_cast<int64_t>(ROWS), static_cast<int64_t>(n) * p.G - row0));
    const bool together = pieces > 16;
    const int j0 = together ? pieces * warp / 16 : 0, j1 = together ? pieces * (warp + 1) / 16 : pieces;
    for (int r = member + (together ? 0 : warp * pieces); r < rows; r += together ? pieces : 16 * pieces) {
      float ref = -INFINITY, l = 0.0f, o[E] = {};
#pragma unroll 4
      for (int j = j0; j < j1; ++j) {
        const float* part = p.part + (static_cast<int64_t>(first + j) * 2 + (j == 0)) * ROWS * (D + 2);
        const float r2 = part[2 * r], l2 = part[2 * r + 1];
        float x[E];
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = part[2 * ROWS + r * D + lane * E + e];
        const float top = fmaxf(ref, r2), zero = top == -INFINITY ? 0.0f : top;
        const float f1 = ptx::ex2_approx(ref - zero), f2 = ptx::ex2_approx(r2 - zero);
        ref = top;
        l = l * f1 + l2 * f2;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = o[e] * f1 + x[e] * f2;
      }
      if (together) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < E; ++e) s_part[warp][lane * E + e] = o[e];
        if (lane == 0) s_part[warp][D] = ref, s_part[warp][D + 1] = l;
        __syncthreads();
        if (warp != 0) continue;
        ref = -INFINITY;
        for (int w = 0; w < 16; ++w) ref = fmaxf(ref, s_part[w][D]);
        l = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = 0.0f;
        for (int w = 0; w < 16; ++w) {
          const float f = ptx::ex2_approx(s_part[w][D] - (ref == -INFINITY ? 0.0f : ref));
          l += s_part[w][D + 1] * f;
#pragma unroll
          for (int e = 0; e < E; ++e) o[e] += s_part[w][lane * E + e] * f;
        }
      }
      const int64_t rr = row0 + r;
      const int64_t at_row = (row_first + rr / p.G) * p.Hq + h * p.G + rr % p.G;
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
      for (int e = 0; e < E; e += 2)
        *reinterpret_cast<uint32_t*>(p.out + at_row * D + lane * E + e) = ptx::pack_bf16x2(o[e] * inv, o[e + 1] * inv);
      if (p.lse && lane == 0) p.lse[at_row] = l == 0.0f ? -INFINITY : (ref + log2f(l)) * 0.6931471805599453f;
    }
  }
}

}  // namespace gdpa
