// gdpa_cache_evict.cuh -- cuts sequences of the cache to their most attended
// tokens: a kernel that chooses them, head by head, and one that moves them.
//
// Choosing.  A weight's bits, turned so that larger numbers have larger unsigned
// keys, are searched for the least key that stays, eight bits a pass: a histogram
// of the keys that agree so far says which digit the k-th largest has.  Tokens that
// stay in any case count as the largest keys.  A last pass over the tokens, in
// order, keeps what is above that key and the first of what equals it.  One CTA a
// sequence and head, or a cluster of up to 16 where those are few (each with a
// part of the tokens; histograms are added through distributed shared memory);
// keys stay in shared memory.  Bound: latency, about 25 barriers and four rounds
// of dependent loads a head: 24 us for 512 heads of 4846 tokens, 19 for 4 heads of
// 130k (under a profiler).  What a CTA keeps in shared memory goes by the table's width:
// a wide one leaves an SM fewer CTAs, and one of more than 40 960 tokens a CTA has every
// digit read the weights anew (those 512 heads with their move 112 us; tables of twice, 4 and
// 16 times the longest sequence 138, 135 and 117).
//
// Moving.  A warp moves 32 tokens of one head, two new blocks, K and then V: their scales,
// the largest of each block, and the codes, which are copied as they are where
// the scale is the same.  Every token is 128 (64) consecutive bytes.  Bound:
// memory: 64 histories cut to 2048 tokens, 8 heads of 128, 87 us (6.2 TB/s).
// Both together take 112 us there and 24 for two histories of 130k tokens cut to
// 16384 (2 heads).
//
// (One kernel that moved each head once it was chosen took 145 us for the 64
// histories: with the registers of both, two CTAs an SM; a warp that looked up the next
// tokens while it moved these 151; a warp a block of 16 tokens 132.)
#pragma once

#include <cooperative_groups.h>

#include "gdpa_cache_append.cuh"

namespace gdpa {

struct EvictParams {
  CacheView cache;
  float* weights;
  const int32_t* kv_lens;
  const int32_t* table;      // [B, max_pages]
  const int32_t* new_table;  // [B, new_max_pages]
  int32_t* kept;             // [B, H, budget]
  int32_t* new_lens;
  int B, max_pages, new_max_pages;
  int budget, sink, recent;
  int most;  // tokens that any sequence keeps, as far as the host knows
  int* status;
};

// Larger weights have larger keys; NaN has the least; both zeros are the same.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (!(w == w)) return 0;
  const uint32_t u = __float_as_uint(w + 0.0f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// A sequence's length, -1 (flagged) where it does not fit the table.
__device__ __forceinline__ int evict_len(const EvictParams& p, int b) {
  const int len = __ldg(p.kv_lens + b);
  if (len >= 0 && len <= static_cast<int64_t>(p.max_pages) << p.cache.lp) return len;
  atomicOr(p.status, kStatusBadPlan);
  return -1;
}

// Token j's row of the cache, -1 on a page out of range (flagged).
__device__ __forceinline__ int64_t token_row(const EvictParams& p, const int32_t* table, int max_pages, int b, int h, int j) {
  const int page = __ldg(table + static_cast<int64_t>(b) * max_pages + (j >> p.cache.lp));
  if (page >= 0 && page < p.cache.num_pages) return cache_row(p.cache, page, h, j & ((1 << p.cache.lp) - 1));
  atomicOr(p.status, kStatusBadPlan);
  return -1;
}

constexpr int kMostKeys = 40960;  // keys that a CTA keeps in shared memory

template <int WARPS>
struct ChooseShared {
  int hist[4][256];  // of each digit, this CTA's
  int total[256];    // the cluster's
  int above[WARPS], same[WARPS];  // each warp's tokens that stay, and those that equal the least key that does
  int cta_above, cta_same;
  uint32_t digit;
  int need, of;  // of the `of` tokens with these digits `need` stay
};

// One sequence and head by a cluster of CTAs, each with an equal part of its
// tokens (a warp with an equal part of those).  `slots`: keys that `keys` holds.
template <int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS == 256 ? 6 : 1)
    gdpa_cache_choose_kernel(const __grid_constant__ EvictParams p, int slots) {
  namespace cg = cooperative_groups;
  extern __shared__ __align__(16) uint32_t keys[];  // (read four at a time)
  constexpr int WARPS = THREADS / 32;
  __shared__ ChooseShared<WARPS> sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t heads = static_cast<int64_t>(p.B) * p.cache.H;
  auto meet = [&]() {
    if (ctas > 1)
      cluster.sync();
    else
      __syncthreads();
  };
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the move may be set up beside this
  for (int64_t bh = blockIdx.x / ctas; bh < heads; bh += gridDim.x / ctas) {
    const int b = static_cast<int>(bh / p.cache.H), h = static_cast<int>(bh - static_cast<int64_t>(b) * p.cache.H);
    const int len = evict_len(p, b), keep = min(len, p.budget);
    if (h == 0 && rank == 0 && tid == 0) p.new_lens[b] = max(keep, 0);
    if (keep <= 0) continue;
    int32_t* const kept = p.kept + bh * p.budget;
    if (keep == len) {
      for (int64_t j = rank * THREADS + tid; j < keep; j += ctas * THREADS) kept[j] = static_cast<int>(j);
      continue;
    }
    // this CTA's tokens: n from j0 on (a multiple of 4 each, but for the last one's)
    const int per = static_cast<int>((static_cast<int64_t>(len) + ctas - 1) / ctas + 3) & ~3;
    const int j0 = static_cast<int>(min(static_cast<int64_t>(len), static_cast<int64_t>(per) * rank)), n = min(len - j0, per);
    const bool held = per <= slots;
    // The first and last ones stay in any case: they count as larger than any
    // number, so that the `keep` largest of all are what stays (sink + recent <=
    // budget).  The others are [free0, free1) of this CTA's.
    const int free0 = max(min(p.sink - j0, n), 0), free1 = max(min(len - p.recent - j0, n), 0);
    const int32_t* const table = p.table + static_cast<int64_t>(b) * p.max_pages;
    const float* const weights = p.weights + (static_cast<int64_t>(h) << p.cache.lp);
    const int64_t page_weights = static_cast<int64_t>(p.cache.H) << p.cache.lp;
    auto load4 = [&](int i) {  // i a multiple of 4: one page
      const int j = j0 + i, page = __ldg(table + (j >> p.cache.lp));
      uint4 k = make_uint4(0, 0, 0, 0);
      if (page >= 0 && page < p.cache.num_pages) {
        const float4 w = *reinterpret_cast<const float4*>(weights + page * page_weights + (j & ((1 << p.cache.lp) - 1)));
        k = make_uint4(weight_key(w.x), weight_key(w.y), weight_key(w.z), weight_key(w.w));
      } else {
        atomicOr(p.status, kStatusBadPlan);
      }
      if (i < free0 || i + 3 >= free1) {
        if (i < free0 || i >= free1) k.x = 0xffffffffu;
        if (i + 1 < free0 || i + 1 >= free1) k.y = 0xffffffffu;
        if (i + 2 < free0 || i + 2 >= free1) k.z = 0xffffffffu;
        if (i + 3 < free0 || i + 3 >= free1) k.w = 0xffffffffu;
      }
      return k;
    };
    auto keys4 = [&](int i) { return held ? *reinterpret_cast<const uint4*>(keys + i) : load4(i); };
    for (int i = tid; i < 1024; i += THREADS) (&sh.hist[0][0])[i] = 0;
    __syncthreads();
    // the first digit's histogram while the keys come
#pragma unroll 4
    for (unsigned i = 4 * tid; i < static_cast<unsigned>(n); i += 4 * THREADS) {
      const uint4 k = load4(i);
      if (held) *reinterpret_cast<uint4*>(keys + i) = k;
      atomicAdd(&sh.hist[0][k.x >> 24], 1);
      if (i + 1 < static_cast<unsigned>(n)) atomicAdd(&sh.hist[0][k.y >> 24], 1);
      if (i + 2 < static_cast<unsigned>(n)) atomicAdd(&sh.hist[0][k.z >> 24], 1);
      if (i + 3 < static_cast<unsigned>(n)) atomicAdd(&sh.hist[0][k.w >> 24], 1);
    }
    uint32_t prefix = 0;  // the digits so far of the least key that stays
    int need = keep;      // how many of those that equal them do
#pragma unroll 1
    for (int d = 0; d < 4; ++d) {
      const int shift = 24 - 8 * d;
      if (d > 0) {
        const uint32_t mask = 0xffffffffu << (shift + 8);
        auto count = [&](uint32_t k) {
          if (((k ^ prefix) & mask) == 0) atomicAdd(&sh.hist[d][k >> shift & 255], 1);
        };
#pragma unroll 2
        for (unsigned i = 4 * tid; i < static_cast<unsigned>(n); i += 4 * THREADS) {
          const uint4 k = keys4(i);
          count(k.x);
          if (i + 1 < static_cast<unsigned>(n)) count(k.y);
          if (i + 2 < static_cast<unsigned>(n)) count(k.z);
          if (i + 3 < static_cast<unsigned>(n)) count(k.w);
        }
      }
      meet();
      if (tid < 256) {
        int c = sh.hist[d][tid];
        if (ctas > 1) {
          c = 0;
          for (int r = 0; r < ctas; ++r) c += *cluster.map_shared_rank(&sh.hist[d][tid], r);
        }
        sh.total[tid] = c;
      }
      __syncthreads();
      if (warp == 0) {  // lane i: digits 255 - 8 i down to 248 - 8 i
        int c[8], mine = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) mine += c[i] = sh.total[255 - 8 * lane - i];
        int before = mine;
#pragma unroll
        for (int s = 1; s < 32; s <<= 1) {
          const int x = __shfl_up_sync(0xffffffffu, before, s);
          if (lane >= s) before += x;
        }
        const int at = __ffs(__ballot_sync(0xffffffffu, before >= need)) - 1;
        if (lane == at) {
          before -= mine;
          int i = 0;
#pragma unroll
          for (int u = 0; u < 7; ++u)
            if (i == u && before + c[u] < need) before += c[u], ++i;
          sh.digit = 255 - 8 * lane - i;
          sh.need = need - before;
          sh.of = sh.total[255 - 8 * lane - i];
        }
      }
      __syncthreads();
      prefix |= sh.digit << shift;
      need = sh.need;
      if (need == sh.of && prefix > 0) {  // all of them stay: the lower digits do not matter
        prefix -= 1;
        need = 0;
        break;
      }
    }
    // Each warp counts what is above the key and what equals it in its part of
    // the tokens, 4 a lane at a time; then it knows its places.
    const int part = ((n - 1) / WARPS + 128) & ~127, w0 = min(n, part * warp), w1 = w0 + min(n - w0, part);
    auto flags = [&](unsigned i) {  // of 4 tokens: bits 0-3 above, 16-19 equal
      if (i >= static_cast<unsigned>(w1)) return 0;
      const uint4 k = keys4(i);
      int f = (k.x > prefix) | (k.y > prefix) << 1 | (k.z > prefix) << 2 | (k.w > prefix) << 3 | (k.x == prefix) << 16 |
              (k.y == prefix) << 17 | (k.z == prefix) << 18 | (k.w == prefix) << 19;
      if (i + 4 > static_cast<unsigned>(w1)) f &= ((1 << (w1 - i)) - 1) * 0x10001;
      return f;
    };
    auto counts = [](int f) { return __popc(f & 0xffff) | __popc(f >> 16) << 16; };
    int mine_above = 0, mine_same = 0;
    for (unsigned i = w0 + 4 * lane; i < static_cast<unsigned>(w1); i += 128) {
      const int c = counts(flags(i));
      mine_above += c & 0xffff;
      mine_same += c >> 16;
    }
    mine_above = __reduce_add_sync(0xffffffffu, mine_above);
    mine_same = __reduce_add_sync(0xffffffffu, mine_same);
    if (lane == 0) sh.above[warp] = mine_above, sh.same[warp] = mine_same;
    __syncthreads();
    int out = 0, equal = 0, all_above = 0, all_same = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      if (w < warp) out += sh.above[w], equal += sh.same[w];
      all_above += sh.above[w], all_same += sh.same[w];
    }
    if (ctas > 1) {
      if (tid == 0) sh.cta_above = all_above, sh.cta_same = all_same;
      cluster.sync();
      for (int r = 0; r < rank; ++r) {
        out += *cluster.map_shared_rank(&sh.cta_above, r);
        equal += *cluster.map_shared_rank(&sh.cta_same, r);
      }
    }
    // `out` counts what is above; of the equal ones the first `need` stay
    for (unsigned i0 = w0; i0 < static_cast<unsigned>(w1); i0 += 128) {  // (a length may be as large as 2^31 - 16)
      const int i = static_cast<int>(i0) + 4 * lane, f = flags(i0 + 4 * lane), mine = counts(f);
      int incl = mine;
#pragma unroll
      for (int s = 1; s < 32; s <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, incl, s);
        if (lane >= s) incl += x;
      }
      const int all = __shfl_sync(0xffffffffu, incl, 31);
      int above = out + ((incl - mine) & 0xffff), same = equal + ((incl - mine) >> 16);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool is_above = f >> e & 1, is_same = f >> (16 + e) & 1;
        const int at = above + min(same, need);
        if ((is_above || (is_same && same < need)) && at < keep) kept[at] = j0 + i + e;
        above += is_above;
        same += is_same;
      }
      out += all & 0xffff;
      equal += all >> 16;
    }
    meet();  // others may still read this CTA's counts
  }
}

// 16 codes to a scale 2^down as large.
__device__ __forceinline__ uint4 rescale16(uint4 x, int down) {
  if (down == 0) return x;
  const float f = sf_value(127 - min(down, 126));
  return make_uint4(rescale4(x.x, f), rescale4(x.y, f), rescale4(x.z, f), rescale4(x.w, f));
}

constexpr int kMoveWarps = 8, kMoveTokens = 32;  // of a CTA; of a warp

template <int D>
__global__ void __launch_bounds__(32 * kMoveWarps) gdpa_cache_move_kernel(const __grid_constant__ EvictParams p) {
  constexpr int LPT = D / 16, TPS = 32 / LPT, STEPS = kMoveTokens / TPS;  // lanes of a token, tokens of a step
  asm volatile("griddepcontrol.wait;" ::: "memory");  // what is kept has been chosen
  const int lane = threadIdx.x & 31, H = p.cache.H;
  const int i0 = (blockIdx.x * kMoveWarps + (threadIdx.x >> 5)) * kMoveTokens;
  const int64_t heads = static_cast<int64_t>(p.B) * H;
  for (int64_t bh = blockIdx.y; bh < heads; bh += gridDim.y) {
    const int b = static_cast<int>(bh / H), h = static_cast<int>(bh - static_cast<int64_t>(b) * H);
    const int keep = min(evict_len(p, b), p.budget);
    if (i0 >= keep) continue;
    // each lane's token: its old row and its new one, -1 where there is none
    int64_t from = -1, to = -1;
    if (i0 + lane < keep) {
      from = token_row(p, p.table, p.max_pages, b, h, p.kept[bh * p.budget + i0 + lane]);
      to = token_row(p, p.new_table, p.new_max_pages, b, h, i0 + lane);
      if (to < 0) from = -1;
    }
    __syncwarp();
    int sf[2] = {-1, -1};
    float w = 0.0f;
    if (from >= 0) {
      sf[0] = __ldg(p.cache.k_sf + (from >> 4));
      sf[1] = __ldg(p.cache.v_sf + (from >> 4));
      w = p.weights[from];
    }
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      uint8_t* const codes = (which ? p.cache.v : p.cache.k) + lane % LPT * 16;
      uint4 x[STEPS];
#pragma unroll
      for (int u = 0; u < STEPS; ++u) {
        const int64_t src = __shfl_sync(0xffffffffu, from, u * TPS + lane / LPT);
        if (src >= 0) x[u] = *reinterpret_cast<const uint4*>(codes + src * D);
      }
      // the largest scale of a new block: of 16 lanes
      int top = sf[which];
#pragma unroll
      for (int d = 8; d > 0; d >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
      if (which == 0 && from >= 0) p.weights[to] = w;
      if ((lane & 15) == 0 && to >= 0 && top >= 0)
        (which ? p.cache.v_sf : p.cache.k_sf)[to >> 4] = static_cast<uint8_t>(top);
      const int below = top - sf[which];  // by how much a token's codes shrink
      const bool any = __any_sync(0xffffffffu, from >= 0 && below != 0);
#pragma unroll
      for (int u = 0; u < STEPS; ++u) {
        const int tok = u * TPS + lane / LPT;
        const int64_t src = __shfl_sync(0xffffffffu, from, tok), dst = __shfl_sync(0xffffffffu, to, tok);
        const int down = any ? __shfl_sync(0xffffffffu, below, tok) : 0;
        if (src >= 0) *reinterpret_cast<uint4*>(codes + dst * D) = rescale16(x[u], down);
      }
    }
  }
}

}  // namespace gdpa
