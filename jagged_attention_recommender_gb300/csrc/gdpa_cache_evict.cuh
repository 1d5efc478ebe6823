// gdpa_cache_evict.cuh -- cuts sequences of the cache to their most attended
// tokens: a kernel that chooses them, head by head, and one that moves them.
//
// Choosing.  One cluster of CTAs a sequence and head (one CTA where there are enough of
// those), its keys in shared memory.  A weight's bits, turned so that larger numbers have larger unsigned
// keys, are searched for the smallest key that is kept, eight bits a pass: a
// histogram of the keys that agree so far says which digit the k-th largest
// has.  A last pass over the tokens, in order, keeps what is above that key and
// the first of what equals it.
//
// Moving.  A warp makes one block of 16 new tokens of one head, for K and for V:
// their scales, the largest of them, and the codes, which are copied as they
// are where the scale is the same.
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

constexpr int kChooseThreads = 512, kChooseWarps = kChooseThreads / 32;
constexpr int kMostKeys = 40960;  // keys that a CTA keeps in shared memory

struct ChooseShared {
  int hist[4][256];  // of each digit, this CTA's
  int total[256];    // the cluster's
  int above[kChooseWarps], same[kChooseWarps];  // each warp's tokens that stay, and those that equal the least key that does
  int cta_above, cta_same;
  uint32_t digit;
  int need;
};

// One sequence and head by a cluster of CTAs, each with an equal part of its
// tokens (a warp with an equal part of those).  `slots`: keys that `keys` holds.
__global__ void __launch_bounds__(kChooseThreads) gdpa_cache_choose_kernel(const __grid_constant__ EvictParams p, int slots) {
  namespace cg = cooperative_groups;
  extern __shared__ uint32_t keys[];
  __shared__ ChooseShared sh;
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
      for (int64_t j = rank * kChooseThreads + tid; j < keep; j += ctas * kChooseThreads) kept[j] = static_cast<int>(j);
      continue;
    }
    // this CTA's tokens [j0, j1), a multiple of 4 but for the last one, and this warp's [w0, w1)
    const int per = static_cast<int>((static_cast<int64_t>(len) + ctas - 1) / ctas + 3) & ~3;
    const int j0 = static_cast<int>(min(static_cast<int64_t>(len), static_cast<int64_t>(per) * rank));
    const int j1 = static_cast<int>(min(static_cast<int64_t>(len), static_cast<int64_t>(j0) + per));
    const int part = ((j1 - j0 + kChooseWarps - 1) / kChooseWarps + 31) & ~31;
    const int w0 = min(j1 - j0, part * warp) + j0, w1 = min(j1 - w0, part) + w0;
    const bool held = per <= slots;
    const int32_t* const table = p.table + static_cast<int64_t>(b) * p.max_pages;
    auto load4 = [&](int j, uint32_t (&k)[4]) {  // j a multiple of 4: one page
      const int page = __ldg(table + (j >> p.cache.lp));
      k[0] = k[1] = k[2] = k[3] = 0;
      if (page >= 0 && page < p.cache.num_pages) {
        const float4 w = *reinterpret_cast<const float4*>(
            p.weights + cache_row(p.cache, page, h, j & ((1 << p.cache.lp) - 1)));
        k[0] = weight_key(w.x), k[1] = weight_key(w.y), k[2] = weight_key(w.z), k[3] = weight_key(w.w);
      } else {
        atomicOr(p.status, kStatusBadPlan);
      }
    };
    for (int i = tid; i < 1024; i += kChooseThreads) (&sh.hist[0][0])[i] = 0;
    __syncthreads();
    // sink + recent <= budget < len: the tokens between them compete for `need` places
    const int lo = p.sink, hi = len - p.recent;
    int need = keep - p.sink - p.recent;
    const bool any = need > 0;  // (none of them stays otherwise)
    uint32_t prefix = 0;
    if (any) {
      // the first digit's histogram while the keys come
#pragma unroll 4
      for (int64_t j = j0 + 4 * tid; j < j1; j += 4 * kChooseThreads) {
        uint32_t k[4];
        load4(static_cast<int>(j), k);
        if (held) *reinterpret_cast<uint4*>(keys + (j - j0)) = make_uint4(k[0], k[1], k[2], k[3]);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (j + i >= lo && j + i < hi && j + i < j1) atomicAdd(&sh.hist[0][k[i] >> 24], 1);
      }
#pragma unroll 1
      for (int d = 0; d < 4; ++d) {
        const int shift = 24 - 8 * d;
        if (d > 0) {
          const uint32_t mask = 0xffffffffu << (shift + 8);
          for (int64_t j = j0 + 4 * tid; j < j1; j += 4 * kChooseThreads) {
            uint32_t k[4];
            if (held) {
              const uint4 u = *reinterpret_cast<const uint4*>(keys + (j - j0));
              k[0] = u.x, k[1] = u.y, k[2] = u.z, k[3] = u.w;
            } else {
              load4(static_cast<int>(j), k);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if ((k[i] & mask) == prefix && j + i >= lo && j + i < hi && j + i < j1)
                atomicAdd(&sh.hist[d][k[i] >> shift & 255], 1);
          }
        }
        meet();
        if (tid < 256) {
          int n = 0;
          for (int r = 0; r < ctas; ++r) n += ctas > 1 ? *cluster.map_shared_rank(&sh.hist[d][tid], r) : sh.hist[d][tid];
          sh.total[tid] = n;
        }
        __syncthreads();
        if (warp == 0) {  // lane i: digits 255 - 8 i down to 248 - 8 i
          int n[8], mine = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) mine += n[i] = sh.total[255 - 8 * lane - i];
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
            while (i < 7 && before + n[i] < need) before += n[i++];
            sh.digit = 255 - 8 * lane - i;
            sh.need = need - before;
          }
        }
        __syncthreads();
        prefix |= sh.digit << shift;
        need = sh.need;  // how many of those that equal the key so far stay
      }
    }
    // what stays whatever its place, and what equals the least key
    auto stays = [&](int j, bool& above, bool& same) {
      above = j < w1 && (j < lo || j >= hi);
      same = false;
      if (any && j < w1 && !above) {
        uint32_t k[4];
        uint32_t key;
        if (held) {
          key = keys[j - j0];
        } else {
          load4(j & ~3, k);
          key = (j & 2) ? ((j & 1) ? k[3] : k[2]) : ((j & 1) ? k[1] : k[0]);
        }
        above = key > prefix;
        same = key == prefix;
      }
    };
    int n_above = 0, n_same = 0;
    for (int64_t j = w0; j < w1; j += 32) {
      bool above, same;
      stays(static_cast<int>(j) + lane, above, same);
      n_above += __popc(__ballot_sync(0xffffffffu, above));
      n_same += __popc(__ballot_sync(0xffffffffu, same));
    }
    if (lane == 0) sh.above[warp] = n_above, sh.same[warp] = n_same;
    __syncthreads();
    int out = 0, equal = 0, all_above = 0, all_same = 0;
    for (int w = 0; w < kChooseWarps; ++w) {
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
    out += min(equal, need);  // (need counts places among equals by now; 0 if nothing competes)
    for (int64_t j = w0; j < w1; j += 32) {
      bool above, same;
      stays(static_cast<int>(j) + lane, above, same);
      const unsigned eq = __ballot_sync(0xffffffffu, same), before = (1u << lane) - 1;
      const bool take = above || (same && equal + __popc(eq & before) < need);
      const unsigned taken = __ballot_sync(0xffffffffu, take);
      const int at = out + __popc(taken & before);
      if (take && at < keep) kept[at] = static_cast<int>(j) + lane;
      out += __popc(taken);
      equal += __popc(eq);
    }
    meet();  // others may still read this CTA's counts
  }
}

// 16 codes from scale `from` to the larger scale `to`.
__device__ __forceinline__ uint4 rescale16(uint4 x, int from, int to) {
  if (from == to) return x;
  const float f = sf_value(127 - min(to - from, 126));
  return make_uint4(rescale4(x.x, f), rescale4(x.y, f), rescale4(x.z, f), rescale4(x.w, f));
}

template <int D>
__global__ void __launch_bounds__(256) gdpa_cache_move_kernel(const __grid_constant__ EvictParams p) {
  constexpr int LPT = D / 16, TPS = 32 / LPT;  // lanes of a token, tokens of a step
  asm volatile("griddepcontrol.wait;" ::: "memory");  // what is kept has been chosen
  const int lane = threadIdx.x & 31, H = p.cache.H;
  const int64_t blocks = (static_cast<int64_t>(p.most) + kCacheBlock - 1) / kCacheBlock;
  const int64_t tasks = blocks * p.B * H, step = gridDim.x * 8ll;
  for (int64_t task = blockIdx.x * 8ll + (threadIdx.x >> 5); task < tasks; task += step) {
    const int64_t bh = task / blocks;
    const int i0 = static_cast<int>(task - bh * blocks) * kCacheBlock;
    const int b = static_cast<int>(bh / H), h = static_cast<int>(bh - static_cast<int64_t>(b) * H);
    const int keep = min(evict_len(p, b), p.budget), cnt = min(keep - i0, kCacheBlock);
    if (cnt <= 0) continue;
    const int64_t to = token_row(p, p.new_table, p.new_max_pages, b, h, i0);
    if (to < 0) continue;
    // lanes 0..15 and 16..31 hold the tokens' old rows
    const int t = lane & 15;
    int64_t from = -1;
    if (t < cnt) from = token_row(p, p.table, p.max_pages, b, h, p.kept[bh * p.budget + i0 + t]);
    int sf = -1;  // of K in the lower lanes, of V in the upper ones
    if (from >= 0) sf = __ldg((lane < 16 ? p.cache.k_sf : p.cache.v_sf) + (from >> 4));
    if (lane < 16 && from >= 0) p.weights[to + t] = p.weights[from];
    int top = sf;
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
    if (t == 0 && top >= 0) (lane < 16 ? p.cache.k_sf : p.cache.v_sf)[to >> 4] = static_cast<uint8_t>(top);
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const uint8_t* const codes = which ? p.cache.v : p.cache.k;
      uint8_t* const dst = which ? p.cache.v : p.cache.k;
      const int most = __shfl_sync(0xffffffffu, top, 16 * which);
#pragma unroll
      for (int u = 0; u < kCacheBlock; u += TPS) {
        const int tok = u + lane / LPT;
        const int64_t src = __shfl_sync(0xffffffffu, from, tok);
        const int old = __shfl_sync(0xffffffffu, sf, 16 * which + tok);
        if (tok < cnt && src >= 0) {
          const uint4 x = *reinterpret_cast<const uint4*>(codes + src * D + lane % LPT * 16);
          *reinterpret_cast<uint4*>(dst + (to + tok) * D + lane % LPT * 16) = rescale16(x, old, most);
        }
      }
    }
  }
}

}  // namespace gdpa
