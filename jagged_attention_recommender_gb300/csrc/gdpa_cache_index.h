// gdpa_cache_index.h -- the paged cache's index arithmetic, free of CUDA: the
// kernels compile it for the device, the tests as plain C++ for the host.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define GDPA_HD __host__ __device__ __forceinline__
#else
#define GDPA_HD inline
#endif

namespace gdpa {

constexpr int kCacheBlock = 16;  // tokens that share a scale, per head

// A sequence of a batch: its rows of the new tokens and its length.  ok = 0
// where its offsets do not describe rows of the tensors, or its length does
// not fit the page table.
struct CacheSeq {
  int first, n, len, ok;
};
GDPA_HD CacheSeq cache_sequence(int first, int end, int len, int T, int64_t most_tokens) {
  CacheSeq s;
  s.first = first;
  s.len = len;
  s.ok = first >= 0 && end >= first && end <= T && len >= 0 && len <= most_tokens;
  s.n = s.ok ? end - first : 0;
  return s;
}

// The part of a scale block that row r of the new tokens begins, if it begins
// one: `cnt` rows from r on, the first at position `pos` of sequence s.  bad:
// the sequence is no valid one or does not hold the row, which happens where
// offsets decrease (the lookup counts the ends in front of a row).
struct OwnedRows {
  int pos, cnt, bad;
};
GDPA_HD OwnedRows owned_rows(const CacheSeq& s, int r) {
  OwnedRows o = {0, 0, 0};
  o.bad = !s.ok || s.len < s.n || r < s.first || r - s.first >= s.n;
  if (o.bad) return o;
  const int at = r - s.first, pos = s.len - s.n + at;
  if (at > 0 && (pos & (kCacheBlock - 1)) != 0) return o;
  const int room = kCacheBlock - (pos & (kCacheBlock - 1)), left = s.n - at;
  o.pos = pos;
  o.cnt = room < left ? room : left;
  return o;
}

// The first key that the row at position `pos` (negative in front of the first
// token) sees through a window of `window` tokens, 0 for none.  (pos - window
// alone can lie below -2^31.)
GDPA_HD int first_key(int pos, int window) { return window > 0 && pos >= window ? pos - window + 1 : 0; }

}  // namespace gdpa
