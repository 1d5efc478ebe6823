// gdpa_cache_index.h -- the paged cache's index arithmetic and the launch's
// angles, free of CUDA: the kernels compile it for the device, the tests as
// plain C++ for the host.
#pragma once

#include <cmath>
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

// x modulo 1 in units of 2^-64, rounded (the difference is exact: x and its
// floor are multiples of x's last bit).
inline uint64_t fraction64(double x) {
  const double a = std::fabs(x), y = (a - std::floor(a)) * 4294967296.0, top = std::floor(y);
  const uint64_t u = (static_cast<uint64_t>(top) << 32) + static_cast<uint64_t>(std::nearbyint((y - top) * 4294967296.0));
  return x < 0 ? ~u + 1 : u;
}

// f / 2 pi modulo 1 in units of 2^-64, off by one of them at most (|f| below
// 2^40): 1 / 2 pi is a sum of two doubles, and the first product's rounding error
// is added.  A position times this, modulo 2^64, is the angle to 2^-32 turns at
// every position below 2^31; a single product's error of 2^-56 grows to 2^-25.
inline uint64_t turn_fraction(double f) {
  constexpr double kHigh = 0.15915494309189535, kLow = -9.839338337591243e-18;  // 1 / 2 pi
  const volatile double product = f * kHigh;  // rounded here (never part of a fused product)
  const double p = product;
  return fraction64(p) + fraction64(std::fma(f, kHigh, -p) + f * kLow);
}

}  // namespace gdpa
