// gdpa_cache_index.h -- the paged cache's index arithmetic and the launch's
// angles, free of CUDA: the kernels compile it for the device, the tests as
// plain C++ for the host.
#pragma once

#include <algorithm>
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

// How an eviction's choice is launched: CTAs of a sequence and head, the most tokens
// that each of them has, and its threads.  Measured (us of a whole eviction in a graph,
// by CTAs a head, with 256 / 1024 threads; heads of 128; the rule's in brackets):
//     heads, tokens          1              2              4              8              16
//       1, 131 072           -              -         51.4 / 28.4    32.1 / 21.6    23.5 / [20.6]
//       4, 131 071           -              -         54.6 / 31.0    34.9 / 25.7    27.9 / [24.4]
//       2, 8192         18.8 / 14.6    15.6 / 14.9   [13.2] / 14.3   12.5 / 14.6    14.2 / 17.3
//       1, 4096         12.8 / 11.8   [11.9] / 12.7   11.0 / 12.8    11.2 / 13.0    12.6 / 15.5
//      16, 32 768       51.9 / 29.2    36.4 / 26.4    27.0 / 21.7   [22.5] / 28.0   24.8 / 45.1
//      72, 16 384       42.2 / 29.4    35.7 / [26.7]  28.9 / 34.8    27.8 / 65.5         -
//     128, 8192         47.4 / [35.8]  40.6 / 44.5    36.8 / 61.2    44.2 / 106          -
//     256, 8192         78.5 / [65.6]  64.7 / 82.6    65.5 / 111          -              -
//     304, 8192        [87.9] / 72.9   71.1 / 91.7    75.2 / 128          -              -
//     512, 8192       [111.8] / 121     114 / 152          -              -              -
//     320, 4096        [43.8] / 50.7   42.8 / 72.6         -              -              -
constexpr int kMostCluster = 16, kEveryCluster = 8;  // CTAs of a cluster: at most; on every device
struct ChooseShape {
  int ctas, threads;
  int64_t part;
};
inline ChooseShape choose_shape(int64_t heads, int64_t most, int sms, int widest) {
  ChooseShape c;
  // one, or where heads are few as many as the SMs hold with 2048 tokens each
  c.ctas = 1;
  while (c.ctas < widest && heads * c.ctas * 2 <= sms && most / (c.ctas * 2) >= 2048) c.ctas *= 2;
  c.part = ((most + c.ctas - 1) / c.ctas + 3) & ~static_cast<int64_t>(3);
  // few tokens do not keep 1024 threads busy, and of many heads several CTAs share an SM
  c.threads = c.part <= 4096 || heads >= 2 * sms ? 256 : 1024;
  return c;
}

// Whether any of T rows of `len` elements, x_stride apart from 0 on, shares an
// element with any of T rows y_stride apart from `apart` on (len <= both strides).
inline bool rows_overlap(int64_t apart, int64_t x_stride, int64_t y_stride, int64_t len, int64_t T) {
  auto floor_div = [](int64_t a, int64_t b) { return a / b - (a % b < 0); };
  const int64_t x_end = (T - 1) * x_stride + len, y_end = apart + (T - 1) * y_stride + len;
  if (T <= 0 || apart >= x_end || y_end <= 0) return false;
  if (x_stride == y_stride) {  // where they begin less than a row apart, modulo the stride
    const int64_t m = apart - floor_div(apart, x_stride) * x_stride;
    return m < len || m > x_stride - len;
  }
  // each row of x that lies among y's, with the first of y's that ends behind its beginning
  for (int64_t i = std::max<int64_t>(0, floor_div(apart - len, x_stride) + 1); i < T && i * x_stride < y_end; ++i) {
    const int64_t at = i * x_stride, j = std::max<int64_t>(0, floor_div(at - len - apart, y_stride) + 1);
    if (j < T && apart + j * y_stride < at + len) return true;
  }
  return false;
}

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
