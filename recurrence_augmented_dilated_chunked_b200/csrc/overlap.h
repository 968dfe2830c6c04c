// overlap.h -- whether two views of head rows share an element (host only).
#pragma once
#include <algorithm>
#include <utility>

#include "ratp.h"

namespace ratp {

// Whether two views share an element: base + sum of index * stride + channel meets
// for both where the difference of the bases, plus every stride times what its
// index can differ by (strides that both have are one term), lies within a row.
// Largest stride first, an index that the smaller ones cannot make up for is
// passed over, so nested strides take a few steps; views that take more than
// kOverlapSteps count as overlapping.
constexpr int kOverlapSteps = 1 << 16;
struct StrideTerm {
  long long stride, lo, hi;
};
inline bool terms_meet(const StrideTerm* t, int n, long long diff, int Dh, int* steps) {
  if (--*steps < 0) return true;
  if (n == 0) return diff > -Dh && diff < Dh;
  long long lo = diff, hi = diff;              // what the smaller strides can make of diff
  for (int i = 1; i < n; ++i) {
    lo += t[i].lo * t[i].stride;
    hi += t[i].hi * t[i].stride;
  }
  const auto floor_div = [](long long a, long long b) { return a / b - (a % b < 0 ? 1 : 0); };
  const long long first = std::max(t[0].lo, -floor_div(Dh - 1 + hi, t[0].stride));
  const long long last = std::min(t[0].hi, floor_div(Dh - 1 - lo, t[0].stride));
  for (long long d = first; d <= last; ++d)
    if (terms_meet(t + 1, n - 1, diff + d * t[0].stride, Dh, steps)) return true;
  return false;
}
inline bool views_overlap(const ratp_view& a, const ratp_view& b, int esize, int B, int T, int Dh) {
  const long long diff = (static_cast<const char*>(a.data) - static_cast<const char*>(b.data)) / esize;
  const auto span = [&](const ratp_view& v) { return (B - 1) * v.stride_b + (T - 1) * v.stride_t + (v.heads - 1) * v.stride_h + Dh; };
  if (diff >= span(b) || -diff >= span(a)) return false;
  const std::pair<int64_t, int> dims[2][3] = {{{a.stride_b, B}, {a.stride_t, T}, {a.stride_h, a.heads}},
                                              {{b.stride_b, B}, {b.stride_t, T}, {b.stride_h, b.heads}}};
  StrideTerm t[6];
  int n = 0;
  for (int v = 0; v < 2; ++v)
    for (const auto& d : dims[v]) {
      if (d.first == 0 || d.second <= 1) continue;
      int i = 0;
      while (i < n && t[i].stride != d.first) ++i;
      if (i == n) t[n++] = {d.first, 0, 0};
      (v == 0 ? t[i].hi : t[i].lo) += v == 0 ? d.second - 1 : 1 - d.second;
    }
  std::sort(t, t + n, [](const StrideTerm& x, const StrideTerm& y) { return x.stride > y.stride; });
  int steps = kOverlapSteps;
  return terms_meet(t, n, diff, Dh, &steps);
}

// The same rows at the same indices: a view and itself.
inline bool same_rows(const ratp_view& a, const ratp_view& b, int B, int T) {
  return a.data == b.data && (B <= 1 || a.stride_b == b.stride_b) && (T <= 1 || a.stride_t == b.stride_t) &&
         (a.heads <= 1 || a.stride_h == b.stride_h);
}

}  // namespace ratp
