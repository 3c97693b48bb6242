// sa_views.h — host-side checks of strided views, shared by the entry points that take them.
#pragma once

#include <algorithm>
#include <numeric>

#include "sa_internal.h"
#include "sparse_attn.h"

namespace sa {

// A [B, H, N, d] view: 16-byte aligned rows, no negative strides.  Strides of
// dimensions of size one are free and are replaced by the row size.  An input
// may repeat a dimension (stride 0) where `repeats`; an output's elements must
// not overlap.  *extent: bytes from the first to behind the last element.
inline bool check_view(const void* p, sa_strides* s, int64_t B, int64_t H, int64_t N, int64_t d, int esz,
                       bool output, bool repeats, uint64_t* extent) {
  if (!p || !aligned(p, 16)) return false;
  struct Dim {
    int64_t n, stride;
  } dims[3] = {{B, s->b}, {H, s->h}, {N, s->n}};
  int64_t last = d;  // elements
  for (Dim& x : dims) {
    if (x.n == 1) x.stride = d;
    if (x.stride < 0 || x.stride >= (int64_t(1) << 38) / esz || (x.stride * esz) % 16) return false;
    if (x.stride == 0 && !repeats) return false;
    if (x.stride > 0 && x.n - 1 > (int64_t(1) << 45) / x.stride) return false;
    last += (x.n - 1) * x.stride;
  }
  s->b = dims[0].stride;
  s->h = dims[1].stride;
  s->n = dims[2].stride;
  if (output) {
    std::sort(dims, dims + 3, [](const Dim& x, const Dim& y) { return x.stride < y.stride; });
    int64_t inner = d;
    for (const Dim& x : dims)
      if (x.n > 1) {
        if (x.stride < inner) return false;
        inner = x.stride * (x.n - 1) + inner;
      }
  }
  *extent = static_cast<uint64_t>(last) * esz;
  return true;
}

inline bool overlap(const void* a, uint64_t na, const void* b, uint64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

// A checked view: its first element, strides, sizes and extent in bytes.
struct View {
  const void* p;
  sa_strides s;
  int64_t B, H, N;
  uint64_t n;
};

// Whether two views (checked by check_view) are the same elements in the same order.
inline bool same_view(const View& a, const View& b) {
  return a.p == b.p && a.s.b == b.s.b && a.s.h == b.s.h && a.s.n == b.s.n;
}

// Whether two views of rows of d elements (checked by check_view) may share an
// element.  With the same strides they may interleave in one buffer (heads of a
// fused projection): rows that follow one another make blocks, and blocks start at
// multiples of the other strides' common divisor g from the view's start, so views
// whose starts differ modulo g by at least the first one's block one way round and
// the second one's the other never meet.  A dimension of size one has no stride of
// its own and takes the other view's.
inline bool views_overlap(const View& a, const View& b, int64_t d, int esz) {
  if (!overlap(a.p, a.n, b.p, b.n)) return false;
  struct Dim {
    int64_t na, nb, sa, sb;
  } dims[3] = {{a.B, b.B, a.s.b, b.s.b}, {a.H, b.H, a.s.h, b.s.h}, {a.N, b.N, a.s.n, b.s.n}};
  for (Dim& x : dims) {
    if (x.na == 1) x.sa = x.sb;
    if (x.nb == 1) x.sb = x.sa;
    if (x.sa != x.sb) return true;
  }
  std::sort(dims, dims + 3, [](const Dim& x, const Dim& y) { return x.sa < y.sa; });
  int64_t block_a = d, block_b = d, g = 0;
  for (const Dim& x : dims) {
    if (x.na == 1 && x.nb == 1) continue;
    if (g == 0 && x.sa == block_a && x.sa == block_b) {
      block_a *= x.na;
      block_b *= x.nb;
    } else {
      g = std::gcd(g, x.sa);
    }
  }
  const int64_t apart = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b.p) - reinterpret_cast<uintptr_t>(a.p)) / esz;
  if (g == 0) return apart < block_a && -apart < block_b;
  const int64_t m = ((apart % g) + g) % g;
  return m < block_a || g - m < block_b;
}

}  // namespace sa
