// sa_mask.cuh — which keys a query row may see, shared by the masked forward
// and the accumulated cache weights.
//
// Every mask the entry points take leaves a row one contiguous span of keys:
// a document is a run of keys, the rows of a document are its last positions,
// a frame-causal row sees up to the end of its own frame (`causal` tokens a
// frame; 1 = token-causal), and a prefix is the document's first keys, which
// every row of the document sees.  Both ends of the span never decrease from
// one row to the next, so the keys that a run of rows needs are
// [span(first).lo, span(last).hi).
#pragma once

#include <stdint.h>

#include "sa_internal.h"

namespace sa {

struct Span {
  int lo, hi;  // visible keys [lo, hi), 0 <= lo <= hi <= Nk whatever the tables hold
  int pos;     // the row's position as a key index (distances are |pos - key|)
};

__device__ __forceinline__ int clamp_int(int x, int lo, int hi) { return min(max(x, lo), hi); }

__device__ __forceinline__ Span row_span(const MaskDev& m, int b, int i) {
  int qs = 0, qe = m.Nq, ks = 0, ke = m.Nk, px = 0;
  if (m.nd > 0) {
    const int32_t* dq = m.dq + static_cast<int64_t>(b) * (m.nd + 1);
    const int32_t* dk = m.dk + static_cast<int64_t>(b) * (m.nd + 1);
    int e = 0, top = m.nd;  // the first document that ends behind row i
    while (e < top) {
      const int mid = (e + top) >> 1;
      if (__ldg(dq + mid + 1) <= i)
        e = mid + 1;
      else
        top = mid;
    }
    if (e == m.nd || __ldg(dq) > i) {  // a row of no document sees nothing
      const int at = clamp_int(__ldg(dk + (e == m.nd ? m.nd : 0)), 0, m.Nk);
      return {at, at, at};
    }
    qs = __ldg(dq + e);
    qe = __ldg(dq + e + 1);
    ks = clamp_int(__ldg(dk + e), 0, m.Nk);
    ke = clamp_int(__ldg(dk + e + 1), ks, m.Nk);
    if (m.px) px = __ldg(m.px + static_cast<int64_t>(b) * m.nd + e);
  } else if (m.len) {
    ke = clamp_int(__ldg(m.len + b), 0, m.Nk);
  }
  const int nk = ke - ks;
  const int p = i - qs + nk - (qe - qs);
  int vis = nk;
  if (m.causal > 0) {
    const int64_t end = p >= 0 ? (static_cast<int64_t>(p / m.causal) + 1) * m.causal : 0;
    vis = static_cast<int>(min(static_cast<int64_t>(nk), max(end, static_cast<int64_t>(px))));
    vis = max(vis, 0);
  }
  return {ks, ks + vis, p + ks};
}

}  // namespace sa
