// sa_ops.cu — the C ABI of the operators around the attention path (rotary
// positions, masked forward, cache weights, eviction): argument checks and
// launches.  The checks run before anything is enqueued.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdlib>
#include <numeric>
#include <utility>

#include "sa_internal.h"
#include "sparse_attn.h"

namespace {

using sa::aligned;
using sa::device_info;
using sa::in_device_allocation;

// (tanh(z)/z - 1)/z^2 as a quadratic in z^2 through its Chebyshev nodes on
// [0, 0.16]: |z| times the error stays below 1.6e-7.
constexpr double kTanh1 = -0.3333307876878961, kTanh2 = 0.13304591654903536, kTanh3 = -0.04907868548467837;

sa_status map_cuda(cudaError_t e) { return e == cudaSuccess ? SA_OK : SA_ERR_CUDA; }

// A [B, H, N, d] view: 16-byte aligned rows, no negative strides.  Strides of
// dimensions of size one are free and are replaced by the row size.  An input
// may repeat a dimension (stride 0) where `repeats`; an output's elements must
// not overlap.  *extent: bytes from the first to behind the last element.
bool check_view(const void* p, sa_strides* s, int64_t B, int64_t H, int64_t N, int64_t d, int esz,
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

bool overlap(const void* a, uint64_t na, const void* b, uint64_t nb) {
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

// Whether two views of rows of d elements (checked by check_view) may share an
// element.  With the same strides they may interleave in one buffer (heads of a
// fused projection): rows that follow one another make blocks, and blocks start at
// multiples of the other strides' common divisor g from the view's start, so views
// whose starts differ modulo g by at least the first one's block one way round and
// the second one's the other never meet.  A dimension of size one has no stride of
// its own and takes the other view's.
bool views_overlap(const View& a, const View& b, int64_t d, int esz) {
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

// f / 2 pi modulo 1 as a 64-bit fraction of a turn, to its last bits for every double f below
// 2^40 or so: 1 / 2 pi is taken to twice a double's digits (a double's alone would leave an error
// that 2^31 positions multiply to f 2^-22 of a radian).
uint64_t turn_fraction(double f) {
  constexpr double kInv1 = 0.15915494309189535, kInv2 = -9.839338337591243e-18;  // their sum is 1 / 2 pi to 2^-108
  volatile double rounded = f * kInv1;  // (not to be fused with what follows)
  const double hi = rounded, lo = std::fma(f, kInv1, -hi) + f * kInv2;
  auto fraction = [](double x) -> uint64_t {
    x -= std::trunc(x);  // exact
    const uint64_t m = static_cast<uint64_t>(std::ldexp(std::fabs(x), 64));
    return x < 0.0 ? 0 - m : m;
  };
  return fraction(hi) + fraction(lo);
}

// Shapes and options of sa_masked; fills everything but the tensor pointers.
sa_status check_masked(const sa_masked* p, sa::MaskedArgs* a) {
  if (!p) return SA_ERR_INVALID_ARG;
  if (p->B < 1 || p->Hq < 1 || p->Hkv < 1 || p->Nq < 1 || p->Nk < 1 || p->d < 1) return SA_ERR_INVALID_ARG;
  if (p->Hq % p->Hkv || p->causal < 0 || p->ndocs < 0) return SA_ERR_INVALID_ARG;
  if (!std::isfinite(p->scale) || p->scale == 0.f || !std::isfinite(p->cap) || p->cap < 0.f)
    return SA_ERR_INVALID_ARG;
  if (p->out_dtype != SA_OUT_BF16 && p->out_dtype != SA_OUT_FP32) return SA_ERR_INVALID_ARG;
  if (p->ndocs > 0 ? (!p->docs_q || !p->docs_k || p->lengths) : (p->docs_q || p->docs_k || p->prefix))
    return SA_ERR_INVALID_ARG;
  for (const void* t : {static_cast<const void*>(p->docs_q), static_cast<const void*>(p->docs_k),
                        static_cast<const void*>(p->prefix), static_cast<const void*>(p->lengths),
                        static_cast<const void*>(p->slopes)})
    if (!aligned(t, 4)) return SA_ERR_INVALID_ARG;
  if (p->d != 64 && p->d != 128) return SA_ERR_UNSUPPORTED;
  const int64_t R = p->Hq / p->Hkv;
  if (R > 128) return SA_ERR_UNSUPPORTED;  // a Q tile holds all of a query's heads
  // key coordinates and numbers of Q tiles are 32-bit with room for a tile behind them
  const int64_t heads = int64_t(p->B) * p->Hkv, qn = 128 / R;
  if (p->Nq > (1 << 30) || p->Nk > (1 << 30) || p->ndocs > (1 << 30) || heads * R > (1 << 24) ||
      heads * ((p->Nq + qn - 1) / qn) > (1 << 30) || R * p->Nq > UINT32_MAX)
    return SA_ERR_UNSUPPORTED;
  a->qs = p->q;
  a->ks = p->k;
  a->vs = p->v;
  a->os = p->o;
  a->slopes = p->slopes;
  a->mask = {p->docs_q, p->docs_k, p->prefix, p->lengths, p->ndocs, p->causal, p->Nq, p->Nk};
  a->B = p->B;
  a->Hq = p->Hq;
  a->Hkv = p->Hkv;
  a->R = static_cast<int32_t>(R);
  a->Nq = p->Nq;
  a->Nk = p->Nk;
  a->d = p->d;
  a->out_fp32 = p->out_dtype == SA_OUT_FP32 ? 1 : 0;
  a->neg_scale = p->scale < 0.f ? 1 : 0;
  const double log2e = 1.4426950408889634, s = std::fabs(static_cast<double>(p->scale));
  a->scale_log2 = static_cast<float>(s * log2e);
  a->cap_log2 = static_cast<float>(p->cap * log2e);
  a->cap_k1 = p->cap > 0.f ? static_cast<float>(2.0 * s * log2e / p->cap) : 0.f;
  // tanh(z) = z (1 + z^2 (c1 + z^2 (c2 + z^2 c3))) for |z| <= 0.4, z = x |scale| / cap
  const double r2 = p->cap > 0.f ? s / p->cap * (s / p->cap) : 0.0;
  a->cap_p1 = static_cast<float>(kTanh1 * s * log2e * r2);
  a->cap_p2 = static_cast<float>(kTanh2 * s * log2e * r2 * r2);
  a->cap_p3 = static_cast<float>(kTanh3 * s * log2e * r2 * r2 * r2);
  // a scale or a ratio to the cap that fp32 cannot hold would turn scores into NaN
  if (!std::isfinite(a->scale_log2) || !std::isfinite(a->cap_log2) || !std::isfinite(a->cap_k1))
    return SA_ERR_INVALID_ARG;
  a->cap_limit = r2 > 0.0 && r2 < 1e6 ? static_cast<float>(0.16 / r2) : -1.f;
  a->total_rows = int64_t(p->B) * p->Hq * p->Nq;
  a->qn = a->tiles = a->unit_rows = a->row_blocks = a->group = a->splits = 1;
  a->quads = a->slots = 0;
  a->full_units = a->split_units = 0;
  a->part_o = nullptr;
  a->part_lse = nullptr;
  a->part_first = nullptr;
  return SA_OK;
}

// The device tables of sa_masked (after device_info).
bool masked_tables(const sa_masked* p) {
  const uint64_t B = p->B, nd = p->ndocs;
  return (!nd || (in_device_allocation(p->docs_q, B * (nd + 1) * 4) &&
                  in_device_allocation(p->docs_k, B * (nd + 1) * 4))) &&
         (!p->prefix || in_device_allocation(p->prefix, B * nd * 4)) &&
         (!p->lengths || in_device_allocation(p->lengths, B * 4)) &&
         (!p->slopes || in_device_allocation(p->slopes, uint64_t(p->Hq) * 4));
}

// The partial outputs, then their lse, then the table of slots (each 256-byte aligned).
size_t part_count(const sa::MaskedArgs& a) { return a.slots ? a.slots : size_t(a.split_units) * a.splits; }
size_t part_bytes(const sa::MaskedArgs& a) { return (part_count(a) * a.unit_rows * a.d * 4 + 255) / 256 * 256; }
size_t part_lse_bytes(const sa::MaskedArgs& a) { return (part_count(a) * a.unit_rows * 4 + 255) / 256 * 256; }

size_t masked_workspace(const sa::MaskedArgs& a) {
  return part_bytes(a) + part_lse_bytes(a) + (a.slots ? (size_t(a.B) * 8 + 255) / 256 * 256 : 0);
}

}  // namespace

extern "C" {

size_t sparse_attn_forward_masked_workspace_size(const sa_masked* p) {
  sa::MaskedArgs a;
  if (check_masked(p, &a) != SA_OK) return 0;
  sa::masked_plan(&a);
  return masked_workspace(a);
}

sa_status sparse_attn_forward_masked(const sa_masked* p, const void* q, const void* k, const void* v, void* o,
                                     float* lse, int32_t* dev_status, void* workspace, size_t workspace_bytes,
                                     sa_stream_t stream) {
  sa::MaskedArgs a;
  sa_status st = check_masked(p, &a);
  if (st != SA_OK) return st;
  uint64_t nq, nk, nv, no;
  if (!check_view(q, &a.qs, p->B, p->Hq, p->Nq, p->d, 2, false, false, &nq) ||
      !check_view(k, &a.ks, p->B, p->Hkv, p->Nk, p->d, 2, false, false, &nk) ||
      !check_view(v, &a.vs, p->B, p->Hkv, p->Nk, p->d, 2, false, false, &nv) ||
      !check_view(o, &a.os, p->B, p->Hq, p->Nq, p->d, a.out_fp32 ? 4 : 2, true, false, &no))
    return SA_ERR_INVALID_ARG;
  if (!aligned(lse, 4) || !aligned(dev_status, 4)) return SA_ERR_INVALID_ARG;
  // Outputs may not share elements with inputs or each other; o may be q's view
  // (a row of q is read only ahead of the row of o that takes its place).
  const int esz = a.out_fp32 ? 4 : 2;
  const View out{o, a.os, p->B, p->Hq, p->Nq, no};
  auto apart = [&](const View& x) {
    return esz == 2 ? !views_overlap(out, x, p->d, 2) : !overlap(o, no, x.p, x.n);
  };
  const bool same = o == q && esz == 2 && a.os.b == a.qs.b && a.os.h == a.qs.h && a.os.n == a.qs.n;
  if ((!same && !apart({q, a.qs, p->B, p->Hq, p->Nq, nq})) || !apart({k, a.ks, p->B, p->Hkv, p->Nk, nk}) ||
      !apart({v, a.vs, p->B, p->Hkv, p->Nk, nv}))
    return SA_ERR_INVALID_ARG;
  const uint64_t nl = lse ? uint64_t(a.total_rows) * 4 : 0;
  if (nl && (overlap(lse, nl, q, nq) || overlap(lse, nl, k, nk) || overlap(lse, nl, v, nv) || overlap(lse, nl, o, no)))
    return SA_ERR_INVALID_ARG;
  sa::masked_plan(&a);
  const size_t need = masked_workspace(a);
  if (need && (!workspace || !aligned(workspace, 256) || workspace_bytes < need)) return SA_ERR_INVALID_ARG;
  if (need)
    for (const auto& x : {std::pair<const void*, uint64_t>{q, nq}, {k, nk}, {v, nv}, {o, no}, {lse, nl}})
      if (x.second && overlap(workspace, need, x.first, x.second)) return SA_ERR_INVALID_ARG;
  int sms = 0;
  if ((st = device_info(&sms)) != SA_OK) return st;
  if (!in_device_allocation(q, nq) || !in_device_allocation(k, nk) || !in_device_allocation(v, nv) ||
      !in_device_allocation(o, no) || (lse && !in_device_allocation(lse, uint64_t(a.total_rows) * 4)) ||
      (dev_status && !in_device_allocation(dev_status, 4)) || (need && !in_device_allocation(workspace, need)) ||
      !masked_tables(p))
    return SA_ERR_INVALID_ARG;
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.o = o;
  a.lse = lse;
  a.status = dev_status;
  if (need) {
    a.part_o = static_cast<float*>(workspace);
    a.part_lse = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + part_bytes(a));
    a.part_first = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) + part_bytes(a) + part_lse_bytes(a));
  }
  sa::NvtxRange range("sparse_attn_forward_masked");
  return map_cuda(sa::launch_masked(a, reinterpret_cast<cudaStream_t>(stream)));
}

sa_status sparse_attn_cache_weights(const sa_masked* p, const void* q, const void* k, const float* lse,
                                    const float* w_in, float* w_out, float decay, int32_t* dev_status,
                                    sa_stream_t stream) {
  sa::WeightArgs w;
  sa::MaskedArgs& a = w.m;
  sa_status st = check_masked(p, &a);
  if (st != SA_OK) return st;
  uint64_t nq, nk;
  if (!check_view(q, &a.qs, p->B, p->Hq, p->Nq, p->d, 2, false, false, &nq) ||
      !check_view(k, &a.ks, p->B, p->Hkv, p->Nk, p->d, 2, false, false, &nk))
    return SA_ERR_INVALID_ARG;
  if (!lse || !w_out || !std::isfinite(decay) || (decay != 0.f && !w_in)) return SA_ERR_INVALID_ARG;
  if (!aligned(lse, 4) || !aligned(w_in, 4) || !aligned(w_out, 4) || !aligned(dev_status, 4))
    return SA_ERR_INVALID_ARG;
  if (int64_t(p->B) * p->Hkv * ((int64_t(p->Nk) + 255) / 256) >= (int64_t(1) << 30)) return SA_ERR_UNSUPPORTED;
  const uint64_t wbytes = uint64_t(p->B) * p->Hkv * p->Nk * 4, lbytes = uint64_t(a.total_rows) * 4;
  if (w_in && w_in != w_out && overlap(w_in, wbytes, w_out, wbytes)) return SA_ERR_INVALID_ARG;
  if (overlap(lse, lbytes, w_out, wbytes) || overlap(q, nq, w_out, wbytes) || overlap(k, nk, w_out, wbytes))
    return SA_ERR_INVALID_ARG;
  int sms = 0;
  if ((st = device_info(&sms)) != SA_OK) return st;
  if (!in_device_allocation(q, nq) || !in_device_allocation(k, nk) || !in_device_allocation(lse, lbytes) ||
      !in_device_allocation(w_out, wbytes) || (w_in && !in_device_allocation(w_in, wbytes)) ||
      (dev_status && !in_device_allocation(dev_status, 4)) || !masked_tables(p))
    return SA_ERR_INVALID_ARG;
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.v = nullptr;
  a.o = nullptr;
  a.lse = nullptr;
  a.status = dev_status;
  w.lse = lse;
  w.w_in = w_in;
  w.w_out = w_out;
  w.decay = decay;
  sa::NvtxRange range("sparse_attn_cache_weights");
  return map_cuda(sa::launch_cache_weights(w, sms, reinterpret_cast<cudaStream_t>(stream)));
}

sa_status sparse_attn_cache_evict(const sa_evict* p, const float* weights, const void* k, const void* v,
                                  int32_t* kept, void* k_out, void* v_out, float* weights_out,
                                  sa_stream_t stream) {
  if (!p || p->B < 1 || p->Hkv < 1 || p->Nk < 1 || p->d < 1) return SA_ERR_INVALID_ARG;
  if (p->budget < 1 || p->sink < 0 || p->recent < 0 || int64_t(p->sink) + p->recent > p->budget)
    return SA_ERR_INVALID_ARG;
  if (p->d != 64 && p->d != 128) return SA_ERR_UNSUPPORTED;
  const int64_t rows = int64_t(p->B) * p->Hkv;
  if (rows > 65535 || p->Nk > (1 << 30) || p->budget > (1 << 30)) return SA_ERR_UNSUPPORTED;  // grid.y, int indexes
  if (!weights || !kept || !aligned(weights, 4) || !aligned(kept, 4) || !aligned(weights_out, 4) ||
      !aligned(p->lengths, 4))
    return SA_ERR_INVALID_ARG;
  const bool kv = k || v || k_out || v_out;
  sa::EvictArgs a;
  a.ks = p->k;
  a.vs = p->v;
  a.kos = p->k_out;
  a.vos = p->v_out;
  uint64_t nk = 0, nv = 0, nko = 0, nvo = 0;
  if (kv && (!check_view(k, &a.ks, p->B, p->Hkv, p->Nk, p->d, 2, false, true, &nk) ||
             !check_view(v, &a.vs, p->B, p->Hkv, p->Nk, p->d, 2, false, true, &nv) ||
             !check_view(k_out, &a.kos, p->B, p->Hkv, p->budget, p->d, 2, true, false, &nko) ||
             !check_view(v_out, &a.vos, p->B, p->Hkv, p->budget, p->d, 2, true, false, &nvo)))
    return SA_ERR_INVALID_ARG;
  const uint64_t wbytes = uint64_t(rows) * p->Nk * 4, obytes = uint64_t(rows) * p->budget * 4;
  // the rows are moved by many blocks at once: nothing may be read where something is written
  struct Span {
    const void* p;
    uint64_t n;
  };
  const Span in[] = {{weights, wbytes}, {k, nk}, {v, nv}};
  const Span out[] = {{kept, obytes}, {k_out, nko}, {v_out, nvo}, {weights_out, weights_out ? obytes : 0}};
  for (int i = 0; i < 4; ++i) {
    if (!out[i].n) continue;
    for (const Span& x : in)
      if (x.n && overlap(x.p, x.n, out[i].p, out[i].n)) return SA_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)  // (k_out and v_out: below)
      if (out[j].n && !(j == 1 && i == 2) && overlap(out[j].p, out[j].n, out[i].p, out[i].n))
        return SA_ERR_INVALID_ARG;
  }
  if (kv && views_overlap({k_out, a.kos, p->B, p->Hkv, p->budget, nko}, {v_out, a.vos, p->B, p->Hkv, p->budget, nvo},
                          p->d, 2))
    return SA_ERR_INVALID_ARG;
  int sms = 0;
  sa_status st = device_info(&sms);
  if (st != SA_OK) return st;
  if (!in_device_allocation(weights, wbytes) || !in_device_allocation(kept, obytes) ||
      (weights_out && !in_device_allocation(weights_out, obytes)) ||
      (p->lengths && !in_device_allocation(p->lengths, uint64_t(p->B) * 4)) ||
      (kv && (!in_device_allocation(k, nk) || !in_device_allocation(v, nv) || !in_device_allocation(k_out, nko) ||
              !in_device_allocation(v_out, nvo))))
    return SA_ERR_INVALID_ARG;
  a.w = weights;
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.k_out = static_cast<uint16_t*>(k_out);
  a.v_out = static_cast<uint16_t*>(v_out);
  a.w_out = weights_out;
  a.kept = kept;
  a.len = p->lengths;
  a.B = p->B;
  a.Hkv = p->Hkv;
  a.Nk = p->Nk;
  a.d = p->d;
  a.budget = p->budget;
  a.sink = p->sink;
  a.recent = p->recent;
  sa::NvtxRange range("sparse_attn_cache_evict");
  return map_cuda(sa::launch_cache_evict(a, sms, reinterpret_cast<cudaStream_t>(stream)));
}

sa_status sparse_attn_rope(const sa_rope* p, int32_t H0, const void* x0, const sa_strides* x0s, void* y0,
                           const sa_strides* y0s, int32_t H1, const void* x1, const sa_strides* x1s, void* y1,
                           const sa_strides* y1s, sa_stream_t stream) {
  if (!p || p->B < 1 || p->N < 1 || p->d < 1 || H0 < 1 || H1 < 0 || !x0s || !y0s) return SA_ERR_INVALID_ARG;
  if (p->axes < 1 || p->axes > 3 || (p->pairing != SA_ROPE_INTERLEAVED && p->pairing != SA_ROPE_HALF) ||
      (p->dtype != SA_OUT_BF16 && p->dtype != SA_OUT_FP32))
    return SA_ERR_INVALID_ARG;
  if (p->d != 64 && p->d != 128) return SA_ERR_UNSUPPORTED;
  if (p->B > 65535 || int64_t(H0) + H1 > 65535) return SA_ERR_UNSUPPORTED;  // grid.z, grid.y
  sa::RopeArgs a;
  a.axes = p->axes;
  a.rot = 0;
  for (int i = 0; i < 4; ++i) a.first[i] = 0;
  for (int i = 0; i < 3; ++i) {
    const int32_t n = i < p->axes ? p->axis_dim[i] : 0;
    if (n < 0 || n % 2 || n > p->d) return SA_ERR_INVALID_ARG;
    a.rot += n;
    a.first[i + 1] = a.rot / 2;
  }
  if (a.rot < 2 || a.rot > p->d) return SA_ERR_INVALID_ARG;
  if (p->pairing == SA_ROPE_HALF && a.rot % 16) return SA_ERR_UNSUPPORTED;  // 16-byte halves
  if (!p->inv_freq && !(std::isfinite(p->theta) && p->theta > 0.0)) return SA_ERR_INVALID_ARG;
  for (int x = 0; x < p->axes; ++x)
    for (int i = a.first[x]; i < a.first[x + 1]; ++i) {
      const double f = p->inv_freq ? p->inv_freq[i]
                                   : std::pow(p->theta, -2.0 * (i - a.first[x]) / p->axis_dim[x]);
      if (!std::isfinite(f)) return SA_ERR_INVALID_ARG;
      a.turn[i] = turn_fraction(f);
    }
  for (int i = a.rot / 2; i < 64; ++i) a.turn[i] = 0;
  a.vox = {};
  a.pos = p->positions;
  a.pos_b = p->positions_b;
  a.voxel_order = 0;
  if (p->positions) {
    if (!aligned(p->positions, 4) || p->positions_b < 0 || (p->B > 1 && p->positions_b > (int64_t(1) << 40)) ||
        (p->positions_b && p->positions_b < int64_t(p->N) * p->axes))
      return SA_ERR_INVALID_ARG;
    for (int i = 0; i < 3; ++i) a.offset[i] = 0;
  } else {
    const sa_voxel_grid& g = p->grid;
    if (p->axes != 3 || g.T < 1 || g.Hh < 1 || g.W < 1 || g.T > p->N || g.Hh > p->N || g.W > p->N)
      return SA_ERR_INVALID_ARG;
    if (int64_t(g.T) * g.Hh > p->N || int64_t(g.T) * g.Hh * g.W != p->N) return SA_ERR_INVALID_ARG;
    if (p->voxel_order && (g.vt < 1 || g.vh < 1 || g.vw < 1)) return SA_ERR_INVALID_ARG;
    const int64_t size[3] = {g.T, g.Hh, g.W};
    for (int i = 0; i < 3; ++i) {
      const int64_t o = p->offset[i];
      if (o < INT32_MIN || o + size[i] - 1 > INT32_MAX) return SA_ERR_INVALID_ARG;
      a.offset[i] = static_cast<int32_t>(o);
    }
    a.vox.T = g.T;
    a.vox.Hh = g.Hh;
    a.vox.W = g.W;
    // a voxel larger than the grid is the grid
    a.vox.vt = p->voxel_order ? std::min(g.vt, g.T) : g.T;
    a.vox.vh = p->voxel_order ? std::min(g.vh, g.Hh) : g.Hh;
    a.vox.vw = p->voxel_order ? std::min(g.vw, g.W) : g.W;
    a.voxel_order = p->voxel_order ? 1 : 0;
  }
  const int esz = p->dtype == SA_OUT_FP32 ? 4 : 2;
  const void* x[2] = {x0, x1};
  void* y[2] = {y0, y1};
  const sa_strides* xs[2] = {x0s, x1s};
  const sa_strides* ys[2] = {y0s, y1s};
  const int32_t H[2] = {H0, H1};
  uint64_t nx[2] = {0, 0}, ny[2] = {0, 0};
  for (int i = 0; i < 2; ++i) {
    a.x[i] = x[i];
    a.y[i] = y[i];
    a.H[i] = H[i];
    if (!H[i]) continue;
    if (!xs[i] || !ys[i]) return SA_ERR_INVALID_ARG;
    a.xs[i] = *xs[i];
    a.ys[i] = *ys[i];
    if (!check_view(x[i], &a.xs[i], p->B, H[i], p->N, p->d, esz, false, true, &nx[i]) ||
        !check_view(y[i], &a.ys[i], p->B, H[i], p->N, p->d, esz, true, false, &ny[i]))
      return SA_ERR_INVALID_ARG;
    // in place (the same view) or apart: a row is read only by the threads that write it
    const bool same = x[i] == y[i] && a.xs[i].b == a.ys[i].b && a.xs[i].h == a.ys[i].h && a.xs[i].n == a.ys[i].n;
    if (!same && views_overlap({x[i], a.xs[i], p->B, H[i], p->N, nx[i]}, {y[i], a.ys[i], p->B, H[i], p->N, ny[i]},
                               p->d, esz))
      return SA_ERR_INVALID_ARG;
  }
  if (H1) {  // one pair's rows are not to be written while the other's are read or written
    const View vx[2] = {{x0, a.xs[0], p->B, H0, p->N, nx[0]}, {x1, a.xs[1], p->B, H1, p->N, nx[1]}};
    const View vy[2] = {{y0, a.ys[0], p->B, H0, p->N, ny[0]}, {y1, a.ys[1], p->B, H1, p->N, ny[1]}};
    if (views_overlap(vy[0], vy[1], p->d, esz) || views_overlap(vy[0], vx[1], p->d, esz) ||
        views_overlap(vx[0], vy[1], p->d, esz))
      return SA_ERR_INVALID_ARG;
  }
  int sms = 0;
  sa_status st = device_info(&sms);
  if (st != SA_OK) return st;
  for (int i = 0; i < 2; ++i)
    if (H[i] && (!in_device_allocation(x[i], nx[i]) || !in_device_allocation(y[i], ny[i])))
      return SA_ERR_INVALID_ARG;
  if (p->positions &&
      !in_device_allocation(p->positions, (uint64_t(p->B - 1) * uint64_t(p->positions_b) + uint64_t(p->N) * p->axes) * 4))
    return SA_ERR_INVALID_ARG;
  a.B = p->B;
  a.N = p->N;
  a.d = p->d;
  a.half = p->pairing == SA_ROPE_HALF;
  a.fp32 = p->dtype == SA_OUT_FP32;
  a.inverse = p->inverse ? 1 : 0;
  sa::NvtxRange range("sparse_attn_rope");
  return map_cuda(sa::launch_rope(a, sms, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
