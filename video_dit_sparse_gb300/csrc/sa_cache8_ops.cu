// sa_cache8_ops.cu — the C ABI of the 8-bit cache: argument checks and launches.  The checks run before anything is
// enqueued.
#include <cuda_runtime.h>

#include <cmath>
#include <utility>

#include "sa_internal.h"
#include "sa_views.h"
#include "sparse_attn.h"

namespace {

using namespace sa;

sa_status map_cuda(cudaError_t e) { return e == cudaSuccess ? SA_OK : SA_ERR_CUDA; }

// A cache's four tensors, as checked views with their extents in bytes.
struct Cache {
  View codes[2];
  const float* scales[2];
  sa_strides ss[2];
  uint64_t sn[2];
};

// Scales [B, H, blocks] with contiguous blocks; apart from one another where `output`.
bool check_scales(const float* p, sa_strides* s, int64_t B, int64_t H, int64_t blocks, bool output, uint64_t* extent) {
  if (!p || !aligned(p, 4)) return false;
  if (B == 1) s->b = 0;
  if (H == 1) s->h = 0;
  for (const auto& x : {std::pair<int64_t, int64_t>{s->b, B}, {s->h, H}})
    if (x.first < 0 || (x.second > 1 && x.first > (int64_t(1) << 40) / (x.second - 1))) return false;
  if (output) {
    const int64_t in = B == 1 || (H > 1 && s->h <= s->b) ? s->h : s->b, out = in == s->h ? s->b : s->h;
    const int64_t n_in = in == s->h ? H : B, n_out = in == s->h ? B : H;
    if ((n_in > 1 && in < blocks) || (n_out > 1 && out < in * (n_in - 1) + blocks)) return false;
  }
  *extent = static_cast<uint64_t>((B - 1) * s->b + (H - 1) * s->h + blocks) * 4;
  return true;
}

// Shapes, views and alignment of a cache that is written to (`output`) or read.
sa_status check_cache(const sa_cache8* c, bool output, Cache* out) {
  if (!c || c->B < 1 || c->Hkv < 1 || c->N < 1 || c->d < 1) return SA_ERR_INVALID_ARG;
  if (c->block != 16 && c->block != 32 && c->block != 64 && c->block != 128) return SA_ERR_INVALID_ARG;
  if (c->d != 64 && c->d != 128) return SA_ERR_UNSUPPORTED;
  if (c->N > (1 << 30) || int64_t(c->B) * c->Hkv > (1 << 24)) return SA_ERR_UNSUPPORTED;
  const void* codes[2] = {c->k, c->v};
  const sa_strides strides[2] = {c->ks, c->vs}, scale_strides[2] = {c->k_scales, c->v_scales};
  const float* scales[2] = {c->k_scale, c->v_scale};
  const int64_t blocks = (int64_t(c->N) + c->block - 1) / c->block;
  for (int i = 0; i < 2; ++i) {
    out->codes[i] = {codes[i], strides[i], c->B, c->Hkv, c->N, 0};
    out->scales[i] = scales[i];
    out->ss[i] = scale_strides[i];
    if (!check_view(codes[i], &out->codes[i].s, c->B, c->Hkv, c->N, c->d, 1, output, false, &out->codes[i].n) ||
        !check_scales(scales[i], &out->ss[i], c->B, c->Hkv, blocks, output, &out->sn[i]))
      return SA_ERR_INVALID_ARG;
  }
  return SA_OK;
}

bool cache_in_device(const Cache& c) {
  for (int i = 0; i < 2; ++i)
    if (!in_device_allocation(c.codes[i].p, c.codes[i].n) || !in_device_allocation(c.scales[i], c.sn[i])) return false;
  return true;
}

// [p, p + n) shares memory with any part of the cache.
bool meets_cache(const Cache& c, const void* p, uint64_t n) {
  for (int i = 0; i < 2; ++i)
    if (overlap(p, n, c.codes[i].p, c.codes[i].n) || overlap(p, n, c.scales[i], c.sn[i])) return true;
  return false;
}

void fill(const sa_cache8* p, const Cache& c, int32_t n, const int32_t* start, int32_t start0, Cache8Args* a) {
  *a = Cache8Args{};
  for (int i = 0; i < 2; ++i) {
    a->codes[i] = static_cast<uint8_t*>(const_cast<void*>(c.codes[i].p));
    a->cs[i] = c.codes[i].s;
    a->scales[i] = const_cast<float*>(c.scales[i]);
    a->ss[i] = c.ss[i];
  }
  a->start = start;
  a->start0 = start0;
  a->B = p->B;
  a->H = p->Hkv;
  a->N = p->N;
  a->d = p->d;
  a->block = p->block;
  a->n = n;
}

}  // namespace

extern "C" {

sa_status sparse_attn_cache8_append(const sa_cache8* p, int32_t n, const void* k, const sa_strides* ks, const void* v,
                                    const sa_strides* vs, const int32_t* start, int32_t start0, const int32_t* counts,
                                    sa_stream_t stream) {
  Cache c;
  sa_status st = check_cache(p, true, &c);
  if (st != SA_OK) return st;
  if (n < 1 || !ks || !vs || !aligned(start, 4) || !aligned(counts, 4)) return SA_ERR_INVALID_ARG;
  if (n > (1 << 30)) return SA_ERR_UNSUPPORTED;
  const int64_t blocks = (int64_t(n) + p->block - 2) / p->block + 1;
  if (int64_t(p->B) * p->Hkv * 2 * blocks >= (int64_t(1) << 31)) return SA_ERR_UNSUPPORTED;  // grid.x
  View x[2] = {{k, *ks, p->B, p->Hkv, n, 0}, {v, *vs, p->B, p->Hkv, n, 0}};
  for (View& y : x)
    if (!check_view(y.p, &y.s, p->B, p->Hkv, n, p->d, 2, false, true, &y.n) || meets_cache(c, y.p, y.n))
      return SA_ERR_INVALID_ARG;
  // the keys' codes, the values' and both scales are apart (views of one buffer may interleave)
  if (views_overlap(c.codes[0], c.codes[1], p->d, 1) || overlap(c.scales[0], c.sn[0], c.scales[1], c.sn[1]))
    return SA_ERR_INVALID_ARG;
  for (const View& y : c.codes)
    for (int i = 0; i < 2; ++i)
      if (overlap(y.p, y.n, c.scales[i], c.sn[i])) return SA_ERR_INVALID_ARG;
  int sms = 0;
  if ((st = device_info(&sms)) != SA_OK) return st;
  if (!cache_in_device(c) || !in_device_allocation(k, x[0].n) || !in_device_allocation(v, x[1].n) ||
      (start && !in_device_allocation(start, uint64_t(p->B) * 4)) ||
      (counts && !in_device_allocation(counts, uint64_t(p->B) * 4)))
    return SA_ERR_INVALID_ARG;
  Cache8Args a;
  fill(p, c, n, start, start0, &a);
  a.counts = counts;
  for (int i = 0; i < 2; ++i) {
    a.x[i] = x[i].p;
    a.xs[i] = x[i].s;
  }
  NvtxRange range("sparse_attn_cache8_append");
  return map_cuda(launch_cache8_append(a, reinterpret_cast<cudaStream_t>(stream)));
}

sa_status sparse_attn_cache8_read(const sa_cache8* p, const int32_t* first, int32_t first0, int32_t n, int32_t out_dtype,
                                  void* k_out, const sa_strides* ks, void* v_out, const sa_strides* vs,
                                  sa_stream_t stream) {
  Cache c;
  sa_status st = check_cache(p, false, &c);
  if (st != SA_OK) return st;
  if (n < 1 || (!k_out && !v_out) || (k_out && !ks) || (v_out && !vs) || !aligned(first, 4)) return SA_ERR_INVALID_ARG;
  if (out_dtype != SA_OUT_BF16 && out_dtype != SA_OUT_FP32) return SA_ERR_INVALID_ARG;
  if (n > (1 << 30) || int64_t(p->B) * p->Hkv * n * (p->d / 16) > (int64_t(1) << 37)) return SA_ERR_UNSUPPORTED;  // grid.x
  const int esz = out_dtype == SA_OUT_FP32 ? 4 : 2;
  View y[2] = {{k_out, {}, p->B, p->Hkv, n, 0}, {v_out, {}, p->B, p->Hkv, n, 0}};
  for (int i = 0; i < 2; ++i) {
    if (!y[i].p) continue;
    y[i].s = *(i ? vs : ks);
    if (!check_view(y[i].p, &y[i].s, p->B, p->Hkv, n, p->d, esz, true, false, &y[i].n) || meets_cache(c, y[i].p, y[i].n))
      return SA_ERR_INVALID_ARG;
  }
  if (k_out && v_out && views_overlap(y[0], y[1], p->d, esz)) return SA_ERR_INVALID_ARG;
  int sms = 0;
  if ((st = device_info(&sms)) != SA_OK) return st;
  if (!cache_in_device(c) || (k_out && !in_device_allocation(k_out, y[0].n)) ||
      (v_out && !in_device_allocation(v_out, y[1].n)) || (first && !in_device_allocation(first, uint64_t(p->B) * 4)))
    return SA_ERR_INVALID_ARG;
  Cache8Args a;
  fill(p, c, n, first, first0, &a);
  for (int i = 0; i < 2; ++i) {
    a.y[i] = const_cast<void*>(y[i].p);
    a.xs[i] = y[i].s;
  }
  NvtxRange range("sparse_attn_cache8_read");
  return map_cuda(launch_cache8_read(a, out_dtype == SA_OUT_FP32, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
