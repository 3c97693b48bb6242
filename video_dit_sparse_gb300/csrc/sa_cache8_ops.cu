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

// Shapes and options of sa_attend8; fills what the plan goes by.
sa_status check_attend(const sa_attend8* p, const sa_cache8* c, Attend8Args* a) {
  if (!p || !c || p->Hq < 1 || p->Nq < 1 || c->B < 1 || c->Hkv < 1 || c->N < 1 || c->d < 1) return SA_ERR_INVALID_ARG;
  if (p->Hq % c->Hkv || p->causal < 0 || !aligned(p->lengths, 4)) return SA_ERR_INVALID_ARG;
  if (p->out_dtype != SA_OUT_BF16 && p->out_dtype != SA_OUT_FP32) return SA_ERR_INVALID_ARG;
  if (!std::isfinite(p->scale) || p->scale == 0.f || !std::isfinite(p->scale * 1.4426950408889634f)) return SA_ERR_INVALID_ARG;
  if (c->block != 16 && c->block != 32 && c->block != 64 && c->block != 128) return SA_ERR_INVALID_ARG;
  if (c->d != 64 && c->d != 128) return SA_ERR_UNSUPPORTED;
  const int64_t R = p->Hq / c->Hkv, heads = int64_t(c->B) * c->Hkv, qn = R > 128 ? 1 : 128 / R;
  // row and tile numbers are 32-bit
  if (R > 128 || p->Nq > (1 << 30) || c->N > (1 << 30) || heads * R > (1 << 24) ||
      heads * ((p->Nq + qn - 1) / qn) > (1 << 30) || R * p->Nq > UINT32_MAX ||
      heads * ((int64_t(c->N) + 127) / 128) > (1 << 30))
    return SA_ERR_UNSUPPORTED;
  *a = Attend8Args{};
  MaskedArgs& m = a->m;
  m.mask = {nullptr, nullptr, nullptr, p->lengths, 0, p->causal, p->Nq, c->N};
  m.qs = p->q;
  m.os = p->o;
  m.B = c->B;
  m.Hq = p->Hq;
  m.Hkv = c->Hkv;
  m.R = static_cast<int32_t>(R);
  m.Nq = p->Nq;
  m.Nk = c->N;
  m.d = c->d;
  m.out_fp32 = p->out_dtype == SA_OUT_FP32;
  m.total_rows = heads * R * p->Nq;
  a->scale_log2 = p->scale * 1.4426950408889634f;
  while ((1 << a->block_log2) < c->block) ++a->block_log2;
  if (!attend8_few(*a)) attend8_many_plan(a);
  return SA_OK;
}

// Partial results (fp32 rows), then their lse: each 256-byte aligned.
struct Parts {
  size_t o, lse;
};
Parts parts_of(const Attend8Args& a) {
  if (attend8_few(a) && attend8_whole(a)) return {0, 0};
  const size_t rows = attend8_few(a) ? (size_t(attend8_few_grid(a)) + size_t(a.m.B) * a.m.Hkv) * a.m.R * a.m.Nq
                                     : size_t(a.m.split_units) * a.m.splits * a.m.unit_rows;
  return {(rows * a.m.d * 4 + 255) / 256 * 256, (rows * 4 + 255) / 256 * 256};
}

}  // namespace

extern "C" {

size_t sparse_attn_forward_cache8_workspace_size(const sa_attend8* p, const sa_cache8* cache) {
  Attend8Args a;
  if (check_attend(p, cache, &a) != SA_OK) return 0;
  const Parts n = parts_of(a);
  return n.o + n.lse;
}

sa_status sparse_attn_forward_cache8(const sa_attend8* p, const sa_cache8* cache, const void* q, void* o, float* lse,
                                     int32_t* dev_status, void* workspace, size_t workspace_bytes, sa_stream_t stream) {
  Attend8Args a;
  sa_status st = check_attend(p, cache, &a);
  if (st != SA_OK) return st;
  MaskedArgs& m = a.m;
  Cache c;
  if ((st = check_cache(cache, false, &c)) != SA_OK) return st;
  const int esz = m.out_fp32 ? 4 : 2;
  View in{q, m.qs, m.B, m.Hq, m.Nq, 0}, out{o, m.os, m.B, m.Hq, m.Nq, 0};
  if (!check_view(q, &in.s, m.B, m.Hq, m.Nq, m.d, 2, false, false, &in.n) ||
      !check_view(o, &out.s, m.B, m.Hq, m.Nq, m.d, esz, true, false, &out.n) || !aligned(lse, 4) || !aligned(dev_status, 4))
    return SA_ERR_INVALID_ARG;
  m.qs = in.s;
  m.os = out.s;
  // Nothing that is written may share memory with anything else of the call, but o may be q's view: a row of q is
  // read ahead of the row of o that takes its place.
  const uint64_t nl = lse ? uint64_t(m.total_rows) * 4 : 0;
  const Parts n = parts_of(a);
  const size_t need = n.o + n.lse;
  if (need && (!workspace || !aligned(workspace, 256) || workspace_bytes < need)) return SA_ERR_INVALID_ARG;
  if (!(esz == 2 && same_view(in, out)) && (esz == 2 ? views_overlap(in, out, m.d, 2) : overlap(q, in.n, o, out.n)))
    return SA_ERR_INVALID_ARG;
  if (meets_cache(c, o, out.n)) return SA_ERR_INVALID_ARG;
  if (nl && (overlap(lse, nl, q, in.n) || overlap(lse, nl, o, out.n) || meets_cache(c, lse, nl))) return SA_ERR_INVALID_ARG;
  if (need && (overlap(workspace, need, q, in.n) || overlap(workspace, need, o, out.n) || meets_cache(c, workspace, need) ||
               (nl && overlap(workspace, need, lse, nl))))
    return SA_ERR_INVALID_ARG;
  int sms = 0;
  if ((st = device_info(&sms)) != SA_OK) return st;
  if (!cache_in_device(c) || !in_device_allocation(q, in.n) || !in_device_allocation(o, out.n) ||
      (nl && !in_device_allocation(lse, nl)) || (dev_status && !in_device_allocation(dev_status, 4)) ||
      (need && !in_device_allocation(workspace, need)) ||
      (p->lengths && !in_device_allocation(p->lengths, uint64_t(m.B) * 4)))
    return SA_ERR_INVALID_ARG;
  m.q = static_cast<const uint16_t*>(q);
  m.o = o;
  m.lse = lse;
  m.status = dev_status;
  m.ks = c.codes[0].s;
  m.vs = c.codes[1].s;
  a.k8 = static_cast<const uint8_t*>(c.codes[0].p);
  a.v8 = static_cast<const uint8_t*>(c.codes[1].p);
  a.k_scale = c.scales[0];
  a.v_scale = c.scales[1];
  a.k_scales = c.ss[0];
  a.v_scales = c.ss[1];
  if (need) {
    m.part_o = static_cast<float*>(workspace);
    m.part_lse = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + n.o);
  }
  NvtxRange range("sparse_attn_forward_cache8");
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return map_cuda(attend8_few(a) ? launch_attend8_few(a, s) : launch_attend8_many(a, s));
}

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
  if (n > (1 << 30) || int64_t(p->B) * p->Hkv * 2 * ((int64_t(n) * (p->d / 16) + 511) / 512) >= (int64_t(1) << 31))
    return SA_ERR_UNSUPPORTED;  // grid.x
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
