// sa_norm_rope.cu — every head's row normalised and rotated by its position in one pass, and the gradient of that.
//
// For a row x of d values (mu = 0 for SA_NORM_RMS, the row's mean for SA_NORM_LAYER):
//     r = 1 / sqrt(mean (x - mu)^2 + eps),  n = (x - mu) r,  y = R (n w + b)
// with R the rotation of sa_rope.cu.  The gradient, with g = R^-1 dy and h = g w:
//     dx = r (h - n mean(h n) - [layer: mean h]),  dw = sum over rows of g n,  db = sum of g.
// r is worked out again from x, which the gradient needs in any case; nothing is kept from the forward pass.
// Values are fp32 from the load to the one rounding at the store; the mean is taken off before the squares are
// summed (their difference would cancel for rows far off centre).
//
// Both are bound by HBM.  As in the rotation, a row is 4 to 16 lanes of two 16-byte pieces each, a row's sums are
// three or four shuffles, and a thread keeps its token's cosines and sines for a run of heads.
//
// dw and db sum over all rows of all heads: each thread of a fixed grid adds up its columns over the rows that it is
// given, a block adds its threads, and a second kernel the blocks, all in a fixed order: the same inputs give the
// same bits.
#include <cmath>

#include "sa_rope.cuh"
#include "sa_views.h"

namespace sa {

struct NormRopeArgs {
  RopeArgs r;           // x: inputs, y: outputs (the gradient's dx)
  const void* g[2];     // the gradient's dy
  sa_strides gs[2];
  const void* w[2];     // [d] or null
  const void* b[2];     // [d] or null
  float* dw[2];         // [d] or null
  float* db[2];
  float* part;          // [blocks][dw | db][d], side 0's blocks and then side 1's
  int32_t blocks[2];    // of each side
  int32_t run[2];       // heads a block takes at a time
  float eps;
  int32_t wide;         // weights and shifts are fp32 (else bf16)
};

namespace {

// The lane's 2 V values of a [d] vector (`none` where it is null).
template <int V>
__device__ __forceinline__ void load_vector(const void* p, bool wide, int e0, int e1, float none, float* f0, float* f1) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    f0[i] = f1[i] = none;
    if (p && wide) {
      f0[i] = __ldg(static_cast<const float*>(p) + e0 + i);
      f1[i] = __ldg(static_cast<const float*>(p) + e1 + i);
    } else if (p) {
      f0[i] = __uint_as_float(uint32_t(__ldg(static_cast<const uint16_t*>(p) + e0 + i)) << 16);
      f1[i] = __uint_as_float(uint32_t(__ldg(static_cast<const uint16_t*>(p) + e1 + i)) << 16);
    }
  }
}

// Sum over the LANES lanes of a row (every lane of the warp takes part).
template <int LANES>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = LANES / 2; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Takes the mean off (LAYER) and returns r.
template <int V, int LANES, bool LAYER>
__device__ __forceinline__ float normalise(float* f0, float* f1, float eps) {
  constexpr float kInv = 1.f / (2 * V * LANES);
  if (LAYER) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) s += f0[i] + f1[i];
    const float mu = row_sum<LANES>(s) * kInv;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      f0[i] -= mu;
      f1[i] -= mu;
    }
  }
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) q = fmaf(f0[i], f0[i], fmaf(f1[i], f1[i], q));
  return rsqrtf(fmaf(row_sum<LANES>(q), kInv, eps));
}

}  // namespace

// V values per 16-byte piece (8: bf16, 4: fp32), LANES threads per row.
template <int V, int LANES, bool HALF, bool LAYER>
__global__ void __launch_bounds__(256, 2) sa_norm_rope_kernel(const __grid_constant__ NormRopeArgs a, int heads_per_block) {
  constexpr int kTokens = 256 / LANES;
  constexpr int kBytes = V == 8 ? 2 : 4;
  const RopeArgs& r = a.r;
  const int c = threadIdx.x % LANES;
  const int64_t tok = int64_t(blockIdx.x) * kTokens + threadIdx.x / LANES;
  const bool valid = tok < r.N;
  const int64_t n = valid ? tok : r.N - 1;  // (every lane takes part in the sums)
  const int b = blockIdx.z;
  const int first = blockIdx.y * heads_per_block, last = min(first + heads_per_block, r.H[0] + r.H[1]);
  int p[3] = {0, 0, 0};
  token_position(r, b, n, p);
  int e0, e1;
  const bool turns = lane_pieces<V, HALF>(r, c, &e0, &e1);
  float cs[V], sn[V];
  lane_angles<V, HALF>(r, p, e0, e1, turns, cs, sn);
  constexpr int U = 4;  // heads in flight
#pragma unroll 1
  for (int s = 0; s < 2; ++s) {
    const int h0 = s ? max(first - r.H[0], 0) : first, h1 = s ? last - r.H[0] : min(last, r.H[0]);
    if (h0 >= h1) continue;
    float w0[V], w1[V], b0[V], b1[V];
    load_vector<V>(a.w[s], a.wide, e0, e1, 1.f, w0, w1);
    load_vector<V>(a.b[s], a.wide, e0, e1, 0.f, b0, b1);
    const char* x = static_cast<const char*>(r.x[s]) + (b * r.xs[s].b + n * r.xs[s].n) * kBytes;
    char* y = static_cast<char*>(r.y[s]) + (b * r.ys[s].b + n * r.ys[s].n) * kBytes;
    for (int h = h0; h < h1; h += U) {
      uint4 u0[U], u1[U];
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (h + i < h1) {
          const char* at = x + (h + i) * r.xs[s].h * kBytes;
          u0[i] = *reinterpret_cast<const uint4*>(at + e0 * kBytes);
          u1[i] = *reinterpret_cast<const uint4*>(at + e1 * kBytes);
        }
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (h + i < h1) {
          float f0[V], f1[V];
          unpack<V>(u0[i], f0);
          unpack<V>(u1[i], f1);
          const float k = normalise<V, LANES, LAYER>(f0, f1, a.eps);
#pragma unroll
          for (int e = 0; e < V; ++e) {
            f0[e] = fmaf(f0[e] * k, w0[e], b0[e]);
            f1[e] = fmaf(f1[e] * k, w1[e], b1[e]);
          }
          turn_pieces<V, HALF>(r, e0, e1, turns, cs, sn, f0, f1);
          char* at = y + (h + i) * r.ys[s].h * kBytes;
          if (valid) {
            *reinterpret_cast<uint4*>(at + e0 * kBytes) = pack<V>(f0);
            *reinterpret_cast<uint4*>(at + e1 * kBytes) = pack<V>(f1);
          }
        }
    }
  }
}

// The gradient.  blockIdx.y: side.  A block takes every gridDim.x-th piece of work: 256 / LANES tokens of a batch
// entry, `run` heads of them.
template <int V, int LANES, bool HALF, bool LAYER>
__global__ void __launch_bounds__(256, 2) sa_norm_rope_grad_kernel(const __grid_constant__ NormRopeArgs a) {
  constexpr int kTokens = 256 / LANES;
  constexpr int kBytes = V == 8 ? 2 : 4;
  constexpr int kRow = 2 * V * LANES;  // d
  constexpr float kInv = 1.f / kRow;
  __shared__ float sums[8][2][kRow];
  const RopeArgs& r = a.r;
  const int s = blockIdx.y;
  if (static_cast<int>(blockIdx.x) >= a.blocks[s]) return;
  const int c = threadIdx.x % LANES, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int e0, e1;
  const bool turns = lane_pieces<V, HALF>(r, c, &e0, &e1);
  float w0[V], w1[V], dw0[V], dw1[V], db0[V], db1[V];
  load_vector<V>(a.w[s], a.wide, e0, e1, 1.f, w0, w1);
#pragma unroll
  for (int i = 0; i < V; ++i) dw0[i] = dw1[i] = db0[i] = db1[i] = 0.f;
  const bool sum_w = a.dw[s] != nullptr, sum_b = a.db[s] != nullptr;
  const uint32_t tiles = (static_cast<uint32_t>(r.N) + kTokens - 1) / kTokens, runs = (r.H[s] + a.run[s] - 1) / a.run[s];
  const int64_t items = int64_t(tiles) * r.B * runs;
  for (int64_t item = blockIdx.x; item < items; item += a.blocks[s]) {
    const int64_t bt = item / runs;
    const int h0 = static_cast<int>(item - bt * runs) * a.run[s], h1 = min(h0 + a.run[s], r.H[s]);
    const int b = static_cast<int>(bt / tiles);
    const int64_t tok = (bt - int64_t(b) * tiles) * kTokens + threadIdx.x / LANES;
    const bool valid = tok < r.N;
    const int64_t n = valid ? tok : r.N - 1;
    int p[3] = {0, 0, 0};
    token_position(r, b, n, p);
    float cs[V], sn[V];
    lane_angles<V, HALF>(r, p, e0, e1, turns, cs, sn);  // (r.inverse is set: R^-1)
    const char* x = static_cast<const char*>(r.x[s]) + (b * r.xs[s].b + n * r.xs[s].n) * kBytes;
    const char* dy = static_cast<const char*>(a.g[s]) + (b * a.gs[s].b + n * a.gs[s].n) * kBytes;
    char* dx = static_cast<char*>(r.y[s]) + (b * r.ys[s].b + n * r.ys[s].n) * kBytes;
    constexpr int U = 2;  // heads in flight
    for (int h = h0; h < h1; h += U) {
      uint4 ux0[U], ux1[U], ug0[U], ug1[U];
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (h + i < h1) {
          const char* at = x + (h + i) * r.xs[s].h * kBytes;
          ux0[i] = *reinterpret_cast<const uint4*>(at + e0 * kBytes);
          ux1[i] = *reinterpret_cast<const uint4*>(at + e1 * kBytes);
          at = dy + (h + i) * a.gs[s].h * kBytes;
          ug0[i] = *reinterpret_cast<const uint4*>(at + e0 * kBytes);
          ug1[i] = *reinterpret_cast<const uint4*>(at + e1 * kBytes);
        }
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (h + i < h1) {
          float f0[V], f1[V], g0[V], g1[V];
          unpack<V>(ux0[i], f0);
          unpack<V>(ux1[i], f1);
          const float k = normalise<V, LANES, LAYER>(f0, f1, a.eps);
          unpack<V>(ug0[i], g0);
          unpack<V>(ug1[i], g1);
          turn_pieces<V, HALF>(r, e0, e1, turns, cs, sn, g0, g1);
          float hn = 0.f, hs = 0.f;
#pragma unroll
          for (int e = 0; e < V; ++e) {
            f0[e] *= k;
            f1[e] *= k;
            if (valid) {  // (a row that is there twice counts once)
              dw0[e] = fmaf(g0[e], f0[e], dw0[e]);
              dw1[e] = fmaf(g1[e], f1[e], dw1[e]);
              db0[e] += g0[e];
              db1[e] += g1[e];
            }
            g0[e] *= w0[e];
            g1[e] *= w1[e];
            hn = fmaf(g0[e], f0[e], fmaf(g1[e], f1[e], hn));
            if (LAYER) hs += g0[e] + g1[e];
          }
          hn = row_sum<LANES>(hn) * kInv;
          if (LAYER) hs = row_sum<LANES>(hs) * kInv;
#pragma unroll
          for (int e = 0; e < V; ++e) {
            f0[e] = k * (fmaf(-hn, f0[e], g0[e]) - hs);
            f1[e] = k * (fmaf(-hn, f1[e], g1[e]) - hs);
          }
          char* at = dx + (h + i) * r.ys[s].h * kBytes;
          if (valid) {
            *reinterpret_cast<uint4*>(at + e0 * kBytes) = pack<V>(f0);
            *reinterpret_cast<uint4*>(at + e1 * kBytes) = pack<V>(f1);
          }
        }
    }
  }
  if (!sum_w && !sum_b) return;
  let_next_kernel_start();
  // the warp's rows, then the block's warps
  auto fold = [&](float v) -> float {
#pragma unroll
    for (int o = 16; o >= LANES; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  };
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float v[4] = {fold(dw0[i]), fold(dw1[i]), fold(db0[i]), fold(db1[i])};
    if (lane < LANES) {
      sums[warp][0][e0 + i] = v[0];
      sums[warp][0][e1 + i] = v[1];
      sums[warp][1][e0 + i] = v[2];
      sums[warp][1][e1 + i] = v[3];
    }
  }
  __syncthreads();
  float* part = a.part + (int64_t(s ? a.blocks[0] : 0) + blockIdx.x) * (2 * kRow);
  for (int i = threadIdx.x; i < 2 * kRow; i += 256) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) v += sums[w][i / kRow][i % kRow];
    part[i] = v;
  }
}

// dw and db from the blocks' sums.  blockIdx.y: side, blockIdx.x: 0 dw, 1 db; eight threads a column.
template <int D>
__global__ void __launch_bounds__(8 * D) sa_norm_rope_sum_kernel(const __grid_constant__ NormRopeArgs a) {
  __shared__ float sums[8][D];
  wait_for_earlier_kernel();
  const int s = blockIdx.y, what = blockIdx.x, c = threadIdx.x % D, k = threadIdx.x / D;
  float* out = what ? a.db[s] : a.dw[s];
  if (!out) return;
  const float* part = a.part + int64_t(s ? a.blocks[0] : 0) * (2 * D) + what * D + c;
  float v = 0.f;
#pragma unroll 8
  for (int i = k; i < a.blocks[s]; i += 8) v += part[int64_t(i) * (2 * D)];
  sums[k][c] = v;
  __syncthreads();
  if (k) return;
#pragma unroll
  for (int i = 1; i < 8; ++i) v += sums[i][c];
  out[c] = v;
}

namespace {

template <int V, int LANES>
cudaError_t launch_n(const NormRopeArgs& a, bool layer, int num_sms, cudaStream_t st) {
  constexpr int kTokens = 256 / LANES;
  const RopeArgs& r = a.r;
  const int64_t tiles = (int64_t(r.N) + kTokens - 1) / kTokens;
  const int heads = r.H[0] + r.H[1];
  // (runs of heads as in the rotation)
  int run = heads;
  while (run > 4 && tiles * r.B * ((heads + run - 1) / run) < int64_t(num_sms) * 2) run = (run + 1) / 2;
  if (tiles * r.B * heads < num_sms * 4) run = 1;
  const dim3 grid(static_cast<unsigned>(tiles), (heads + run - 1) / run, r.B);
  if (r.half)
    (layer ? sa_norm_rope_kernel<V, LANES, true, true> : sa_norm_rope_kernel<V, LANES, true, false>)<<<grid, 256, 0, st>>>(a, run);
  else
    (layer ? sa_norm_rope_kernel<V, LANES, false, true> : sa_norm_rope_kernel<V, LANES, false, false>)<<<grid, 256, 0, st>>>(a, run);
  return cudaGetLastError();
}

// Blocks of each side: two an SM for both sides together, by their heads, and no more than there is work for.
// Runs of heads as long as that leaves work for all of them.
void grad_plan(NormRopeArgs* a, int num_sms) {
  const RopeArgs& r = a->r;
  const int tokens = r.fp32 ? (r.d == 128 ? 16 : 32) : (r.d == 128 ? 32 : 64);
  const int64_t tiles = (int64_t(r.N) + tokens - 1) / tokens * r.B;
  for (int s = 0; s < 2; ++s) {
    const int H = r.H[s];
    a->run[s] = 1;
    a->blocks[s] = 0;
    if (!H) continue;
    const int64_t share = std::max<int64_t>(1, int64_t(num_sms) * 2 * H / (r.H[0] + r.H[1]));
    int run = H;
    while (run > 1 && tiles * ((H + run - 1) / run) < share) run = (run + 1) / 2;
    a->run[s] = run;
    a->blocks[s] = static_cast<int32_t>(std::min<int64_t>(share, tiles * ((H + run - 1) / run)));
  }
}

template <int V, int LANES>
cudaError_t launch_g(const NormRopeArgs& a, bool layer, cudaStream_t st) {
  constexpr int D = 2 * V * LANES;
  const dim3 grid(std::max(a.blocks[0], a.blocks[1]), a.r.H[1] ? 2 : 1);
  if (a.r.half)
    (layer ? sa_norm_rope_grad_kernel<V, LANES, true, true> : sa_norm_rope_grad_kernel<V, LANES, true, false>)<<<grid, 256, 0, st>>>(a);
  else
    (layer ? sa_norm_rope_grad_kernel<V, LANES, false, true> : sa_norm_rope_grad_kernel<V, LANES, false, false>)<<<grid, 256, 0, st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !(a.dw[0] || a.dw[1] || a.db[0] || a.db[1])) return e;
  return launch_early(sa_norm_rope_sum_kernel<D>, dim3(2, grid.y), 8 * D, 0, st, a);
}

sa_status map_cuda(cudaError_t e) { return e == cudaSuccess ? SA_OK : SA_ERR_CUDA; }

// Options; fills the positions, eps and the weights' type.
sa_status check_norm(const sa_norm_rope* p, int32_t H0, int32_t H1, NormRopeArgs* a) {
  if (!p) return SA_ERR_INVALID_ARG;
  if (p->norm != SA_NORM_RMS && p->norm != SA_NORM_LAYER) return SA_ERR_INVALID_ARG;
  if (p->weight_dtype != SA_OUT_BF16 && p->weight_dtype != SA_OUT_FP32) return SA_ERR_INVALID_ARG;
  if (!std::isfinite(p->eps) || p->eps < 0.f || p->rope.inverse) return SA_ERR_INVALID_ARG;
  *a = NormRopeArgs{};
  a->eps = p->eps;
  a->wide = p->weight_dtype == SA_OUT_FP32;
  return check_rope(&p->rope, H0, H1, &a->r);
}

// Workspace of the gradient: the blocks' sums, for as many SMs as the GPU can have.
constexpr int kMostSms = 152;
size_t grad_workspace(const NormRopeArgs& a) { return size_t(a.blocks[0] + a.blocks[1]) * 2 * a.r.d * 4; }

}  // namespace

}  // namespace sa

extern "C" {

sa_status sparse_attn_norm_rope(const sa_norm_rope* p, const sa_norm_side* side0, const sa_norm_side* side1,
                                sa_stream_t stream) {
  using namespace sa;
  if (!side0) return SA_ERR_INVALID_ARG;
  NormRopeArgs a;
  sa_status st = check_norm(p, side0->H, side1 ? side1->H : 0, &a);
  if (st != SA_OK) return st;
  const sa_norm_side* sides[2] = {side0, side1};
  const sa_rope& q = p->rope;
  const int esz = a.r.fp32 ? 4 : 2, wsz = a.wide ? 4 : 2;
  View x[2] = {}, y[2] = {};
  for (int i = 0; i < 2; ++i) {
    a.r.H[i] = sides[i] ? sides[i]->H : 0;
    if (!a.r.H[i]) continue;
    const sa_norm_side& s = *sides[i];
    x[i] = {s.x, s.xs, q.B, s.H, q.N, 0};
    y[i] = {s.y, s.ys, q.B, s.H, q.N, 0};
    if (!check_view(s.x, &x[i].s, q.B, s.H, q.N, q.d, esz, false, true, &x[i].n) ||
        !check_view(s.y, &y[i].s, q.B, s.H, q.N, q.d, esz, true, false, &y[i].n) || !aligned(s.weight, wsz) ||
        !aligned(s.bias, wsz))
      return SA_ERR_INVALID_ARG;
    a.r.x[i] = s.x;
    a.r.y[i] = s.y;
    a.r.xs[i] = x[i].s;
    a.r.ys[i] = y[i].s;
    a.w[i] = s.weight;
    a.b[i] = s.bias;
    // in place (the same view) or apart: a row is read only by the threads that write it
    if (!same_view(x[i], y[i]) && views_overlap(x[i], y[i], q.d, esz)) return SA_ERR_INVALID_ARG;
  }
  for (int i = 0; i < 2; ++i) {
    if (!a.r.H[i]) continue;
    if (a.r.H[i ^ 1] && (views_overlap(y[i], x[i ^ 1], q.d, esz) || (i && views_overlap(y[0], y[1], q.d, esz))))
      return SA_ERR_INVALID_ARG;
    for (int j = 0; j < 2; ++j)
      for (const void* v : {a.w[j], a.b[j]})
        if (v && overlap(v, uint64_t(q.d) * wsz, y[i].p, y[i].n)) return SA_ERR_INVALID_ARG;
  }
  int sms = 0;
  if ((st = device_info(&sms)) != SA_OK) return st;
  for (int i = 0; i < 2; ++i)
    if (a.r.H[i] && (!in_device_allocation(x[i].p, x[i].n) || !in_device_allocation(y[i].p, y[i].n) ||
                     (a.w[i] && !in_device_allocation(a.w[i], uint64_t(q.d) * wsz)) ||
                     (a.b[i] && !in_device_allocation(a.b[i], uint64_t(q.d) * wsz))))
      return SA_ERR_INVALID_ARG;
  if (!rope_positions(&q)) return SA_ERR_INVALID_ARG;
  NvtxRange range("sparse_attn_norm_rope");
  const bool layer = p->norm == SA_NORM_LAYER;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (a.r.fp32) return map_cuda(q.d == 128 ? launch_n<4, 16>(a, layer, sms, s) : launch_n<4, 8>(a, layer, sms, s));
  return map_cuda(q.d == 128 ? launch_n<8, 8>(a, layer, sms, s) : launch_n<8, 4>(a, layer, sms, s));
}

size_t sparse_attn_norm_rope_backward_workspace_size(const sa_norm_rope* p, int32_t H0, int32_t H1) {
  sa::NormRopeArgs a;
  if (sa::check_norm(p, H0, H1, &a) != SA_OK) return 0;
  a.r.H[0] = H0;
  a.r.H[1] = H1;
  sa::grad_plan(&a, sa::kMostSms);
  return sa::grad_workspace(a);
}

sa_status sparse_attn_norm_rope_backward(const sa_norm_rope* p, const sa_norm_grad_side* side0,
                                         const sa_norm_grad_side* side1, void* workspace, size_t workspace_bytes,
                                         sa_stream_t stream) {
  using namespace sa;
  if (!side0) return SA_ERR_INVALID_ARG;
  NormRopeArgs a;
  sa_status st = check_norm(p, side0->H, side1 ? side1->H : 0, &a);
  if (st != SA_OK) return st;
  a.r.inverse = 1;
  const sa_norm_grad_side* sides[2] = {side0, side1};
  const sa_rope& q = p->rope;
  const int esz = a.r.fp32 ? 4 : 2, wsz = a.wide ? 4 : 2;
  const uint64_t wn = uint64_t(q.d) * wsz, dn = uint64_t(q.d) * 4;
  View x[2] = {}, g[2] = {}, y[2] = {};
  bool sums = false;
  for (int i = 0; i < 2; ++i) {
    a.r.H[i] = sides[i] ? sides[i]->H : 0;
    if (!a.r.H[i]) continue;
    const sa_norm_grad_side& s = *sides[i];
    x[i] = {s.x, s.xs, q.B, s.H, q.N, 0};
    g[i] = {s.dy, s.dys, q.B, s.H, q.N, 0};
    y[i] = {s.dx, s.dxs, q.B, s.H, q.N, 0};
    if (!check_view(s.x, &x[i].s, q.B, s.H, q.N, q.d, esz, false, true, &x[i].n) ||
        !check_view(s.dy, &g[i].s, q.B, s.H, q.N, q.d, esz, false, true, &g[i].n) ||
        !check_view(s.dx, &y[i].s, q.B, s.H, q.N, q.d, esz, true, false, &y[i].n) || !aligned(s.weight, wsz) ||
        !aligned(s.dweight, 4) || !aligned(s.dbias, 4))
      return SA_ERR_INVALID_ARG;
    a.r.x[i] = s.x;
    a.r.y[i] = s.dx;
    a.r.xs[i] = x[i].s;
    a.r.ys[i] = y[i].s;
    a.g[i] = s.dy;
    a.gs[i] = g[i].s;
    a.w[i] = s.weight;
    a.dw[i] = s.dweight;
    a.db[i] = s.dbias;
    sums |= s.dweight || s.dbias;
    if ((!same_view(x[i], y[i]) && views_overlap(x[i], y[i], q.d, esz)) ||
        (!same_view(g[i], y[i]) && views_overlap(g[i], y[i], q.d, esz)))
      return SA_ERR_INVALID_ARG;
  }
  grad_plan(&a, kMostSms);
  const size_t need = sums ? grad_workspace(a) : 0;
  if (need && (!workspace || !aligned(workspace, 256) || workspace_bytes < need)) return SA_ERR_INVALID_ARG;
  // Nothing that is written may share memory with anything else of the call.
  struct Span {
    const void* p;
    uint64_t n;
  };
  const Span flat[] = {{a.dw[0], dn}, {a.db[0], dn}, {a.dw[1], dn}, {a.db[1], dn}, {need ? workspace : nullptr, need}};
  for (int i = 0; i < 5; ++i) {
    if (!flat[i].p) continue;
    for (int j = 0; j < i; ++j)
      if (flat[j].p && overlap(flat[i].p, flat[i].n, flat[j].p, flat[j].n)) return SA_ERR_INVALID_ARG;
    for (int s = 0; s < 2; ++s) {
      if (!a.r.H[s]) continue;
      for (const View* v : {&x[s], &g[s], &y[s]})
        if (overlap(flat[i].p, flat[i].n, v->p, v->n)) return SA_ERR_INVALID_ARG;
      if (a.w[s] && overlap(flat[i].p, flat[i].n, a.w[s], wn)) return SA_ERR_INVALID_ARG;
    }
  }
  for (int i = 0; i < 2; ++i) {
    if (!a.r.H[i]) continue;
    for (int j = 0; j < 2; ++j)
      if (a.w[j] && overlap(a.w[j], wn, y[i].p, y[i].n)) return SA_ERR_INVALID_ARG;
    if (a.r.H[i ^ 1] && (views_overlap(y[i], x[i ^ 1], q.d, esz) || views_overlap(y[i], g[i ^ 1], q.d, esz) ||
                         (i && views_overlap(y[0], y[1], q.d, esz))))
      return SA_ERR_INVALID_ARG;
  }
  int sms = 0;
  if ((st = device_info(&sms)) != SA_OK) return st;
  for (int i = 0; i < 2; ++i)
    if (a.r.H[i] && (!in_device_allocation(x[i].p, x[i].n) || !in_device_allocation(g[i].p, g[i].n) ||
                     !in_device_allocation(y[i].p, y[i].n) || (a.w[i] && !in_device_allocation(a.w[i], wn)) ||
                     (a.dw[i] && !in_device_allocation(a.dw[i], dn)) || (a.db[i] && !in_device_allocation(a.db[i], dn))))
      return SA_ERR_INVALID_ARG;
  if (!rope_positions(&q) || (need && !in_device_allocation(workspace, need))) return SA_ERR_INVALID_ARG;
  a.part = static_cast<float*>(workspace);
  NvtxRange range("sparse_attn_norm_rope_backward");
  const bool layer = p->norm == SA_NORM_LAYER;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (a.r.fp32) return map_cuda(q.d == 128 ? launch_g<4, 16>(a, layer, s) : launch_g<4, 8>(a, layer, s));
  return map_cuda(q.d == 128 ? launch_g<8, 8>(a, layer, s) : launch_g<8, 4>(a, layer, s));
}

}  // extern "C"
