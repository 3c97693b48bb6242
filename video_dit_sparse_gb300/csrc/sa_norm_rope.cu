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
#include <type_traits>

#include "sa_rope.cuh"
#include "sa_views.h"

namespace sa {

// Heads on their way in the gradient: this one and seven more (a power of two), 128 KB for the one block that an SM has.
// (24 + 24 heads x 16384 x 128, token-major: 97 us; four heads and two blocks an SM 110; the next head in registers 120.)
constexpr int kAhead = 8;

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

// A lane's piece of V values is V / 2 packed pairs of fp32.

// Both of the lane's pieces of a [d] vector (`none` where it is null).
template <int V>
__device__ __forceinline__ void load_vector(const void* p, bool wide, int e0, int e1, float none, uint64_t* v0, uint64_t* v1) {
#pragma unroll
  for (int i = 0; i < V; i += 2) {
    float f[4] = {none, none, none, none};
    const int at[4] = {e0 + i, e0 + i + 1, e1 + i, e1 + i + 1};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (p && wide) f[e] = __ldg(static_cast<const float*>(p) + at[e]);
      if (p && !wide) f[e] = __uint_as_float(uint32_t(__ldg(static_cast<const uint16_t*>(p) + at[e])) << 16);
    }
    v0[i / 2] = f2(f[0], f[1]);
    v1[i / 2] = f2(f[2], f[3]);
  }
}

template <int V>
__device__ __forceinline__ void unpack2(const uint4& u, uint64_t* v) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  if (V == 8) {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) v[i] = f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
  } else {
    v[0] = f2(__uint_as_float(w[0]), __uint_as_float(w[1]));
    v[1] = f2(__uint_as_float(w[2]), __uint_as_float(w[3]));
  }
}
template <int V>
__device__ __forceinline__ uint4 pack2(const uint64_t* v) {
  if (V == 8)
    return make_uint4(pack_bf16(f2lo(v[0]), f2hi(v[0])), pack_bf16(f2lo(v[1]), f2hi(v[1])),
                      pack_bf16(f2lo(v[V / 2 - 2]), f2hi(v[V / 2 - 2])), pack_bf16(f2lo(v[V / 2 - 1]), f2hi(v[V / 2 - 1])));
  return make_uint4(f2lo_bits(v[0]), f2hi_bits(v[0]), f2lo_bits(v[1]), f2hi_bits(v[1]));
}

// Cosines and sines as `turn` wants them: HALF: of the pairs (i, i + 1); else pair by pair, in both halves.
template <int V, bool HALF>
struct Angles {
  uint64_t cs[V / 2], sn[V / 2];
  __device__ __forceinline__ void load(const RopeArgs& a, int b, int64_t n, int e0, int e1, bool turns) {
    int p[3] = {0, 0, 0};
    token_position(a, b, n, p);
    float c[V], s[V];
    lane_angles<V, HALF>(a, p, e0, e1, turns, c, s);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      cs[i] = f2(c[2 * i], c[2 * i + 1]);
      sn[i] = f2(s[2 * i], s[2 * i + 1]);
    }
  }
  // Turns the two pieces; `part`: not all of a row turns (what does not is kept as it is).
  __device__ __forceinline__ void turn(const RopeArgs& a, int e0, int e1, bool turns, bool part, uint64_t* x0, uint64_t* x1) const {
    if (HALF) {
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        const uint64_t y0 = sub2(mul2(x0[i], cs[i]), mul2(x1[i], sn[i])), y1 = fma2(x0[i], sn[i], mul2(x1[i], cs[i]));
        x0[i] = turns ? y0 : x0[i];
        x1[i] = turns ? y1 : x1[i];
      }
      return;
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      uint64_t* x = k ? x1 : x0;
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {  // pair number i of the piece: angle i (k = 0) or V / 2 + i
        const int at = k * (V / 2) + i;
        const float c = at & 1 ? f2hi(cs[at / 2]) : f2lo(cs[at / 2]), s = at & 1 ? f2hi(sn[at / 2]) : f2lo(sn[at / 2]);
        const float u = f2lo(x[i]), v = f2hi(x[i]);
        const uint64_t y = f2(u * c - v * s, u * s + v * c);
        x[i] = part && (k ? e1 : e0) + 2 * i >= a.rot ? x[i] : y;
      }
    }
  }
};

// Sum over the LANES lanes of a row (every lane of the warp takes part).
template <int LANES>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = LANES / 2; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
__device__ __forceinline__ float both(uint64_t v) { return f2lo(v) + f2hi(v); }

// Takes the mean off (LAYER) and returns r.
template <int V, int LANES, bool LAYER>
__device__ __forceinline__ float normalise(uint64_t* v0, uint64_t* v1, float eps) {
  constexpr float kInv = 1.f / (2 * V * LANES);
  if (LAYER) {
    uint64_t s = add2(v0[0], v1[0]);
#pragma unroll
    for (int i = 1; i < V / 2; ++i) s = add2(s, add2(v0[i], v1[i]));
    const float mu = row_sum<LANES>(both(s)) * kInv;
    const uint64_t m = f2(mu, mu);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      v0[i] = sub2(v0[i], m);
      v1[i] = sub2(v1[i], m);
    }
  }
  uint64_t q = 0;
#pragma unroll
  for (int i = 0; i < V / 2; ++i) q = fma2(v0[i], v0[i], fma2(v1[i], v1[i], q));
  return rsqrtf(fmaf(row_sum<LANES>(both(q)), kInv, eps));
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
  // (Every lane takes part in the sums.  Those past the last token read the last row and use none of it: in place it may be
  // half written.  Returning early spills: 12 + 12 heads of 7040 tokens, pairs by halves, 18.7 -> 20.6 us.)
  const int64_t n = valid ? tok : r.N - 1;
  const int b = blockIdx.z;
  const int first = blockIdx.y * heads_per_block, last = min(first + heads_per_block, r.H[0] + r.H[1]);
  int e0, e1;
  const bool turns = lane_pieces<V, HALF>(r, c, &e0, &e1), part = r.rot < 2 * V * LANES;
  Angles<V, HALF> angles;
  angles.load(r, b, n, e0, e1, turns);
  constexpr int U = 4;  // heads in flight
#pragma unroll 1
  for (int s = 0; s < 2; ++s) {
    const int h0 = s ? max(first - r.H[0], 0) : first, h1 = s ? last - r.H[0] : min(last, r.H[0]);
    if (h0 >= h1) continue;
    uint64_t w0[V / 2], w1[V / 2], b0[V / 2], b1[V / 2];
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
          uint64_t v0[V / 2], v1[V / 2];
          unpack2<V>(u0[i], v0);
          unpack2<V>(u1[i], v1);
          const float k = normalise<V, LANES, LAYER>(v0, v1, a.eps);
          const uint64_t kk = f2(k, k);
#pragma unroll
          for (int e = 0; e < V / 2; ++e) {
            v0[e] = fma2(mul2(v0[e], kk), w0[e], b0[e]);
            v1[e] = fma2(mul2(v1[e], kk), w1[e], b1[e]);
          }
          angles.turn(r, e0, e1, turns, part, v0, v1);
          char* at = y + (h + i) * r.ys[s].h * kBytes;
          if (valid) {
            *reinterpret_cast<uint4*>(at + e0 * kBytes) = pack2<V>(v0);
            *reinterpret_cast<uint4*>(at + e1 * kBytes) = pack2<V>(v1);
          }
        }
    }
  }
}

// The gradient.  blockIdx.y: side.  A block takes every blocks[side]-th piece of work: 256 / LANES tokens of a batch
// entry, `run` heads of them.  BIAS: db is wanted.
template <int V, int LANES, bool HALF, bool LAYER, bool BIAS>
__global__ void __launch_bounds__(256, 1) sa_norm_rope_grad_kernel(const __grid_constant__ NormRopeArgs a) {
  constexpr int kTokens = 256 / LANES;
  constexpr int kBytes = V == 8 ? 2 : 4;
  constexpr int kRow = 2 * V * LANES;  // d
  constexpr float kInv = 1.f / kRow;
  __shared__ float sums[8][2][kRow];
  extern __shared__ uint4 ring[];  // [kAhead][x piece 0, 1, dy piece 0, 1][thread]
  const RopeArgs& r = a.r;
  const int s = blockIdx.y;
  if (static_cast<int>(blockIdx.x) >= a.blocks[s]) return;
  const int c = threadIdx.x % LANES, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int e0, e1;
  const bool turns = lane_pieces<V, HALF>(r, c, &e0, &e1), part_turns = r.rot < kRow;
  uint64_t w0[V / 2], w1[V / 2], dw0[V / 2], dw1[V / 2], db0[V / 2], db1[V / 2];
  load_vector<V>(a.w[s], a.wide, e0, e1, 1.f, w0, w1);
#pragma unroll
  for (int i = 0; i < V / 2; ++i) dw0[i] = dw1[i] = db0[i] = db1[i] = 0;
  const uint32_t tiles = (static_cast<uint32_t>(r.N) + kTokens - 1) / kTokens, runs = (r.H[s] + a.run[s] - 1) / a.run[s];
  const int64_t items = int64_t(tiles) * r.B * runs;
  for (int64_t item = blockIdx.x; item < items; item += a.blocks[s]) {
    const int64_t bt = item / runs;
    const int h0 = static_cast<int>(item - bt * runs) * a.run[s], h1 = min(h0 + a.run[s], r.H[s]);
    const int b = static_cast<int>(bt / tiles);
    const int64_t tok = (bt - int64_t(b) * tiles) * kTokens + threadIdx.x / LANES;
    const bool valid = tok < r.N;
    const int64_t n = valid ? tok : r.N - 1;
    const char* x = static_cast<const char*>(r.x[s]) + (b * r.xs[s].b + n * r.xs[s].n) * kBytes;
    const char* dy = static_cast<const char*>(a.g[s]) + (b * a.gs[s].b + n * a.gs[s].n) * kBytes;
    char* dx = static_cast<char*>(r.y[s]) + (b * r.ys[s].b + n * r.ys[s].n) * kBytes;
    // The thread's pieces of the next heads are on their way to places of its own in shared memory.
    // (Past the last token: zeros.  In place, the last row is being written by its own lanes.)
    const uint32_t bytes = valid ? 16 : 0;
    auto fetch = [&](int h) {
      if (h < h1) {
        const uint32_t to = smem_u32(ring + ((h & (kAhead - 1)) * 4) * 256 + threadIdx.x);
        const char* at = x + h * r.xs[s].h * kBytes;
        cp_async16(to, at + e0 * kBytes, bytes);
        cp_async16(to + 4096, at + e1 * kBytes, bytes);
        at = dy + h * a.gs[s].h * kBytes;
        cp_async16(to + 8192, at + e0 * kBytes, bytes);
        cp_async16(to + 12288, at + e1 * kBytes, bytes);
      }
      cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kAhead - 1; ++i) fetch(h0 + i);
    Angles<V, HALF> angles;
    angles.load(r, b, n, e0, e1, turns);  // (r.inverse is set: R^-1)
    for (int h = h0; h < h1; ++h) {
      uint64_t v0[V / 2], v1[V / 2], g0[V / 2], g1[V / 2];
      fetch(h + kAhead - 1);
      cp_async_wait<kAhead - 1>();
      const uint4* here = ring + ((h & (kAhead - 1)) * 4) * 256 + threadIdx.x;
      unpack2<V>(here[0], v0);
      unpack2<V>(here[256], v1);
      unpack2<V>(here[512], g0);
      unpack2<V>(here[768], g1);
      const float k = normalise<V, LANES, LAYER>(v0, v1, a.eps);
      const uint64_t kk = f2(k, k);
      angles.turn(r, e0, e1, turns, part_turns, g0, g1);
      uint64_t hn = 0, hs = 0;
#pragma unroll
      for (int e = 0; e < V / 2; ++e) {
        v0[e] = mul2(v0[e], kk);
        v1[e] = mul2(v1[e], kk);
        if (valid) {
          dw0[e] = fma2(g0[e], v0[e], dw0[e]);
          dw1[e] = fma2(g1[e], v1[e], dw1[e]);
          if (BIAS) {
            db0[e] = add2(g0[e], db0[e]);
            db1[e] = add2(g1[e], db1[e]);
          }
        }
        g0[e] = mul2(g0[e], w0[e]);
        g1[e] = mul2(g1[e], w1[e]);
        hn = fma2(g0[e], v0[e], fma2(g1[e], v1[e], hn));
        if (LAYER) hs = add2(hs, add2(g0[e], g1[e]));
      }
      const float mn = -row_sum<LANES>(both(hn)) * kInv, ms = LAYER ? row_sum<LANES>(both(hs)) * kInv : 0.f;
      const uint64_t mn2 = f2(mn, mn), ms2 = f2(ms, ms);
#pragma unroll
      for (int e = 0; e < V / 2; ++e) {
        uint64_t y0 = fma2(mn2, v0[e], g0[e]), y1 = fma2(mn2, v1[e], g1[e]);
        if (LAYER) y0 = sub2(y0, ms2), y1 = sub2(y1, ms2);
        v0[e] = mul2(kk, y0);
        v1[e] = mul2(kk, y1);
      }
      char* at = dx + h * r.ys[s].h * kBytes;
      if (valid) {
        *reinterpret_cast<uint4*>(at + e0 * kBytes) = pack2<V>(v0);
        *reinterpret_cast<uint4*>(at + e1 * kBytes) = pack2<V>(v1);
      }
    }
  }
  cp_async_wait<0>();
  if (!a.dw[s] && !a.db[s]) return;
  let_next_kernel_start();
  // the warp's rows, then the block's warps
  auto fold = [&](float v) -> float {
#pragma unroll
    for (int o = 16; o >= LANES; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  };
#pragma unroll
  for (int i = 0; i < V; ++i) {
    auto value = [&](const uint64_t* v) -> float { return fold(i & 1 ? f2hi(v[i / 2]) : f2lo(v[i / 2])); };
    const float v[4] = {value(dw0), value(dw1), BIAS ? value(db0) : 0.f, BIAS ? value(db1) : 0.f};
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

// Blocks of each side: one an SM (of a GB300, whatever the device) for both sides together, by their heads, and no more
// than there is work for.  Runs of heads as long as that leaves work for all of them.
void grad_plan(NormRopeArgs* a) {
  const RopeArgs& r = a->r;
  const int tokens = r.fp32 ? (r.d == 128 ? 16 : 32) : (r.d == 128 ? 32 : 64);
  const int64_t tiles = (int64_t(r.N) + tokens - 1) / tokens * r.B;
  for (int s = 0; s < 2; ++s) {
    const int H = r.H[s];
    a->run[s] = 1;
    a->blocks[s] = 0;
    if (!H) continue;
    const int64_t share = std::max<int64_t>(1, int64_t(kSms) * H / (r.H[0] + r.H[1]));
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
  const bool bias = a.db[0] || a.db[1];
  constexpr int kSmem = kAhead * 4 * 256 * 16;
  cudaError_t e = cudaSuccess;
  auto go = [&](auto half, auto lay) {
    constexpr bool kHalf = decltype(half)::value, kLayer = decltype(lay)::value;
    auto kern = bias ? sa_norm_rope_grad_kernel<V, LANES, kHalf, kLayer, true> : sa_norm_rope_grad_kernel<V, LANES, kHalf, kLayer, false>;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e == cudaSuccess) kern<<<grid, 256, kSmem, st>>>(a);
  };
  if (a.r.half)
    layer ? go(std::true_type(), std::true_type()) : go(std::true_type(), std::false_type());
  else
    layer ? go(std::false_type(), std::true_type()) : go(std::false_type(), std::false_type());
  if (e == cudaSuccess) e = cudaGetLastError();
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

// Workspace of the gradient: the blocks' sums.
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
  sa::grad_plan(&a);
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
  grad_plan(&a);
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
