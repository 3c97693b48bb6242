// sa_rope.cu — rotary positions along up to three axes (time, height, width).
//
// Pair i of a row turns by t = p * f_i, where p is the token's position along
// the pair's axis:  (a, b) -> (a cos t - b sin t, a sin t + b cos t).  The
// gradient (and the way back) is the same rotation by -t.
//
// Angles.  p f_i reaches thousands of turns for far positions, where an fp32
// product keeps no digit of the fraction.  The host passes f_i / 2 pi as a
// 64-bit fixed-point fraction of a turn (below 2^-62 off, whatever f_i); p times
// that, modulo 2^64, is the fraction of a turn that p f_i ends on (positions are
// whole numbers), whose top 32 bits go to sincospi.  Error: 2^-30 of a half turn
// from the product at |p| = 2^31, 2^-31 from the bits left out and 2^-25 from the
// conversion to fp32: below 2^-24 of a half turn at any 32-bit position.
//
// The kernel is bound by HBM (each row is read and written once; 24 + 24 heads of
// 69120 rows of 128: 259 us, 97 % of the measured copy rate).  A thread
// owns the same two 16-byte pieces of a token's row in every head of its run,
// so one set of cosines and sines in registers serves them all; four heads'
// loads are in flight at a time.  Pieces c and c + half a row are a thread's
// two, so that eight (or four, sixteen) lanes read contiguous lines, and with
// the half-row pairing of a fully rotated row both partners are in the thread.
#include "sa_device.cuh"
#include "sa_internal.h"

namespace sa {

namespace {

// (t, h, w) of token n of the grid.
__device__ __forceinline__ void grid_position(const RopeArgs& a, uint32_t n, int* p) {
  const VoxArgs& g = a.vox;
  const uint32_t HW = g.Hh * g.W;
  if (!a.voxel_order) {
    const uint32_t t = n / HW, r = n - t * HW;
    p[0] = t;
    p[1] = r / g.W;
    p[2] = r - p[1] * g.W;
    return;
  }
  // voxels in raster order, tokens in raster order inside a voxel; all voxels
  // before the last along an axis are full
  const uint32_t ta = n / (g.vt * HW), r0 = n - ta * g.vt * HW;
  const uint32_t st = min(g.vt, g.T - ta * g.vt);
  const uint32_t ha = r0 / (st * g.vh * g.W), r1 = r0 - ha * st * g.vh * g.W;
  const uint32_t sh = min(g.vh, g.Hh - ha * g.vh);
  const uint32_t wa = r1 / (st * sh * g.vw), r2 = r1 - wa * st * sh * g.vw;
  const uint32_t sw = min(g.vw, g.W - wa * g.vw);
  const uint32_t t = r2 / (sh * sw), r3 = r2 - t * sh * sw, h = r3 / sw;
  p[0] = ta * g.vt + t;
  p[1] = ha * g.vh + h;
  p[2] = wa * g.vw + r3 - h * sw;
}

// 16 bytes as V values of fp32.
template <int V>
__device__ __forceinline__ void unpack(const uint4& u, float* f) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (V == 8) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    } else {
      f[i] = __uint_as_float(w[i]);
    }
  }
}
template <int V>
__device__ __forceinline__ uint4 pack(const float* f) {
  if (V == 8)
    return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
  return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}

}  // namespace

// V values per 16-byte piece (8: bf16, 4: fp32), LANES threads per row.
template <int V, int LANES, bool HALF>
__global__ void __launch_bounds__(256) sa_rope_kernel(const __grid_constant__ RopeArgs a, int heads_per_block) {
  constexpr int kTokens = 256 / LANES;
  constexpr int kBytes = V == 8 ? 2 : 4;
  const int c = threadIdx.x % LANES;
  const int64_t n = int64_t(blockIdx.x) * kTokens + threadIdx.x / LANES;
  const int b = blockIdx.z;
  const int h0 = blockIdx.y * heads_per_block;
  const int h1 = min(h0 + heads_per_block, a.H[0] + a.H[1]);
  if (n >= a.N) return;
  int p[3] = {0, 0, 0};
  if (a.pos) {
    const int32_t* src = a.pos + b * a.pos_b + n * a.axes;
    for (int x = 0; x < a.axes; ++x) p[x] = __ldg(src + x);
  } else {
    grid_position(a, static_cast<uint32_t>(n), p);
#pragma unroll
    for (int x = 0; x < 3; ++x) p[x] += a.offset[x];
  }
  // The thread's two pieces (first elements e0, e1) and its V pairs.  HALF:
  // pair i is elements (i, i + rot/2); pieces past the rotated part are copied
  // two by two.  Else pair i is elements (2i, 2i + 1).
  int e0, e1;
  bool turns = true;
  if (HALF) {
    if (c * V < a.rot / 2) {
      e0 = c * V;
      e1 = e0 + a.rot / 2;
    } else {
      e0 = a.rot + 2 * (c * V - a.rot / 2);
      e1 = e0 + V;
      turns = false;
    }
  } else {
    e0 = c * V;
    e1 = e0 + a.d / 2;
  }
  float cs[V], sn[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int pair = HALF ? e0 + i : (i < V / 2 ? e0 / 2 + i : e1 / 2 + i - V / 2);
    cs[i] = 1.f;
    sn[i] = 0.f;
    if (turns && pair < a.rot / 2) {
      const int pp = pair >= a.first[2] ? p[2] : pair >= a.first[1] ? p[1] : p[0];
      const uint64_t turn = static_cast<uint64_t>(static_cast<int64_t>(pp)) * a.turn[pair];
      const float x = static_cast<float>(static_cast<int32_t>(turn >> 32)) * 4.6566128730773926e-10f;  // 2^-31 half turns
      sincospif(x, &sn[i], &cs[i]);
      if (a.inverse) sn[i] = -sn[i];
    }
  }
  constexpr int U = 4;  // heads in flight
  for (int h = h0; h < h1; h += U) {
    uint4 u0[U], u1[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (h + i < h1) {
        const int s = h + i >= a.H[0];
        const int hh = h + i - (s ? a.H[0] : 0);
        const char* x = static_cast<const char*>(a.x[s]) +
                        (b * a.xs[s].b + hh * a.xs[s].h + n * a.xs[s].n) * kBytes;
        u0[i] = *reinterpret_cast<const uint4*>(x + e0 * kBytes);
        u1[i] = *reinterpret_cast<const uint4*>(x + e1 * kBytes);
      }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (h + i < h1) {
        float f0[V], f1[V];
        unpack<V>(u0[i], f0);
        unpack<V>(u1[i], f1);
        if (HALF) {
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float x0 = f0[e], x1 = f1[e];
            f0[e] = turns ? x0 * cs[e] - x1 * sn[e] : x0;
            f1[e] = turns ? x0 * sn[e] + x1 * cs[e] : x1;
          }
        } else {
          // (a pair past the rotated part has cos 1, sin 0: kept as it is
          // unless its partner is infinite, which the copy below avoids)
#pragma unroll
          for (int e = 0; e < V / 2; ++e) {
            const float x0 = f0[2 * e], x1 = f0[2 * e + 1], y0 = f1[2 * e], y1 = f1[2 * e + 1];
            f0[2 * e] = x0 * cs[e] - x1 * sn[e];
            f0[2 * e + 1] = x0 * sn[e] + x1 * cs[e];
            f1[2 * e] = y0 * cs[e + V / 2] - y1 * sn[e + V / 2];
            f1[2 * e + 1] = y0 * sn[e + V / 2] + y1 * cs[e + V / 2];
            if (e0 + 2 * e >= a.rot) f0[2 * e] = x0, f0[2 * e + 1] = x1;
            if (e1 + 2 * e >= a.rot) f1[2 * e] = y0, f1[2 * e + 1] = y1;
          }
        }
        const int s = h + i >= a.H[0];
        const int hh = h + i - (s ? a.H[0] : 0);
        char* y = static_cast<char*>(a.y[s]) + (b * a.ys[s].b + hh * a.ys[s].h + n * a.ys[s].n) * kBytes;
        *reinterpret_cast<uint4*>(y + e0 * kBytes) = pack<V>(f0);
        *reinterpret_cast<uint4*>(y + e1 * kBytes) = pack<V>(f1);
      }
    }
  }
}

template <int V, int LANES>
static cudaError_t launch_r(const RopeArgs& a, int num_sms, cudaStream_t st) {
  constexpr int kTokens = 256 / LANES;
  const int64_t tiles = (int64_t(a.N) + kTokens - 1) / kTokens;
  const int heads = a.H[0] + a.H[1];
  // Runs of heads as long as possible (the angles are worked out once a run)
  // while the grid still has two blocks for every SM (12 + 12 heads of 7040 tokens:
  // 12.0 us; with eight blocks for every SM 17.2, most of it angles).
  int run = heads;
  while (run > 4 && tiles * a.B * ((heads + run - 1) / run) < int64_t(num_sms) * 2) run = (run + 1) / 2;
  if (tiles * a.B * heads < num_sms * 4) run = 1;
  const dim3 grid(static_cast<unsigned>(tiles), (heads + run - 1) / run, a.B);
  if (a.half)
    sa_rope_kernel<V, LANES, true><<<grid, 256, 0, st>>>(a, run);
  else
    sa_rope_kernel<V, LANES, false><<<grid, 256, 0, st>>>(a, run);
  return cudaGetLastError();
}

cudaError_t launch_rope(const RopeArgs& a, int num_sms, cudaStream_t st) {
  if (a.fp32) return a.d == 128 ? launch_r<4, 16>(a, num_sms, st) : launch_r<4, 8>(a, num_sms, st);
  return a.d == 128 ? launch_r<8, 8>(a, num_sms, st) : launch_r<8, 4>(a, num_sms, st);
}

}  // namespace sa
