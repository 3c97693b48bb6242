// sa_rope.cuh — positions, angles and 16-byte pieces, shared by the rotation and the normalised rotation.
#pragma once

#include "sa_device.cuh"
#include "sa_internal.h"

namespace sa {

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

// Token n's position along each axis.
__device__ __forceinline__ void token_position(const RopeArgs& a, int b, int64_t n, int* p) {
  if (a.pos) {
    const int32_t* src = a.pos + b * a.pos_b + n * a.axes;
    for (int x = 0; x < a.axes; ++x) p[x] = __ldg(src + x);
  } else {
    grid_position(a, static_cast<uint32_t>(n), p);
#pragma unroll
    for (int x = 0; x < 3; ++x) p[x] += a.offset[x];
  }
}

// The two pieces of a row, of V values each, that lane c of its LANES has: their first
// elements.  HALF: pair i is elements (i, i + rot/2); pieces past the rotated part are
// taken two by two (returns false: they do not turn).  Else pair i is elements (2i, 2i + 1).
template <int V, bool HALF>
__device__ __forceinline__ bool lane_pieces(const RopeArgs& a, int c, int* e0, int* e1) {
  if (!HALF) {
    *e0 = c * V;
    *e1 = *e0 + a.d / 2;
    return true;
  }
  if (c * V < a.rot / 2) {
    *e0 = c * V;
    *e1 = *e0 + a.rot / 2;
    return true;
  }
  *e0 = a.rot + 2 * (c * V - a.rot / 2);
  *e1 = *e0 + V;
  return false;
}

// Cosines and sines of the lane's V pairs (1 and 0 for pairs past the rotated part).
template <int V, bool HALF>
__device__ __forceinline__ void lane_angles(const RopeArgs& a, const int* p, int e0, int e1, bool turns, float* cs, float* sn) {
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
}

// Turns the pairs of the two pieces f0 (at e0) and f1 (at e1).
template <int V, bool HALF>
__device__ __forceinline__ void turn_pieces(const RopeArgs& a, int e0, int e1, bool turns, const float* cs, const float* sn,
                                            float* f0, float* f1) {
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
}

}  // namespace sa
