// sa_cache8.cu — a key-value cache in e4m3 codes with a scale for each head and block of tokens: new tokens in,
// tokens out.
//
// A value is code * scale.  A block's scale is a power of two, the least one that brings the block's largest
// magnitude to 448 or below: for a floating-point code that gives up nothing against scale = top / 448 but up to one
// binade at the bottom of its 16, dividing by it is exact, and a block whose scale grows when a larger token joins it
// moves its other codes by whole binades, so that only values next to e4m3's smallest are rounded a second time.
// Codes are rounded to nearest: off by at most 2^-4 of the value, 2^-10 of the scale at the bottom.
//
// Bound by HBM: 2 bytes read and 1 written for each new value.  A block of tokens is a run of threads with 64 values
// each, so that its largest magnitude is known before anything is written and each value is loaded once.
#include <algorithm>

#include "sa_device.cuh"
#include "sa_e4m3.cuh"
#include "sa_internal.h"

namespace sa {

namespace {

struct Tokens {
  int64_t lo, hi;  // tokens of the cache that a batch entry's call covers
};
__device__ __forceinline__ Tokens covered(const Cache8Args& a, int b) {
  const int64_t first = a.start ? __ldg(a.start + b) : a.start0;
  const int64_t n = a.counts ? min(max(__ldg(a.counts + b), 0), a.n) : a.n;
  return {max(first, int64_t(0)), min(first + n, int64_t(a.N))};
}

}  // namespace

// T = block d / 64 threads for a block of tokens; a.blocks: blocks that the call can touch in a head.
template <int T>
__global__ void __launch_bounds__(256) sa_cache8_append_kernel(const __grid_constant__ Cache8Args a) {
  constexpr int kItems = 256 / T, kWarps = T > 32 ? T / 32 : 1;
  __shared__ uint32_t tops[8];
  const int t = threadIdx.x % T, row16 = a.d / 8;  // 16-byte pieces of a new row
  const int64_t item = int64_t(blockIdx.x) * kItems + threadIdx.x / T, head2 = item / a.blocks;
  bool live = item < a.items;
  const int which = static_cast<int>(head2 & 1), h = static_cast<int>((head2 >> 1) % a.H), b = live ? static_cast<int>((head2 >> 1) / a.H) : 0;
  const Tokens tk = covered(a, b);
  const int64_t first = a.start ? __ldg(a.start + b) : a.start0;
  const int64_t j = tk.lo / a.block + (item - head2 * a.blocks);
  const int64_t t0 = j * a.block, t1 = min(t0 + a.block, int64_t(a.N));  // the block's tokens
  const int64_t w0 = max(t0, tk.lo), w1 = min(t1, tk.hi);                // those written
  live = live && w0 < w1;
  const char* x = static_cast<const char*>(a.x[which]) + (b * a.xs[which].b + h * a.xs[which].h) * 2;
  uint8_t* codes = a.codes[which] + b * a.cs[which].b + h * a.cs[which].h;
  float* scale = a.scales[which] + b * a.ss[which].b + h * a.ss[which].h + j;
  uint4 u[8];
  uint32_t top = 0;  // the largest finite magnitude's bits
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int p = t + i * T, r = p / row16;
    u[i] = make_uint4(0, 0, 0, 0);
    if (live && t0 + r >= w0 && t0 + r < w1)
      u[i] = *reinterpret_cast<const uint4*>(x + ((t0 + r - first) * a.xs[which].n + (p - r * row16) * 8) * 2);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t lo = (w[e] & 0x7FFFu) << 16, hi = w[e] & 0x7FFF0000u;
      top = max(top, lo < 0x7F800000u ? lo : 1u);  // (what is not finite is held as a NaN: the scale may not be 0)
      top = max(top, hi < 0x7F800000u ? hi : 1u);
    }
  }
#pragma unroll
  for (int o = (T < 32 ? T : 32) / 2; o; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (kWarps > 1) {
    if ((threadIdx.x & 31) == 0) tops[threadIdx.x >> 5] = top;
    __syncthreads();
    top = tops[threadIdx.x / T * kWarps];
#pragma unroll
    for (int i = 1; i < kWarps; ++i) top = max(top, tops[threadIdx.x / T * kWarps + i]);
  }
  const bool whole = w0 == t0 && w1 == t1;
  const float had = live ? held_scale(*scale) : 0.f, old = whole ? 0.f : had;
  const float s = fmaxf(old, scale_for(__uint_as_float(top)));
  __syncthreads();  // (every thread has read the old scale)
  if (!live) return;
  const uint32_t sb = __float_as_uint(s);
  // a power of two is divided by exactly; a scale that the caller brought along need not be one
  const bool two = (sb & 0x7FFFFFu) == 0 && sb >= 0x00800000u && sb < 0x7E800000u;
  const float inv = two ? __uint_as_float(0x7F000000u - sb) : 0.f;
  auto code = [&](float lo, float hi) -> uint32_t {
    if (s != 0.f) {  // (else all are zeros)
      lo = fabsf(lo) <= 3.4028234663852886e38f ? (two ? lo * inv : __fdiv_rn(lo, s)) : __uint_as_float(0x7FC00000u);
      hi = fabsf(hi) <= 3.4028234663852886e38f ? (two ? hi * inv : __fdiv_rn(hi, s)) : __uint_as_float(0x7FC00000u);
    }
    return encode2(lo, hi);
  };
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int p = t + i * T, r = p / row16;
    const int64_t at = (t0 + r) * a.cs[which].n + (p - r * row16) * 8;
    if (t0 + r >= w0 && t0 + r < w1) {
      const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
      uint32_t c[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) c[e] = code(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xFFFF0000u));
      *reinterpret_cast<uint2*>(codes + at) = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
    } else if (t0 + r < t1 && s != old) {  // the block's other tokens keep their values
      const uint2 had8 = *reinterpret_cast<const uint2*>(codes + at);
      const uint32_t w[4] = {had8.x & 0xFFFFu, had8.x >> 16, had8.y & 0xFFFFu, had8.y >> 16};
      uint32_t c[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t f = old == 0.f ? 0u : decode2(w[e]);
        c[e] = code(half_lo(f) * old, half_hi(f) * old);
      }
      *reinterpret_cast<uint2*>(codes + at) = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
    }
  }
  if (t == 0) *scale = s;
}

// Tokens first[b] .. first[b] + n - 1 of every head as bf16 (exact where the scale is a power of two) or fp32 values;
// 0 where the cache has no such token.  A thread takes 16 codes.
template <bool WIDE>
__global__ void __launch_bounds__(256) sa_cache8_read_kernel(const __grid_constant__ Cache8Args a) {
  const int pieces = a.d / 16;
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x, row = i / pieces, head2 = row / a.n;
  if (i >= a.items) return;
  const int c = static_cast<int>(i - row * pieces);
  const int64_t at = row - head2 * a.n;
  int which = static_cast<int>(head2 & 1);
  int64_t bh = head2 >> 1;
  if (!a.y[0] || !a.y[1]) {
    which = a.y[0] ? 0 : 1;
    bh = head2;
  }
  const int h = static_cast<int>(bh % a.H), b = static_cast<int>(bh / a.H);
  const int64_t tok = (a.start ? __ldg(a.start + b) : a.start0) + at;
  uint4 u = make_uint4(0, 0, 0, 0);
  float s = 0.f;
  if (tok >= 0 && tok < a.N) {
    u = *reinterpret_cast<const uint4*>(a.codes[which] + b * a.cs[which].b + h * a.cs[which].h + tok * a.cs[which].n + c * 16);
    s = held_scale(a.scales[which][b * a.ss[which].b + h * a.ss[which].h + tok / a.block]);
  }
  if (s == 0.f) u = make_uint4(0, 0, 0, 0);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  float f[16];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t lo = decode2(w[e] & 0xFFFFu), hi = decode2(w[e] >> 16);
    f[4 * e] = half_lo(lo) * s;
    f[4 * e + 1] = half_hi(lo) * s;
    f[4 * e + 2] = half_lo(hi) * s;
    f[4 * e + 3] = half_hi(hi) * s;
  }
  char* y = static_cast<char*>(a.y[which]) +
            (b * a.xs[which].b + h * a.xs[which].h + at * a.xs[which].n + c * 16) * (WIDE ? 4 : 2);
  uint4* out = reinterpret_cast<uint4*>(y);
  if (WIDE) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      out[e] = make_uint4(__float_as_uint(f[4 * e]), __float_as_uint(f[4 * e + 1]), __float_as_uint(f[4 * e + 2]),
                          __float_as_uint(f[4 * e + 3]));
  } else {
#pragma unroll
    for (int e = 0; e < 2; ++e)
      out[e] = make_uint4(pack_bf16(f[8 * e], f[8 * e + 1]), pack_bf16(f[8 * e + 2], f[8 * e + 3]),
                          pack_bf16(f[8 * e + 4], f[8 * e + 5]), pack_bf16(f[8 * e + 6], f[8 * e + 7]));
  }
}

cudaError_t launch_cache8_append(Cache8Args a, cudaStream_t st) {
  // blocks that n tokens can touch, wherever they start
  a.blocks = static_cast<int32_t>(std::min<int64_t>((int64_t(a.N) + a.block - 1) / a.block, (int64_t(a.n) + a.block - 2) / a.block + 1));
  a.items = int64_t(a.B) * a.H * 2 * a.blocks;
  const int T = a.block * a.d / 64;
  const unsigned grid = static_cast<unsigned>((a.items + 256 / T - 1) / (256 / T));
  switch (T) {
    case 16: sa_cache8_append_kernel<16><<<grid, 256, 0, st>>>(a); break;
    case 32: sa_cache8_append_kernel<32><<<grid, 256, 0, st>>>(a); break;
    case 64: sa_cache8_append_kernel<64><<<grid, 256, 0, st>>>(a); break;
    case 128: sa_cache8_append_kernel<128><<<grid, 256, 0, st>>>(a); break;
    default: sa_cache8_append_kernel<256><<<grid, 256, 0, st>>>(a);
  }
  return cudaGetLastError();
}

cudaError_t launch_cache8_read(Cache8Args a, bool wide, cudaStream_t st) {
  a.items = int64_t(a.B) * a.H * (a.y[0] && a.y[1] ? 2 : 1) * a.n * (a.d / 16);
  const unsigned grid = static_cast<unsigned>((a.items + 255) / 256);
  if (wide)
    sa_cache8_read_kernel<true><<<grid, 256, 0, st>>>(a);
  else
    sa_cache8_read_kernel<false><<<grid, 256, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace sa
