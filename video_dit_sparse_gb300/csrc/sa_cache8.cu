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

// The larger of each half, as unsigned 16-bit numbers.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

}  // namespace

// T = block d / 64 threads for a block of tokens, ROW of them (d / 8) side by side in a token's row: a thread has the
// same eight columns of every (block / 8)-th token.  a.blocks: blocks that the call can touch in a head.
template <int T, int ROW>
__global__ void __launch_bounds__(256, 4) sa_cache8_append_kernel(const __grid_constant__ Cache8Args a) {
  constexpr int kItems = 256 / T, kWarps = T > 32 ? T / 32 : 1, kStep = T / ROW;  // kStep: block / 8
  constexpr int kBlock = 8 * kStep;
  __shared__ uint32_t tops[8];
  const int t = threadIdx.x % T, r0 = t / ROW, col = t % ROW * 8;
  const uint32_t item = blockIdx.x * kItems + threadIdx.x / T, head2 = item / a.blocks;
  bool live = item < a.items;
  const int which = static_cast<int>(head2 & 1), bh = live ? static_cast<int>(head2 >> 1) : 0, b = bh / a.H, h = bh - b * a.H;
  const int64_t first = a.start ? __ldg(a.start + b) : a.start0;
  const Tokens tk = covered(a, b);
  const int64_t j = tk.lo / kBlock + (item - head2 * a.blocks), t0 = j * kBlock;  // the block and its first token
  const int64_t end = min(t0 + kBlock, int64_t(a.N)), w0 = max(t0, tk.lo), w1 = min(end, tk.hi);
  live = live && w0 < w1;
  // its tokens, and those written, as rows of the block
  const int rows = static_cast<int>(end - t0), lo = live ? static_cast<int>(w0 - t0) : 0, hi = live ? static_cast<int>(w1 - t0) : 0;
  const char* x = static_cast<const char*>(a.x[which]) +
                  (b * a.xs[which].b + h * a.xs[which].h + (t0 + r0 - first) * a.xs[which].n + col) * 2;
  const int64_t xstep = a.xs[which].n * (2 * kStep), cstep = a.cs[which].n * kStep;
  uint8_t* codes = a.codes[which] + b * a.cs[which].b + h * a.cs[which].h + (t0 + r0) * a.cs[which].n + col;
  float* scale = a.scales[which] + b * a.ss[which].b + h * a.ss[which].h + j;
  uint4 u[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = r0 + i * kStep;
    u[i] = r >= lo && r < hi ? *reinterpret_cast<const uint4*>(x + i * xstep) : make_uint4(0, 0, 0, 0);
  }
  // The largest magnitude, as bf16 bits in both halves; from 0x7F80 on something is not finite.
  uint32_t pair = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    pair = max_u16x2(max_u16x2(pair, max_u16x2(u[i].x & 0x7FFF7FFFu, u[i].y & 0x7FFF7FFFu)),
                     max_u16x2(u[i].z & 0x7FFF7FFFu, u[i].w & 0x7FFF7FFFu));
  uint32_t top = max(pair & 0xFFFFu, pair >> 16);
  const bool finite = top < 0x7F80u;
  if (!finite) {  // the largest finite one (what is not finite is held as a NaN: the scale may not be 0)
    top = 1;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
      for (int e = 0; e < 4; ++e) {
        const uint32_t v0 = w[e] & 0x7FFFu, v1 = w[e] >> 16 & 0x7FFFu;
        top = max(top, max(v0 < 0x7F80u ? v0 : 0u, v1 < 0x7F80u ? v1 : 0u));
      }
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
  const bool whole = lo == 0 && hi == rows;
  const float old = live && !whole ? held_scale(*scale) : 0.f;
  const float s = fmaxf(old, scale_for(__uint_as_float(top << 16)));
  if (kWarps > 1)
    __syncthreads();  // (every thread has read the old scale)
  else
    __syncwarp();
  if (!live) return;
  const uint32_t sb = __float_as_uint(s);
  // a power of two is divided by exactly; a scale that the caller brought along need not be one
  const bool two = s == 0.f || ((sb & 0x7FFFFFu) == 0 && sb >= 0x00800000u && sb < 0x7E800000u);
  const float inv = s == 0.f ? 0.f : __uint_as_float(0x7F000000u - sb);
  auto code = [&](float lo_, float hi_) -> uint32_t {  // of any values, by any scale but 0
    const float none = __uint_as_float(0x7FC00000u);
    return encode2(fabsf(lo_) <= 3.4028234663852886e38f ? __fdiv_rn(lo_, s) : none,
                   fabsf(hi_) <= 3.4028234663852886e38f ? __fdiv_rn(hi_, s) : none);
  };
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = r0 + i * kStep;
    uint2* at = reinterpret_cast<uint2*>(codes + i * cstep);
    if (r >= lo && r < hi) {
      const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
      uint32_t c[4];
      if (two && finite) {
#pragma unroll
        for (int e = 0; e < 4; ++e) c[e] = encode2(__uint_as_float(w[e] << 16) * inv, __uint_as_float(w[e] & 0xFFFF0000u) * inv);
      } else {
        for (int e = 0; e < 4; ++e) c[e] = code(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xFFFF0000u));
      }
      *at = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
    } else if (s != old && r < rows) {  // the block's other tokens keep their values
      const uint2 had = *at;
      const uint32_t w[4] = {had.x & 0xFFFFu, had.x >> 16, had.y & 0xFFFFu, had.y >> 16};
      uint32_t c[4];
      for (int e = 0; e < 4; ++e) {
        const uint32_t f = old == 0.f ? 0u : decode2(w[e]);
        c[e] = code(half_lo(f) * old, half_hi(f) * old);
      }
      *at = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
    }
  }
  if (t == 0) *scale = s;
}

// Tokens first[b] .. first[b] + n - 1 of every head as bf16 (exact where the scale is a power of two) or fp32 values;
// 0 where the cache has no such token.  A thread takes twice 16 codes; a.blocks: blocks of a head.
template <bool WIDE, int PIECES>
__global__ void __launch_bounds__(256) sa_cache8_read_kernel(const __grid_constant__ Cache8Args a) {
  constexpr int U = 2, kTokens = 256 / PIECES;  // tokens that the block's threads have at a time
  // (a block is a whole number of tokens: pieces of a head, counted through, pass 32 bits from 2^29 tokens of d = 128 on)
  const uint32_t head2 = blockIdx.x / a.blocks;
  const int at0 = static_cast<int>(blockIdx.x - head2 * a.blocks) * (kTokens * U) + static_cast<int>(threadIdx.x) / PIECES;
  const bool two = a.y[0] && a.y[1];
  const int which = two ? static_cast<int>(head2 & 1) : a.y[0] ? 0 : 1, bh = static_cast<int>(two ? head2 >> 1 : head2);
  const int b = bh / a.H, h = bh - b * a.H, c = threadIdx.x % PIECES;
  const int64_t first = a.start ? __ldg(a.start + b) : a.start0;
  const uint8_t* codes = a.codes[which] + b * a.cs[which].b + h * a.cs[which].h + c * 16;
  const float* scales = a.scales[which] + b * a.ss[which].b + h * a.ss[which].h;
  char* y = static_cast<char*>(a.y[which]) + (b * a.xs[which].b + h * a.xs[which].h + c * 16) * (WIDE ? 4 : 2);
  uint4 u[U];
  float s[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int at = at0 + i * kTokens;
    const int64_t tok = first + at;
    u[i] = make_uint4(0, 0, 0, 0);
    s[i] = 0.f;
    if (at < a.n && tok >= 0 && tok < a.N) {
      u[i] = *reinterpret_cast<const uint4*>(codes + tok * a.cs[which].n);
      s[i] = held_scale(scales[static_cast<int>(tok) / a.block]);
    }
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int at = at0 + i * kTokens;
    if (at >= a.n) return;
    if (s[i] == 0.f) u[i] = make_uint4(0, 0, 0, 0);
    const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
    float f[16];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t lo = decode2(w[e] & 0xFFFFu), hi = decode2(w[e] >> 16);
      f[4 * e] = half_lo(lo) * s[i];
      f[4 * e + 1] = half_hi(lo) * s[i];
      f[4 * e + 2] = half_lo(hi) * s[i];
      f[4 * e + 3] = half_hi(hi) * s[i];
    }
    uint4* out = reinterpret_cast<uint4*>(y + at * a.xs[which].n * (WIDE ? 4 : 2));
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
}

namespace {

template <int T, int ROW>
void launch_append(const Cache8Args& a, cudaStream_t st) {
  sa_cache8_append_kernel<T, ROW><<<static_cast<unsigned>((a.items + 256 / T - 1) / (256 / T)), 256, 0, st>>>(a);
}

}  // namespace

cudaError_t launch_cache8_append(Cache8Args a, cudaStream_t st) {
  // blocks that n tokens can touch, wherever they start
  a.blocks = static_cast<int32_t>(std::min<int64_t>((int64_t(a.N) + a.block - 1) / a.block, (int64_t(a.n) + a.block - 2) / a.block + 1));
  a.items = int64_t(a.B) * a.H * 2 * a.blocks;
  const bool wide = a.d == 128;
  switch (a.block) {
    case 16: wide ? launch_append<32, 16>(a, st) : launch_append<16, 8>(a, st); break;
    case 32: wide ? launch_append<64, 16>(a, st) : launch_append<32, 8>(a, st); break;
    case 64: wide ? launch_append<128, 16>(a, st) : launch_append<64, 8>(a, st); break;
    default: wide ? launch_append<256, 16>(a, st) : launch_append<128, 8>(a, st);
  }
  return cudaGetLastError();
}

cudaError_t launch_cache8_read(Cache8Args a, bool wide, cudaStream_t st) {
  a.blocks = static_cast<int32_t>((int64_t(a.n) * (a.d / 16) + 511) / 512);
  const unsigned grid = static_cast<unsigned>(int64_t(a.B) * a.H * (a.y[0] && a.y[1] ? 2 : 1) * a.blocks);
  if (a.d == 128)
    (wide ? sa_cache8_read_kernel<true, 8> : sa_cache8_read_kernel<false, 8>)<<<grid, 256, 0, st>>>(a);
  else
    (wide ? sa_cache8_read_kernel<true, 4> : sa_cache8_read_kernel<false, 4>)<<<grid, 256, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace sa
