// sa_attend8.cuh — what the kernels that attend over an 8-bit cache share: the operands' descriptors, the tensor maps
// and the query rows in two e4m3 terms.
//
// Products of e4m3 codes run on the tensor cores as they are (kind::f8f6f4), at twice the rate of 16-bit operands.  A
// query row is bf16 and may not lose digits, so it is held as two e4m3 terms of a scaled row: with f the power of two
// that brings the row's largest magnitude into [128, 256), hi = e4m3(q f) and lo = e4m3(q f - hi).  hi is off by half of
// its last of four digits, so what is left is a multiple of bf16's last place of at most four digits: lo holds
// it exactly, down to e4m3's smallest step of 2^-9.  q f is exact above 2^-10 of the row's largest value and off
// by 2^-10 (2^-17 of the largest value) below.  Two products at twice the rate cost what one of bf16 does.
// Where the products of the terms are kept apart, lo is held times 2^5 (it is 8 at most): off by 2^-15, 2^-22 of the
// largest value.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "sa_device.cuh"
#include "sa_e4m3.cuh"
#include "sa_internal.h"
#include "sa_mask.cuh"
#include "sa_tma.h"

namespace sa {

// Instruction descriptor for kind::f8f6f4 with fp32 accumulate: formats 0 e4m3, 1 e5m2; a_mn, b_mn: MN-major operands.
__host__ __device__ constexpr uint32_t idesc_f8(int M, int N, int a_format, int b_format, bool a_mn, bool b_mn) {
  return (1u << 4) | (static_cast<uint32_t>(a_format) << 7) | (static_cast<uint32_t>(b_format) << 10) |
         ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

// D(tmem) (+)= A(smem) * B(smem), 8-bit operands; descriptors as in mma_ss_w.
__device__ __forceinline__ void mma8_ss_w(uint32_t d_tmem, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "mov.b64 da, {%1, %2};\n\t"
      "mov.b64 db, {%3, %4};\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %5, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 32 lanes x 8 columns; tmem_ld_wait() before use.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}

// Tiles of rows of D bytes, D = 128 or 64: the swizzle is as wide as a row, eight rows follow one another.
template <int D>
__device__ __forceinline__ uint64_t rows8_desc(uint32_t saddr, uint32_t lbo) {
  uint64_t d = sw128_desc(saddr, lbo, 8 * D);
  if (D == 64) d = (d & ~(static_cast<uint64_t>(7) << 61)) | (static_cast<uint64_t>(4) << 61);  // 64-byte swizzle
  return d;
}

// Byte offset of byte c of row r in such a tile.
template <int D>
__device__ __forceinline__ uint32_t rows8_offset(int r, int c) {
  const int x = D == 128 ? r & 7 : (r >> 1) & 3;
  return static_cast<uint32_t>(r * D + ((((c >> 4) ^ x) << 4) | (c & 15)));
}

// The codes [B, H, N, d] of a cache as boxes of d bytes x `box` tokens of one head, swizzled as rows8_desc reads them
// (or not).  Tokens past N read as zeros.
inline bool make_codes_map(CUtensorMap* map, const void* base, uint32_t d, uint64_t N, uint64_t H, uint64_t B,
                           const sa_strides& s, uint32_t box, bool swizzled) {
  const EncodeTiledFn fn = encode_tiled_fn();
  if (!fn) return false;
  const cuuint64_t dims[4] = {d, N, H, B};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(s.n), static_cast<cuuint64_t>(s.h), static_cast<cuuint64_t>(s.b)};
  const cuuint32_t boxes[4] = {d, box, 1, 1};
  const cuuint32_t elem[4] = {1, 1, 1, 1};
  const CUtensorMapSwizzle sw = !swizzled ? CU_TENSOR_MAP_SWIZZLE_NONE
                                : d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(base), dims, strides, boxes, elem,
            CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Brings a tensor map near ahead of the first copy.
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// The power of two that brings a row's largest finite magnitude (its fp32 bits) into [128, 256); 1 for 0.
__device__ __forceinline__ float row_factor(uint32_t top) {
  const int e = static_cast<int>(top >> 23);
  if (top == 0) return 1.f;
  return __uint_as_float(static_cast<uint32_t>(min(254, 127 + 7 + 127 - e)) << 23);
}

// Eight bf16 values times f as their two terms, the second one times `lift`.
__device__ __forceinline__ void two_terms(const uint4& u, float f, float lift, uint2* hi, uint2* lo) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = __uint_as_float(w[i] << 16), b = __uint_as_float(w[i] & 0xFFFF0000u);
    // (an infinity is to be no number, not the largest one)
    const float x = (a - a) + a * f, y = (b - b) + b * f;
    h[i] = encode2(x, y);
    const uint32_t back = decode2(h[i]);
    l[i] = encode2((x - half_lo(back)) * lift, (y - half_hi(back)) * lift);
  }
  *hi = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
  *lo = make_uint2(l[0] | l[1] << 16, l[2] | l[3] << 16);
}

// Keys of an empty value block add their weights to a row's sum and nothing to its output (their values are cleared).  The
// row's reference is there for the output, whose weights carry the value scales, any powers of two: as large as the others',
// an empty block's would push these to the bottom of the second product's 8 or 16 bits.  So they count for the reference
// less by 2^kEmptyBelow: far enough for blocks 2^100 apart (2^-16 of the reference at least where their weights are as
// large), near enough for fp32 to hold the sum (2^(84 + 15) a tile, 2^23 tiles); their weights saturate on the way into the
// product.  As long as a run has seen empty blocks alone they set the reference like any others.
constexpr float kEmptyBelow = 84.f;

// The first of a head's scales that holds anything, of the blocks of a tile's `keys` keys from k0 on that begin ahead of
// `end`; 0: none.  One load a lane, the warp together.
__device__ __forceinline__ float first_scale(const float* scales, int k0, int keys, int end, int block_log2) {
  const int lane = threadIdx.x & 31, key = k0 + (lane << block_log2);
  const float s = lane < (keys >> block_log2) && key < end ? held_scale(__ldg(scales + (key >> block_log2))) : 0.f;
  const uint32_t has = __ballot_sync(0xffffffffu, s > 0.f);
  return __shfl_sync(0xffffffffu, s, has ? __ffs(has) - 1 : 0);
}

// A pair of weights as fp16; past 65504: 65504.
__device__ __forceinline__ uint32_t pack_weights(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// ln of 2^m sum.  A sum far from 1 (value scales or empty blocks far from the reference) gives its exponent to m first: added
// up as logarithms the two would cancel in the digits that fp32 has at their size.
__device__ __forceinline__ float ln_of(float m, float sum) {
  const int e = (static_cast<int>(__float_as_uint(sum) >> 23) - 127) / 16 * 16;  // (0 for sums from 2^-15 to 2^16)
  return 0.69314718055994531f * ((m + e) + log2f(sum * __uint_as_float(static_cast<uint32_t>(127 - e) << 23)));
}

// Largest finite magnitude (bits) of eight bf16 values.
__device__ __forceinline__ uint32_t top_of(const uint4& u, uint32_t top) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = (w[i] & 0x7FFFu) << 16, hi = w[i] & 0x7FFF0000u;
    top = max(top, lo < 0x7F800000u ? lo : 0u);
    top = max(top, hi < 0x7F800000u ? hi : 0u);
  }
  return top;
}

}  // namespace sa
