// sa_attend8_few.cu — attention of few query rows (a new token's heads, or a few tokens) over an 8-bit cache.
//
// The cache is read once and decides the time, so nothing is done to it but what the tensor cores do: its codes go by
// TMA into shared memory and from there, as they are, into both products.  Keys are the rows of the first,
//     S^T [128 keys x rows] = K Q^T  (rows in two e4m3 terms: sa_attend8.cuh),
// so that its cost goes with the rows there are, and a thread owns a key: the key's scale is one factor, a row's sum
// of weights stays in the thread until the end, and the mask is a comparison.  The second is
//     O^T [d x rows] = V^T P^T,
// with V's codes as the MN-major operand.  Its other operand has 8 bits too: a weight u = 2^12 p vs (vs: the value
// block's scale; p counts from the row's reference, so that u <= 2^15) is rounded to fp16 and cut into three e5m2 terms,
// whose exponent reaches from 2^-16 to 2^15: three digits each, which hold an fp16 value exactly from 2^-6 on.  Off by
// 2^-11 of u, or by 2^-29 of the row's largest.
// The terms are columns of their own, added up at the end.
//
// Work is cut evenly whatever the lengths: the key tiles of all heads of all sequences are one row of tiles, and every
// block takes an equal part of it.  A run that covers a head in part leaves a normalised fp32 partial result and its
// lse; a second kernel joins them.
//
// The row's reference is that of its run's first tile and moves when a weight passes 2^15 (eight times the first
// tile's largest).  Keys of empty value blocks count less for it: sa_attend8.cuh.
#include <algorithm>
#include <atomic>

#include "sa_attend8.cuh"

namespace sa {

namespace {

constexpr int kKeys = 128;  // keys of a tile
// A row's weights count from the largest of its first tile, so that neither a weight's exponent nor the sum's logarithm
// carries an offset that its rounding would pay for (2^-20 of lse); the product takes them times 2^12.
constexpr float kUnit = 4096.f;
constexpr float kMostWeight = 8.f;  // (2^15 in the product: an exponent of 3 and more, as `moved` says it)
constexpr float kLift = 32.f;  // of a row's second term (its products are columns of their own)
constexpr int kNever = 0x7FFFFFFF;

template <int D, int RP>
struct FCfg {
  static constexpr int kTile = kKeys * D;
  static constexpr int kStages = D == 128 ? 10 : 18;
  static constexpr int kQRows = 2 * RP;                       // hi rows, then lo rows
  static constexpr int kPRows = RP == 8 ? 32 : 3 * RP;        // columns of O^T (a multiple of 16)
  static constexpr int kQBytes = kQRows * D, kPBytes = kPRows * kKeys;
  static constexpr int kRing = 0, kQ = kStages * kTile, kP = kQ + (kQBytes + 1023) / 1024 * 1024, kEnd = kP + 2 * kPBytes;
  static constexpr int kSmemBytes = 1024 + kEnd;
  static constexpr int kOCol = 2 * kQRows;
  static constexpr int kTmemCols = kOCol + kPRows <= 64 ? 64 : kOCol + kPRows <= 128 ? 128 : 256;
  static constexpr int kThreads = 192;  // four softmax warps, one for the MMAs, one for the loads
  static_assert(kSmemBytes <= 220 * 1024, "shared memory");
  static_assert(kStages <= 32, "a warp makes the ring's barriers");
};

// What the blocks of a launch share out: places, of which a head has one for each of its key tiles and kRunCost in
// front of them (if it has any tiles).  A run's start and output take as long as that many tiles: with tiles alone to go
// by, the blocks that end one head and begin another came last by a fifth (4 sequences of 24 heads on 6, up to 28160
// keys).
constexpr int kRunCost = 6;
struct Run {
  int b, hk, j0, n, tiles;  // entry, key head, first tile, tiles, tiles of the head
};

__device__ __forceinline__ int keys_of(const Attend8Args& a, int b) { return row_span(a.m.mask, b, a.m.Nq - 1).hi; }
__device__ __forceinline__ int tiles_of_entry(const Attend8Args& a, int b) { return (keys_of(a, b) + kKeys - 1) / kKeys; }
__device__ __forceinline__ int places_of_head(int tiles) { return tiles ? tiles + kRunCost : 0; }

// Any of `count` threads' flags, on hardware barrier `id`.
__device__ __forceinline__ bool any_of(int id, int count, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\t"
      "barrier.cta.red.or.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(count), "r"(static_cast<uint32_t>(x))
      : "memory");
  return r != 0;
}

// A pair of fp16 values to the nearest e5m2 codes.
__device__ __forceinline__ uint32_t encode_e5m2(uint32_t pair) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(r) : "r"(pair));
  return r;
}
__device__ __forceinline__ uint32_t half_sub(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

}  // namespace

template <int D, int RP>
__global__ void __launch_bounds__(FCfg<D, RP>::kThreads, 1)
    sa_attend8_few_kernel(const __grid_constant__ Attend8Args a, bool whole, const __grid_constant__ CUtensorMap tm_k,
                          const __grid_constant__ CUtensorMap tm_v) {
  using C = FCfg<D, RP>;
  constexpr int S = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ uint64_t full[S], empty[S], sfull[2], pfull[2], pdone[2], qfull, drain;
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag;
  __shared__ int before[kMostEntries + 1];  // places of the entries ahead of each
  __shared__ float rowf[2][RP], rowm[RP], red[4][RP];  // (two: this run's and the next one's)
  __shared__ int rowhi[2][RP], nan_at[2][D];
  volatile int* abort = &abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nr = a.m.R * a.m.Nq;  // rows of a key head

  if (threadIdx.x < S) {
    mbar_init(&full[threadIdx.x], 1);
    mbar_init(&empty[threadIdx.x], 1);
    fence_mbar_init();
  } else if (threadIdx.x >= 32 && threadIdx.x < 34) {
    const int i = threadIdx.x - 32;
    mbar_init(&sfull[i], 1);
    mbar_init(&pfull[i], 4);
    mbar_init(&pdone[i], 1);
    fence_mbar_init();
  } else if (threadIdx.x == 64) {
    mbar_init(&qfull, 4);
    mbar_init(&drain, 1);
    abort_flag = 0;
    fence_mbar_init();
  } else if (threadIdx.x == 160) {
    prefetch_map(&tm_k);
    prefetch_map(&tm_v);
  }
  for (int b = threadIdx.x; b < a.m.B; b += C::kThreads) before[b + 1] = places_of_head(tiles_of_entry(a, b)) * a.m.Hkv;
  for (int i = threadIdx.x; i < 2 * C::kPBytes / 16; i += C::kThreads)  // (columns that no term fills stay 0)
    reinterpret_cast<uint4*>(smem + C::kP)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  if (warp == 4) {
    tmem_alloc(&tmem_base, C::kTmemCols);
    tmem_relinquish();
  }
  __syncthreads();
  if (warp == 5) {  // running sums
    int sum = 0;
    for (int b0 = 0; b0 < a.m.B; b0 += 32) {
      int x = b0 + lane < a.m.B ? before[b0 + lane + 1] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (b0 + lane < a.m.B) before[b0 + lane + 1] = sum + x;
      sum += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) before[0] = 0;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  const int total = before[a.m.B], heads = a.m.B * a.m.Hkv;
  int g0, g1, v0 = 0, v1 = 0;  // the block's places, and its heads where they are not cut
  if (whole) {
    v0 = static_cast<int>(int64_t(blockIdx.x) * heads / gridDim.x);
    v1 = static_cast<int>(int64_t(blockIdx.x + 1) * heads / gridDim.x);
    auto place_of = [&](int v) -> int {  // head v's first place
      const int b = v / a.m.Hkv;
      return b == a.m.B ? total : before[b] + (v - b * a.m.Hkv) * ((before[b + 1] - before[b]) / a.m.Hkv);
    };
    g0 = place_of(v0);
    g1 = place_of(v1);
  } else {
    const int blocks = min(static_cast<int>(gridDim.x), total);
    const bool works = static_cast<int>(blockIdx.x) < blocks;
    g0 = works ? static_cast<int>(int64_t(blockIdx.x) * total / blocks) : 0;
    g1 = works ? static_cast<int>(int64_t(blockIdx.x + 1) * total / blocks) : 0;
    let_next_kernel_start();
  }
  // The run that begins at place *g or behind it, which moves on; none: n = 0.
  auto next_run = [&](int* g) -> Run {
    Run x = {};
    while (*g < g1 && x.n == 0) {
      int b = 0, top = a.m.B - 1;  // the last entry that starts there or before and has places
      while (b < top) {
        const int mid = (b + top + 1) >> 1;
        if (before[mid] <= *g)
          b = mid;
        else
          top = mid - 1;
      }
      const int per = (before[b + 1] - before[b]) / a.m.Hkv;
      x.b = b;
      x.tiles = per - kRunCost;
      x.hk = (*g - before[b]) / per;
      const int at = *g - before[b] - x.hk * per, len = min(per - at, g1 - *g);
      x.j0 = max(at - kRunCost, 0);
      x.n = max(at + len - kRunCost, 0) - x.j0;
      *g += len;
    }
    return x;
  };

  if (warp < 4) {
    // ------------------------------------------------------------ softmax: thread = key of a tile
    // (A wait that gives up lets the thread go on: all meet at the same barriers to the end.)
    const int t = threadIdx.x;
    const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
    uint32_t c = 0;  // tiles so far
    uint32_t runs = 0;
    // A run's rows, in two terms: RP rows of D / 8 pieces of eight values.  (The last run's products have read the
    // old ones: its last S is here.)
    // What else a run needs from memory is asked for ahead of the rows, all at once: one after the other the loads took
    // longer than the first S.
    const float *ksc = nullptr, *vsc = nullptr;  // the head's scales
    int most_next = 0, at_block = 0;             // keys that any row sees; the thread's key's block
    float s0_next = 0.f, ks_next = 0.f, vs_next = 0.f;
    const int last_block = (a.m.Nk - 1) >> a.block_log2, block_step = kKeys >> a.block_log2;
    auto fetch = [&]() {  // (past the cache's end: its last block; no row sees that key)
      const int at = min(at_block, last_block);
      ks_next = __ldg(ksc + at);
      vs_next = __ldg(vsc + at);
      at_block += block_step;
    };
    auto prepare = [&](const Run& x, int at) {
      ksc = a.k_scale + int64_t(x.b) * a.k_scales.b + int64_t(x.hk) * a.k_scales.h;
      vsc = a.v_scale + int64_t(x.b) * a.v_scales.b + int64_t(x.hk) * a.v_scales.h;
      s0_next = __ldg(vsc + (x.j0 * kKeys >> a.block_log2));
      at_block = (x.j0 * kKeys + t) >> a.block_log2;
      fetch();
      most_next = keys_of(a, x.b);
      constexpr int kPieces = D / 8;
#pragma unroll
      for (int f0 = 0; f0 < RP * kPieces; f0 += 128) {
        const int f = f0 + t, r = f / kPieces, p = f % kPieces;
        const int qi = r / a.m.R, h = x.hk * a.m.R + r - qi * a.m.R;
        const bool there = RP * kPieces % 128 == 0 || r < RP;
        const int sees = r < nr ? row_span(a.m.mask, x.b, qi).hi : 0;
        uint4 u = make_uint4(0, 0, 0, 0);
        if (r < nr)
          u = *reinterpret_cast<const uint4*>(a.m.q + int64_t(x.b) * a.m.qs.b + int64_t(h) * a.m.qs.h + int64_t(qi) * a.m.qs.n + p * 8);
        uint32_t top = top_of(u, 0);
#pragma unroll
        for (int o = kPieces / 2; o; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float fac = row_factor(top);
        uint2 hi, lo;
        two_terms(u, fac, kLift, &hi, &lo);
        if (there) {
          *reinterpret_cast<uint2*>(smem + C::kQ + rows8_offset<D>(r, p * 8)) = hi;
          *reinterpret_cast<uint2*>(smem + C::kQ + rows8_offset<D>(RP + r, p * 8)) = lo;
        }
        if (there && p == 0) {
          rowf[at][r] = r < nr ? a.scale_log2 / fac : 0.f;
          rowhi[at][r] = sees;
        }
      }
      if (t < D) nan_at[at][t] = kNever;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&qfull);
    };
    int g = g0;
    Run next = next_run(&g);
    if (next.n) {
      prepare(next, 0);
      named_barrier(1, 128);
    }
    for (; next.n; ++runs) {
      const Run x = next;
      const float* rowf_ = rowf[runs & 1];
      const int* rowhi_ = rowhi[runs & 1];
      int* nan_at_ = nan_at[runs & 1];
      int least = kNever;
      for (int r = 0; r < nr; ++r) least = min(least, rowhi_[r]);
      const int most = most_next;
      // value scales count from that of the run's first block that holds anything (0: none so far)
      float s0 = held_scale(s0_next), lref = s0 > 0.f ? __log2f(s0) : 0.f;
      float l[RP];
#pragma unroll
      for (int r = 0; r < RP; ++r) l[r] = 0.f;
      for (int j = 0; j < x.n; ++j, ++c) {
        const int k0 = (x.j0 + j) * kKeys, key = k0 + t;
        const float ks = held_scale(ks_next), vs = held_scale(vs_next);
        // (ahead of the next loads, which this one would wait for; all threads alike)
        bool first_values = false;  // behind tiles of empty blocks alone
        if (s0 == 0.f) {
          s0 = first_scale(vsc, k0, kKeys, most, a.block_log2);
          if (s0 > 0.f) lref = __log2f(s0);
          first_values = j > 0 && s0 > 0.f;
        }
        if (j + 1 < x.n) fetch();
        const float lv = vs > 0.f ? fminf(fmaxf(__log2f(vs) - lref, -100.f), 100.f) : 0.f, iv = fast_exp2(-lv);
        const uint32_t sb = c & 1;
        const bool edge = k0 + kKeys > least;  // some row does not see the whole tile
        mbar_wait(&sfull[sb], (c >> 1) & 1, abort);
        __syncwarp();
        tc_fence_after();
        float y[RP];
        {
          float s[2 * RP];
          uint32_t* w = reinterpret_cast<uint32_t*>(s);
          const uint32_t at = tmem + lanes + sb * C::kQRows;
          if (RP == 8) {
            tmem_ld16(at, w);
          } else {
#pragma unroll
            for (int i = 0; i < 2 * RP; i += 32) tmem_ld32(at + i, w + i);
          }
          tmem_ld_wait();
#pragma unroll
          for (int r = 0; r < RP; ++r) y[r] = fmaf(fmaf(s[RP + r], 1.f / kLift, s[r]), rowf_[r] * ks, lv);
        }
        if (ks == 0.f) {  // (an empty block's keys are zeros, whatever their codes)
#pragma unroll
          for (int r = 0; r < RP; ++r) y[r] = lv;
        }
        if (edge) {
#pragma unroll
          for (int r = 0; r < RP; ++r) y[r] = key < rowhi_[r] ? y[r] : -INFINITY;
        }
        float u[RP];
        auto weights = [&]() -> bool {  // false: one is too large
          float top = 0.f;
#pragma unroll
          for (int r = 0; r < RP; ++r) {
            u[r] = fast_exp2(y[r] - rowm[r]);
            top = u[r] <= kMostWeight ? top : 1.f;
          }
          return top == 0.f;
        };
        // A row's new reference: it moves if a weight passed 8 (each row by itself: its bits do not go by the others), and
        // where empty blocks alone have set it so far.
        auto moved = [&](int r, float m0, bool start, int rows) -> float {
          if (first_values) m0 -= kEmptyBelow;
          const float mx = fmaxf(fmaxf(red[0][r], red[1][r]), fmaxf(red[2][r], red[3][r]));
          const float mn = start || mx - m0 > 3.f ? mx : m0;
          return r >= rows || mn == -INFINITY ? INFINITY : mn;
        };
        bool fits = true;
        if (j > 0) fits = weights() && !first_values;
        if (j == 0 || any_of(2, 128, !fits || (vs == 0.f && key < most)) || edge) {
          const bool raise = j == 0 || any_of(2, 128, !fits);
          if (raise) {
            const float below = vs == 0.f && s0 > 0.f ? kEmptyBelow : 0.f;
#pragma unroll
            for (int r = 0; r < RP; ++r) {
              const uint32_t o = __reduce_max_sync(0xffffffffu, y[r] == y[r] ? order_key(y[r] - below) : 0u);
              if (lane == 0) red[warp][r] = o ? key_value(o) : -INFINITY;
            }
            named_barrier(1, 128);
            float alpha[RP];
#pragma unroll
            for (int r = 0; r < RP; ++r) {
              // (a row that sees nothing of the run's first tile sees nothing of the run; rows that are not there: 0 weights)
              const float m0 = j == 0 ? -INFINITY : rowm[r], mn = moved(r, m0, j == 0, nr);
              alpha[r] = j == 0 || mn == m0 ? 1.f : fast_exp2(m0 - mn);
              l[r] *= alpha[r];
              y[r] -= mn;  // (rowm changes behind the barrier)
            }
            named_barrier(1, 128);
            if (t < RP) {
              rowm[t] = moved(t, j == 0 ? -INFINITY : rowm[t], j == 0, nr);
            }
            if (j > 0) {  // O holds the tiles so far
              mbar_wait(&pdone[(c - 1) & 1], ((c - 1) >> 1) & 1, abort);
              __syncwarp();
              tc_fence_after();
#pragma unroll
              for (int k = 0; k < 3; ++k) {
#pragma unroll
                for (int r0 = 0; r0 < RP; r0 += 8) {
                  const uint32_t at = tmem + lanes + C::kOCol + k * RP + r0;
                  uint32_t o[8];
                  tmem_ld8(at, o);
                  tmem_ld_wait();
#pragma unroll
                  for (int i = 0; i < 8; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha[r0 + i]);
                  tmem_st8(at, o);
                }
              }
              tmem_st_wait();
            }
#pragma unroll
            for (int r = 0; r < RP; ++r) u[r] = fast_exp2(y[r]);
            named_barrier(1, 128);
          }
          // Values of tokens that some row does not see, or of empty blocks, must not reach O by 0 times NaN: what no
          // row sees is cleared, a NaN that some do is noted by its column (rows see the first keys, so its first
          // key says which) and cleared.
          const bool clean = edge || any_of(2, 128, vs == 0.f && key < most);
          const uint32_t iv_at = (2 * c + 1) % S;
          if (clean) mbar_wait(&full[iv_at], ((2 * c + 1) / S) & 1, abort);
          uint8_t* vt = smem + C::kRing + iv_at * C::kTile;
          auto piece = [&](int p) -> uint4* { return reinterpret_cast<uint4*>(vt + rows8_offset<D>(t, p * 16)); };
          if (clean && (key >= most || vs == 0.f)) {
#pragma unroll
            for (int p = 0; p < D / 16; ++p) *piece(p) = make_uint4(0, 0, 0, 0);
          } else if (clean) {
            uint32_t bad = 0;
#pragma unroll
            for (int p = 0; p < D / 16; ++p) {
              const uint4 w = *piece(p);
              bad |= ((w.x & 0x7F7F7F7Fu) + 0x01010101u) | ((w.y & 0x7F7F7F7Fu) + 0x01010101u) |
                     ((w.z & 0x7F7F7F7Fu) + 0x01010101u) | ((w.w & 0x7F7F7F7Fu) + 0x01010101u);
            }
            if (bad & 0x80808080u) {
              for (int q = 0; q < D; ++q) {
                uint8_t* code = vt + rows8_offset<D>(t, q);
                if ((*code & 127) == 127) {
                  atomicMin(&nan_at_[q], key);
                  *code = 0;
                }
              }
            }
          }
        }
#pragma unroll
        for (int r = 0; r < RP; ++r) l[r] = fmaf(u[r], iv, l[r]);
        // (The buffer's last reader, the product of tile c - 2, was issued ahead of this tile's S and is done with it.)
        uint8_t* sp = smem + C::kP + sb * C::kPBytes;
        auto put = [&](int n, uint32_t code) {
          sp[n * kKeys + ((((t >> 4) ^ (n & 7)) << 4) | (t & 15))] = static_cast<uint8_t>(code);
        };
#pragma unroll
        for (int r = 0; r < RP; r += 2) {
          uint32_t h = pack_weights(u[r] * kUnit, u[r + 1] * kUnit);
#pragma unroll
          for (int k = 0; k < 3; ++k) {
            const uint32_t e = encode_e5m2(h);
            put(k * RP + r, e);
            put(k * RP + r + 1, e >> 8);
            if (k < 2) h = half_sub(h, __byte_perm(e, 0, 0x1404));
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pfull[sb]);
      }
      next = next_run(&g);
      if (next.n) prepare(next, (runs + 1) & 1);  // its first S is computed beside this run's output
      // ---------------------------------------------------------- output: thread = column of d
#pragma unroll
      for (int r = 0; r < RP; ++r) {
        float v = l[r];
#pragma unroll
        for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (lane == 0) red[warp][r] = v;
      }
      mbar_wait(&pdone[(c - 1) & 1], ((c - 1) >> 1) & 1, abort);
      named_barrier(1, 128);
      tc_fence_after();
      const bool all = x.n == x.tiles;
      const int64_t slot = int64_t(blockIdx.x) + int64_t(x.b) * a.m.Hkv + x.hk;
      const float unit = s0 > 0.f ? s0 : 1.f;
      const int nan = t < D ? nan_at_[t] : kNever;
#pragma unroll 1
      for (int r0 = 0; r0 < RP; r0 += 8) {
        if (r0 >= nr) break;
        uint32_t o[3][8];
#pragma unroll
        for (int k = 0; k < 3; ++k) tmem_ld8(tmem + lanes + C::kOCol + k * RP + r0, o[k]);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = r0 + i;
          if (r >= nr) continue;
          const float sum = (red[0][r] + red[1][r]) + (red[2][r] + red[3][r]);
          float v = __uint_as_float(o[0][i]) + (__uint_as_float(o[1][i]) + __uint_as_float(o[2][i]));
          // (one after the other: the smallest scales by a row's sum are no normal number)
          v = sum == 0.f ? 0.f : v * ((1.f / kUnit) / sum) * unit;
          if (nan < rowhi_[r]) v = __uint_as_float(0x7FC00000u);
          const int qi = r / a.m.R, h = x.hk * a.m.R + r - qi * a.m.R;
          if (t < D) {
            if (!all)
              a.m.part_o[(slot * nr + r) * D + t] = v;
            else {
              const int64_t at = int64_t(x.b) * a.m.os.b + int64_t(h) * a.m.os.h + int64_t(qi) * a.m.os.n + t;
              if (a.m.out_fp32)
                static_cast<float*>(a.m.o)[at] = v;
              else
                static_cast<uint16_t*>(a.m.o)[at] = static_cast<uint16_t>(pack_bf16(v, 0.f));
            }
          }
        }
      }
      if (t < nr) {
        const float sum = (red[0][t] + red[1][t]) + (red[2][t] + red[3][t]), lse = sum == 0.f ? -INFINITY : ln_of(rowm[t], sum);
        if (!all)
          a.m.part_lse[slot * nr + t] = lse;
        else if (a.m.lse)
          a.m.lse[(int64_t(x.b) * a.m.Hq + x.hk * a.m.R + t % a.m.R) * a.m.Nq + t / a.m.R] = lse;
      }
      tc_fence_before();
      named_barrier(1, 128);  // (the next run writes rowm and red, and reads its rows)
    }
    for (int v = v0; v < v1; ++v) {  // heads without keys
      const int b = v / a.m.Hkv, hk = v - b * a.m.Hkv;
      if (before[b + 1] != before[b]) continue;
      for (int f = t; f < nr * D; f += 128) {
        const int r = f / D, qi = r / a.m.R, h = hk * a.m.R + r - qi * a.m.R;
        const int64_t at = int64_t(b) * a.m.os.b + int64_t(h) * a.m.os.h + int64_t(qi) * a.m.os.n + f % D;
        if (a.m.out_fp32)
          static_cast<float*>(a.m.o)[at] = 0.f;
        else
          static_cast<uint16_t*>(a.m.o)[at] = 0;
        if (f % D == 0 && a.m.lse) a.m.lse[(int64_t(b) * a.m.Hq + h) * a.m.Nq + qi] = -INFINITY;
      }
    }
  } else if (warp == 4) {
    // ------------------------------------------------------------ MMA issue
    constexpr uint32_t kIdescS = idesc_f8(128, C::kQRows, 0, 0, false, false);
    constexpr uint32_t kIdescO = idesc_f8(128, C::kPRows, 0, 1, true, false);
    // (d = 64: V^T has 64 rows; the MMA's other 64 repeat them and are not read)
    const uint64_t dk = rows8_desc<D>(smem_u32(smem + C::kRing), 16), dv = rows8_desc<D>(smem_u32(smem + C::kRing), 0);
    const uint64_t dq = rows8_desc<D>(smem_u32(smem + C::kQ), 16), dp = sw128_desc(smem_u32(smem + C::kP), 16, 1024);
    const uint32_t k_lo = static_cast<uint32_t>(dk), k_hi = static_cast<uint32_t>(dk >> 32);
    const uint32_t v_lo = static_cast<uint32_t>(dv), v_hi = static_cast<uint32_t>(dv >> 32);
    const uint32_t q_lo = static_cast<uint32_t>(dq), q_hi = static_cast<uint32_t>(dq >> 32);
    const uint32_t p_lo = static_cast<uint32_t>(dp), p_hi = static_cast<uint32_t>(dp >> 32);
    auto ready = [&](uint32_t i) -> bool { return mbar_wait(&full[i % S], (i / S) & 1, abort); };
    auto first = [&](uint32_t c) {  // S^T of tile number c
      const uint32_t at = (((2 * c) % S) * C::kTile) >> 4;
#pragma unroll
      for (int kk = 0; kk < D / 32; ++kk)
        mma8_ss_w(tmem + (c & 1) * C::kQRows, k_lo + at + kk * 2, k_hi, q_lo + kk * 2, q_hi, kIdescS, kk > 0);
      mma_commit(&sfull[c & 1]);
      mma_commit(&empty[(2 * c) % S]);
    };
    if (lane == 0) {
      bool ok = true;
      uint32_t c = 0, runs = 0;
      for (int g = g0; ok; ++runs) {
        const Run x = next_run(&g);
        if (!x.n) break;
        if (!(ok = mbar_wait(&qfull, runs & 1, abort)) || !(ok = ready(2 * c))) break;
        tc_fence_after();
        first(c);
        for (int j = 0; j < x.n; ++j, ++c) {
          // (S^T's other buffer: its tile's P is here already)
          if (j + 1 < x.n) {
            if (!(ok = ready(2 * c + 2))) break;
            first(c + 1);
          }
          if (!(ok = ready(2 * c + 1)) || !(ok = mbar_wait(&pfull[c & 1], (c >> 1) & 1, abort))) break;
          tc_fence_after();
          const uint32_t at = (((2 * c + 1) % S) * C::kTile) >> 4, bt = ((c & 1) * C::kPBytes) >> 4;
#pragma unroll
          for (int kk = 0; kk < kKeys / 32; ++kk)
            mma8_ss_w(tmem + C::kOCol, v_lo + at + ((kk * 32 * D) >> 4), v_hi, p_lo + bt + kk * 2, p_hi, kIdescO, j > 0 || kk > 0);
          mma_commit(&pdone[c & 1]);
          mma_commit(&empty[(2 * c + 1) % S]);
        }
      }
      // Every MMA issued above must finish before TMEM is released.
      mma_commit(&drain);
      const long long t0 = clock64();
      while (!mbar_test(&drain, 0) && clock64() - t0 < kWaitLimitCycles) {
      }
    }
  } else if (lane == 0) {
    // ------------------------------------------------------------ loads
    uint32_t it = 0;
    bool ok = true;
    for (int g = g0; ok;) {
      const Run x = next_run(&g);
      if (!x.n) break;
      for (int f = 0; f < 2 * x.n; ++f, ++it) {
        const uint32_t s = it % S;
        if (!(ok = mbar_wait(&empty[s], ((it / S) & 1) ^ 1, abort))) break;
        mbar_expect_tx(&full[s], C::kTile);
        tma_load_4d(smem_u32(smem + C::kRing) + s * C::kTile, (f & 1) ? &tm_v : &tm_k, 0, (x.j0 + (f >> 1)) * kKeys, x.hk, x.b,
                    &full[s]);
      }
    }
    if (*abort) {  // what is in flight lands before the block ends
      for (uint32_t f = it > S ? it - S : 0; f < it; ++f) {
        const long long t0 = clock64();
        while (!mbar_test(&full[f % S], (f / S) & 1) && clock64() - t0 < kWaitLimitCycles) {
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && abort_flag) report(a.m.status, SA_DEVERR_TIMEOUT);
  if (warp == 4) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// A block joins a row's partial results (or writes that it saw nothing): lse = ln sum_p e^(lse_p), o = sum_p
// e^(lse_p - lse) o_p.  Every column has four threads, each takes every fourth partial result, eight at a time.
template <int D>
__global__ void __launch_bounds__(4 * D) sa_attend8_join_kernel(const __grid_constant__ Attend8Args a, int grid) {
  __shared__ int sums[2][4 * D / 32];
  __shared__ float s_acc[4][D], s_sum[4], s_mx[4];
  const int nr = a.m.R * a.m.Nq, v = blockIdx.x / nr, r = blockIdx.x - v * nr, b = v / a.m.Hkv, hk = v - b * a.m.Hkv;
  int ahead = 0, total = 0;  // places of the entries ahead of b, and of all
  for (int i = threadIdx.x; i < a.m.B; i += 4 * D) {
    const int n = places_of_head(tiles_of_entry(a, i)) * a.m.Hkv;
    total += n;
    if (i < b) ahead += n;
  }
  ahead = __reduce_add_sync(0xffffffffu, ahead);
  total = __reduce_add_sync(0xffffffffu, total);
  if ((threadIdx.x & 31) == 0) {
    sums[0][threadIdx.x >> 5] = ahead;
    sums[1][threadIdx.x >> 5] = total;
  }
  __syncthreads();
  ahead = total = 0;
#pragma unroll
  for (int i = 0; i < 4 * D / 32; ++i) {
    ahead += sums[0][i];
    total += sums[1][i];
  }
  const int tiles = tiles_of_entry(a, b), blocks = min(grid, total);
  int first = 0, parts = 0;
  if (tiles > 0) {
    const int64_t t0 = ahead + int64_t(hk) * (tiles + kRunCost) + kRunCost;  // the head's first tile's place
    first = static_cast<int>(((t0 + 1) * blocks - 1) / total);
    parts = static_cast<int>(((t0 + tiles) * blocks - 1) / total) - first + 1;
  }
  // (the partial results are read by plain loads, which stay behind the wait; every block waits)
  wait_for_earlier_kernel();
  if (parts == 1) return;  // one block did it all
  const int k = threadIdx.x / D, c = threadIdx.x % D;
  const int64_t row0 = (int64_t(first) + v) * nr + r;
  float mx = -INFINITY, sum = 0.f, o = 0.f;
  for (int p0 = k; p0 < parts; p0 += 32) {
    float l[8], f[8], top = mx;
    bool none = false;  // a partial result that is not a number makes the row none (fmaxf drops it)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int p = p0 + 4 * i;
      const int64_t row = row0 + int64_t(p) * nr;
      l[i] = p < parts ? a.m.part_lse[row] : -INFINITY;
      f[i] = p < parts ? a.m.part_o[row * D + c] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      top = fmaxf(top, l[i]);
      none |= l[i] != l[i];
    }
    if (top == -INFINITY && !none) continue;
    const float keep = __expf(mx - top);
    mx = top;
    sum *= keep;
    o *= keep;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float w = __expf(l[i] - mx);
      sum += w;
      o = fmaf(w, f[i], o);
    }
  }
  s_acc[k][c] = o;
  if (c == 0) {
    s_sum[k] = sum;
    s_mx[k] = mx;
  }
  __syncthreads();
  if (k) return;
  const float all = fmaxf(fmaxf(s_mx[0], s_mx[1]), fmaxf(s_mx[2], s_mx[3]));
  sum = o = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (s_sum[i] != 0.f) {  // (a NaN is not 0)
      const float w = __expf(s_mx[i] - all);
      sum = fmaf(w, s_sum[i], sum);
      o = fmaf(w, s_acc[i][c], o);
    }
  o = sum == 0.f ? 0.f : o / sum;
  const int qi = r / a.m.R, h = hk * a.m.R + r - qi * a.m.R;
  const int64_t at = int64_t(b) * a.m.os.b + int64_t(h) * a.m.os.h + int64_t(qi) * a.m.os.n + c;
  if (a.m.out_fp32)
    static_cast<float*>(a.m.o)[at] = o;
  else
    static_cast<uint16_t*>(a.m.o)[at] = static_cast<uint16_t>(pack_bf16(o, 0.f));
  if (c == 0 && a.m.lse) a.m.lse[(int64_t(b) * a.m.Hq + h) * a.m.Nq + qi] = sum == 0.f ? -INFINITY : all + logf(sum);
}

namespace {

template <int D, int RP>
cudaError_t launch_f(const Attend8Args& a, int grid, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t st) {
  using C = FCfg<D, RP>;
  auto kern = sa_attend8_few_kernel<D, RP>;
  // at least half the SM's shared memory: one block per SM owns its TMEM
  const int smem = C::kSmemBytes > 120 * 1024 ? C::kSmemBytes : 120 * 1024;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kern<<<grid, C::kThreads, smem, st>>>(a, attend8_whole(a), tk, tv);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_d8(const Attend8Args& a, int grid, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t st) {
  const int nr = a.m.R * a.m.Nq;
  cudaError_t e = nr <= 8 ? launch_f<D, 8>(a, grid, tk, tv, st) : launch_f<D, 16>(a, grid, tk, tv, st);
  if (e != cudaSuccess || attend8_whole(a)) return e;
  return launch_early(sa_attend8_join_kernel<D>, dim3(a.m.B * a.m.Hkv * nr), 4 * D, 0, st, a, grid);
}

}  // namespace

// Blocks of the few-row kernel: one an SM, or a tile (a head, where they are not cut) each.
int attend8_few_grid(const Attend8Args& a) {
  const int64_t heads = int64_t(a.m.B) * a.m.Hkv, tiles = heads * ((int64_t(a.m.Nk) + kKeys - 1) / kKeys);
  return static_cast<int>(std::min<int64_t>(attend8_whole(a) ? heads : tiles, kSms));
}

cudaError_t launch_attend8_few(const Attend8Args& a, cudaStream_t st) {
  CUtensorMap tk, tv;
  if (!make_codes_map(&tk, a.k8, a.m.d, a.m.Nk, a.m.Hkv, a.m.B, a.m.ks, kKeys, true) ||
      !make_codes_map(&tv, a.v8, a.m.d, a.m.Nk, a.m.Hkv, a.m.B, a.m.vs, kKeys, true))
    return cudaErrorInvalidValue;
  const int grid = attend8_few_grid(a);
  return a.m.d == 128 ? launch_d8<128>(a, grid, tk, tv, st) : launch_d8<64>(a, grid, tk, tv, st);
}

}  // namespace sa
