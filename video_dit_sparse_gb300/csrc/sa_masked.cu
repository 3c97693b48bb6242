// sa_masked.cu — attention with masks, capped scores and a distance bias.
//
// For a query row at position p and a visible key j (sa_mask.cuh):
//     s_j = cap tanh(scale q.k_j / cap) - slope_h |p - j|
// (without a cap: scale q.k_j; without slopes: no bias),
//     o = sum_j e^(s_j - lse) v_j,   lse = ln sum_j e^(s_j).
// A row that sees no key gets o = 0 and lse = -inf.
//
// Rows of one key head are packed, row = query * R + head-in-group (R = Hq/Hkv
// query heads share a key head), so that K and V are read once for all of
// them.  A block takes 256 packed rows as two 128-row Q tiles (128 rows and one
// tile when a key head has no more).  K and V stream through one ring of
// 128-row tiles by TMA; S = Q K^T and O stay in TMEM, P (bf16) overwrites its S.
// The MMA thread issues PV(j) of a tile and then S(j+1) of the same tile, so
// while one tile's softmax runs the tensor core works for the other.  TMEM is
// full (2 S + 2 O of 128 columns), so a tile's own S cannot be a step ahead:
// the tensor core stays busy only if a softmax takes no longer than the other
// tile's two products (1024 cycles).  One warp needs about 1600 cycles for 32
// rows x 128 columns whatever else runs, so two warps share each row, 64
// columns each (16 softmax warps for two tiles).  They keep separate sums and
// agree on the row's reference through a pair barrier each step.
// Only the key span that the block's rows see is read; tiles that every row
// sees whole skip the mask.
//
// Units that do not fill a last wave of SMs (all of them, for a new token over
// a long cache) are cut into `splits` runs of key tiles; each writes a
// normalised fp32 partial and its lse, and a second kernel joins them:
// o = sum_s e^(lse_s - lse) o_s.
#include <atomic>
#include <cmath>

#include "sa_device.cuh"
#include "sa_internal.h"
#include "sa_mask.cuh"
#include "sa_tma.h"

namespace sa {

namespace {

constexpr int BN = 128;
constexpr int64_t kSms = 152;
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kLog2e = 1.4426950408889634f;
// P is computed against a row reference m that only moves when a tile's sum
// of P passes this (the fp32 sums and O have room for far more).
constexpr float kRaiseLimit = 4294967296.f;

template <int D, int T>
struct MCfg {
  static constexpr int kSoftWarps = 8 * T;  // per Q tile two sets of four: column halves
  static constexpr int kMmaWarp = kSoftWarps, kTmaWarp = kSoftWarps + 1;
  // whole warpgroups: setmaxnreg acts on aligned groups of four warps
  static constexpr int kThreads = 32 * (kSoftWarps + 4);
  static constexpr bool kRegSplit = T == 2;
  // 640 threads launch with 96 registers each = 61440 = 512 * 104 + 128 * 64
  // (fewer than 64 make the MMA thread spill)
  static constexpr int kRegSoft = 104, kRegOther = 64;
  static constexpr int kTile = BN * D * 2;
  static constexpr int kQBytes = T * 128 * D * 2;
  static constexpr int kStages = D == 128 ? (T == 2 ? 4 : 5) : 8;
  static constexpr int kXch = T * 2 * 2 * 128 * 8;  // [slot][tile][half][row] float2
  static constexpr int kSmemBytes = 1024 + kQBytes + kStages * kTile + kXch + 1024;
  static constexpr int kOCol = T * 128;
  static constexpr int kTmemCols = T == 2 ? 512 : 256;
  static_assert(kSmemBytes <= 232448, "shared memory");
};

template <int T, int STAGES>
struct MBars {
  uint64_t full[STAGES], empty[STAGES];
  uint64_t qfull[T], sfull[T], pfull[T], pair[T * 4], drain;
  int flag[T * 4][2];
  uint32_t tmem_base;
  int abort;
};

}  // namespace

template <int D, int T, bool CAP, bool BIAS>
__global__ void __launch_bounds__(MCfg<D, T>::kThreads, 1)
    sa_masked_kernel(const MaskedArgs a, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v) {
  using C = MCfg<D, T>;
  constexpr int S = C::kStages;
  constexpr int W = BIAS ? 16 : 32;  // S columns in registers at a time
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sQ = smem;
  uint8_t* sKV = sQ + C::kQBytes;
  float2* sX = reinterpret_cast<float2*>(sKV + S * C::kTile);
  MBars<T, S>* bars = reinterpret_cast<MBars<T, S>*>(reinterpret_cast<uint8_t*>(sX) + C::kXch);
  volatile int* abort = &bars->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // The block's unit: heads outermost (their K and V stay in L2), row blocks
  // from the last (with a causal mask the longest) to the first.  Units from
  // full_units on are split over their keys.
  int64_t u = blockIdx.x;
  int split = 0, splits = 1;
  int64_t part = -1;  // partial result number
  if (u >= a.full_units) {
    part = u - a.full_units;
    splits = a.splits;
    split = static_cast<int>(part % splits);
    u = a.full_units + part / splits;
  }
  const int rb = a.row_blocks - 1 - static_cast<int>(u % a.row_blocks);
  const int bh = static_cast<int>(u / a.row_blocks);
  const int b = bh / a.Hkv, hk = bh % a.Hkv;
  const int64_t row0 = int64_t(rb) * (128 * T);
  const int rows = static_cast<int>(min64(128 * T, a.rows - row0));

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&bars->full[s], 1);
      mbar_init(&bars->empty[s], 1);
    }
    for (int i = 0; i < T; ++i) {
      mbar_init(&bars->qfull[i], 256);
      mbar_init(&bars->sfull[i], 1);
      mbar_init(&bars->pfull[i], 256);
    }
    for (int i = 0; i < T * 4; ++i) {
      mbar_init(&bars->pair[i], 64);
      bars->flag[i][0] = bars->flag[i][1] = 0;
    }
    mbar_init(&bars->drain, 1);
    bars->abort = 0;
    fence_mbar_init();
  }
  if (warp == C::kMmaWarp) {
    tmem_alloc(&bars->tmem_base, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;

  // Keys that any of the block's rows sees, and this split's run of tiles.
  const int ulo = row_span(a.mask, b, static_cast<int>(row0 / a.R)).lo;
  const int uhi = row_span(a.mask, b, static_cast<int>((row0 + rows - 1) / a.R)).hi;
  const int ntiles = uhi > ulo ? (uhi - ulo + BN - 1) / BN : 0;
  const int j0 = static_cast<int>(int64_t(ntiles) * split / splits);
  const int n = static_cast<int>(int64_t(ntiles) * (split + 1) / splits) - j0;
  const int key0 = ulo + j0 * BN;

  if (C::kRegSplit) {
    if (warp < C::kSoftWarps)
      reg_alloc<C::kRegSoft>();
    else
      reg_dealloc<C::kRegOther>();
  }

  if (warp < C::kSoftWarps) {
    // ------------------------------------------------------------ softmax
    // Warps 8t .. 8t+3 take columns 0-63 of tile t's S (half 0), 8t+4 .. 8t+7
    // columns 64-127; warps of both halves with the same lane quarter share rows.
    const int t = warp >> 3, half = (warp >> 2) & 1, quarter = warp & 3;
    constexpr int H = BN / 2;
    const int tid = threadIdx.x & 255;                  // among the tile's 256 threads
    const int trow = quarter * 32 + lane;               // row of the tile
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const int wrow0 = t * 128 + quarter * 32;           // the warp's first row in the block
    const bool idle = wrow0 >= rows;                    // none of its rows exists
    const bool valid = wrow0 + lane < rows;
    const int64_t grow = row0 + wrow0 + lane;
    const int qi = valid ? static_cast<int>(grow / a.R) : 0;
    const int hq = hk * a.R + (valid ? static_cast<int>(grow % a.R) : 0);
    if (n > 0) {
      // The tile's Q rows, swizzled as the MMA reads them (missing rows zero).
      const uint32_t q_addr = smem_u32(sQ) + t * 128 * D * 2;
      constexpr int kCh = D / 8;  // 16-byte pieces of a row
#pragma unroll 4
      for (int c = 0; c < kCh / 2; ++c) {
        const int e = c * 256 + tid, r = e / kCh, ch = e % kCh;
        const bool ok = t * 128 + r < rows;
        const int64_t g = row0 + t * 128 + r;
        const int64_t q = ok ? g / a.R : 0;
        const int64_t h = hk * a.R + (ok ? g % a.R : 0);
        cp_async16(q_addr + sw128_offset(r, ch, 128),
                   a.q + int64_t(b) * a.qs.b + h * a.qs.h + q * a.qs.n + ch * 8, ok ? 16u : 0u);
      }
      cp_async_commit();
      cp_async_wait<0>();
      fence_proxy_async_smem();
      mbar_arrive(&bars->qfull[t]);
    }
    Span sp = {0, 0, 0};
    if (valid) sp = row_span(a.mask, b, qi);
    const float sl = a.scale_log2;
    float nslope = 0.f;
    if (BIAS && valid) nslope = -__ldg(a.slopes + hq) * kLog2e;
    float m = -INFINITY, l = 0.f, lr = 0.f;
    const uint32_t sbase = tmem + lane_base + t * 128 + half * H;
    uint64_t* pair = &bars->pair[t * 4 + quarter];
    volatile int* flag = bars->flag[t * 4 + quarter];
    uint32_t xn = 0;  // pair exchanges so far
    // Slot of exchange xn: this half's value, and the other half's.
    auto mine = [&]() -> float2* { return sX + (((xn & 1) * T + t) * 2 + half) * 128 + trow; };
    auto other = [&]() -> float2* { return sX + (((xn & 1) * T + t) * 2 + (half ^ 1)) * 128 + trow; };
    auto pair_sync = [&]() -> bool {
      mbar_arrive(pair);
      const bool ok = mbar_wait(pair, xn & 1, abort);
      return ok;
    };
    constexpr bool kUnits = CAP || BIAS;  // scores are brought to exp2 units first
    for (int j = 0; j < n; ++j) {
      if (!mbar_wait(&bars->sfull[t], j & 1, abort)) goto done;
      if (idle) {
        mbar_arrive(&bars->pfull[t]);
        continue;
      }
      __syncwarp();
      tc_fence_after();
      const int c0 = key0 + j * BN + half * H;  // key of the half's first column
      const int va = sp.lo - c0, vb = sp.hi - c0;
      const bool edge = __any_sync(0xffffffffu, va > 0 || vb < H);
      // W raw scores -> capped, biased and masked ones (in place)
      auto prepare = [&](float* x, int base) {
        if constexpr (CAP) {
          // cap tanh(y) = cap (1 - 2 / (1 + e^2y)), in exp2 units; exact at both
          // ends (e^2y = inf or 0), absolute error about 1e-7 cap
          const uint64_t k1 = f2(a.cap_k1, a.cap_k1), one = f2(1.f, 1.f);
          const uint64_t cc = f2(a.cap_log2, a.cap_log2), mc = f2(-2.f * a.cap_log2, -2.f * a.cap_log2);
#pragma unroll
          for (int c = 0; c < W; c += 2) {
            const uint64_t e = mul2(f2(x[c], x[c + 1]), k1);
            const uint64_t d1 = add2(f2(fast_exp2(f2lo(e)), fast_exp2(f2hi(e))), one);
            const uint64_t y = fma2(f2(fast_rcp(f2lo(d1)), fast_rcp(f2hi(d1))), mc, cc);
            x[c] = f2lo(y);
            x[c + 1] = f2hi(y);
          }
        }
        if constexpr (BIAS) {
          const float t0 = static_cast<float>(sp.pos - c0 - base);
          const uint64_t ns2 = f2(nslope, nslope), sl2 = f2(sl, sl);
#pragma unroll
          for (int c = 0; c < W; c += 2) {
            const uint64_t dist = f2(fabsf(t0 - static_cast<float>(c)), fabsf(t0 - static_cast<float>(c + 1)));
            uint64_t y = f2(x[c], x[c + 1]);
            if (!CAP) y = mul2(y, sl2);
            y = fma2(ns2, dist, y);
            x[c] = f2lo(y);
            x[c + 1] = f2hi(y);
          }
        }
        if (edge) {
#pragma unroll
          for (int c = 0; c < W; ++c)
            if (base + c < va || base + c >= vb) x[c] = -INFINITY;
        }
      };
      auto load = [&](float* x, int base) {
        if constexpr (W == 32)
          tmem_ld32(sbase + base, reinterpret_cast<uint32_t*>(x));
        else
          tmem_ld16(sbase + base, reinterpret_cast<uint32_t*>(x));
      };
      // The row's largest score so far in this tile, over both halves.
      auto row_max = [&](float* res) -> bool {
        float mx = -INFINITY;
#pragma unroll
        for (int base = 0; base < H; base += W) {
          float x[W];
          load(x, base);
          tmem_ld_wait();
          prepare(x, base);
#pragma unroll
          for (int c = 0; c < W; c += 2) mx = fmax3(mx, x[c], x[c + 1]);
        }
        *mine() = make_float2(kUnits ? mx : sl * mx, 0.f);
        if (!pair_sync()) return false;
        *res = fmaxf(mine()->x, other()->x);
        ++xn;
        return true;
      };
      // P = exp2(x - mm) as bf16 pairs, its fp32 sum (for lse) and the sum of
      // the rounded values, which normalises O (so that O stays a convex
      // combination of V rows whatever the rounding of P to bf16).
      uint32_t p[H / 2];
      float ts, tr;
      auto exps = [&](float mm) {
        const uint64_t sl2 = f2(sl, sl), nm2 = f2(-mm, -mm);
        uint64_t ps[2] = {0, 0};
        float pr[2] = {0.f, 0.f};
        auto some = [&](const float* x, uint32_t* pp) {
#pragma unroll
          for (int c = 0; c < W / 2; ++c) {
            const uint64_t xx = f2(x[2 * c], x[2 * c + 1]);
            const uint64_t y = kUnits ? add2(xx, nm2) : fma2(xx, sl2, nm2);
            const float p0 = fast_exp2(f2lo(y)), p1 = fast_exp2(f2hi(y));
            pp[c] = pack_bf16(p0, p1);
            ps[c & 1] = add2(ps[c & 1], f2(p0, p1));
            pr[c & 1] = add_bf16x2(pp[c], pr[c & 1]);
          }
        };
#pragma unroll
        for (int base = 0; base < H; base += W) {
          float x[W];
          load(x, base);
          tmem_ld_wait();
          prepare(x, base);
          some(x, p + base / 2);
        }
        const uint64_t s2 = add2(ps[0], ps[1]);
        ts = f2lo(s2) + f2hi(s2);
        tr = pr[0] + pr[1];
      };
      // The first tile that shows a row a key sets its reference; later tiles
      // raise it only when needed.  (A row without one has P = 0, l = 0, O = 0.)
      // Both warps of a pair hold the same references and spans, so they agree.
      const bool first = j == 0 || __any_sync(0xffffffffu, m == -INFINITY && sp.hi > sp.lo);
      if (first) {
        float mx;
        if (!row_max(&mx)) goto done;
        if (m == -INFINITY) m = mx;
      }
      exps(m == -INFINITY ? 0.f : m);
      {
        // either half's sum too large: both raise
        const bool bad = j > 0 && __any_sync(0xffffffffu, !(ts <= kRaiseLimit));
        if (bad && lane == 0) flag[xn & 1] = j + 1;
        __syncwarp();
        if (!pair_sync()) goto done;
        const bool raise = flag[xn & 1] == j + 1;
        ++xn;
        if (raise) {
          float mx;
          if (!row_max(&mx)) goto done;
          const float mn = fmaxf(m, mx);
          const float alpha = m == mn ? 1.f : fast_exp2(m - mn);
          m = mn;
          l *= alpha;
          lr *= alpha;
          // O holds PV of every earlier tile: its commit came with this S.
          const uint32_t obase = tmem + lane_base + C::kOCol + t * D + half * (D / 2);
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {
            uint32_t r[32];
            tmem_ld32(obase + c * 32, r);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * alpha);
            tmem_st32(obase + c * 32, r);
          }
          exps(m == -INFINITY ? 0.f : m);
        }
      }
      l += ts;
      lr += tr;
      tmem_st32(sbase, p);
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&bars->pfull[t]);
    }
    if (n > 0) {
      if (!mbar_wait(&bars->sfull[t], n & 1, abort)) goto done;
      __syncwarp();
      tc_fence_after();
    }
    if (!idle) {
      // both halves' sums; each half writes its half of the row
      *mine() = make_float2(l, lr);
      if (!pair_sync()) goto done;
      l += other()->x;
      lr += other()->y;
      ++xn;
      const float inv = l == 0.f ? 0.f : 1.f / lr;
      if (valid && half == 0) {
        const float lse = l == 0.f ? -INFINITY : m * kLn2 + logf(l);
        if (part >= 0)
          a.part_lse[part * (128 * T) + wrow0 + lane] = lse;
        else if (a.lse)
          a.lse[(int64_t(b) * a.Hq + hq) * a.Nq + qi] = lse;
      }
      const uint32_t obase = tmem + lane_base + C::kOCol + t * D + half * (D / 2);
      const int64_t oo = int64_t(b) * a.os.b + int64_t(hq) * a.os.h + int64_t(qi) * a.os.n + half * (D / 2);
      float* dst32 = part >= 0 ? a.part_o + (part * (128 * T) + wrow0 + lane) * D + half * (D / 2)
                               : static_cast<float*>(a.o) + oo;
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        float v[32];
        if (n > 0) {
          tmem_ld32(obase + c * 32, reinterpret_cast<uint32_t*>(v));
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = inv == 0.f ? 0.f : v[e] * inv;
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = 0.f;
        }
        if (valid && (part >= 0 || a.out_fp32)) {
          float4* dst = reinterpret_cast<float4*>(dst32 + c * 32);
#pragma unroll
          for (int e = 0; e < 8; ++e) dst[e] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
        } else if (valid) {
          uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.o) + oo + c * 32);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            dst[e] = make_uint4(pack_bf16(v[8 * e], v[8 * e + 1]), pack_bf16(v[8 * e + 2], v[8 * e + 3]),
                                pack_bf16(v[8 * e + 4], v[8 * e + 5]), pack_bf16(v[8 * e + 6], v[8 * e + 7]));
        }
        __syncwarp();
      }
    }
  } else if (warp == C::kMmaWarp) {
    // ------------------------------------------------------------ MMA issue
    const uint32_t kIdescS = a.neg_scale ? idesc_negate_b(idesc_bf16(128, BN, false, false))
                                         : idesc_bf16(128, BN, false, false);
    constexpr uint32_t kIdescPV = idesc_bf16(128, D, false, true);
    const uint32_t q_addr = smem_u32(sQ), kv_addr = smem_u32(sKV);
    bool ok = n > 0;
    auto ready = [&](int i) -> bool { return mbar_wait(&bars->full[i % S], (i / S) & 1, abort); };
    auto qk = [&](int t, int i) {
      const uint32_t ka = kv_addr + (i % S) * C::kTile, qa = q_addr + t * 128 * D * 2;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = (kk >> 2) * 128 * 128 + (kk & 3) * 32;
        mma_ss(tmem + t * 128, sw128_desc(qa + off, 16, 1024), sw128_desc(ka + off, 16, 1024), kIdescS,
               kk > 0 ? 1u : 0u);
      }
    };
    auto pv = [&](int t, int i, bool first) {
      const uint32_t va = kv_addr + (i % S) * C::kTile;
#pragma unroll
      for (int kk = 0; kk < BN / 16; ++kk)
        // P of keys 0-63 lies in S columns 0-31, of keys 64-127 in 64-95
        mma_ts(tmem + C::kOCol + t * D, tmem + t * 128 + (kk >> 2) * 64 + (kk & 3) * 8, sw128_desc(va + kk * 2048, BN * 128, 1024),
               kIdescPV, (!first || kk > 0) ? 1u : 0u);
    };
    // Ring entries: K(j) is number 2j, V(j) is 2j + 1.
    if (ok) ok = ready(0);
    if (ok) {
      for (int t = 0; t < T && ok; ++t) {
        ok = mbar_wait(&bars->qfull[t], 0, abort);
        if (!ok) break;
        tc_fence_after();
        if (lane == 0) {
          qk(t, 0);
          mma_commit(&bars->sfull[t]);
        }
      }
      if (ok && lane == 0) mma_commit(&bars->empty[0]);
    }
    for (int j = 0; j < n && ok; ++j) {
      const bool more = j + 1 < n;
      if (!(ok = ready(2 * j + 1)) || (more && !(ok = ready(2 * j + 2)))) break;
      // V rows past the span (another document's, or a cache's unused rows)
      // meet P = 0, but 0 times a NaN or an infinity would still reach O.
      const int live = uhi - (key0 + j * BN);
      if (live < BN) {
        uint8_t* vt = sKV + ((2 * j + 1) % S) * C::kTile;
        for (int e = lane; e < (BN - live) * (D / 8); e += 32) {
          const int r = live + e / (D / 8), ch = e % (D / 8);
          *reinterpret_cast<uint4*>(vt + (ch >> 3) * BN * 128 + r * 128 + (ch & 7) * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
      }
      for (int t = 0; t < T && ok; ++t) {
        ok = mbar_wait(&bars->pfull[t], j & 1, abort);
        if (!ok) break;
        tc_fence_after();
        if (lane == 0) {
          pv(t, 2 * j + 1, j == 0);
          if (more) qk(t, 2 * j + 2);
          mma_commit(&bars->sfull[t]);
        }
      }
      if (ok && lane == 0) {
        mma_commit(&bars->empty[(2 * j + 1) % S]);
        if (more) mma_commit(&bars->empty[(2 * j + 2) % S]);
      }
      __syncwarp();
    }
    if (lane == 0) {
      // Every MMA issued above must finish before TMEM is released.
      mma_commit(&bars->drain);
      const long long t0 = clock64();
      while (!mbar_test(&bars->drain, 0) && clock64() - t0 < kWaitLimitCycles) {
      }
    }
  } else if (warp == C::kTmaWarp && lane == 0) {
    // ------------------------------------------------------------ loads (TMA)
    const uint32_t kv_addr = smem_u32(sKV);
    int issued = 0;
    for (int i = 0; i < 2 * n; ++i) {
      const int s = i % S;
      if (!mbar_wait(&bars->empty[s], ((i / S) & 1) ^ 1, abort)) break;
      mbar_expect_tx(&bars->full[s], C::kTile);
      const int key = key0 + (i >> 1) * BN;
#pragma unroll
      for (int cb = 0; cb < D / 64; ++cb)
        tma_load_4d(kv_addr + s * C::kTile + cb * BN * 128, (i & 1) ? &tm_v : &tm_k, 64 * cb, key, hk, b,
                    &bars->full[s]);
      issued = i + 1;
    }
    // After an abort: the copies in flight land before the block ends.
    if (*abort)
      for (int i = issued > S ? issued - S : 0; i < issued; ++i) {
        const long long t0 = clock64();
        while (!mbar_test(&bars->full[i % S], (i / S) & 1) && clock64() - t0 < kWaitLimitCycles) {
        }
      }
  }
done:
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && bars->abort) report(a.status, SA_DEVERR_TIMEOUT);
  if (warp == C::kMmaWarp) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// One warp per row of a split unit: lse = ln sum_s e^(lse_s),
// o = sum_s e^(lse_s - lse) o_s.
template <int D>
__global__ void __launch_bounds__(256) sa_masked_join_kernel(const MaskedArgs a, int unit_rows) {
  const int64_t i = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int64_t su = i / unit_rows;  // split unit
  const int r = static_cast<int>(i % unit_rows);
  const int64_t u = a.full_units + su;
  const int64_t bh = u / a.row_blocks;
  if (bh >= int64_t(a.B) * a.Hkv) return;
  const int64_t row = (a.row_blocks - 1 - u % a.row_blocks) * unit_rows + r;
  if (row >= a.rows) return;
  const float* pl = a.part_lse + su * a.splits * unit_rows + r;
  float mx = -INFINITY;
  for (int s = lane; s < a.splits; s += 32) mx = fmaxf(mx, __ldg(pl + s * unit_rows));
#pragma unroll
  for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  constexpr int V = D / 32;
  float acc[V] = {}, sum = 0.f;
  if (mx != -INFINITY)
    for (int s = 0; s < a.splits; ++s) {
      const float w = __expf(__ldg(pl + s * unit_rows) - mx);
      sum += w;
      const float* src = a.part_o + ((su * a.splits + s) * unit_rows + r) * D + lane * V;
#pragma unroll
      for (int e = 0; e < V; ++e) acc[e] += w * src[e];
    }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const int64_t q = row / a.R, h = (bh % a.Hkv) * a.R + row % a.R, b = bh / a.Hkv;
  const int64_t oo = b * a.os.b + h * a.os.h + q * a.os.n + lane * V;
#pragma unroll
  for (int e = 0; e < V; e += 2) {
    if (a.out_fp32)
      *reinterpret_cast<float2*>(static_cast<float*>(a.o) + oo + e) = make_float2(acc[e] * inv, acc[e + 1] * inv);
    else
      *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.o) + oo + e) = pack_bf16(acc[e] * inv, acc[e + 1] * inv);
  }
  if (lane == 0 && a.lse) a.lse[(b * a.Hq + h) * a.Nq + q] = sum == 0.f ? -INFINITY : mx + logf(sum);
}

// Units that fill whole waves of SMs run whole; the rest (all, if they are
// fewer than the SMs) are split into the number of key runs that ends first by
// this count of tile times: a wave costs its tiles plus a block's start, a
// split the join.
void masked_plan(MaskedArgs* a) {
  const int T = a->rows > 128 ? 2 : 1;
  a->unit_rows = 128 * T;
  a->row_blocks = static_cast<int32_t>((a->rows + a->unit_rows - 1) / a->unit_rows);
  const int64_t units = int64_t(a->B) * a->Hkv * a->row_blocks, rest = units % kSms;
  const int64_t tiles = (int64_t(a->Nk) + BN - 1) / BN;
  constexpr int64_t kStart = 5, kJoin = 8;
  int64_t best = 1, cost = tiles + kStart;
  for (int64_t s = 2; s <= tiles && s <= 64 && rest; ++s) {
    const int64_t c = (rest * s + kSms - 1) / kSms * ((tiles + s - 1) / s + kStart) + kJoin;
    if (c < cost) {
      cost = c;
      best = s;
    }
  }
  a->splits = static_cast<int32_t>(best);
  a->full_units = best == 1 ? units : units - rest;
  a->split_units = units - a->full_units;
}

template <int D, int T, bool CAP, bool BIAS>
static cudaError_t launch_m(const MaskedArgs& a, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t st) {
  using C = MCfg<D, T>;
  auto kern = sa_masked_kernel<D, T, CAP, BIAS>;
  // at least half the SM's shared memory: one block per SM owns its TMEM
  const int smem = C::kSmemBytes > 120 * 1024 ? C::kSmemBytes : 120 * 1024;
  static std::atomic<int> regs_ok{0};  // 0 unknown, 1 enough, 2 too few
  if (regs_ok.load() == 0) {
    cudaFuncAttributes attr;
    cudaError_t e = cudaFuncGetAttributes(&attr, kern);
    if (e != cudaSuccess) return e;
    // setmaxnreg.inc waits until the block's launch registers cover the split
    const long need = long(C::kRegSoft) * C::kSoftWarps * 32 + long(C::kRegOther) * 128;
    regs_ok.store(!C::kRegSplit || long(attr.numRegs) * C::kThreads >= need ? 1 : 2);
  }
  if (regs_ok.load() != 1) return cudaErrorLaunchOutOfResources;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int64_t grid = a.full_units + a.split_units * a.splits;
  kern<<<static_cast<unsigned>(grid), C::kThreads, smem, st>>>(a, tk, tv);
  return cudaGetLastError();
}

template <int D, int T>
static cudaError_t launch_t(const MaskedArgs& a, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t st) {
  const bool cap = a.cap_log2 > 0.f, bias = a.slopes != nullptr;
  if (cap) return bias ? launch_m<D, T, true, true>(a, tk, tv, st) : launch_m<D, T, true, false>(a, tk, tv, st);
  return bias ? launch_m<D, T, false, true>(a, tk, tv, st) : launch_m<D, T, false, false>(a, tk, tv, st);
}

cudaError_t launch_masked(const MaskedArgs& a, cudaStream_t st) {
  CUtensorMap tk, tv;
  if (!make_view_map(&tk, a.k, a.d, a.Nk, a.Hkv, a.B, a.ks.n, a.ks.h, a.ks.b, BN, 1, false) ||
      !make_view_map(&tv, a.v, a.d, a.Nk, a.Hkv, a.B, a.vs.n, a.vs.h, a.vs.b, BN, 1, false))
    return cudaErrorInvalidValue;
  const bool two = a.unit_rows == 256;
  cudaError_t e = a.d == 128 ? (two ? launch_t<128, 2>(a, tk, tv, st) : launch_t<128, 1>(a, tk, tv, st))
                             : (two ? launch_t<64, 2>(a, tk, tv, st) : launch_t<64, 1>(a, tk, tv, st));
  if (e != cudaSuccess || a.split_units == 0) return e;
  const unsigned blocks = static_cast<unsigned>((a.split_units * a.unit_rows + 7) / 8);
  if (a.d == 128)
    sa_masked_join_kernel<128><<<blocks, 256, 0, st>>>(a, a.unit_rows);
  else
    sa_masked_join_kernel<64><<<blocks, 256, 0, st>>>(a, a.unit_rows);
  return cudaGetLastError();
}

}  // namespace sa
