// sa_attend8_many.cu — attention of many query rows over an 8-bit cache.
//
// Rows of one key head are packed, row = query * R + head-in-group, and a unit is two tiles of up to 128 packed rows that
// take K and V from one ring, as in sa_masked.cu.  What differs is how eight bits reach the tensor cores.
//
// S = Q K^T takes K's codes as they are (kind::f8f6f4) and the query rows in two e4m3 terms (sa_attend8.cuh): two
// products at twice the rate.  K's scale belongs to a column: it is a factor of the row's multiplier, the same for
// the 16 columns that a chunk of the softmax works on.
//
// O = P V cannot have P in eight bits (a term holds four digits, and cutting P in terms would cost the softmax more
// than its exponentials).  So V's codes become fp16 on the way: one instruction for two of them, exact.
// V's scale goes into P's exponent, P = 2^(x + log2 vs - m), where it is free, and comes out of the row's sum as
// one factor a chunk.  P in fp16 keeps eleven digits; its range holds because a row's largest weight starts at 2^6 and
// the reference m moves before a half row's sum passes 2^15: what is lost lies below 2^-31 of the row's largest.
//
// A V tile is cleared where no row of the unit sees it and where a block is empty (whose keys count less for the
// reference: sa_attend8.cuh); a NaN among its codes is cleared too and noted by its column: rows see the first keys of the
// cache, so a column's first NaN says which rows get one.
//
// Warps: sixteen softmax warps (two a row, 64 columns each), an MMA warp a tile taking turns, one for units and loads.
// The softmax warps convert V too, a sixteenth of the next tile each behind their P, while they would wait for S
// (a warp of its own for it took 5000 cycles a tile: 12 heads, 7040 rows x 28160 keys 1124 us), and make the next
// unit's query terms between their last tile and the output, so that its first S is computed beside the output.
#include <atomic>

#include "sa_attend8.cuh"

namespace sa {

namespace {

constexpr int BN = 128;  // keys of a tile
constexpr int kRing = 2;  // units in flight
constexpr float kTop = 6.f;            // a row's largest weight of its first tile is 2^6
constexpr float kUnit = 64.f;          // 2^kTop
constexpr float kMostSum = 32768.f;    // of half a row's weights in a tile
constexpr float kNoScale = INFINITY;   // of a unit that no block with values has shown up in

template <int D>
struct ACfg {
  static constexpr int kSoftWarps = 16, kMmaWarp = 16, kTmaWarp = 18;
  static constexpr int kThreads = 640;
  // 640 threads launch with 96 registers each = 61440 = 512 * 104 + 128 * 64
  static constexpr int kRegSoft = 104, kRegOther = 64;
  static constexpr int kTile = BN * D;  // bytes of a tile of codes
  static constexpr int kKStages = D == 128 ? 2 : 4, kCStages = D == 128 ? 2 : 3, kVStages = D == 128 ? 2 : 4;
  static constexpr int kQ = 0, kK = kQ + 4 * kTile, kC = kK + kKStages * kTile, kV = kC + kCStages * kTile,
                       kX = kV + kVStages * 2 * kTile;
  static constexpr int kWarpBytes = 2048;  // a softmax warp's own: exchange slots, output staging
  static constexpr int kSmemBytes = 1024 + kX + kSoftWarps * kWarpBytes;
  static constexpr int kOCol = 256, kTmemCols = 512;
  static_assert(kSmemBytes <= 232448 - 2048, "shared memory (beside 2 KB of barriers)");
};

struct AUnit {
  int go;              // 0: no more units
  int key0, n, uhi;    // first key, key tiles, end of the rows' keys
  int part, q0, b, hk; // partial result (-1: whole), first query, batch entry, key head
  int two;             // the second tile has rows
};

template <int D>
struct ABars {
  using C = ACfg<D>;
  uint64_t kfull[C::kKStages], kempty[C::kKStages], cfull[C::kCStages], cempty[C::kCStages], vfull[C::kVStages],
      vempty[C::kVStages];
  uint64_t qfull[2], sfull[2], pfull[2], ofull[2], ofree[2], turn[2], drain[2], next, ring_full[kRing], ring_empty[kRing];
  uint4 answer;
  AUnit ring[kRing];
  int nans[kRing];  // a unit's values hold a NaN
  uint32_t tmem_base;
  int abort;
};

// How many of `count` threads say so, on hardware barrier `id`.
__device__ __forceinline__ uint32_t count_of(int id, int count, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %3, 0;\n\t"
      "barrier.cta.red.popc.u32 %0, %1, %2, p;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(count), "r"(static_cast<uint32_t>(x))
      : "memory");
  return r;
}

template <class T, T N>
struct Constant {
  static constexpr T value = N;
};

}  // namespace

// NB: scales that a warp's 64 columns have (blocks of 64 and more: 1; 32: 2; 16: 4).
template <int D, int NB>
__global__ void __launch_bounds__(ACfg<D>::kThreads, 1)
    sa_attend8_many_kernel(const __grid_constant__ Attend8Args a, const __grid_constant__ CUtensorMap tm_k,
                           const __grid_constant__ CUtensorMap tm_v) {
  using C = ACfg<D>;
  constexpr int W = 16;      // S columns a register buffer holds; a chunk has one scale
  constexpr int H = BN / 2;  // columns of a warp
  static_assert(sizeof(ABars<D>) + kRing * D * 4 <= 2048, "shared memory");
  extern __shared__ uint8_t smem_raw[];
  __shared__ ABars<D> bars;
  __shared__ int nan_at[kRing][D];  // a unit's first key with a NaN in each column of V
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  volatile int* abort = &bars.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const MaskedArgs& m_ = a.m;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kKStages; ++s) {
      mbar_init(&bars.kfull[s], 1);
      mbar_init(&bars.kempty[s], 2);
    }
    for (int s = 0; s < C::kCStages; ++s) {
      mbar_init(&bars.cfull[s], 1);
      mbar_init(&bars.cempty[s], C::kSoftWarps);
    }
    for (int s = 0; s < C::kVStages; ++s) {
      mbar_init(&bars.vfull[s], C::kSoftWarps);
      mbar_init(&bars.vempty[s], 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.qfull[i], 8);
      mbar_init(&bars.sfull[i], 1);
      mbar_init(&bars.pfull[i], 8);
      mbar_init(&bars.ofull[i], 1);
      mbar_init(&bars.ofree[i], 8);
      mbar_init(&bars.turn[i], 1);
      mbar_init(&bars.drain[i], 1);
    }
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&bars.ring_full[i], 1);
      mbar_init(&bars.ring_empty[i], C::kSoftWarps + 2);
    }
    mbar_init(&bars.next, 1);
    bars.abort = 0;
    fence_mbar_init();
  }
  if (warp == C::kMmaWarp) {
    tmem_alloc(&bars.tmem_base, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars.tmem_base;
  if (warp < C::kSoftWarps)
    reg_alloc<C::kRegSoft>();
  else
    reg_dealloc<C::kRegOther>();

  auto unit_here = [&](uint32_t i) -> bool { return mbar_wait(&bars.ring_full[i % kRing], (i / kRing) & 1, abort); };

  if (warp < C::kSoftWarps) {
    // ------------------------------------------------------------ softmax
    const int t = warp >> 3, half = (warp >> 2) & 1, quarter = warp & 3;
    const int col0 = half * H;
    const int trow = quarter * 32 + lane;  // row of the tile
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t sbase = tmem + lane_base + t * 128 + col0;
    const uint32_t obase = tmem + lane_base + C::kOCol + t * D + half * (D / 2);
    const int rq = trow / m_.R, rh = trow - rq * m_.R;  // its query and head in the tile
    const bool in_tile = trow < m_.qn * m_.R;
    uint32_t xn = 0;          // pair exchanges so far
    uint32_t tc = 0, uc = 0;  // key tiles and units with keys of this Q tile so far
    uint8_t* own = smem + C::kX + warp * C::kWarpBytes;
    auto mine = [&]() -> float2* { return reinterpret_cast<float2*>(own) + (xn & 1) * 32 + lane; };
    auto other = [&]() -> float2* {
      return reinterpret_cast<float2*>(smem + C::kX + (warp ^ 4) * C::kWarpBytes) + (xn & 1) * 32 + lane;
    };
    // A warp's arrival (a barrier counts its warps: 256 threads' arrivals one by one took as long as the store of P).
    auto arrive = [&](uint64_t* bar) {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    // Meets the other half's warp: how many of the two ask for something (one of their lanes counts).  At its end a
    // warp meets it once more, and all its lanes count: whoever it meets elsewhere gives up too.
    bool alone = false;  // the other warp has given up, and waits no more
    auto meet = [&](bool ask) -> uint32_t {
      const uint32_t n = count_of(1 + t * 4 + quarter, 64, ask && lane == 0);
      alone = n >= 32;
      return n;
    };
    auto pair_sync = [&]() -> bool { return meet(false) < 32; };
    // Scales that the warp needs of a tile, fetched a tile ahead: lanes 0-3 the key scales of its four chunks of columns,
    // lanes 4-7 the value scales, lane 8 that of the eight keys whose values it converts.
    const float* scales = nullptr;
    float ahead = 0.f;
    auto fetch = [&](int k0) -> float {
      const int key = min(k0 + (lane < 8 ? col0 + (lane & 3) * W : warp * 8), m_.Nk - 1);
      return __ldg(scales + (key >> a.block_log2));  // (as it is: a look at it here would wait for it)
    };
    // The warp's eight keys of a tile's values from codes to fp16.
    uint32_t vc = 0;  // tiles converted so far
    auto convert = [&](uint32_t slot, int k0) -> bool {
      constexpr int kLanes = D / 16, kRows = 32 / kLanes;  // lanes a row, rows at a time
      // d = 128: eight lanes load and store 16-byte pieces without bank conflicts if they are four of row r and four of
      // row r ^ 5, the codes as the 128-byte swizzle has them
      const int r_lane = D == 128 ? lane >> 3 ^ ((lane & 4) ? 5 : 0) : lane / kLanes, p_lane = lane & 3;
      auto row_of = [&](int y) -> int { return warp * 8 + r_lane + (D == 128 ? 0 : y * kRows); };
      auto piece_of = [&](int y) -> int { return D == 128 ? p_lane + 4 * y : p_lane; };
      const uint32_t cs = vc % C::kCStages, vs = vc % C::kVStages;
      const bool filled = held_scale(__shfl_sync(0xffffffffu, ahead, 8)) > 0.f;
      const int live = filled ? bars.ring[slot].uhi - k0 : 0;
      if (!mbar_wait(&bars.cfull[cs], (vc / C::kCStages) & 1, abort) ||
          !mbar_wait(&bars.vempty[vs], ((vc / C::kVStages) & 1) ^ 1, abort))
        return false;
      __syncwarp();
      uint4 w[8 / kRows];
      uint32_t bad = 0;
#pragma unroll
      for (int y = 0; y < 8 / kRows; ++y) {
        const int r = row_of(y);
        w[y] = *reinterpret_cast<const uint4*>(smem + C::kC + cs * C::kTile +
                                               (D == 128 ? rows8_offset<D>(r, piece_of(y) * 16) : r * D + p_lane * 16));
        if (r >= live) w[y] = make_uint4(0, 0, 0, 0);
        bad |= ((w[y].x & 0x7F7F7F7Fu) + 0x01010101u) | ((w[y].y & 0x7F7F7F7Fu) + 0x01010101u) |
               ((w[y].z & 0x7F7F7F7Fu) + 0x01010101u) | ((w[y].w & 0x7F7F7F7Fu) + 0x01010101u);
      }
      if (bad & 0x80808080u) {
        bars.nans[slot] = 1;
#pragma unroll
        for (int y = 0; y < 8 / kRows; ++y) {
          auto sift = [&](uint32_t e, int p) -> uint32_t {
            for (int b = 0; b < 4; ++b)
              if ((e >> (8 * b) & 127) == 127) {
                atomicMin(&nan_at[slot][piece_of(y) * 16 + p + b], k0 + row_of(y));
                e &= ~(255u << (8 * b));
              }
            return e;
          };
          w[y] = make_uint4(sift(w[y].x, 0), sift(w[y].y, 4), sift(w[y].z, 8), sift(w[y].w, 12));
        }
      }
#pragma unroll
      for (int y = 0; y < 8 / kRows; ++y) {
        const int r = row_of(y), ch = p_lane * 2;
        uint8_t* row = smem + C::kV + vs * 2 * C::kTile + (piece_of(y) >> 2) * BN * 128 + r * 128;
        *reinterpret_cast<uint4*>(row + ((ch ^ (r & 7)) << 4)) =
            make_uint4(decode2(w[y].x & 0xFFFFu), decode2(w[y].x >> 16), decode2(w[y].y & 0xFFFFu), decode2(w[y].y >> 16));
        *reinterpret_cast<uint4*>(row + (((ch + 1) ^ (r & 7)) << 4)) =
            make_uint4(decode2(w[y].z & 0xFFFFu), decode2(w[y].z >> 16), decode2(w[y].w & 0xFFFFu), decode2(w[y].w >> 16));
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&bars.vfull[vs]);
        mbar_arrive(&bars.cempty[cs]);
      }
      ++vc;
      return true;
    };
    // log2 of what value scales count from, as a tile of unit x has it (of keys that some row of the unit sees).
    auto scale_from = [&](const AUnit& x, int k0) -> float {
      const float s = first_scale(a.v_scale + int64_t(x.b) * a.v_scales.b + int64_t(x.hk) * a.v_scales.h, k0, BN, x.uhi, a.block_log2);
      return s > 0.f ? __log2f(s) : kNoScale;
    };
    // The row of the next unit: keys it sees, its multiplier, what value scales count from.
    int hi_next = 0;
    float rf_next = 0.f, lref_next = 0.f;
    // The next unit's query terms into shared memory, and its first values.  (The last unit's products have read
    // the old terms: its last S is here.)
    auto prepare = [&](uint32_t slot) -> bool {
      const AUnit& x = bars.ring[slot];
      hi_next = 0;
      if (x.n == 0) return true;
      scales = lane < 4 ? a.k_scale + int64_t(x.b) * a.k_scales.b + int64_t(x.hk) * a.k_scales.h
                        : a.v_scale + int64_t(x.b) * a.v_scales.b + int64_t(x.hk) * a.v_scales.h;
      ahead = fetch(x.key0);
      if (t == 0 || x.two) {
        const int qi = x.q0 + t * m_.qn + rq;
        const bool valid = in_tile && qi < m_.Nq;
        uint4 u[D / 16];
        uint32_t top = 0;
        const uint16_t* q = m_.q + int64_t(x.b) * m_.qs.b + int64_t(x.hk * m_.R + rh) * m_.qs.h + int64_t(qi) * m_.qs.n + half * (D / 2);
#pragma unroll
        for (int p = 0; p < D / 16; ++p) u[p] = valid ? *reinterpret_cast<const uint4*>(q + p * 8) : make_uint4(0, 0, 0, 0);
        if (valid) hi_next = row_span(m_.mask, x.b, qi).hi;
#pragma unroll
        for (int p = 0; p < D / 16; ++p) top = top_of(u[p], top);
        *mine() = make_float2(__uint_as_float(top), 0.f);
        if (!pair_sync()) return false;
        top = max(top, __float_as_uint(other()->x));
        ++xn;
        const float f = row_factor(top);
        rf_next = a.scale_log2 / f;
        uint8_t* sq = smem + C::kQ + t * 2 * C::kTile;
#pragma unroll
        for (int p = 0; p < D / 16; p += 2) {
          uint2 h0, l0, h1, l1;
          two_terms(u[p], f, 1.f, &h0, &l0);
          two_terms(u[p + 1], f, 1.f, &h1, &l1);
          const uint32_t at = rows8_offset<D>(trow, half * (D / 2) + p * 8);
          *reinterpret_cast<uint4*>(sq + at) = make_uint4(h0.x, h0.y, h1.x, h1.y);
          *reinterpret_cast<uint4*>(sq + C::kTile + at) = make_uint4(l0.x, l0.y, l1.x, l1.y);
        }
        fence_proxy_async_smem();
        arrive(&bars.qfull[t]);
        lref_next = scale_from(x, x.key0);
      }
      return convert(slot, x.key0);
    };
    if (!unit_here(0)) goto end;
    if (bars.ring[0].go && !prepare(0)) goto end;
    for (uint32_t i = 0;; ++i) {
      const AUnit& x = bars.ring[i % kRing];
      if (!x.go) break;
      const int hi = hi_next;
      const float rf = rf_next;
      float lref = lref_next;
      const bool here = t == 0 || x.two;  // the tile has rows
      const int n = x.n, key0 = x.key0;
      const bool valid = in_tile && x.q0 + t * m_.qn + rq < m_.Nq;
      const bool idle = !__any_sync(0xffffffffu, valid);
      float m = -INFINITY, l = 0.f;  // reference (less kTop) and sum
      {
        for (int j = 0; j < n; ++j) {
          const int k0 = key0 + j * BN, c0 = k0 + col0;  // the tile's and the warp's first key
          const float sc = held_scale(ahead);
          // (ahead of the next load, which this one would wait for)
          bool first_values = false;  // behind tiles of empty blocks alone
          if (here && lref == kNoScale) {
            lref = scale_from(x, k0);
            first_values = j > 0 && lref != kNoScale;
          }
          if (j + 1 < n) ahead = fetch(k0 + BN);
          auto step = [&]() -> bool {
          const int vb = hi - c0;
          const bool special = __any_sync(0xffffffffu, (valid && vb < H) || (lane < 4 && sc == 0.f));
          // lanes 4-7: the value scale's exponent and its inverse (1 for an empty block)
          const float lv_ = sc > 0.f && lane >= 4 ? fminf(fmaxf(__log2f(sc) - lref, -100.f), 100.f) : 0.f;
          const float iv_ = fast_exp2(-lv_);
          if (!mbar_wait(&bars.sfull[t], (tc + j) & 1, abort)) return false;
          if (idle) {
            arrive(&bars.pfull[t]);
            return true;
          }
          __syncwarp();
          tc_fence_after();
          auto load = [&](float* s, int base) { tmem_ld16(sbase + base, reinterpret_cast<uint32_t*>(s)); };
          // The row's largest exponent in this tile, over both halves, and whether either half's `over` is set.
          auto row_max = [&](float* res, bool* over) -> bool {
            float mx = -INFINITY;
            const float lm_ = lane >= 4 && sc == 0.f && lref != kNoScale ? -kEmptyBelow : lv_;
#pragma unroll 1
            for (int base = 0; base < H; base += W) {
              float s[W];
              load(s, base);
              const float ks = __shfl_sync(0xffffffffu, sc, base / W), lv = __shfl_sync(0xffffffffu, lm_, 4 + base / W);
              tmem_ld_wait();
#pragma unroll
              for (int c = 0; c < W; ++c) {
                const float y = ks == 0.f ? lv : fmaf(s[c], rf * ks, lv);
                mx = fmaxf(mx, base + c < vb ? y : -INFINITY);
              }
            }
            *mine() = make_float2(mx, *over ? 1.f : 0.f);
            if (!pair_sync()) return false;
            *res = fmaxf(mx, other()->x) - kTop;
            *over |= other()->y != 0.f;
            ++xn;
            return true;
          };
          // P = 2^(y - mm) as fp16 pairs, its sum `ts` and that without the value scales `tl`, in fp32.
          uint32_t p[H / 2];
          float ts, tl;
          auto exps = [&](float mm, auto special) {  // special: columns are hidden, or a block of keys is empty
            constexpr bool kSpecial = decltype(special)::value != 0;
            ts = tl = 0.f;
            float buf[2][W];  // the next columns load while these are worked on
            load(buf[0], 0);
            float ks = 0.f, iv = 0.f;
            uint64_t f_2 = 0, g_2 = 0, ps[2] = {0, 0};
#pragma unroll
            for (int base = 0; base < H; base += W) {
              if (base % (H / NB) == 0) {
                ks = __shfl_sync(0xffffffffu, sc, base / W);
                iv = __shfl_sync(0xffffffffu, iv_, 4 + base / W);
                const float f = rf * ks, g = __shfl_sync(0xffffffffu, lv_, 4 + base / W) - mm;
                f_2 = f2(f, f);
                g_2 = f2(g, g);
              }
              float* s = buf[(base / W) & 1];
              tmem_ld_wait();
              if (base + W < H) load(buf[(base / W + 1) & 1], base + W);
#pragma unroll
              for (int c = 0; c < W / 2; ++c) {
                // (an empty block's keys are zeros, whatever their codes)
                if (kSpecial) s[2 * c] = ks == 0.f ? 0.f : s[2 * c], s[2 * c + 1] = ks == 0.f ? 0.f : s[2 * c + 1];
                const uint64_t y = fma2(f2(s[2 * c], s[2 * c + 1]), f_2, g_2);
                float y0 = f2lo(y), y1 = f2hi(y);
                if (kSpecial) {
                  y0 = base + 2 * c < vb ? y0 : -INFINITY;
                  y1 = base + 2 * c + 1 < vb ? y1 : -INFINITY;
                }
                const float p0 = fast_exp2(y0), p1 = fast_exp2(y1);
                p[base / 2 + c] = pack_weights(p0, p1);
                ps[c & 1] = add2(ps[c & 1], f2(p0, p1));
              }
              if ((base + W) % (H / NB) == 0) {
                const uint64_t two = add2(ps[0], ps[1]);
                const float sum = f2lo(two) + f2hi(two);
                ts += sum;
                tl = fmaf(sum, iv, tl);
                ps[0] = ps[1] = 0;
              }
            }
          };
          // The run's first tile sets the reference: a row that sees nothing of it sees nothing of the run.
          // Both warps of a pair hold the same references, so they agree.
          if (j == 0) {
            bool over = false;
            if (!row_max(&m, &over)) return false;
          }
          const float mm = m == -INFINITY ? 0.f : m;
          if (special)
            exps(mm, Constant<int, 1>());
          else
            exps(mm, Constant<int, 0>());
          // A row whose sum is too large in either half moves its reference (the others keep theirs: a row's bits
          // do not go by its neighbours).
          if (j > 0) {
            bool over = !(ts <= kMostSum) || first_values;
            const uint32_t asked = meet(__any_sync(0xffffffffu, valid && over));
            if (asked >= 32) return false;
            const bool raise = asked != 0;
            if (raise) {
              float mx;
              if (!row_max(&mx, &over)) return false;
              const float mn = over ? fmaxf(first_values ? m - kEmptyBelow : m, mx) : m;
              const float alpha = m == mn ? 1.f : fast_exp2(m - mn);
              m = mn;
              l *= alpha;
              // O holds PV of every earlier tile: its commit came with this S.
#pragma unroll
              for (int c = 0; c < D / 64; ++c) {
                uint32_t r[32];
                tmem_ld32(obase + c * 32, r);
                tmem_ld_wait();
#pragma unroll
                for (int y = 0; y < 32; ++y) r[y] = __float_as_uint(__uint_as_float(r[y]) * alpha);
                tmem_st32(obase + c * 32, r);
              }
              exps(m == -INFINITY ? 0.f : m, Constant<int, 1>());
            }
          }
          l += tl;
          tmem_st32(sbase, p);
          tmem_st_wait();
          tc_fence_before();
          arrive(&bars.pfull[t]);
          return true;
          };
          if (here && !step()) goto end;
          if (j + 1 < n && !convert(i % kRing, k0 + BN)) goto end;
        }
      }
      if (here) tc += n;
      // the next unit's query terms, ahead of this one's output
      if (!unit_here(i + 1)) goto end;
      if (bars.ring[(i + 1) % kRing].go && !prepare((i + 1) % kRing)) goto end;
      if (here && n > 0) {
        if (!mbar_wait(&bars.ofull[t], uc & 1, abort)) goto end;
        ++uc;
        __syncwarp();
        tc_fence_after();
      }
      if (here && !idle) {
        const int qi = x.q0 + t * m_.qn + rq, hq = x.hk * m_.R + rh;
        // both halves' sums; each half writes its half of the row
        *mine() = make_float2(l, 0.f);
        if (!pair_sync()) goto end;
        l += other()->x;
        ++xn;
        // (two factors: the smallest scales by a row's sum are no normal number)
        const float inv = l == 0.f ? 0.f : 1.f / l, unit = lref == kNoScale ? 1.f : exp2f(lref);
        const int64_t prow = int64_t(x.part) * m_.unit_rows + t * 128 + trow;
        if (valid && half == 0) {
          const float lse = l == 0.f ? -INFINITY : ln_of(m + kTop, l * (1.f / kUnit));
          if (x.part >= 0)
            m_.part_lse[prow] = lse;
          else if (m_.lse)
            m_.lse[(int64_t(x.b) * m_.Hq + hq) * m_.Nq + qi] = lse;
        }
        // The warp's 32 half rows go out through its own shared memory, so that consecutive lanes write
        // consecutive bytes of a row.
        const bool wide = x.part >= 0 || m_.out_fp32;
        char* base = x.part >= 0 ? reinterpret_cast<char*>(m_.part_o) : static_cast<char*>(m_.o);
        int64_t at = x.part >= 0 ? prow * D : int64_t(x.b) * m_.os.b + int64_t(hq) * m_.os.h + int64_t(qi) * m_.os.n;
        at = valid ? (at + half * (D / 2)) * (wide ? 4 : 2) : -1;
        uint32_t v[D / 2];
        if (n > 0) {
#pragma unroll
          for (int c = 0; c < D / 64; ++c) tmem_ld32(obase + c * 32, v + c * 32);
          tmem_ld_wait();
          tc_fence_before();
          arrive(&bars.ofree[t]);
#pragma unroll
          for (int y = 0; y < D / 2; ++y) v[y] = inv == 0.f ? 0 : __float_as_uint(__uint_as_float(v[y]) * inv * unit);
          if (*static_cast<volatile int*>(&bars.nans[i % kRing])) {
            const volatile int* na = nan_at[i % kRing] + half * (D / 2);
#pragma unroll
            for (int y = 0; y < D / 2; ++y) v[y] = na[y] < hi ? 0x7FC00000u : v[y];
          }
        } else {
#pragma unroll
          for (int y = 0; y < D / 2; ++y) v[y] = 0;
        }
        if (!pair_sync()) goto end;  // (the other half has read this warp's slot)
        auto put = [&](auto words) {  // words per half row
          constexpr int PC = decltype(words)::value / 4;  // 16-byte pieces of it
          constexpr int kRows = C::kWarpBytes / 16 / PC;  // rows at a time
          uint4* st = reinterpret_cast<uint4*>(own);
          auto cell = [&](int r, int c) -> uint4* {  // (no bank conflicts either way)
            return st + r * PC + (PC >= 8 ? (c & ~7) | ((c ^ r) & 7) : c ^ ((r >> 1) & 3));
          };
#pragma unroll
          for (int r0 = 0; r0 < 32; r0 += kRows) {
            if (lane >= r0 && lane < r0 + kRows) {
#pragma unroll
              for (int c = 0; c < PC; ++c) *cell(lane - r0, c) = make_uint4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
            }
            __syncwarp();
#pragma unroll 1
            for (int f = 0; f < kRows * PC; f += 32) {
              const int r = (f + lane) / PC, c = (f + lane) % PC;
              const int64_t to = __shfl_sync(0xffffffffu, at, r0 + r);
              const uint4 w = *cell(r, c);
              if (to >= 0) *reinterpret_cast<uint4*>(base + to + c * 16) = w;
            }
            __syncwarp();
          }
        };
        if (wide) {
          put(Constant<int, D / 2>());
        } else {
#pragma unroll
          for (int y = 0; y < D / 4; ++y)
            v[y] = pack_bf16(__uint_as_float(v[2 * y]), __uint_as_float(v[2 * y + 1]));
          put(Constant<int, D / 4>());
        }
      } else if (here && n > 0) {
        arrive(&bars.ofree[t]);
      }
      arrive(&bars.ring_empty[i % kRing]);
    }
  end:
    // (Also without a fault: one of the two may end as usual where the other gives up.)
    if (!alone) count_of(1 + t * 4 + quarter, 64, true);
  } else if (warp < C::kTmaWarp) {
    // ------------------------------------------------------------ MMA issue, a warp for each Q tile
    const int t = warp - C::kMmaWarp;
    constexpr uint32_t kIdescS = idesc_f8(128, BN, 0, 0, false, false);
    // (kind::f16 with both operands fp16; V is MN-major)
    constexpr uint32_t kIdescPV = idesc_bf16(128, D, false, true) & ~((1u << 7) | (1u << 10));
    const uint64_t dq = rows8_desc<D>(smem_u32(smem + C::kQ) + t * 2 * C::kTile, 16);
    const uint64_t dk = rows8_desc<D>(smem_u32(smem + C::kK), 16), dv = sw128_desc(smem_u32(smem + C::kV), BN * 128, 1024);
    const uint32_t q_lo = static_cast<uint32_t>(dq), q_hi = static_cast<uint32_t>(dq >> 32);
    const uint32_t k_lo = static_cast<uint32_t>(dk), k_hi = static_cast<uint32_t>(dk >> 32);
    const uint32_t v_lo = static_cast<uint32_t>(dv), v_hi = static_cast<uint32_t>(dv >> 32);
    const uint32_t o_tmem = tmem + C::kOCol + t * D, s_tmem = tmem + t * 128;
    if (lane == 0) {
      bool ok = true, two = false;
      uint32_t tc = 0, uc = 0;  // key tiles (of the ring) and units of this tile so far
      uint32_t pc = 0, ts = 0;  // key tiles of this Q tile, steps taken in turns
      auto pass = [&]() { mbar_arrive(&bars.turn[t ^ 1]); };
      auto qk = [&](uint32_t c, bool turn) {
        const uint32_t kl = k_lo + (((c % C::kKStages) * C::kTile) >> 4);
        constexpr int kSteps = 2 * (D / 32);
#pragma unroll
        for (int kk = 0; kk < kSteps; ++kk) {
          const uint32_t off = (kk % (D / 32)) * 2, term = kk < D / 32 ? 0 : C::kTile >> 4;
          mma8_ss_w(s_tmem, q_lo + term + off, q_hi, kl + off, k_hi, kIdescS, kk > 0);
          if (kk == kSteps - 3 && turn) pass();  // (two MMAs cover the hand-over)
        }
        mma_commit(&bars.sfull[t]);
      };
      for (uint32_t i = 0; ok; ++i) {
        if (!unit_here(i)) break;
        const AUnit& u = bars.ring[i % kRing];
        const int go = u.go, n = u.n;
        two = u.two;
        mbar_arrive(&bars.ring_empty[i % kRing]);
        if (!go) break;
        if (n == 0) continue;
        if (t && !two) {  // no rows: K and V pass by (tile by tile: a wait for the next unit could outlast its limit)
          for (int j = 0; ok && j < n; ++j, ++tc) {
            if (!(ok = mbar_wait(&bars.kfull[tc % C::kKStages], (tc / C::kKStages) & 1, abort))) break;
            mbar_arrive(&bars.kempty[tc % C::kKStages]);
            if (!(ok = mbar_wait(&bars.vfull[tc % C::kVStages], (tc / C::kVStages) & 1, abort))) break;
            mbar_arrive(&bars.vempty[tc % C::kVStages]);
          }
          continue;
        }
        if (!(ok = mbar_wait(&bars.qfull[t], uc & 1, abort)) ||
            !(ok = mbar_wait(&bars.kfull[tc % C::kKStages], (tc / C::kKStages) & 1, abort)))
          break;
        tc_fence_after();
        qk(tc, false);
        mma_commit(&bars.kempty[tc % C::kKStages]);
        for (int j = 0; j < n; ++j) {
          const uint32_t c = tc + j, s = ts + j;
          const bool more = j + 1 < n;
          if (!(ok = mbar_wait(&bars.vfull[c % C::kVStages], (c / C::kVStages) & 1, abort)) ||
              (more && !(ok = mbar_wait(&bars.kfull[(c + 1) % C::kKStages], ((c + 1) / C::kKStages) & 1, abort))))
            break;
          if (j == 0 && uc > 0 && !(ok = mbar_wait(&bars.ofree[t], (uc - 1) & 1, abort))) break;
          // Turns: the tiles' steps alternate (side by side they would fall into step and leave the tensor core
          // idle during both softmaxes).
          if (two && s + t > 0 && !(ok = mbar_wait(&bars.turn[t], (s + t - 1) & 1, abort))) break;
          if (!(ok = mbar_wait(&bars.pfull[t], (pc + j) & 1, abort))) break;
          tc_fence_after();
          const uint32_t vl = v_lo + (((c % C::kVStages) * 2 * C::kTile) >> 4);
#pragma unroll
          for (int kk = 0; kk < BN / 16; ++kk)
            // P of keys 0-63 lies in S columns 0-31, of keys 64-127 in 64-95
            mma_ts_w(o_tmem, s_tmem + (kk >> 2) * 64 + (kk & 3) * 8, vl + ((kk * 2048) >> 4), v_hi, kIdescPV, j > 0 || kk > 0);
          if (more)
            qk(c + 1, two);
          else if (two)
            pass();
          if (!more) mma_commit(&bars.ofull[t]);
          mma_commit(&bars.vempty[c % C::kVStages]);
          if (more) mma_commit(&bars.kempty[(c + 1) % C::kKStages]);
        }
        tc += n;
        pc += n;
        if (two) ts += n;
        ++uc;
      }
      // Every MMA issued above must finish before TMEM is released.
      mma_commit(&bars.drain[t]);
      const long long t0 = clock64();
      while (!mbar_test(&bars.drain[t], 0) && clock64() - t0 < kWaitLimitCycles) {
      }
    }
  } else if (warp == C::kTmaWarp && lane == 0) {
    // ------------------------------------------------------------ units and loads
    int64_t g = blockIdx.x;
    uint32_t c = 0, i = 0;
    bool ok = true;
    for (; ok; ++i) {
      AUnit x = {};
      if (g >= 0) {
        mbar_expect_tx(&bars.next, 16);
        request_block(&bars.answer, &bars.next);
        // (the order of units and their splits: masked_plan)
        int u = static_cast<int>(g), split = 0, splits = 1;
        x.go = 1;
        x.part = -1;
        if (g >= m_.full_units) {
          splits = m_.splits;
          x.part = static_cast<int>(g - m_.full_units);
          split = x.part % splits;
          u = static_cast<int>(m_.full_units) + x.part / splits;
        }
        const MaskedPlace at = masked_place(m_, u);
        x.b = at.bh / m_.Hkv;
        x.hk = at.bh - x.b * m_.Hkv;
        x.q0 = at.rb * (m_.tiles * m_.qn);
        const int q1 = min(x.q0 + m_.tiles * m_.qn, m_.Nq);
        x.two = m_.tiles == 2 && x.q0 + m_.qn < q1;
        x.uhi = row_span(m_.mask, x.b, q1 - 1).hi;
        const int tiles = (x.uhi + BN - 1) / BN;
        const int j0 = static_cast<int>(int64_t(tiles) * split / splits);
        x.n = static_cast<int>(int64_t(tiles) * (split + 1) / splits) - j0;
        x.key0 = j0 * BN;
      }
      if (i >= kRing && !mbar_wait(&bars.ring_empty[i % kRing], ((i / kRing) - 1) & 1, abort)) break;
      bars.ring[i % kRing] = x;
      for (int y = 0; y < D; ++y) nan_at[i % kRing][y] = 0x7FFFFFFF;
      bars.nans[i % kRing] = 0;
      mbar_arrive(&bars.ring_full[i % kRing]);
      if (g < 0) break;
      for (int j = 0; j < x.n; ++j, ++c) {
        const uint32_t ks = c % C::kKStages, cs = c % C::kCStages;
        if (!(ok = mbar_wait(&bars.kempty[ks], ((c / C::kKStages) & 1) ^ 1, abort))) break;
        mbar_expect_tx(&bars.kfull[ks], C::kTile);
        tma_load_4d(smem_u32(smem + C::kK) + ks * C::kTile, &tm_k, 0, x.key0 + j * BN, x.hk, x.b, &bars.kfull[ks]);
        if (!(ok = mbar_wait(&bars.cempty[cs], ((c / C::kCStages) & 1) ^ 1, abort))) {
          // (the K tile lands before the block ends)
          const long long t0 = clock64();
          while (!mbar_test(&bars.kfull[ks], (c / C::kKStages) & 1) && clock64() - t0 < kWaitLimitCycles) {
          }
          break;
        }
        mbar_expect_tx(&bars.cfull[cs], C::kTile);
        tma_load_4d(smem_u32(smem + C::kC) + cs * C::kTile, &tm_v, 0, x.key0 + j * BN, x.hk, x.b, &bars.cfull[cs]);
      }
      if (!ok) break;
      if (!(ok = mbar_wait(&bars.next, i & 1, abort))) break;
      g = answered_block(&bars.answer);
      fence_proxy_async_smem();  // read before the next answer is written
    }
    if (*abort) {
      // After an abort: what is in flight lands before the block ends.
      auto settle = [&](uint64_t* bar, uint32_t parity) {
        const long long t0 = clock64();
        while (!mbar_test(bar, parity) && clock64() - t0 < kWaitLimitCycles) {
        }
      };
      for (uint32_t f = c > C::kKStages ? c - C::kKStages : 0; f < c; ++f)
        settle(&bars.kfull[f % C::kKStages], (f / C::kKStages) & 1);
      for (uint32_t f = c > C::kCStages ? c - C::kCStages : 0; f < c; ++f)
        settle(&bars.cfull[f % C::kCStages], (f / C::kCStages) & 1);
      if (g >= 0) settle(&bars.next, i & 1);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && bars.abort) report(m_.status, SA_DEVERR_TIMEOUT);
  if (warp == C::kMmaWarp) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// Units, splits and their order are the masked forward's.
void attend8_many_plan(Attend8Args* a) {
  masked_plan(&a->m);
  a->m.quads = a->m.slots = 0;
  a->m.unit_rows = 128 * a->m.tiles;
}

template <int D, int NB>
static cudaError_t launch_a(const Attend8Args& a, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t st) {
  using C = ACfg<D>;
  auto kern = sa_attend8_many_kernel<D, NB>;
  // at least half the SM's shared memory: one block per SM owns its TMEM
  const int smem = C::kSmemBytes > 120 * 1024 ? C::kSmemBytes : 120 * 1024;
  static std::atomic<int> regs_ok{0};  // 0 unknown, 1 enough, 2 too few
  if (regs_ok.load() == 0) {
    cudaFuncAttributes attr;
    cudaError_t e = cudaFuncGetAttributes(&attr, kern);
    if (e != cudaSuccess) return e;
    // setmaxnreg.inc waits until the block's launch registers cover the split
    const long need = long(C::kRegSoft) * C::kSoftWarps * 32 + long(C::kRegOther) * 128;
    regs_ok.store(long(attr.numRegs) * C::kThreads >= need ? 1 : 2);
  }
  if (regs_ok.load() != 1) return cudaErrorLaunchOutOfResources;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int64_t grid = a.m.full_units + a.m.split_units * a.m.splits;
  kern<<<static_cast<unsigned>(grid), C::kThreads, smem, st>>>(a, tk, tv);
  if ((e = cudaGetLastError()) != cudaSuccess || a.m.split_units == 0) return e;
  return launch_masked_join(a.m, st);
}

cudaError_t launch_attend8_many(const Attend8Args& a, cudaStream_t st) {
  CUtensorMap tk, tv;
  if (!make_codes_map(&tk, a.k8, a.m.d, a.m.Nk, a.m.Hkv, a.m.B, a.m.ks, BN, true) ||
      !make_codes_map(&tv, a.v8, a.m.d, a.m.Nk, a.m.Hkv, a.m.B, a.m.vs, BN, a.m.d == 128))
    return cudaErrorInvalidValue;
  if (a.m.d == 128)
    return a.block_log2 >= 6   ? launch_a<128, 1>(a, tk, tv, st)
           : a.block_log2 == 5 ? launch_a<128, 2>(a, tk, tv, st)
                               : launch_a<128, 4>(a, tk, tv, st);
  return a.block_log2 >= 6   ? launch_a<64, 1>(a, tk, tv, st)
         : a.block_log2 == 5 ? launch_a<64, 2>(a, tk, tv, st)
                             : launch_a<64, 4>(a, tk, tv, st);
}

}  // namespace sa
