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
// them.  A unit is two Q tiles of up to 128 packed rows (whole queries), or one
// when a key head has no more.  K and V stream through one ring of 128-row
// tiles by TMA; S = Q K^T and O stay in TMEM, P (bf16) overwrites its S.
// The MMA thread issues PV(j) of a tile and then S(j+1) of the same tile, so
// while one tile's softmax runs the tensor core works for the other.  TMEM is
// full (2 S + 2 O of 128 columns), so a tile's own S cannot be a step ahead:
// the tensor core stays busy only if a softmax takes no longer than the other
// tile's two products (1024 cycles).  One warp needs about 1600 cycles for 32
// rows x 128 columns whatever else runs, so two warps share each row, 64
// columns each (16 softmax warps for two tiles).  They keep separate sums and
// agree on the row's reference through a pair barrier each step.
// Tiles are taken from the last key to the first: a distance bias is strongest
// there, so the first tile's reference holds (from the far end every tile would
// raise it).
// Only the key span that the unit's rows see is read; tiles that every row
// sees whole skip the mask.  A step of both tiles takes 1.59 us, 1.1 of them MMAs
// (12 heads, 7040 rows x 28160 keys, frame-causal: 791 us, 71 % of the measured
// bf16 rate).
//
// A block starts with its own unit and then takes units of blocks that have not
// started (cluster launch control), so the next unit's Q, K and V load and its
// first S is computed while the last one's softmax and output finish; with one
// unit a block, each unit paid about 10 us for its start and end.  Units differ
// in length (causal rows, documents); taking the next free one balances them.
//
// Units that do not fill a last wave of SMs (all of them, for a new token over
// a long cache) are cut into `splits` runs of key tiles; each writes a
// normalised fp32 partial and its lse, and a second kernel joins them:
// o = sum_s e^(lse_s - lse) o_s.
// A new token's few rows would leave all but two softmax warps idle, and those two
// 64 columns a tile each (1.26 us a tile of 128 keys with a cap).  With up to 32 rows
// the tile holds them four times, once per TMEM lane quarter, and each quarter's two
// warps take 32 of the 128 keys; the other keys' P is 0 there, so the quarters' O and
// sums are those of four splits, and are joined like them (1.01 us a tile; with a
// warp for each of the two products 0.73, K and V at 90 GB/s a SM, twice an even share
// of the HBM).
#include <atomic>
#include <cmath>

#include "sa_device.cuh"
#include "sa_internal.h"
#include "sa_mask.cuh"
#include "sa_tma.h"

namespace sa {

namespace {

constexpr int BN = 128;
constexpr int kSms = 152;
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kLog2e = 1.4426950408889634f;
// P is computed against a row reference m that only moves when a tile's sum
// of P passes this (the fp32 sums and O have room for far more).
constexpr float kRaiseLimit = 4294967296.f;

template <int D, int T>
struct MCfg {
  static constexpr int kSoftWarps = 8 * T;  // per Q tile two sets of four: column halves
  static constexpr int kMmaWarp = kSoftWarps, kTmaWarp = kSoftWarps + T,  // one MMA warp a tile
                       kTailWarp = kTmaWarp + 1, kPvWarp = kTailWarp + 1;  // (one tile: PV has its own)
  // whole warpgroups: setmaxnreg acts on aligned groups of four warps
  static constexpr int kThreads = 32 * (kSoftWarps + 4);
  static constexpr bool kRegSplit = T == 2;
  // 640 threads launch with 96 registers each = 61440 = 512 * 104 + 128 * 64
  // (fewer than 64 make the MMA thread spill)
  static constexpr int kRegSoft = 104, kRegOther = 64;
  static constexpr int kTile = BN * D * 2;
  static constexpr int kQBytes = T * 128 * D * 2;
  static constexpr int kStages = D == 128 ? (T == 2 ? 4 : 5) : 8;
  static constexpr int kWarpBytes = 2048;  // a softmax warp's own: exchange slots, output staging
  static constexpr int kXch = kSoftWarps * kWarpBytes;
  static constexpr int kSmemBytes = 1024 + kQBytes + kStages * kTile + kXch + 1024 + (T == 1 ? 2048 : 0);
  // one tile: two S buffers, so that S(j+1) is computed beside softmax(j) and PV(j)
  static constexpr int kOCol = 256;
  static constexpr int kPCol = 384;  // quads: P has columns of its own, 64 for each S buffer
  static constexpr int kTmemCols = 512;
  static_assert(kSmemBytes <= 232448, "shared memory");
};

template <int T, int STAGES>
struct MBars {
  uint64_t full[STAGES], empty[STAGES];
  uint64_t sfull[2], pfull[2], pvdone[2], ofull[T], ofree[T];
  uint64_t qfull, qempty, next, tail, tail_here, turn[T], ring_full[2], ring_empty[2], drain[2];
  uint4 answer;   // of the request for the next unit
  struct Unit {
    int go;                // 0: no more units
    int key0, n, uhi;      // first key, key tiles, end of the rows' span
    int part, q0, b, hk;   // partial result (-1: whole), first query, batch entry, key head
  } ring[2];
  int flag[T * 4][2];
  uint32_t again[T * 8]; // rows that each softmax warp computes once more
  int first[T == 1 ? kSms : 1], runs[T == 1 ? kSms : 1];  // slots of each batch entry (share_out)
  int used;
  uint32_t tmem_base;
  int abort, steps;  // steps: of rows_again
};

// Unit number -> key head of the batch and row block.
struct Place {
  int bh, rb;
};
__host__ __device__ __forceinline__ Place place_of(const MaskedArgs& a, int u) {
  const int per = a.group * a.row_blocks, grp = u / per, r = u - grp * per;
  const int heads = a.B * a.Hkv - grp * a.group < a.group ? a.B * a.Hkv - grp * a.group : a.group;
  const int k = r / heads;
  return {grp * a.group + (r - k * heads), a.row_blocks - 1 - k};
}

// Key tiles that the rows of a unit with the queries q0 .. q1 see.
__device__ __forceinline__ int tiles_of(const MaskedArgs& a, int b, int q0, int q1, int* lo, int* hi) {
  *lo = row_span(a.mask, b, q0).lo;
  *hi = row_span(a.mask, b, q1).hi;
  return *hi > *lo ? (*hi - *lo + BN - 1) / BN : 0;
}

// Shares the slots out among the units of a batch of at most kSms, by one warp: the
// shortest run L for which sum_b Hkv ceil(tiles_b / L) slots are enough, ceil(tiles_b / L)
// runs for each head of entry b.  (With as many for each, whatever its length, 4 sequences
// of 28160, 7041, 20000 and 27999 keys took as long as 4 of 28160: 60.5 us, now 54.8.)
template <typename Bars>
__device__ __forceinline__ void share_out(const MaskedArgs& a, Bars* bars, int lane) {
  constexpr int N = (kSms + 31) / 32;
  int t[N], sum = 0, most = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int b = i * 32 + lane;
    int lo, hi;
    t[i] = b < a.B ? tiles_of(a, b, 0, a.Nq - 1, &lo, &hi) : 0;
    sum += t[i];
    most = max(most, t[i]);
  }
  sum = __reduce_add_sync(0xffffffffu, sum) * a.Hkv;
  most = __reduce_max_sync(0xffffffffu, most);
  int L = max(1, (sum + a.slots - 1) / a.slots), top = max(most, 1);  // (at `top` a run a head)
  // sum_b Hkv ceil(t_b / L) < sum / L + units
  const int spare = a.slots - a.B * a.Hkv;
  if (spare > 0) top = min(top, max(1, (sum + spare - 1) / spare));
  while (L < top) {
    const int mid = (L + top) >> 1;
    int n = 0;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i * 32 < a.B) n += (t[i] + mid - 1) / mid;
    if (static_cast<int>(__reduce_add_sync(0xffffffffu, n)) * a.Hkv <= a.slots)
      top = mid;
    else
      L = mid + 1;
  }
  int at = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (i * 32 >= a.B) break;
    const int b = i * 32 + lane, runs = (t[i] + L - 1) / L;
    int inc = runs * a.Hkv;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    if (b < a.B) {
      bars->first[b] = at + inc - runs * a.Hkv;
      bars->runs[b] = runs;
    }
    at += __shfl_sync(0xffffffffu, inc, 31);
  }
  if (lane == 0) bars->used = at;
  __syncwarp();
}

// Waits as mbar_wait does, but only gives up after kWaitLimitCycles in which no warp computed
// rows again: abort[1] counts their steps.
__device__ __forceinline__ bool bar_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  if (mbar_test(bar, parity)) return true;
  long long t0 = clock64();
  int steps = 0;
  while (true) {
    if (mbar_test(bar, parity)) return true;
    if (*abort) return false;
    if (clock64() - t0 > kWaitLimitCycles) {
      if (abort[1] == steps) {
        *abort = 1;
        return false;
      }
      steps = abort[1];
      t0 = clock64();
    }
  }
}

// Rows whose o is computed again, from the keys they see alone.  The second product meets every
// key of a tile, and P = 0 times a NaN or an infinity is a NaN; so rows whose o is not finite,
// though their scores are, and that do not see every key of their unit's run (or, in quads, take
// a quarter of it) are worked out here, in fp32 with P rounded to bf16 as there.  Nothing calls
// this on finite values (looking for others costs two operations an output value, where rows may
// need it).  A warp takes the rows of `again` one by one, 32 keys at a time, for its half of the
// columns; eight lanes share a key's products.  The partner warp, which has the other half,
// calls it with the same rows: o may be in q's place, so a row is written when both have read
// q.  False: to give up.
struct AgainRow {
  int hq, qi;
  float m;     // the row's reference
  int unused;
  int64_t at;  // where its half row goes, in bytes
};
template <int D, bool QUADS>
__device__ __noinline__ bool rows_again(const MaskedArgs& a, const AgainRow* rows, uint32_t again, int b, int part,
                                        int key0, int n, int barrier, volatile int* abort) {
  constexpr int V = D / 64;  // columns a lane, and pieces of 16 bytes of a key
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, half = (warp >> 2) & 1;
  constexpr int kStep = QUADS ? BN : 32;  // (quads: the quarter's 32 of each tile's keys)
  const int first = key0 + (QUADS ? (warp & 3) * 32 : 0);
  for (; again; again &= again - 1) {
    const AgainRow x = rows[__ffs(again) - 1];
    const Span sp = row_span(a.mask, b, x.qi);
    const float nslope = a.slopes ? -__ldg(a.slopes + x.hq) * kLog2e : 0.f;
    const int hk = x.hq / a.R, end = min(key0 + n * BN, sp.hi);
    const uint16_t* q = a.q + int64_t(b) * a.qs.b + int64_t(x.hq) * a.qs.h + int64_t(x.qi) * a.qs.n + (lane & 7) * 8;
    const uint16_t* k = a.k + int64_t(b) * a.ks.b + int64_t(hk) * a.ks.h + (lane & 7) * 8;
    const uint16_t* v = a.v + int64_t(b) * a.vs.b + int64_t(hk) * a.vs.h + half * (D / 2) + lane * V;
    uint4 qr[V];
#pragma unroll
    for (int e = 0; e < V; ++e) qr[e] = *reinterpret_cast<const uint4*>(q + e * 64);
    float acc[V] = {}, sum = 0.f;
    for (int c0 = first + (sp.lo > first ? (sp.lo - first) / kStep * kStep : 0); c0 < end; c0 += kStep) {
      if (lane == 0) atomicAdd(const_cast<int*>(abort) + 1, 1);
      float s = 0.f;  // of key c0 + lane
#pragma unroll 4
      for (int i = 0; i < 8; ++i) {  // keys 4 i .. 4 i + 3
        const int c = c0 + 4 * i + (lane >> 3);
        float d = 0.f;
        if (c < end) {
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const uint4 kr = __ldg(reinterpret_cast<const uint4*>(k + c * a.ks.n + e * 64));
            const uint32_t qw[4] = {qr[e].x, qr[e].y, qr[e].z, qr[e].w}, kw[4] = {kr.x, kr.y, kr.z, kr.w};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              d = fmaf(__uint_as_float(qw[w] << 16), __uint_as_float(kw[w] << 16), d);
              d = fmaf(__uint_as_float(qw[w] & 0xFFFF0000u), __uint_as_float(kw[w] & 0xFFFF0000u), d);
            }
          }
        }
#pragma unroll
        for (int o = 4; o; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
        d = __shfl_sync(0xffffffffu, d, (lane & 3) * 8);
        if (lane >> 2 == i) s = d;
      }
      const int c = c0 + lane;
      const bool sees = c >= sp.lo && c < end;
      if (a.neg_scale) s = -s;
      float y = s * a.scale_log2;
      if (a.cap_log2 > 0.f) y = fmaf(-2.f * a.cap_log2, fast_rcp(1.f + fast_exp2(s * a.cap_k1)), a.cap_log2);
      y = fmaf(nslope, fabsf(static_cast<float>(sp.pos - c)), y);
      const float p = sees ? __uint_as_float(pack_bf16(fast_exp2(y - x.m), 0.f) << 16) : 0.f;
      sum += p;
      const uint32_t some = __ballot_sync(0xffffffffu, sees);
#pragma unroll 8
      for (int i = 0; i < 32; ++i) {
        const float w = __shfl_sync(0xffffffffu, p, i);
        if (!(some >> i & 1)) continue;
        const uint16_t* row = v + (c0 + i) * a.vs.n;
        if (V == 2) {
          const uint32_t z = __ldg(reinterpret_cast<const uint32_t*>(row));
          acc[0] = fmaf(w, __uint_as_float(z << 16), acc[0]);
          acc[V - 1] = fmaf(w, __uint_as_float(z & 0xFFFF0000u), acc[V - 1]);
        } else {
          acc[0] = fmaf(w, __uint_as_float(uint32_t(__ldg(row)) << 16), acc[0]);
        }
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float2 y = make_float2(acc[0] / sum, acc[V - 1] / sum);
    named_barrier(barrier, 64);
    if (*abort) return false;  // (as after any meeting of the pair)
    const bool wide = part >= 0 || a.out_fp32;
    char* to = (part >= 0 ? reinterpret_cast<char*>(a.part_o) : static_cast<char*>(a.o)) + x.at + lane * V * (wide ? 4 : 2);
    if (V == 2 && wide)
      *reinterpret_cast<float2*>(to) = y;
    else if (V == 2)
      *reinterpret_cast<uint32_t*>(to) = pack_bf16(y.x, y.y);
    else if (wide)
      *reinterpret_cast<float*>(to) = y.x;
    else
      *reinterpret_cast<uint16_t*>(to) = static_cast<uint16_t>(pack_bf16(y.x, 0.f));
  }
  return true;
}

template <bool M>
struct Masked {
  static constexpr bool value = M;
};
template <int N>
struct Words {
  static constexpr int value = N;
};

}  // namespace

template <int D, int T, bool QUADS, bool CAP, bool BIAS>
__global__ void __launch_bounds__(MCfg<D, T>::kThreads, 1)
    sa_masked_kernel(const __grid_constant__ MaskedArgs a, const __grid_constant__ CUtensorMap tm_q,
                     const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v) {
  using C = MCfg<D, T>;
  constexpr int S = C::kStages;
  constexpr int W = 16;  // S columns a register buffer holds
  static_assert(!QUADS || T == 1, "quads have one tile");
  static_assert(sizeof(MBars<T, S>) <= 1024 + (T == 1 ? 2048 : 0), "shared memory");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sQ = smem;
  uint8_t* sKV = sQ + C::kQBytes;
  uint8_t* sX = sKV + S * C::kTile;
  MBars<T, S>* bars = reinterpret_cast<MBars<T, S>*>(sX + C::kXch);
  volatile int* abort = &bars->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&bars->full[s], 1);
      mbar_init(&bars->empty[s], T);
    }
    for (int i = 0; i < T; ++i) {
      mbar_init(&bars->ofull[i], 1);
      mbar_init(&bars->ofree[i], 256);
    }
    for (int i = 0; i < T * 4; ++i) {
      bars->flag[i][0] = bars->flag[i][1] = 0;
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->sfull[i], 1);  // S and P of each S buffer
      mbar_init(&bars->pfull[i], 256);
      mbar_init(&bars->ring_full[i], 1);
      mbar_init(&bars->ring_empty[i], C::kSoftWarps + T + 1 + (T == 1 ? 1 : 0));
      mbar_init(&bars->pvdone[i], 1);
      mbar_init(&bars->drain[i], 1);
    }
    mbar_init(&bars->qfull, 1);
    mbar_init(&bars->qempty, T);
    mbar_init(&bars->next, 1);
    mbar_init(&bars->tail, 1);
    mbar_init(&bars->tail_here, T);
    for (int i = 0; i < T; ++i) mbar_init(&bars->turn[i], 1);
    bars->abort = bars->steps = 0;
    fence_mbar_init();
  }
  if (a.qn * a.R < 128) {  // Q rows that no copy fills are zero for good
    for (int i = threadIdx.x; i < C::kQBytes / 16; i += C::kThreads)
      reinterpret_cast<uint4*>(sQ)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
  }
  if (QUADS && a.slots && warp == C::kTmaWarp) share_out(a, bars, lane);
  if (warp == C::kMmaWarp) {
    tmem_alloc(&bars->tmem_base, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;

  if (C::kRegSplit) {
    if (warp < C::kSoftWarps)
      reg_alloc<C::kRegSoft>();
    else
      reg_dealloc<C::kRegOther>();
  }

  using Unit = typename MBars<T, S>::Unit;

  if (warp < C::kSoftWarps) {
    // ------------------------------------------------------------ softmax
    // Warps 8t .. 8t+3 take columns 0-63 of tile t's S (half 0), 8t+4 .. 8t+7
    // columns 64-127; warps of both halves with the same lane quarter share rows.
    const int t = warp >> 3, half = (warp >> 2) & 1, quarter = warp & 3;
    // Quads: the tile's up to 32 rows stand in each lane quarter, whose two warps take
    // 32 of the columns, 16 each; the quarters' results are joined like splits.
    constexpr int H = QUADS ? 16 : BN / 2;
    const int col0 = (QUADS ? quarter * 2 + half : half) * H;
    const int trow = QUADS ? lane : quarter * 32 + lane;  // row of the tile
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const int rq = trow / a.R, rh = trow - rq * a.R;  // its query and head in the tile
    const bool in_tile = trow < a.qn * a.R;
    const float sl = a.scale_log2;
    uint32_t sbase = tmem + lane_base + t * 128 + col0;
    const uint32_t obase = tmem + lane_base + C::kOCol + t * D + half * (D / 2);
    volatile int* flag = bars->flag[t * 4 + quarter];
    uint32_t xn = 0;           // pair exchanges so far
    uint32_t tc = 0, uc = 0;   // key tiles and units with keys so far
    if (QUADS) {  // the other quarters' columns of P stay 0
      uint32_t zero[32] = {};
      tmem_st32(tmem + lane_base + C::kPCol + half * 64, zero);
      tmem_st32(tmem + lane_base + C::kPCol + half * 64 + 32, zero);
      tmem_st_wait();
    }
    // Slot of exchange xn: this half's value, and the other half's.
    uint8_t* own = sX + warp * C::kWarpBytes;
    auto mine = [&]() -> float2* { return reinterpret_cast<float2*>(own) + (xn & 1) * 32 + lane; };
    auto other = [&]() -> float2* {
      return reinterpret_cast<float2*>(sX + (warp ^ 4) * C::kWarpBytes) + (xn & 1) * 32 + lane;
    };
    // Meets the other half's warp.  A warp that gives up sets *abort and arrives
    // once (below `done`), and whoever it releases gives up too.
    auto pair_sync = [&]() -> bool {
      named_barrier(1 + t * 4 + quarter, 64);
      return *abort == 0;
    };
    for (uint32_t i = 0;; ++i) {
      if (!bar_wait(&bars->ring_full[i & 1], (i >> 1) & 1, abort)) goto done;
      const Unit x = bars->ring[i & 1];
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->ring_empty[i & 1]);
      if (!x.go) break;
      const int key0 = x.key0, n = x.n;
      const int qi = x.q0 + t * a.qn + rq, hq = x.hk * a.R + rh;
      const bool valid = in_tile && qi < a.Nq;
      const bool idle = !__any_sync(0xffffffffu, valid);
      Span sp = {0, 0, 0};
      if (valid) sp = row_span(a.mask, x.b, qi);
      float nslope = 0.f;
      if (BIAS && valid) nslope = -__ldg(a.slopes + hq) * kLog2e;
      float m = -INFINITY, l = 0.f, lr = 0.f;
      for (int j = 0; j < n; ++j) {
        const int k0 = key0 + (n - 1 - j) * BN, c0 = k0 + col0;  // first keys of the tile and of the warp's columns
        const int va = sp.lo - c0, vb = sp.hi - c0;
        const bool edge = __any_sync(0xffffffffu, valid && (va > 0 || vb < H));
        // The first tile that shows a row a key sets its reference.
        const bool first = j == 0 || __any_sync(0xffffffffu, m == -INFINITY && sp.lo < k0 + BN && sp.hi > k0);
        // S buffer and its phase: one buffer a tile, or one tile's two in turn
        const uint32_t sb = T == 2 ? t : (tc + j) & 1;
        if (T == 1) sbase = tmem + lane_base + sb * 128 + col0;
        if (!bar_wait(&bars->sfull[sb], (T == 2 ? tc + j : (tc + j) >> 1) & 1, abort)) goto done;
        if (idle) {
          mbar_arrive(&bars->pfull[sb]);
          continue;
        }
        __syncwarp();
        tc_fence_after();
        auto load = [&](float* s, int base) { tmem_ld16(sbase + base, reinterpret_cast<uint32_t*>(s)); };
        auto hidden = [&](int c) -> bool { return c < va || c >= vb; };
        // cap tanh(x scale / cap) = cap (1 - 2 / (1 + e^2y)) in exp2 units; exact at
        // both ends (e^2y = inf or 0), absolute error about 1e-7 cap
        auto capped = [&](float s) -> float {
          return fmaf(-2.f * a.cap_log2, fast_rcp(1.f + fast_exp2(s * a.cap_k1)), a.cap_log2);
        };
        // W raw scores -> scores in exp2 units with cap, bias and mask.
        auto exact = [&](float* s, int base) {
          const float t0 = static_cast<float>(sp.pos - c0 - base);
#pragma unroll
          for (int c = 0; c < W; ++c) {
            float y = CAP ? capped(s[c]) : s[c] * sl;
            if (BIAS) y = fmaf(nslope, fabsf(t0 - static_cast<float>(c)), y);
            s[c] = edge && hidden(base + c) ? -INFINITY : y;
          }
        };
        // The row's largest score in this tile, over both halves (without a bias
        // the largest product has the largest score).
        auto row_max = [&](float* res) -> bool {
          float mx = -INFINITY;
#pragma unroll 1
          for (int base = 0; base < H; base += W) {
            float s[W];
            load(s, base);
            tmem_ld_wait();
            if (BIAS) {
              exact(s, base);
            } else if (edge) {
#pragma unroll
              for (int c = 0; c < W; ++c)
                if (hidden(base + c)) s[c] = -INFINITY;
            }
#pragma unroll
            for (int c = 0; c < W; c += 2) mx = fmax3(mx, s[c], s[c + 1]);
          }
          if (!BIAS && mx != -INFINITY) mx = CAP ? capped(mx) : sl * mx;
          *mine() = make_float2(mx, 0.f);
          if (!pair_sync()) return false;
          *res = fmaxf(mx, other()->x);
          ++xn;
          return true;
        };
        // P = exp2(score - mm) as bf16 pairs (the second product's two operands have one type, V's:
        // half a step of 2^-8 of each weight), its fp32 sum (for lse) and the sum of the rounded values, which normalises O (so that O stays a convex
        // combination of V rows whatever the rounding of P to bf16).
        uint32_t p[H / 2];
        uint64_t ps[2];
        float pr[2];
        float ts, tr;
        auto zero = [&]() {
          ps[0] = ps[1] = 0;
          pr[0] = pr[1] = 0.f;
        };
        auto take = [&](float y0, float y1, int c) {  // a pair of exponents
          const float p0 = fast_exp2(y0), p1 = fast_exp2(y1);
          p[c] = pack_bf16(p0, p1);
          ps[c & 1] = add2(ps[c & 1], f2(p0, p1));
          pr[c & 1] = add_bf16x2(p[c], pr[c & 1]);
        };
        // Most tiles: every visible key on one side of its row (`behind`: none after the
        // row's position; else none before it), where the bias is linear in the column.
        // The exponent is then one multiply-add a pair:
        // x * f + g with g = -mm or, with a bias, a pair that steps along the
        // columns.  With a cap, f is tanh(z)/z as a polynomial in z^2 (|z| <= 0.4,
        // error below 1.6e-7 cap); false if a score is larger.
        const int far = sp.pos - c0;  // distance of the half's first column
        const bool behind = !BIAS || far >= min(vb, H) - 1;
        auto fast = [&](float mm, auto masked) -> bool {
          zero();
          const float ns = behind ? nslope : -nslope;  // of (far - c)
          const float g0 = BIAS ? fmaf(ns, static_cast<float>(far), -mm) : -mm;
          uint64_t g = BIAS ? f2(g0, g0 - ns) : f2(g0, g0);
          const uint64_t step = f2(-2.f * ns, -2.f * ns);
          const uint64_t sl2 = f2(sl, sl), k1 = f2(a.cap_p1, a.cap_p1), k2 = f2(a.cap_p2, a.cap_p2),
                         k3 = f2(a.cap_p3, a.cap_p3);
          float wm = 0.f;
          float buf[QUADS ? 1 : 2][W];  // the next columns load while these are worked on
          load(buf[0], 0);
#pragma unroll
          for (int base = 0; base < H; base += W) {
            float* s = buf[QUADS ? 0 : (base / W) & 1];
            tmem_ld_wait();
            if (base + W < H) load(buf[QUADS ? 0 : (base / W + 1) & 1], base + W);
            if (BIAS && base) g = f2(g0 - static_cast<float>(base) * ns, g0 - static_cast<float>(base + 1) * ns);
            auto columns = [&](auto some) {
#pragma unroll
              for (int c = 0; c < W / 2; ++c) {
                const uint64_t xx = f2(s[2 * c], s[2 * c + 1]);
                uint64_t f = sl2;
                if (CAP) {
                  const uint64_t w = mul2(xx, xx);
                  wm = fmax3(wm, f2lo(w), f2hi(w));
                  f = fma2(w, fma2(w, fma2(w, k3, k2), k1), sl2);
                }
                const uint64_t y = fma2(xx, f, g);
                if (decltype(some)::value)
                  take(hidden(base + 2 * c) ? -INFINITY : f2lo(y), hidden(base + 2 * c + 1) ? -INFINITY : f2hi(y),
                       base / 2 + c);
                else
                  take(f2lo(y), f2hi(y), base / 2 + c);
                if (BIAS) g = add2(g, step);
              }
            };
            // Of a tile at the mask's edge, columns that no row sees cost nothing
            // and those that every row sees what they always do.
            if (!decltype(masked)::value) {
              columns(Masked<false>());
            } else if (!__any_sync(0xffffffffu, valid && va < base + W && vb > base)) {
#pragma unroll
              for (int c = 0; c < W / 2; ++c) p[base / 2 + c] = 0;
            } else if (__any_sync(0xffffffffu, valid && (va > base || vb < base + W))) {
              columns(Masked<true>());
            } else {
              columns(Masked<false>());
            }
          }
          return !CAP || !__any_sync(0xffffffffu, valid && !(wm <= a.cap_limit));
        };
        auto exps = [&](float mm) {
          bool ok = true;
          if (BIAS) ok = __all_sync(0xffffffffu, !valid || behind || far <= max(va, 0));
          if (ok) ok = edge ? fast(mm, Masked<true>()) : fast(mm, Masked<false>());
          if ((CAP || BIAS) && !ok) {
            zero();
#pragma unroll
            for (int base = 0; base < H; base += W) {
              float s[W];
              load(s, base);
              tmem_ld_wait();
              exact(s, base);
#pragma unroll
              for (int c = 0; c < W / 2; ++c) take(s[2 * c] - mm, s[2 * c + 1] - mm, base / 2 + c);
            }
          }
          const uint64_t s2 = add2(ps[0], ps[1]);
          ts = f2lo(s2) + f2hi(s2);
          tr = pr[0] + pr[1];
        };
        // Later tiles raise the reference only when needed.  (A row without one has
        // P = 0, l = 0, O = 0.)  Both warps of a pair hold the same references and
        // spans, so they agree.
        if (first) {
          float mx;
          if (!row_max(&mx)) goto done;
          if (m == -INFINITY) m = mx;
        }
        exps(m == -INFINITY ? 0.f : m);
        // either half's sum too large: both raise
        if (j > 0 && __any_sync(0xffffffffu, valid && !(ts <= kRaiseLimit)) && lane == 0) flag[xn & 1] = tc + j + 1;
        __syncwarp();
        if (!pair_sync()) goto done;
        const bool raise = flag[xn & 1] == static_cast<int>(tc + j + 1);
        ++xn;
        if (raise) {
          float mx;
          if (!row_max(&mx)) goto done;
          const float mn = fmaxf(m, mx);
          const float alpha = m == mn ? 1.f : fast_exp2(m - mn);
          m = mn;
          l *= alpha;
          lr *= alpha;
          // O holds PV of every earlier tile: with two Q tiles its commit came with
          // this S.  (j > 0, and no later PV has been issued.)
          if (T == 1 && !bar_wait(&bars->pvdone[(tc + j - 1) & 1], ((tc + j - 1) >> 1) & 1, abort)) goto done;
          __syncwarp();
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {
            uint32_t r[32];
            tmem_ld32(obase + c * 32, r);
            tmem_ld_wait();
#pragma unroll
            for (int y = 0; y < 32; ++y) r[y] = __float_as_uint(__uint_as_float(r[y]) * alpha);
            tmem_st32(obase + c * 32, r);
          }
          exps(m == -INFINITY ? 0.f : m);
        }
        l += ts;
        lr += tr;
        if (QUADS)
          tmem_st8(tmem + lane_base + C::kPCol + sb * 64 + col0 / 2, p);
        else
          tmem_st32(sbase, p);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&bars->pfull[sb]);
      }
      tc += n;
      if (n > 0) {
        if (!bar_wait(&bars->ofull[t], uc & 1, abort)) goto done;
        ++uc;
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
        const int64_t prow = QUADS ? int64_t(x.part) * a.unit_rows + quarter * (a.qn * a.R) + trow
                                   : int64_t(x.part) * (128 * T) + t * 128 + trow;
        if (valid && half == 0) {
          const float lse = l == 0.f ? -INFINITY : m * kLn2 + logf(l);
          if (x.part >= 0)
            a.part_lse[prow] = lse;
          else if (a.lse)
            a.lse[(int64_t(x.b) * a.Hq + hq) * a.Nq + qi] = lse;
        }
        // The warp's 32 half rows go out through its own shared memory, so that
        // consecutive lanes write consecutive bytes of a row (a store of 16 bytes
        // from each of 32 rows touches 32 lines; the output of a unit took 3.5 us).
        const bool wide = x.part >= 0 || a.out_fp32;
        char* base = x.part >= 0 ? reinterpret_cast<char*>(a.part_o) : static_cast<char*>(a.o);
        int64_t at = x.part >= 0 ? prow * D : int64_t(x.b) * a.os.b + int64_t(hq) * a.os.h + int64_t(qi) * a.os.n;
        at = valid ? (at + half * (D / 2)) * (wide ? 4 : 2) : -1;
        uint32_t v[D / 2], again = 0;  // again: rows to be computed once more (rows_again)
        if (n > 0) {
#pragma unroll
          for (int c = 0; c < D / 64; ++c) tmem_ld32(obase + c * 32, v + c * 32);
          tmem_ld_wait();
          tc_fence_before();
          mbar_arrive(&bars->ofree[t]);
#pragma unroll
          for (int y = 0; y < D / 2; ++y) v[y] = __float_as_uint(__uint_as_float(v[y]) * inv);
          if (__any_sync(0xffffffffu, inv == 0.f)) {  // (a row that saw nothing: 0 whatever O holds)
#pragma unroll
            for (int y = 0; y < D / 2; ++y) v[y] = inv == 0.f ? 0 : v[y];
          }
          // Values that are not finite may be those of keys that the row does not see (quads: that
          // the quarter does not take, where an infinity would become a NaN).
          const bool blind = valid && (QUADS || sp.lo > key0 || sp.hi < min(key0 + n * BN, x.uhi));
          if (__any_sync(0xffffffffu, blind)) {
            uint32_t top[2] = {0, 0};  // the largest magnitude's bits
#pragma unroll
            for (int y = 0; y < D / 2; ++y) top[y & 1] = max(top[y & 1], v[y] & 0x7FFFFFFFu);
            again = __ballot_sync(0xffffffffu, blind && max(top[0], top[1]) >= 0x7F800000u && inv != 0.f && isfinite(l));
          }
        } else {
#pragma unroll
          for (int y = 0; y < D / 2; ++y) v[y] = 0;
        }
        if (lane == 0) bars->again[warp] = again;
        if (!pair_sync()) goto done;  // (also: the other half has read this warp's slot)
        again |= bars->again[warp ^ 4];
        if (again >> lane & 1) at = -1;
        auto put = [&](auto words) {  // words per half row
          constexpr int P = decltype(words)::value / 4;                // 16-byte pieces of it
          constexpr int kRows = C::kWarpBytes / 16 / P;                // rows at a time
          uint4* st = reinterpret_cast<uint4*>(own);
          auto cell = [&](int r, int c) -> uint4* {  // (no bank conflicts either way)
            return st + r * P + (P >= 8 ? (c & ~7) | ((c ^ r) & 7) : c ^ ((r >> 1) & 3));
          };
#pragma unroll
          for (int r0 = 0; r0 < 32; r0 += kRows) {
            if (lane >= r0 && lane < r0 + kRows) {
#pragma unroll
              for (int c = 0; c < P; ++c) *cell(lane - r0, c) = make_uint4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
            }
            __syncwarp();
#pragma unroll 1
            for (int f = 0; f < kRows * P; f += 32) {
              const int r = (f + lane) / P, c = (f + lane) % P;
              const int64_t to = __shfl_sync(0xffffffffu, at, r0 + r);
              const uint4 w = *cell(r, c);
              if (to >= 0) *reinterpret_cast<uint4*>(base + to + c * 16) = w;
            }
            __syncwarp();
          }
        };
        if (wide) {
          put(Words<D / 2>());
        } else {
#pragma unroll
          for (int y = 0; y < D / 4; ++y)
            v[y] = pack_bf16(__uint_as_float(v[2 * y]), __uint_as_float(v[2 * y + 1]));
          put(Words<D / 4>());
        }
        if (again) {
          AgainRow* rows = reinterpret_cast<AgainRow*>(own);
          const int64_t row = x.part >= 0 ? prow * D : int64_t(x.b) * a.os.b + int64_t(hq) * a.os.h + int64_t(qi) * a.os.n;
          rows[lane] = {hq, qi, m, 0, (row + half * (D / 2)) * (wide ? 4 : 2)};
          __syncwarp();
          if (!rows_again<D, QUADS>(a, rows, again, x.b, x.part, key0, n, 1 + t * 4 + quarter, abort)) goto done;
          __syncwarp();
        }
      } else if (n > 0) {
        mbar_arrive(&bars->ofree[t]);
      }
    }
  } else if (warp < C::kTmaWarp || (T == 1 && warp == C::kPvWarp)) {
    // ------------------------------------------------------------ MMA issue
    // One warp per Q tile: issuing an MMA blocks while the tensor core is busy,
    // so one thread for both tiles left it idle (1000 of 3600 cycles a step)
    // whenever that thread waited for a barrier or committed.  One tile: a warp for
    // the first product and one for the second (12 heads of 880 keys: 13.2 -> 11.9 us, 128
    // of 8000 83.5 -> 79.4; a step of quads 0.98 -> 0.73).
    const bool second = T == 1 && warp == C::kPvWarp;
    const int t = T == 1 ? 0 : warp - C::kMmaWarp;
    const uint32_t kIdescS = a.neg_scale ? idesc_negate_b(idesc_bf16(128, BN, false, false))
                                         : idesc_bf16(128, BN, false, false);
    constexpr uint32_t kIdescPV = idesc_bf16(128, D, false, true);
    // Descriptor halves: stepping through a tile only adds to the low word.
    const uint64_t dq = sw128_desc(smem_u32(sQ) + t * 128 * D * 2, 16, 1024);
    const uint64_t dk = sw128_desc(smem_u32(sKV), 16, 1024), dv = sw128_desc(smem_u32(sKV), BN * 128, 1024);
    const uint32_t q_lo = static_cast<uint32_t>(dq), q_hi = static_cast<uint32_t>(dq >> 32);
    const uint32_t k_lo = static_cast<uint32_t>(dk), k_hi = static_cast<uint32_t>(dk >> 32);
    const uint32_t v_lo = static_cast<uint32_t>(dv), v_hi = static_cast<uint32_t>(dv >> 32);
    const uint32_t o_tmem = tmem + C::kOCol + t * D;
    auto ready = [&](uint32_t i) -> bool { return bar_wait(&bars->full[i % S], (i / S) & 1, abort); };
    auto pass = [&]() { mbar_arrive(&bars->turn[t ^ 1]); };  // the other tile's turn
    auto sbuf = [&](uint32_t step) -> uint32_t { return T == 2 ? t : step & 1; };
    auto qk = [&](uint32_t i, uint32_t step, bool turn) {
      const uint32_t s_tmem = tmem + sbuf(step) * 128;
      const uint32_t kl = k_lo + (((i % S) * C::kTile) >> 4);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = ((kk >> 2) * 128 * 128 + (kk & 3) * 32) >> 4;
        mma_ss_w(s_tmem, q_lo + off, q_hi, kl + off, k_hi, kIdescS, kk > 0 ? 1u : 0u);
        if (kk == D / 16 - 3 && turn) pass();  // (two MMAs cover the hand-over)
      }
      mma_commit(&bars->sfull[sbuf(step)]);
    };
    auto pv = [&](uint32_t i, uint32_t step, bool first) {
      const uint32_t s_tmem = tmem + sbuf(step) * 128, p_tmem = tmem + C::kPCol + sbuf(step) * 64;
      const uint32_t vl = v_lo + (((i % S) * C::kTile) >> 4);
#pragma unroll
      for (int kk = 0; kk < BN / 16; ++kk)
        // P of keys 0-63 lies in S columns 0-31, of keys 64-127 in 64-95
        mma_ts_w(o_tmem, QUADS ? p_tmem + kk * 8 : s_tmem + (kk >> 2) * 64 + (kk & 3) * 8, vl + ((kk * 2048) >> 4),
                 v_hi, kIdescPV, (!first || kk > 0) ? 1u : 0u);
    };
    if (lane == 0) {
      bool ok = true;
      uint32_t tc = 0, uc = 0, zc = 0;  // key tiles, units with keys and cleared tails so far
      for (uint32_t i = 0; ok; ++i) {
        if (!bar_wait(&bars->ring_full[i & 1], (i >> 1) & 1, abort)) break;
        const Unit x = bars->ring[i & 1];
        mbar_arrive(&bars->ring_empty[i & 1]);
        if (!x.go) break;
        const int key0 = x.key0, n = x.n, uhi = x.uhi;
        if (n == 0) continue;
        // Ring entries: K(j) is number 2 (tc + j), V(j) the one behind it.
        if (T == 1 && !second) {
          if (!(ok = bar_wait(&bars->qfull, uc & 1, abort))) break;
          for (int j = 0; j < n; ++j) {
            const uint32_t step = tc + j, ik = 2 * step, was = step - 2;
            // (the second product of two steps ago is done: S and P of this buffer are free)
            if (!(ok = ready(ik)) || (step >= 2 && !(ok = bar_wait(&bars->pvdone[was & 1], (was >> 1) & 1, abort)))) break;
            tc_fence_after();
            qk(ik, step, false);
            mma_commit(&bars->empty[ik % S]);
          }
          if (ok) mma_commit(&bars->qempty);
          tc += n;
          ++uc;
          continue;
        }
        if (second) {
          for (int j = 0; j < n; ++j) {
            const uint32_t step = tc + j, iv = 2 * step + 1;
            if (!(ok = ready(iv))) break;
            if (j == 0 && uhi - (key0 + (n - 1) * BN) < BN) {  // to be cleared behind the span
              mbar_arrive(&bars->tail_here);
              if (!(ok = bar_wait(&bars->tail, zc++ & 1, abort))) break;
            }
            if (j == 0 && uc > 0 && !(ok = bar_wait(&bars->ofree[t], (uc - 1) & 1, abort))) break;
            if (!(ok = bar_wait(&bars->pfull[step & 1], (step >> 1) & 1, abort))) break;
            tc_fence_after();
            pv(iv, step, j == 0);
            mma_commit(&bars->pvdone[step & 1]);
            mma_commit(&bars->empty[iv % S]);
          }
          if (ok) mma_commit(&bars->ofull[t]);
          tc += n;
          ++uc;
          continue;
        }
        if (!(ok = bar_wait(&bars->qfull, uc & 1, abort)) || !(ok = ready(2 * tc))) break;
        tc_fence_after();
        qk(2 * tc, tc, false);
        mma_commit(&bars->empty[(2 * tc) % S]);
        if (n == 1) mma_commit(&bars->qempty);
        for (int j = 0; j < n; ++j) {
          const bool more = j + 1 < n;
          const uint32_t iv = 2 * (tc + j) + 1, ik = iv + 1;
          if (!(ok = ready(iv)) || (more && !(ok = ready(ik)))) break;
          const bool tail = j == 0 && uhi - (key0 + (n - 1) * BN) < BN;  // to be cleared behind the span
          if (tail) mbar_arrive(&bars->tail_here);
          if (tail && !(ok = bar_wait(&bars->tail, zc++ & 1, abort))) break;
          if (j == 0 && uc > 0 && !(ok = bar_wait(&bars->ofree[t], (uc - 1) & 1, abort))) break;
          // Turns: the tiles' steps alternate (side by side they would fall into
          // step and leave the tensor core idle during both softmaxes).
          if (tc + j + t > 0 && !(ok = bar_wait(&bars->turn[t], (tc + j + t - 1) & 1, abort))) break;
          // (P last: even a wait for what is long done takes about 100 cycles)
          if (!(ok = bar_wait(&bars->pfull[t], (tc + j) & 1, abort))) break;
          tc_fence_after();
          pv(iv, tc + j, j == 0);
          if (more)
            qk(ik, tc + j + 1, true);
          else
            pass();
          if (!more) mma_commit(&bars->ofull[t]);
          mma_commit(&bars->empty[iv % S]);
          if (more) mma_commit(&bars->empty[ik % S]);
          if (j + 2 == n) mma_commit(&bars->qempty);
        }
        tc += n;
        ++uc;
      }
      // Every MMA issued above must finish before TMEM is released.
      const int at = second ? 1 : t;
      mma_commit(&bars->drain[at]);
      const long long t0 = clock64();
      while (!mbar_test(&bars->drain[at], 0) && clock64() - t0 < kWaitLimitCycles) {
      }
    }
  } else if (warp == C::kTailWarp) {
    // ------------------------------------------------------------ tails
    // V rows past the span (another document's, or a cache's unused rows) meet
    // P = 0, but 0 times a NaN or an infinity would still reach O of every row: cleared.
    // The MMA warps say when such a tile has landed.  (Rows inside the span that only
    // some of the unit's rows see: rows_again.)
    uint32_t tc = 0, zc = 0;
    for (uint32_t i = 0;; ++i) {
      if (!bar_wait(&bars->ring_full[i & 1], (i >> 1) & 1, abort)) break;
      const Unit x = bars->ring[i & 1];
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->ring_empty[i & 1]);
      if (!x.go) break;
      // The join's table, by the block that runs the first slot (block 0 may never start:
      // any block may take its slot over).
      if (QUADS && a.slots && x.part == 0)
        for (int b = lane; b < a.B; b += 32) {
          a.part_first[b] = bars->first[b];
          a.part_first[a.B + b] = bars->runs[b];
        }
      const uint32_t iv = 2 * tc + 1;  // the unit's first V: tiles come last first
      tc += x.n;
      const int live = x.uhi - (x.key0 + (x.n - 1) * BN);
      if (x.n == 0 || live >= BN) continue;
      if (!bar_wait(&bars->tail_here, zc++ & 1, abort)) break;
      uint8_t* vt = sKV + (iv % S) * C::kTile;
      for (int f = lane; f < (BN - live) * (D / 8); f += 32) {
        const int r = live + f / (D / 8), ch = f % (D / 8);
        *reinterpret_cast<uint4*>(vt + (ch >> 3) * BN * 128 + r * 128 + (ch & 7) * 16) = make_uint4(0, 0, 0, 0);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->tail);
    }
  } else if (warp == C::kTmaWarp) {
    // ------------------------------------------------------------ units and loads
    if (lane) goto done;
    const uint32_t q_addr = smem_u32(sQ), kv_addr = smem_u32(sKV);
    int64_t g = blockIdx.x;
    uint32_t it = 0, uc = 0;
    bool ok = true;
    uint32_t i = 0;
    for (; ok; ++i) {
      Unit x = {};
      if (g >= 0) {
        mbar_expect_tx(&bars->next, 16);
        request_block(&bars->answer, &bars->next);
        // Heads in groups whose K and V stay in L2; in a group the row blocks from
        // the last (with a causal mask the longest) to the first, each of all its
        // heads: long units start first and short ones fill the end (one head
        // after the other left a fifth of the time to the last head's long units).
        // Units from full_units on are split over their keys.
        int u = static_cast<int>(g), split = 0, splits = 1;
        x.go = 1;
        x.part = -1;
        bool none = false;  // a slot that no unit has
        if (QUADS && a.slots) {
          x.part = u;
          none = u >= bars->used;
          int e = 0, top = none ? 0 : a.B - 1;  // the last batch entry that starts here or before
          while (e < top) {
            const int mid = (e + top + 1) >> 1;
            if (bars->first[mid] <= u)
              e = mid;
            else
              top = mid - 1;
          }
          splits = max(bars->runs[e], 1);
          const int in = u - bars->first[e], h = in / splits;
          split = in - h * splits;
          u = none ? 0 : e * a.Hkv + h;
        } else if (g >= a.full_units) {
          splits = a.splits;
          x.part = static_cast<int>(g - a.full_units);
          split = x.part % splits;
          u = static_cast<int>(a.full_units) + x.part / splits;
        }
        const Place at = place_of(a, u);
        const int bh = at.bh;
        x.q0 = at.rb * (T * a.qn);
        x.b = bh / a.Hkv;
        x.hk = bh - x.b * a.Hkv;
        // keys that any of the unit's rows sees, and this split's run of tiles
        int ulo;
        const int ntiles = none ? 0 : tiles_of(a, x.b, x.q0, min(x.q0 + T * a.qn, a.Nq) - 1, &ulo, &x.uhi);
        const int j0 = static_cast<int>(int64_t(ntiles) * split / splits);
        x.n = static_cast<int>(int64_t(ntiles) * (split + 1) / splits) - j0;
        x.key0 = none ? 0 : ulo + j0 * BN;
      }
      const int key0 = x.key0, n = x.n;
      if (i >= 2 && !bar_wait(&bars->ring_empty[i & 1], ((i >> 1) - 1) & 1, abort)) break;
      bars->ring[i & 1] = x;
      mbar_arrive(&bars->ring_full[i & 1]);
      if (g < 0) break;
      if (n > 0) {
        if (uc > 0 && !bar_wait(&bars->qempty, (uc - 1) & 1, abort)) break;
        ++uc;
        constexpr int kCopies = QUADS ? 4 : T;  // of one tile, or of each
        mbar_expect_tx(&bars->qfull, kCopies * a.qn * a.R * D * 2);
#pragma unroll
        for (int t = 0; t < kCopies; ++t)
#pragma unroll
          for (int cb = 0; cb < D / 64; ++cb)
            tma_load_4d(q_addr + (QUADS ? t * 32 * 128 : t * 128 * D * 2) + cb * 128 * 128, &tm_q, 64 * cb, x.hk * a.R,
                        x.q0 + (QUADS ? 0 : t * a.qn), x.b, &bars->qfull);
        for (int f = 0; f < 2 * n; ++f, ++it) {
          const uint32_t s = it % S;
          if (!(ok = bar_wait(&bars->empty[s], ((it / S) & 1) ^ 1, abort))) break;
          mbar_expect_tx(&bars->full[s], C::kTile);
          const int key = key0 + (n - 1 - (f >> 1)) * BN;
#pragma unroll
          for (int cb = 0; cb < D / 64; ++cb)
            tma_load_4d(kv_addr + s * C::kTile + cb * BN * 128, (f & 1) ? &tm_v : &tm_k, 64 * cb, key, x.hk, x.b,
                        &bars->full[s]);
        }
        if (!ok) break;
      }
      if (!(ok = bar_wait(&bars->next, i & 1, abort))) break;
      g = answered_block(&bars->answer);
      fence_proxy_async_smem();  // read before the next answer is written
    }
    if (*abort) {
      // After an abort: what is in flight lands before the block ends.
      auto settle = [&](uint64_t* bar, uint32_t parity) {
        const long long t0 = clock64();
        while (!mbar_test(bar, parity) && clock64() - t0 < kWaitLimitCycles) {
        }
      };
      for (uint32_t f = it > S ? it - S : 0; f < it; ++f) settle(&bars->full[f % S], (f / S) & 1);
      if (uc > 0) settle(&bars->qfull, (uc - 1) & 1);
      if (g >= 0) settle(&bars->next, i & 1);
    }
  }
done:
  if (warp < C::kSoftWarps && *abort) named_barrier_arrive(1 + (warp >> 3) * 4 + (warp & 3), 64);
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
// o = sum_s e^(lse_s - lse) o_s.  Bound by its launch and two rounds of loads.
template <int D>
__global__ void __launch_bounds__(128) sa_masked_join_kernel(const __grid_constant__ MaskedArgs a) {
  // (launched while the partial results are still being made: read by plain loads, which stay behind the wait)
  wait_for_earlier_kernel();
  const uint32_t i = blockIdx.x * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const uint32_t tile_rows = a.qn * a.R, unit_rows = a.tiles * tile_rows;  // that exist
  const uint32_t su = i / unit_rows, r = i - su * unit_rows, t = r / tile_rows, tr = r - t * tile_rows;
  if (su >= a.split_units) return;
  const Place at = place_of(a, static_cast<int>(a.full_units + su));
  const int q = at.rb * (a.tiles * a.qn) + t * a.qn + tr / a.R;
  if (q >= a.Nq) return;
  const int64_t row0 = int64_t(su) * a.splits * a.unit_rows + t * 128 + tr;
  float mx = -INFINITY;
  bool none = false;  // a partial result that is not a number makes the row none (fmaxf drops it)
  for (int s = lane; s < a.splits; s += 32) {
    const float l = a.part_lse[row0 + s * a.unit_rows];
    mx = fmaxf(mx, l);
    none |= l != l;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  constexpr int V = D / 32;
  float acc[V] = {}, sum = 0.f;
  if (mx != -INFINITY || __any_sync(0xffffffffu, none)) {
#pragma unroll 8
    for (int s = 0; s < a.splits; ++s) {
      const int64_t row = row0 + s * a.unit_rows;
      const float w = __expf(a.part_lse[row] - mx);
      float f[V];
      if (V == 4) {
        const float4 x = reinterpret_cast<const float4*>(a.part_o + row * D)[lane];
        f[0] = x.x, f[1] = x.y, f[V - 2] = x.z, f[V - 1] = x.w;
      } else {
        const float2 x = reinterpret_cast<const float2*>(a.part_o + row * D)[lane];
        f[0] = x.x, f[1] = x.y;
      }
      sum += w;
#pragma unroll
      for (int e = 0; e < V; ++e) acc[e] += w * f[e];
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const int h = (at.bh % a.Hkv) * a.R + tr % a.R, b = at.bh / a.Hkv;
  const int64_t oo = int64_t(b) * a.os.b + int64_t(h) * a.os.h + int64_t(q) * a.os.n + lane * V;
#pragma unroll
  for (int e = 0; e < V; e += 2) {
    if (a.out_fp32)
      *reinterpret_cast<float2*>(static_cast<float*>(a.o) + oo + e) = make_float2(acc[e] * inv, acc[e + 1] * inv);
    else
      *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.o) + oo + e) = pack_bf16(acc[e] * inv, acc[e + 1] * inv);
  }
  if (lane == 0 && a.lse) a.lse[(int64_t(b) * a.Hq + h) * a.Nq + q] = sum == 0.f ? -INFINITY : mx + logf(sum);
}

// The same for quads, whose rows have four partial results a split (up to 608 in all):
// a block per row, each warp every sixteenth of them.
template <int D>
__global__ void __launch_bounds__(512) sa_masked_join_quads_kernel(const __grid_constant__ MaskedArgs a) {
  constexpr int V = D / 32, WARPS = 16;
  __shared__ float s_mx[WARPS], s_sum[WARPS], s_acc[WARPS][D];
  wait_for_earlier_kernel();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rows = a.qn * a.R, su = blockIdx.x / rows, tr = blockIdx.x - su * rows;
  const int bh = place_of(a, su).bh, b = bh / a.Hkv, hk = bh - b * a.Hkv;
  int parts = a.splits;
  int64_t first = int64_t(su) * parts;
  if (a.slots) {
    // (within the workspace even if the attention gave up before it wrote the table)
    parts = min(max(a.part_first[a.B + b], 0), a.slots);
    first = min(max(int64_t(a.part_first[b]) + int64_t(hk) * parts, int64_t(0)), int64_t(a.slots - parts));
  }
  parts *= 4;
  const int64_t row0 = first * a.unit_rows + tr;
  float mx = -INFINITY, sum = 0.f, acc[V] = {};
  for (int p = warp; p < parts; p += WARPS * 8) {  // eight at a time
    float l[8], top = mx, f[8][V];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int at = p + i * WARPS;
      l[i] = at < parts ? a.part_lse[row0 + at * rows] : -INFINITY;
#pragma unroll
      for (int e = 0; e < V; ++e) f[i][e] = 0.f;
      if (at < parts) {
        const float* o = a.part_o + (row0 + at * rows) * D + lane * V;
        const float2 x = *reinterpret_cast<const float2*>(o), y = *reinterpret_cast<const float2*>(o + V - 2);
        f[i][0] = x.x, f[i][1] = x.y, f[i][V - 2] = y.x, f[i][V - 1] = y.y;
      }
    }
    bool none = false;  // (fmaxf drops what is not a number; it makes the sums none)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      top = fmaxf(top, l[i]);
      none |= l[i] != l[i];
    }
    if (top == -INFINITY && !none) continue;
    const float keep = __expf(mx - top);
    mx = top;
    sum *= keep;
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] *= keep;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float w = __expf(l[i] - mx);
      sum += w;
#pragma unroll
      for (int e = 0; e < V; ++e) acc[e] += w * f[i][e];
    }
  }
  if (lane == 0) {
    s_mx[warp] = mx;
    s_sum[warp] = sum;
  }
#pragma unroll
  for (int e = 0; e < V; ++e) s_acc[warp][lane * V + e] = acc[e];
  __syncthreads();
  const int c = threadIdx.x;
  if (c >= D) return;
  float all = -INFINITY, total = 0.f, x = 0.f;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) all = fmaxf(all, s_mx[w]);
#pragma unroll
  for (int w = 0; w < WARPS; ++w)
    if (s_sum[w] != 0.f) {  // (a NaN is not 0)
      const float e = __expf(s_mx[w] - all);
      total += e * s_sum[w];
      x += e * s_acc[w][c];
    }
  x = total == 0.f ? 0.f : x / total;
  const int h = hk * a.R + tr % a.R, q = tr / a.R;
  const int64_t at = int64_t(b) * a.os.b + int64_t(h) * a.os.h + int64_t(q) * a.os.n + c;
  if (a.out_fp32)
    static_cast<float*>(a.o)[at] = x;
  else
    static_cast<uint16_t*>(a.o)[at] = static_cast<uint16_t>(pack_bf16(x, 0.f));
  if (c == 0 && a.lse) a.lse[(int64_t(b) * a.Hq + h) * a.Nq + q] = total == 0.f ? -INFINITY : all + logf(total);
}

// Units that fill whole waves of SMs run whole; the rest (all, if they are
// fewer than the SMs) are split into the number of key runs that ends first by
// this count of tile times: a wave costs its tiles plus a block's start, a
// split the join.  What the host knows of their tiles: the mask without
// documents and lengths (a causal mask leaves little to the last units).
void masked_plan(MaskedArgs* a) {
  a->qn = 128 / a->R;
  const int T = a->tiles = a->Nq > a->qn ? 2 : 1;
  a->unit_rows = 128 * T;
  const int64_t unit_q = int64_t(T) * a->qn;
  a->row_blocks = static_cast<int32_t>((a->Nq + unit_q - 1) / unit_q);
  if (a->qn > a->Nq) a->qn = a->Nq;
  // Heads that are worked on at a time.  Units of one length: as many as keep K
  // and V in half the L2 (24 heads of 16384 x 16384: 2.17 ms, 2.23 with all at
  // once).  Units of different lengths (causal, documents) want more of them to
  // choose from: K and V up to twice the L2 (24 packed heads of 16384 tokens, 201
  // MB: 598 us at once, 647 in groups of 64 MB; 24 causal ones 1127 and 1141).
  const bool even = !a->mask.causal && !a->mask.nd;
  const int64_t heads = int64_t(a->B) * a->Hkv,
                fit = (int64_t(even ? 64 : 256) << 20) / (int64_t(a->Nk) * a->d * 4);
  const int64_t groups = fit < 1 ? heads : (heads + fit - 1) / fit;
  a->group = static_cast<int32_t>((heads + groups - 1) / groups);
  const int64_t units = heads * a->row_blocks, rest = units % kSms;
  int64_t seen = 0;  // keys that the last units see
  for (int64_t u = units - rest; u < units; ++u) {
    const int64_t q1 = min64(a->Nq, (place_of(*a, static_cast<int>(u)).rb + 1) * unit_q);
    int64_t hi = a->Nk;
    if (a->mask.causal) {
      const int64_t pos = q1 - 1 + a->Nk - a->Nq;
      hi = pos < 0 ? 0 : min64(hi, (pos / a->mask.causal + 1) * a->mask.causal);
    }
    seen += hi;
  }
  const int64_t tiles = rest ? (seen / rest + BN - 1) / BN : 0;
  constexpr int64_t kStart = 5, kJoin = 8;
  int64_t best = 1, cost = tiles + kStart;
  for (int64_t s = 2; s <= tiles && s <= 64; ++s) {
    const int64_t c = (rest * s + kSms - 1) / kSms * ((tiles + s - 1) / s + kStart) + kJoin;
    if (c < cost) {
      cost = c;
      best = s;
    }
  }
  a->splits = static_cast<int32_t>(best);
  a->full_units = best == 1 ? units : units - rest;
  a->split_units = units - a->full_units;
  // Few rows, all units split: quads (6 key heads of 28160 keys, 4 rows each: 19.0 us then, 22.2
  // with the rows in one lane quarter).  Where lengths may differ the device shares the
  // runs out, which costs a start of 1.7 us: not for short runs (16 key heads of 4000 keys
  // in runs of 4 tiles: 15.8 us shared out, 14.2 not).
  a->quads = T == 1 && a->full_units == 0 && a->qn * a->R <= 32;
  if (a->quads) {
    a->unit_rows = 4 * a->qn * a->R;
    if ((a->mask.nd || a->mask.len) && tiles >= 8 * best)
      a->slots = static_cast<int32_t>(min64(units * ((int64_t(a->Nk) + BN - 1) / BN), kSms));
  }
}

template <int D, int T, bool QUADS, bool CAP, bool BIAS>
static cudaError_t launch_m(const MaskedArgs& a, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                            cudaStream_t st) {
  using C = MCfg<D, T>;
  auto kern = sa_masked_kernel<D, T, QUADS, CAP, BIAS>;
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
  const int64_t grid = a.slots ? a.slots : a.full_units + a.split_units * a.splits;
  kern<<<static_cast<unsigned>(grid), C::kThreads, smem, st>>>(a, tq, tk, tv);
  return cudaGetLastError();
}

template <int D, int T, bool QUADS>
static cudaError_t launch_t(const MaskedArgs& a, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                            cudaStream_t st) {
  const bool cap = a.cap_log2 > 0.f, bias = a.slopes != nullptr;
  if (cap)
    return bias ? launch_m<D, T, QUADS, true, true>(a, q, k, v, st) : launch_m<D, T, QUADS, true, false>(a, q, k, v, st);
  return bias ? launch_m<D, T, QUADS, false, true>(a, q, k, v, st) : launch_m<D, T, QUADS, false, false>(a, q, k, v, st);
}

template <int D>
static cudaError_t launch_d(const MaskedArgs& a, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                            cudaStream_t st) {
  const cudaError_t e = a.tiles == 2 ? launch_t<D, 2, false>(a, q, k, v, st)
                        : a.quads    ? launch_t<D, 1, true>(a, q, k, v, st)
                                     : launch_t<D, 1, false>(a, q, k, v, st);
  if (e != cudaSuccess || a.split_units == 0) return e;
  const int64_t rows = a.split_units * a.tiles * a.qn * a.R;
  if (a.quads)
    return launch_early(sa_masked_join_quads_kernel<D>, dim3(static_cast<unsigned>(rows)), 512, 0, st, a);
  return launch_early(sa_masked_join_kernel<D>, dim3(static_cast<unsigned>((rows + 3) / 4)), 128, 0, st, a);
}

cudaError_t launch_masked(const MaskedArgs& a, cudaStream_t st) {
  CUtensorMap tq, tk, tv;
  if (!make_view_map(&tq, a.q, a.d, a.Nq, a.Hq, a.B, a.qs.n, a.qs.h, a.qs.b, a.qn, a.R, true) ||
      !make_view_map(&tk, a.k, a.d, a.Nk, a.Hkv, a.B, a.ks.n, a.ks.h, a.ks.b, BN, 1, false) ||
      !make_view_map(&tv, a.v, a.d, a.Nk, a.Hkv, a.B, a.vs.n, a.vs.h, a.vs.b, BN, 1, false))
    return cudaErrorInvalidValue;
  return a.d == 128 ? launch_d<128>(a, tq, tk, tv, st) : launch_d<64>(a, tq, tk, tv, st);
}

}  // namespace sa
