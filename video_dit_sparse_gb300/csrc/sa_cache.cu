// sa_cache.cu — which cached keys matter, and the eviction of the others.
//
//  * sa_cache_weights_kernel:  w_out[j] = decay w_in[j] + sum over the query
//    heads that share the key head, and their rows i, of p_ij = e^(s_ij - lse_i):
//    the attention weight key j received, in one pass over the scores.  s is
//    the masked forward's (mask, cap, bias); a masked pair adds nothing.
//  * sa_evict_select_kernel:  of a head's n entries keep the first `sink`, the
//    last `recent` and the highest weights in between (ties: lowest index).
//  * sa_evict_gather_kernel:  the kept rows of K, V and w, in their order.
//
// Weights.  S^T = K Q^T puts keys on the 128 TMEM lanes and query rows on the
// columns, so an epilogue thread owns one key and sums over queries in its own
// registers: no cross-lane reduction, no atomics, a fixed order.  A unit is 256
// keys, two tiles that stay in shared memory while Q tiles of up to 256 packed
// rows (query * R + head-in-group) stream by, each read once for both (with one
// 128-key tile a unit, Q came from L2 at 51 bytes a cycle and SM, its limit).
// Each key tile has its own TMEM buffer, its own MMA warp (its waits and commits
// overlap the other's MMAs; they take turns, so that one buffer's sums run
// beside the other's MMA) and two sets of four epilogue warps, one per half of
// the columns.  With many rows the tensor core is the floor, and two things come
// near it: an exponential a pair (0.8 of its time on the MUFU) and shared memory
// (both MMA operands, 3/4 of the time, and the reads of lse): 12 heads of 7040 rows x
// 35200 keys take 590 us, 61 % of the measured bf16 rate.  (With a cap 932; with two or
// three documents 525 to 610; with a bias 2960, every tile by column: `careful`.)  With one token per
// sequence the bound is the read of K (256-key units of one Q tile: 83 200 keys of 6
// heads, 128 MB, in 27 us).
#include <cooperative_groups.h>

#include <atomic>
#include <climits>

#include "sa_device.cuh"
#include "sa_internal.h"
#include "sa_mask.cuh"
#include "sa_tma.h"

namespace sa {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kMaxStages = 6;

struct WCfg {
  static constexpr int kEpiWarps = 16, kMmaWarp = 16, kTmaWarp = 18;
  // 640 threads launch with 96 registers each = 61440 = 512 * 104 + 128 * 64
  static constexpr int kThreads = 640, kRegEpi = 104, kRegOther = 64;
  static constexpr int kCols = 256;  // columns of a TMEM buffer
};

// What a launch fixes: the Q tile (qn queries x R heads = rows, NR columns),
// the rings and the units.
struct WPlan {
  int32_t qn, rows, NR, qtiles, qst, kst, kqbytes, ktile;
  int32_t units, kunits;  // in all, and per head
  int32_t parts;          // blocks (a cluster) that share a unit's Q tiles
};
constexpr int kUnitKeys = 256;

struct WUnit {
  int go;              // 0: no more units
  int b, hk, k0, len;  // len: keys of the batch entry
  int t0, t1;          // Q tiles with a row that sees one of the unit's keys
  int rot;             // taken from t0 + rot on, round
  __device__ __forceinline__ int tile(int s) const { return t0 + rot + s < t1 ? t0 + rot + s : rot + s + t0 - (t1 - t0); }
};
struct WBars {
  uint64_t kfull[kMaxStages], kempty[kMaxStages], qfull[kMaxStages], qempty[kMaxStages];
  uint64_t dfull[2], dempty[2], hfull[2], hempty[2], turn[2], drain[2];
  uint64_t next, ring_full[2], ring_empty[2];
  uint4 answer;  // of the request for the next unit
  WUnit ring[2];
  uint32_t tmem_base;
  int abort;
};

// Unit u, and of its Q tiles the run that block `rank` of its cluster takes.
__device__ __forceinline__ WUnit unit_at(const MaskedArgs& a, const WPlan& p, int u, int rank) {
  WUnit x;
  x.go = 1;
  const int bh = u / p.kunits;
  x.k0 = (u - bh * p.kunits) * kUnitKeys;
  x.b = bh / a.Hkv;
  x.hk = bh - x.b * a.Hkv;
  const MaskDev& m = a.mask;
  x.len = m.len ? clamp_int(__ldg(m.len + x.b), 0, m.Nk) : m.Nk;
  x.t0 = 0;
  x.t1 = x.k0 < x.len ? p.qtiles : 0;
  // Both ends of the rows' spans never decrease, so the tiles form a run.
  if (m.causal || m.nd)
    for (int top = x.t1; x.t0 < top;) {  // the first tile that sees a key of the unit or behind it
      const int mid = (x.t0 + top) >> 1;
      if (row_span(m, x.b, min((mid + 1) * p.qn, m.Nq) - 1).hi <= x.k0)
        x.t0 = mid + 1;
      else
        top = mid;
    }
  if (m.nd)
    for (int low = x.t0; low < x.t1;) {  // the first one that sees only keys behind the unit
      const int mid = (low + x.t1) >> 1;
      if (row_span(m, x.b, mid * p.qn).lo >= x.k0 + kUnitKeys)
        x.t1 = mid;
      else
        low = mid + 1;
    }
  const int n = x.t1 - x.t0;
  x.t1 = x.t0 + n * (rank + 1) / p.parts;
  x.t0 += n * rank / p.parts;
  // Blocks that work on the same head's keys start at different Q tiles (in step
  // they would all ask L2 for the same lines).
  x.rot = (u & 15) * (x.t1 - x.t0) / 16;
  return x;
}

// A key's sum over the rows from column `first` on that have a finite lse (L: theirs in exp2
// units, negated; -inf: another column), without a cap: for tiles whose plain sum is no number.
__device__ __noinline__ float sum_of_rows(float scale_log2, uint32_t sbase, int H, int first, const float* L) {
  float sum = 0.f;
  for (int c = 0; c < H; c += 16) {
    float x[16];
    tmem_ld16(sbase + c, reinterpret_cast<uint32_t*>(x));
    tmem_ld_wait();
#pragma unroll
    for (int e = 0; e < 16; ++e)
      if (c + e >= first && L[c + e] != -INFINITY) sum += fast_exp2(fmaf(x[e], scale_log2, L[c + e]));
  }
  return sum;
}

}  // namespace

template <int D, bool CAP, bool BIAS>
__global__ void __launch_bounds__(WCfg::kThreads, 1)
    sa_cache_weights_kernel(const __grid_constant__ WeightArgs wa, const __grid_constant__ WPlan p,
                            const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k) {
  const MaskedArgs& a = wa.m;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sK = smem;
  uint8_t* sQ = sK + p.kst * p.ktile;
  float* sL = reinterpret_cast<float*>(sQ + p.qst * p.kqbytes);  // [2][4 sets][128] -lse in exp2 units
  int* sD = reinterpret_cast<int*>(sL + 2 * 4 * 128);            // [2][4 sets][4 warps] a row without lse
  float* sX = reinterpret_cast<float*>(sD + 2 * 4 * 4);          // [2][128] half 1's sums of each key tile; [2][128] the block's
  WBars* bars = reinterpret_cast<WBars*>(sX + 4 * 128);
  volatile int* abort = &bars->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = blockIdx.x % p.parts;
  if (threadIdx.x < 256) sX[2 * 128 + threadIdx.x] = 0.f;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(&bars->kfull[s], 1);
      mbar_init(&bars->kempty[s], 1);
      mbar_init(&bars->qfull[s], 1);
      mbar_init(&bars->qempty[s], 2);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&bars->dfull[b], 1);
      mbar_init(&bars->dempty[b], 256);
      mbar_init(&bars->hfull[b], 128);
      mbar_init(&bars->hempty[b], 128);
      mbar_init(&bars->turn[b], 1);
      mbar_init(&bars->ring_full[b], 1);
      mbar_init(&bars->ring_empty[b], WCfg::kEpiWarps + 2);
      mbar_init(&bars->drain[b], 1);
    }
    mbar_init(&bars->next, 1);
    bars->abort = 0;
    fence_mbar_init();
  }
  // Q rows that no copy fills are zero for good (their columns count nothing,
  // but what they hold must not be a NaN).
  for (int i = threadIdx.x; i < p.qst * p.kqbytes / 16; i += WCfg::kThreads)
    reinterpret_cast<uint4*>(sQ)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  if (warp == WCfg::kMmaWarp) {
    tmem_alloc(&bars->tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;

  if (warp < WCfg::kEpiWarps)
    reg_alloc<WCfg::kRegEpi>();
  else
    reg_dealloc<WCfg::kRegOther>();

  if (warp < WCfg::kEpiWarps) {
    // ------------------------------------------------------------ epilogue
    // Set = warp / 4: key tile set / 2, columns' half set % 2.
    const int set = warp >> 2, d = set >> 1, half = set & 1, tid = threadIdx.x & 127;
    const int H = p.NR / 2, col0 = half * H;
    const uint32_t sbase = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + d * WCfg::kCols + col0;
    // The set's thread tid holds column col0 + tid: query tile * qn + qo of a head.
    const int cr = col0 + tid;
    const bool has = tid < H && cr < p.rows;
    const int qo = has ? cr / a.R : INT_MAX / 2;
    const uint32_t off = has ? uint32_t(cr % a.R) * uint32_t(a.Nq) + uint32_t(qo) : 0;
    const float sl = a.scale_log2;
    const bool docs = a.mask.nd > 0;  // (a length alone only decides which keys are written)
    uint32_t it = 0, hn = 0;  // Q tiles, and sums handed on so far
    // What a unit needs first is loaded while the unit before it is worked on.
    WUnit nu = {};
    uint32_t un = 0;  // units read from the ring
    float nwas = 0.f, next = 0.f;  // its entry as it was; lse of the coming tile's column
    auto fetch = [&](const WUnit& x, int t) {
      next = qo < a.Nq - t * p.qn
                 ? __ldg(wa.lse + (int64_t(x.b) * a.Hq + int64_t(x.hk) * a.R) * a.Nq + int64_t(t) * p.qn + off)
                 : 0.f;
    };
    auto look = [&]() -> bool {
      if (!mbar_wait(&bars->ring_full[un & 1], (un >> 1) & 1, abort)) return false;
      nu = bars->ring[un & 1];
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->ring_empty[un & 1]);
      ++un;
      nwas = 0.f;
      if (!nu.go) return true;
      const int key = nu.k0 + d * 128 + tid;
      if (p.parts == 1 && !half && key < a.Nk && wa.w_in && (key >= nu.len || wa.decay != 0.f))
        nwas = wa.w_in[(int64_t(nu.b) * a.Hkv + nu.hk) * a.Nk + key];
      if (nu.t0 < nu.t1) fetch(nu, nu.tile(0));
      return true;
    };
    if (!look()) goto done;
    while (nu.go) {
      const WUnit x = nu;
      const float was = nwas;
      const int b = x.b, key = x.k0 + d * 128 + tid;
      const float* slopes = BIAS ? a.slopes + x.hk * a.R : nullptr;
      float total = 0.f;
      // Without documents a key is seen from one query on.
      int from = INT_MIN / 2;
      if (a.mask.causal && !docs) from = key / a.mask.causal * a.mask.causal - (x.len - a.Nq);
      if (x.t0 >= x.t1 && !look()) goto done;
      for (int s = 0; s < x.t1 - x.t0; ++s, ++it) {
        const int t = x.tile(s);
        // lse of this tile's columns, by all of the set; a row without a finite one
        // adds nothing.  (A warp that gives up arrives once, below `done`.)
        float* wL = sL + ((it & 1) * 4 + set) * 128;
        int* wD = sD + ((it & 1) * 4 + set) * 4;
        const bool row = qo < a.Nq - t * p.qn, fin = isfinite(next);
        wL[tid] = row && fin ? -next * kLog2e : -INFINITY;
        const bool none = __any_sync(0xffffffffu, row && !fin);
        if (lane == 0) wD[warp & 3] = none;
        named_barrier(1 + set, 128);
        if (*abort) goto done;
        const int4 dead4 = *reinterpret_cast<const int4*>(wD);
        const bool dead = (dead4.x | dead4.y | dead4.z | dead4.w) != 0;
        const int qa = t * p.qn, qz = min(qa + p.qn, a.Nq) - 1, kt = x.k0 + d * 128;
        bool edge = false;
        if (docs)
          edge = row_span(a.mask, b, qz).lo > kt || row_span(a.mask, b, qa).hi < min(kt + 128, a.Nk);
        const int first = from > qa ? (min(from - qa, p.qn) * a.R) - col0 : 0;  // the half's first column to count
        const bool cut = __any_sync(0xffffffffu, first > 0);
        if (s + 1 < x.t1 - x.t0)
          fetch(x, x.tile(s + 1));
        else if (!look())
          goto done;
        if (!mbar_wait(&bars->dfull[d], it & 1, abort)) goto done;
        __syncwarp();
        tc_fence_after();
        uint64_t acc[2] = {0, 0};
        // An exponent from its raw product and -lse (-inf: no row's).  With a cap: exactly (three MUFU
        // results), or (`quick`) tanh(z)/z by the masked forward's polynomial for
        // |z| <= 0.4; a tile with a larger score is summed again exactly.
        auto exponent = [&](float x, float L) -> float {
          if (CAP) {
            const float y = fmaf(-2.f * a.cap_log2, fast_rcp(1.f + fast_exp2(x * a.cap_k1)), a.cap_log2) + L;
            return L == -INFINITY ? L : y;
          }
          return fmaf(x, sl, L);
        };
        // The plain columns of the tile: the next 32 load while 32 are summed.
        bool quick = CAP;
        float wm = 0.f;
        auto sum = [&](const float* x, int c, int count) {
          const uint64_t sl2 = f2(sl, sl);
          const uint64_t k1 = f2(a.cap_p1, a.cap_p1), k2 = f2(a.cap_p2, a.cap_p2), k3 = f2(a.cap_p3, a.cap_p3);
          auto bent = [&](float x0, float x1, uint64_t L) -> uint64_t {
            const uint64_t xx = f2(x0, x1), w = mul2(xx, xx);
            wm = fmax3_nan(wm, f2lo(w), f2hi(w));
            return fma2(xx, fma2(w, fma2(w, fma2(w, k3, k2), k1), sl2), L);
          };
#pragma unroll
          for (int e = 0; e < count; e += 4) {
            const ulonglong2 L = *reinterpret_cast<const ulonglong2*>(wL + c + e);
            uint64_t y0, y1;
            if (CAP && quick) {
              y0 = bent(x[e], x[e + 1], L.x);
              y1 = bent(x[e + 2], x[e + 3], L.y);
            } else if (CAP) {
              y0 = f2(exponent(x[e], f2lo(L.x)), exponent(x[e + 1], f2hi(L.x)));
              y1 = f2(exponent(x[e + 2], f2lo(L.y)), exponent(x[e + 3], f2hi(L.y)));
            } else {
              y0 = fma2(f2(x[e], x[e + 1]), sl2, L.x);
              y1 = fma2(f2(x[e + 2], x[e + 3]), sl2, L.y);
            }
            acc[0] = add2(acc[0], f2(fast_exp2(f2lo(y0)), fast_exp2(f2hi(y0))));
            acc[1] = add2(acc[1], f2(fast_exp2(f2lo(y1)), fast_exp2(f2hi(y1))));
          }
        };
        // Columns before each key's first one are left out.
        auto after_first = [&]() {
          for (int c = 0; c < H; c += 16) {
            if (!__any_sync(0xffffffffu, first < c + 16)) continue;
            float x[16];
            tmem_ld16(sbase + c, reinterpret_cast<uint32_t*>(x));
            tmem_ld_wait();
            const int f = first - c;
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              const float2 L = *reinterpret_cast<const float2*>(wL + c + e);
              const float y0 = exponent(x[e], L.x), y1 = exponent(x[e + 1], L.y);
              acc[0] = add2(acc[0], f2(fast_exp2(e < f ? -INFINITY : y0), fast_exp2(e + 1 < f ? -INFINITY : y1)));
            }
          }
        };
        auto plain = [&]() {
          if (H == 128) {
            float buf[2][32];
            tmem_ld32(sbase, reinterpret_cast<uint32_t*>(buf[0]));
#pragma unroll
            for (int c = 0; c < 128; c += 32) {
              tmem_ld_wait();
              if (c + 32 < 128) tmem_ld32(sbase + c + 32, reinterpret_cast<uint32_t*>(buf[(c / 32 + 1) & 1]));
              sum(buf[(c / 32) & 1], c, 32);
            }
          } else {
            for (int c = 0; c < H; c += 16) {
              float x[16];
              tmem_ld16(sbase + c, reinterpret_cast<uint32_t*>(x));
              tmem_ld_wait();
              sum(x, c, 16);
            }
          }
        };
        // With masked or dead columns, or a bias: each column's span, position
        // and slope come from the lane that holds them.
        auto careful = [&]() {
          for (int c = 0; c < H; c += 16) {
            float x[16];
            int lo = 0, hi = INT_MAX, pos = 0;
            float slope = 0.f;
            const int rr = col0 + c + (lane & 15);
            if (rr < p.rows && qa + rr / a.R < a.Nq) {
              const Span sp = row_span(a.mask, b, qa + rr / a.R);
              lo = sp.lo;
              hi = sp.hi;
              pos = sp.pos;
              if (BIAS) slope = -__ldg(slopes + rr % a.R) * kLog2e;
            }
            __syncwarp();
            tmem_ld16(sbase + c, reinterpret_cast<uint32_t*>(x));
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              float y[2];
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const float L = wL[c + e + i];
                y[i] = exponent(x[e + i], L);
                const int clo = __shfl_sync(0xffffffffu, lo, e + i), chi = __shfl_sync(0xffffffffu, hi, e + i);
                if (BIAS) {
                  const float s = __shfl_sync(0xffffffffu, slope, e + i);
                  const int cp = __shfl_sync(0xffffffffu, pos, e + i);
                  y[i] = fmaf(s, fabsf(static_cast<float>(cp - key)), y[i]);
                }
                if (key < clo || key >= chi || L == -INFINITY) y[i] = -INFINITY;
              }
              acc[0] = add2(acc[0], f2(fast_exp2(y[0]), fast_exp2(y[1])));
            }
          }
        };
        if (BIAS || edge || dead)
          careful();
        else if (cut)
          after_first();
        else
          plain();
        // (keys behind the tensor are zeros; what lies behind a sequence may hold anything)
        if (CAP && !(BIAS || edge || dead || cut) &&
            __any_sync(0xffffffffu, key < x.len && !(wm <= a.cap_limit))) {
          quick = false;
          acc[0] = acc[1] = 0;
          plain();
        }
        // Columns of no row are zeros, which an infinity or a NaN in K turns into NaN.  (Under a cap
        // the exact form leaves them out: the square of such a product is past the limit.)
        if (!CAP && !(BIAS || edge || dead)) {
          const uint64_t s2 = add2(acc[0], acc[1]);
          const float is = f2lo(s2) + f2hi(s2);
          if (__any_sync(0xffffffffu, key < x.len && is != is)) {
            acc[0] = f2(sum_of_rows(sl, sbase, H, first, wL), 0.f);
            acc[1] = 0;
          }
        }
        tc_fence_before();
        mbar_arrive(&bars->dempty[d]);
        const uint64_t s2 = add2(acc[0], acc[1]);
        total += f2lo(s2) + f2hi(s2);
      }
      if (x.t0 < x.t1) {  // half 1 hands its sums to half 0
        if (half) {
          if (!mbar_wait(&bars->hempty[d], (hn & 1) ^ 1, abort)) goto done;
          sX[d * 128 + tid] = total;
          mbar_arrive(&bars->hfull[d]);
        } else {
          if (!mbar_wait(&bars->hfull[d], hn & 1, abort)) goto done;
          total += sX[d * 128 + tid];
          mbar_arrive(&bars->hempty[d]);
        }
        ++hn;
      }
      if (p.parts > 1) {
        if (!half) sX[(2 + d) * 128 + tid] = total;  // joined below
      } else if (!half && key < a.Nk) {
        const int64_t wi = (int64_t(b) * a.Hkv + x.hk) * a.Nk + key;
        if (key < x.len)
          wa.w_out[wi] = wa.decay != 0.f ? fmaf(wa.decay, was, total) : total;
        else if (wa.w_in && wa.w_in != wa.w_out)
          wa.w_out[wi] = was;  // an entry past the sequence stays as it was
      }
    }
  } else if (warp < WCfg::kTmaWarp) {
    // ------------------------------------------------------------ MMA issue
    const int d = warp - WCfg::kMmaWarp;  // the key tile
    if (lane == 0) {
      const uint32_t base = idesc_bf16(128, p.NR, false, false);
      const uint32_t kIdesc = a.neg_scale ? idesc_negate_b(base) : base;
      const uint64_t dq = sw128_desc(smem_u32(sQ), 16, 1024), dk = sw128_desc(smem_u32(sK), 16, 1024);
      const uint32_t q_lo = static_cast<uint32_t>(dq), q_hi = static_cast<uint32_t>(dq >> 32);
      const uint32_t k_lo = static_cast<uint32_t>(dk), k_hi = static_cast<uint32_t>(dk >> 32);
      const uint32_t qstep = (p.NR * 128) >> 4;
      uint32_t it = 0, kn = d;  // Q tiles so far; this warp's key tile in the ring
      bool ok = true;
      for (uint32_t i = 0; ok; ++i) {
        if (!mbar_wait(&bars->ring_full[i & 1], (i >> 1) & 1, abort)) break;
        const WUnit x = bars->ring[i & 1];
        mbar_arrive(&bars->ring_empty[i & 1]);
        if (!x.go) break;
        if (x.t1 <= x.t0) continue;
        const uint32_t ks = kn % p.kst;
        if (!mbar_wait(&bars->kfull[ks], (kn / p.kst) & 1, abort)) break;
        const uint32_t kl = k_lo + ((ks * p.ktile) >> 4);
        for (int t = x.t0; t < x.t1; ++t, ++it) {
          const uint32_t qs = it % p.qst;
          // (the buffer last: even a wait for what is long done takes 100 cycles)
          if (!mbar_wait(&bars->qfull[qs], (it / p.qst) & 1, abort) ||
              (it + d > 0 && !mbar_wait(&bars->turn[d], (it + d - 1) & 1, abort)) ||
              !mbar_wait(&bars->dempty[d], (it & 1) ^ 1, abort)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t ql = q_lo + ((qs * p.kqbytes) >> 4);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t in = ((kk & 3) * 32) >> 4;
            mma_ss_w(tmem + d * WCfg::kCols, kl + (((kk >> 2) * 128 * 128) >> 4) + in, k_hi,
                     ql + (kk >> 2) * qstep + in, q_hi, kIdesc, kk > 0 ? 1u : 0u);
            if (kk == D / 16 - 2) mbar_arrive(&bars->turn[d ^ 1]);  // (an MMA covers the hand-over)
          }
          mma_commit(&bars->dfull[d]);
          mma_commit(&bars->qempty[qs]);
        }
        if (ok) mma_commit(&bars->kempty[ks]);
        kn += 2;
      }
      mma_commit(&bars->drain[d]);
      const long long c0 = clock64();
      while (!mbar_test(&bars->drain[d], 0) && clock64() - c0 < kWaitLimitCycles) {
      }
    }
  } else if (warp == WCfg::kTmaWarp && lane == 0) {
    // ------------------------------------------------------------ units and loads
    const uint32_t q_addr = smem_u32(sQ), k_addr = smem_u32(sK);
    uint32_t it = 0, un = 0;  // Q tiles and key tiles loaded
    bool ok = true;
    auto load_q = [&](const WUnit& x, int t) -> bool {
      const uint32_t qs = it % p.qst;
      if (!mbar_wait(&bars->qempty[qs], ((it / p.qst) & 1) ^ 1, abort)) return false;
      mbar_expect_tx(&bars->qfull[qs], p.rows * D * 2);
#pragma unroll
      for (int cb = 0; cb < D / 64; ++cb)
        tma_load_4d(q_addr + qs * p.kqbytes + cb * p.NR * 128, &tm_q, 64 * cb, x.hk * a.R, t * p.qn, x.b,
                    &bars->qfull[qs]);
      ++it;
      return true;
    };
    // The block's own unit, then (unless units are shared) units of blocks that
    // have not started.
    int64_t u = blockIdx.x / p.parts;
    uint32_t i = 0;
    for (; ok; ++i) {
      WUnit x = {};
      if (u >= 0) {
        if (p.parts == 1) {
          mbar_expect_tx(&bars->next, 16);
          request_block(&bars->answer, &bars->next);
        }
        x = unit_at(a, p, static_cast<int>(u), rank);
      }
      if (i >= 2 && !mbar_wait(&bars->ring_empty[i & 1], ((i >> 1) - 1) & 1, abort)) break;
      bars->ring[i & 1] = x;
      mbar_arrive(&bars->ring_full[i & 1]);
      if (u < 0) break;
      auto following = [&]() -> bool {
        if (p.parts > 1) {
          u = -1;
          return true;
        }
        if (!mbar_wait(&bars->next, i & 1, abort)) return false;
        u = answered_block(&bars->answer);
        fence_proxy_async_smem();  // read before the next answer is written
        return true;
      };
      if (x.t1 <= x.t0) {
        ok = following();
        continue;
      }
      // the first Q tile ahead of K, whose place may still be in use
      if (!(ok = load_q(x, x.tile(0)))) break;
      for (int d = 0; d < 2 && ok; ++d) {
        const uint32_t ks = un % p.kst;
        if (!(ok = mbar_wait(&bars->kempty[ks], ((un / p.kst) & 1) ^ 1, abort))) break;
        mbar_expect_tx(&bars->kfull[ks], p.ktile);
#pragma unroll
        for (int cb = 0; cb < D / 64; ++cb)
          tma_load_4d(k_addr + ks * p.ktile + cb * 128 * 128, &tm_k, 64 * cb, x.k0 + d * 128, x.hk, x.b,
                      &bars->kfull[ks]);
        ++un;
      }
      for (int s = 1; s < x.t1 - x.t0 && ok; ++s) ok = load_q(x, x.tile(s));
      if (ok) ok = following();
    }
    // After an abort: the copies in flight land before the block ends.
    if (*abort) {
      for (uint32_t f = it > uint32_t(p.qst) ? it - p.qst : 0; f < it; ++f) {
        const long long c0 = clock64();
        while (!mbar_test(&bars->qfull[f % p.qst], (f / p.qst) & 1) && clock64() - c0 < kWaitLimitCycles) {
        }
      }
      for (uint32_t f = un > uint32_t(p.kst) ? un - p.kst : 0; f < un; ++f) {
        const long long c0 = clock64();
        while (!mbar_test(&bars->kfull[f % p.kst], (f / p.kst) & 1) && clock64() - c0 < kWaitLimitCycles) {
        }
      }
      if (u >= 0 && p.parts == 1) {
        const long long c0 = clock64();
        while (!mbar_test(&bars->next, i & 1) && clock64() - c0 < kWaitLimitCycles) {
        }
      }
    }
  }
done:
  if (warp < WCfg::kEpiWarps && *abort) named_barrier_arrive(1 + (warp >> 2), 128);
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && bars->abort) report(a.status, SA_DEVERR_TIMEOUT);
  if (p.parts > 1) {
    // The blocks' sums, in the order of their ranks.
    const cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
    cluster.sync();
    const WUnit x = unit_at(a, p, blockIdx.x / p.parts, rank);
    const int key = x.k0 + threadIdx.x;
    if (rank == 0 && threadIdx.x < kUnitKeys && key < a.Nk) {
      float total = 0.f;
      for (int r = 0; r < p.parts; ++r) total += cluster.map_shared_rank(sX, r)[2 * 128 + threadIdx.x];
      const int64_t wi = (int64_t(x.b) * a.Hkv + x.hk) * a.Nk + key;
      if (key < x.len)
        wa.w_out[wi] = wa.decay != 0.f ? fmaf(wa.decay, wa.w_in[wi], total) : total;
      else if (wa.w_in && wa.w_in != wa.w_out)
        wa.w_out[wi] = wa.w_in[wi];
    }
    cluster.sync();  // no block leaves while its sums are read
  }
  if (warp == WCfg::kMmaWarp) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool CAP, bool BIAS>
static cudaError_t launch_w(const WeightArgs& a, const WPlan& p, const CUtensorMap& tq, const CUtensorMap& tk,
                            cudaStream_t st) {
  auto kern = sa_cache_weights_kernel<D, CAP, BIAS>;
  int smem = 1024 + p.kst * p.ktile + p.qst * p.kqbytes + 2 * 4 * 128 * 4 + 2 * 4 * 4 * 4 + 4 * 128 * 4 +
             static_cast<int>(sizeof(WBars)) + 64;
  if (smem < 120 * 1024) smem = 120 * 1024;  // one block per SM owns its TMEM
  static std::atomic<int> regs_ok{0};  // 0 unknown, 1 enough, 2 too few
  if (regs_ok.load() == 0) {
    cudaFuncAttributes attr;
    cudaError_t e = cudaFuncGetAttributes(&attr, kern);
    if (e != cudaSuccess) return e;
    // setmaxnreg.inc waits until the block's launch registers cover the split
    regs_ok.store(long(attr.numRegs) * WCfg::kThreads >= 512L * WCfg::kRegEpi + 128L * WCfg::kRegOther ? 1 : 2);
  }
  if (regs_ok.load() != 1) return cudaErrorLaunchOutOfResources;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(p.units * p.parts);
  c.blockDim = dim3(WCfg::kThreads);
  c.dynamicSmemBytes = smem;
  c.stream = st;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = p.parts;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  c.attrs = &attr;
  c.numAttrs = p.parts > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&c, kern, a, p, tq, tk);
}

cudaError_t launch_cache_weights(const WeightArgs& a, int num_sms, cudaStream_t st) {
  const MaskedArgs& m = a.m;
  WPlan p;
  p.qn = 256 / m.R < m.Nq ? 256 / m.R : m.Nq;
  p.rows = p.qn * m.R;
  p.NR = (p.rows + 31) / 32 * 32;
  p.qtiles = (m.Nq + p.qn - 1) / p.qn;
  p.ktile = 128 * m.d * 2;
  p.kqbytes = p.NR * m.d * 2;
  p.qst = p.NR <= 64 ? 4 : 2;
  const int room = 212 * 1024 - p.qst * p.kqbytes;  // the rest is under 15 KB
  p.kst = room / p.ktile < kMaxStages ? room / p.ktile : kMaxStages;
  p.kst &= ~1;  // whole units
  p.kunits = (m.Nk + kUnitKeys - 1) / kUnitKeys;
  p.units = m.B * m.Hkv * p.kunits;  // (the entry point checks that it fits)
  // Few keys and many rows: up to eight blocks share a unit's Q tiles (four SMs in
  // five can hold such a cluster, so the SMs are not filled to the last).
  p.parts = 1;
  while (p.parts < 8 && p.units * p.parts * 2 <= num_sms * 4 / 5 && p.parts * 2 <= p.qtiles) p.parts *= 2;
  CUtensorMap tq, tk;
  if (!make_view_map(&tq, m.q, m.d, m.Nq, m.Hq, m.B, m.qs.n, m.qs.h, m.qs.b, p.qn, m.R, true) ||
      !make_view_map(&tk, m.k, m.d, m.Nk, m.Hkv, m.B, m.ks.n, m.ks.h, m.ks.b, 128, 1, false))
    return cudaErrorInvalidValue;
  const bool cap = m.cap_log2 > 0.f, bias = m.slopes != nullptr;
  if (m.d == 128) {
    if (cap) return bias ? launch_w<128, true, true>(a, p, tq, tk, st) : launch_w<128, true, false>(a, p, tq, tk, st);
    return bias ? launch_w<128, false, true>(a, p, tq, tk, st) : launch_w<128, false, false>(a, p, tq, tk, st);
  }
  if (cap) return bias ? launch_w<64, true, true>(a, p, tq, tk, st) : launch_w<64, true, false>(a, p, tq, tk, st);
  return bias ? launch_w<64, false, true>(a, p, tq, tk, st) : launch_w<64, false, false>(a, p, tq, tk, st);
}

// ---------------------------------------------------------------- eviction

namespace {

constexpr int kSelThreads = 1024;
constexpr int kBins = 2048;
constexpr int kCached = 48 * 1024;  // weights of a row kept in shared memory

// Order of weights: larger first, -0 equal to +0, a NaN below everything.
__device__ __forceinline__ uint32_t weight_key(float w) { return w != w ? 0u : order_key(w + 0.f); }

}  // namespace

// C blocks (a cluster) per row, each with a run of the row's entries in its shared
// memory.  They add up their histograms through distributed shared memory, so that all
// of them find the same digit.  Bound by latency: three passes, each a histogram, a scan
// and two cluster barriers (12 rows of 35200 entries: 14 us).
template <int C>
__global__ void __cluster_dims__(C, 1, 1) __launch_bounds__(kSelThreads) sa_evict_select_kernel(const EvictArgs a) {
  let_next_kernel_start();  // (the gather's rows that need no choice move meanwhile)
  extern __shared__ uint32_t s_keys[];
  __shared__ __align__(8) uint32_t hist[kBins];
  __shared__ uint32_t wsum[32], weq[32], s_total[2];
  __shared__ uint32_t s_digit, s_left;
  namespace cg = cooperative_groups;
  const cg::cluster_group cluster = cg::this_cluster();
  auto sync_all = [&]() {
    if (C == 1)
      __syncthreads();
    else
      cluster.sync();
  };
  const int rank = C == 1 ? 0 : static_cast<int>(cluster.block_rank());
  const int64_t row = blockIdx.x / C;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int first = rank * kSelThreads + tid;  // among the row's threads
  int32_t* kept = a.kept + row * a.budget;
  const int n = a.len ? min(max(__ldg(a.len + row / a.Hkv), 0), a.Nk) : a.Nk;
  // (n and what depends on it is the same in every block of the cluster)
  if (n <= a.budget) {
    for (int i = first; i < a.budget; i += C * kSelThreads) kept[i] = i < n ? i : -1;
    return;
  }
  const int middle = n - a.recent - a.sink;
  const uint32_t want = a.budget - a.sink - a.recent;  // of the ones in between: 0 <= want < middle
  for (int i = first; i < a.sink; i += C * kSelThreads) kept[i] = i;
  for (int i = first; i < a.recent; i += C * kSelThreads) kept[a.budget - a.recent + i] = n - a.recent + i;
  if (want == 0) return;
  // This block's run of them.
  const int per = ((middle + C - 1) / C + 31) / 32 * 32;
  const int lo = a.sink + min(rank * per, middle), M = min((rank + 1) * per, middle) - min(rank * per, middle);
  const float* w = a.w + row * a.Nk + lo;
  const bool cached = M <= kCached;
  auto key_at = [&](int i) -> uint32_t { return cached ? s_keys[i] : weight_key(__ldg(w + i)); };
  if (cached)
    for (int i = tid; i < M; i += kSelThreads) s_keys[i] = weight_key(__ldg(w + i));

  // Radix selection from the top: 11, 11 and 10 bits.
  uint32_t prefix = 0, mask = 0, left = want;
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t dmask = pass == 2 ? 1023u : 2047u;
    for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0;
    __syncthreads();
    // (adding a warp's equal digits at once, by a match, took twice as long)
    for (int i = tid; i < M; i += kSelThreads) {
      const uint32_t k = key_at(i);
      if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & dmask], 1u);
    }
    sync_all();
    // suffix sums over the row: thread t holds bins 2047 - 2t and 2046 - 2t
    uint32_t h0 = 0, h1 = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const uint32_t* h = C == 1 ? hist : cluster.map_shared_rank(hist, c);
      const uint2 x = *reinterpret_cast<const uint2*>(h + kBins - 2 - 2 * tid);
      h0 += x.y;
      h1 += x.x;
    }
    uint32_t inc = h0 + h1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    if (warp == 0) {
      uint32_t v = wsum[lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += x;
      }
      wsum[lane] = v;
    }
    __syncthreads();
    const uint32_t above = inc - h0 - h1 + (warp ? wsum[warp - 1] : 0);
    if (above < left && left <= above + h0) {
      s_digit = kBins - 1 - 2 * tid;
      s_left = left - above;
    } else if (above + h0 < left && left <= above + h0 + h1) {
      s_digit = kBins - 2 - 2 * tid;
      s_left = left - above - h0;
    }
    sync_all();  // (and every block has read this one's histogram)
    prefix |= s_digit << shift;
    mask |= dmask << shift;
    left = s_left;
  }
  // Keep every key above the cut, and the first `left` of those at it.  Each
  // warp owns a run of the block's entries; the counts of the runs before it, in
  // this block and in the blocks before it, place its own.
  const uint32_t cut = prefix;
  const int run = ((M + 31) / 32 + 31) / 32 * 32;
  const int i0 = warp * run, i1 = min(i0 + run, M);
  uint32_t gt = 0, eq = 0;
  for (int i = i0 + lane; i < i1; i += 32) {
    const uint32_t k = key_at(i);
    gt += k > cut;
    eq += k == cut;
  }
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  if (lane == 0) {
    wsum[warp] = gt;
    weq[warp] = eq;
  }
  __syncthreads();
  uint32_t gb = 0, eb = 0;
  if (C > 1) {
    if (warp == 0) {
      const uint32_t g = __reduce_add_sync(0xffffffffu, wsum[lane]), e = __reduce_add_sync(0xffffffffu, weq[lane]);
      if (lane == 0) {
        s_total[0] = g;
        s_total[1] = e;
      }
    }
    cluster.sync();
    for (int c = 0; c < rank; ++c) {
      const uint32_t* t = cluster.map_shared_rank(s_total, c);
      gb += t[0];
      eb += t[1];
    }
  }
  for (int x = 0; x < warp; ++x) {
    gb += wsum[x];
    eb += weq[x];
  }
  const uint32_t below = (1u << lane) - 1;
  for (int base = i0; base < i1; base += 32) {
    const int i = base + lane;
    const uint32_t k = i < i1 ? key_at(i) : 0;
    const bool g = i < i1 && k > cut, e = i < i1 && k == cut;
    const uint32_t bg = __ballot_sync(0xffffffffu, g), be = __ballot_sync(0xffffffffu, e);
    const uint32_t ge = gb + __popc(bg & below), ee = eb + __popc(be & below);
    if (g || (e && ee < left)) kept[a.sink + ge + min(ee, left)] = lo + i;
    gb += __popc(bg);
    eb += __popc(be);
  }
  if (C > 1) cluster.sync();  // no block leaves while another may read its totals
}

// PIECES 16-byte pieces per row (d / 8); U slots per thread in flight.  Bound by
// HBM: 12 heads x 28160 rows of K and V, 173 MB each way, at 6.5 TB/s.
template <int PIECES>
__global__ void __launch_bounds__(256) sa_evict_gather_kernel(const EvictArgs a, int rows, int tiles) {
  constexpr int U = 4, kSlots = 256 / PIECES, kTile = kSlots * U;
  const int piece = threadIdx.x % PIECES;
  const uint32_t turn = blockIdx.x / uint32_t(rows);
  const int64_t row = blockIdx.x - turn * uint32_t(rows), b = row / a.Hkv, h = row % a.Hkv;
  const int32_t* kept = a.kept + row * a.budget;
  // Tiles of slots: first those that only hold the first entries or the newest, which
  // need not wait for the choice of the others.
  const int sinks = a.sink / kTile, last = (a.budget - a.recent + kTile - 1) / kTile, fixed = sinks + tiles - last;
  const int t = static_cast<int>(turn);
  const bool early = t < fixed;
  const int tile = t < sinks ? t : early ? last + t - sinks : sinks + t - fixed;
  const int j0 = tile * kTile + threadIdx.x / PIECES;
  int idx[U];
  if (early) {
    const int n = a.len ? min(max(__ldg(a.len + b), 0), a.Nk) : a.Nk;
    const int shift = tile < sinks || n <= a.budget ? 0 : n - a.budget;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int j = j0 + i * kSlots;
      idx[i] = j < min(a.budget, n) ? j + shift : -1;
    }
  } else {
    wait_for_earlier_kernel();
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int j = j0 + i * kSlots;
      idx[i] = j < a.budget ? kept[j] : -1;  // (a plain load: the selection may still run beside this kernel)
    }
  }
  if (a.k) {
    const uint16_t* k = a.k + b * a.ks.b + h * a.ks.h + piece * 8;
    const uint16_t* v = a.v + b * a.vs.b + h * a.vs.h + piece * 8;
    uint16_t* ko = a.k_out + b * a.kos.b + h * a.kos.h + piece * 8;
    uint16_t* vo = a.v_out + b * a.vos.b + h * a.vos.h + piece * 8;
    uint4 kr[U], vr[U];
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (idx[i] >= 0) {
        kr[i] = __ldg(reinterpret_cast<const uint4*>(k + idx[i] * a.ks.n));
        vr[i] = __ldg(reinterpret_cast<const uint4*>(v + idx[i] * a.vs.n));
      }
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (idx[i] >= 0) {
        const int64_t j = j0 + i * kSlots;
        *reinterpret_cast<uint4*>(ko + j * a.kos.n) = kr[i];
        *reinterpret_cast<uint4*>(vo + j * a.vos.n) = vr[i];
      }
  }
  if (a.w_out && piece == 0) {
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (idx[i] >= 0) a.w_out[row * a.budget + j0 + i * kSlots] = __ldg(a.w + row * a.Nk + idx[i]);
  }
  // (this kernel's end is to mean the other's, too; a block that waits holds its place)
  if (early && t == tiles - 1) wait_for_earlier_kernel();
}

cudaError_t launch_cache_evict(const EvictArgs& a, int num_sms, cudaStream_t st) {
  const int64_t rows = int64_t(a.B) * a.Hkv;
  // Blocks a row: one is enough for a short row; four, of which every SM holds one, as
  // long as they all run at once (clusters fill about four SMs in five); eight when a
  // fourth of a row is more than half of what a block keeps.  Selection alone, one /
  // two / four / eight: 12 rows of 35200 entries 22.5 / 17.6 / 14.3 / 17.9 us, 48 rows
  // (21120 to choose from) 16.3 / 14.8 / 26.1 / 63, 4 rows of 100000 116 / 33 / 21.9 / 20.7.
  const int64_t room = num_sms * 4 / 5;
  const int blocks = a.Nk <= 8192 || rows * 2 > room           ? 1
                     : rows * 4 > room                         ? 2
                     : rows * 8 > room || a.Nk <= 2 * kCached ? 4
                                                               : 8;
  const int run = blocks == 1 ? a.Nk : (a.Nk + blocks - 1) / blocks + 32;
  const int smem = (run < kCached ? run : kCached) * 4;
  auto kern = blocks == 8   ? sa_evict_select_kernel<8>
              : blocks == 4 ? sa_evict_select_kernel<4>
              : blocks == 2 ? sa_evict_select_kernel<2>
                            : sa_evict_select_kernel<1>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kCached * 4);
  if (e != cudaSuccess) return e;
  kern<<<static_cast<unsigned>(rows * blocks), kSelThreads, smem, st>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if (!a.k && !a.w_out) return cudaSuccess;
  const int slots = 4 * (256 / (a.d / 8)), tiles = (a.budget + slots - 1) / slots;
  return launch_early(a.d == 128 ? sa_evict_gather_kernel<16> : sa_evict_gather_kernel<8>,
                      dim3(static_cast<unsigned>(rows * tiles)), 256, 0, st, a, static_cast<int>(rows), tiles);
}

}  // namespace sa
