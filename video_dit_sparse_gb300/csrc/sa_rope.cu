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
#include "sa_rope.cuh"

namespace sa {

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
  token_position(a, b, n, p);
  int e0, e1;
  const bool turns = lane_pieces<V, HALF>(a, c, &e0, &e1);
  float cs[V], sn[V];
  lane_angles<V, HALF>(a, p, e0, e1, turns, cs, sn);
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
        turn_pieces<V, HALF>(a, e0, e1, turns, cs, sn, f0, f1);
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
