// sa_internal.h — launch interfaces between the C ABI (sa_api.cu) and the
// kernel translation units.  Not part of the public interface.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "sparse_attn.h"

namespace sa {

struct FwdArgs {
  const uint16_t* q;  // bf16 bits [B,H,Nq,d]
  const uint16_t* k;  // bf16 bits [B,H,Nk,d]
  const uint16_t* v;
  const int64_t* row_ptr;
  const int32_t* col_idx;
  int64_t nnz;
  void* o;            // [B,H,Nq,d]: bf16 bits, or fp32 when out_fp32
  float* lse;         // [B,H,Nq] or null
  int32_t* status;    // device status word or null
  int64_t units;      // B*H*G
  int64_t G;
  int32_t Nq, Nk, M;
  int32_t out_fp32;
  int32_t neg_scale;  // scale < 0: the QK MMA negates K, and scale_log2 = |scale| log2(e)
  float scale_log2;   // |scale| * log2(e)
  int32_t dense = 0;  // no lists: every unit keeps keys 0 .. Nk-1
  // unit counter of the launch (zero when it starts), or null: static schedule
  uint32_t* sched = nullptr;
  // sparse delta (launch_forward_delta): o = base + sign * sum_j exp(l_ij - lse_i) v_j
  const float* lse_ref = nullptr;  // [B,H,Nq] natural-log normaliser per query row
  const float* base = nullptr;     // [B,H,Nq,d] fp32 or null (zero)
  float sign = 1.f;
};

cudaError_t launch_forward(const FwdArgs& a, int d, int num_sms, cudaStream_t stream);
cudaError_t launch_forward_delta(const FwdArgs& a, int d, int num_sms, cudaStream_t stream);

// Index builder.  The workspace holds, in order (each 256-byte aligned):
//   qhi, qlo   bf16 [rows, d]   mean query split as hi + lo
//   scores     fp32 [rows, ld]  ld = Nk rounded up to a multiple of 4
//   cut        uint32 [rows]    order-preserving key of the selection cut
//   ties       int32 [rows]     keys equal to the cut that are kept
//   counts     int64 [rows]     kept keys per row
//   misc       int64 nnz, int32 status
//   fail       int32 count (own 256 bytes), int32 [rows] rows, int32 [rows] units:
//              rows the TOPK path without a score matrix leaves to the select
//              kernel, and the (head, 128-row chunk) units whose scores they need
// The TOPK path without a score matrix keeps its sample scores, brackets,
// keep-masks and candidates inside the scores region.
struct BuildLayout {
  size_t qhi, qlo, scores, cut, ties, counts, misc, fail, total;
  int64_t ld;
};
BuildLayout build_layout(int64_t rows, int32_t Nk, int32_t d);

struct BuildArgs {
  const uint16_t* q;
  const uint16_t* k;
  // dense-step lists: stat >= 0 ranks keys by ln max_i / ln sum_i of
  // exp(scale q_i.k_j - lse_i) over the group's rows instead of the mean-query
  // score, and THRESHOLD compares that statistic itself with the threshold
  const float* lse = nullptr;
  int32_t stat = -1;  // -1 mean query, 0 column max, 1 column sum
  int64_t* row_ptr;
  int32_t* col_idx;
  int64_t col_capacity;
  uint8_t* ws;
  BuildLayout L;
  int64_t rows, G;
  int32_t BH, Nq, Nk, d, M;
  float scale;
  int32_t mode;
  int64_t topk;
  double threshold, mass;
};

cudaError_t launch_build_index(const BuildArgs& a, int num_sms, cudaStream_t stream);

// Voxel reordering of [BH, N, d] bf16 rows (N = T*Hh*W < 2^31).
struct VoxArgs {
  const uint4* x;
  uint4* y;
  int64_t BH;
  uint32_t N, T, Hh, W, vt, vh, vw;
  int32_t pieces;   // 16-byte pieces per row: d / 8 (a divisor of 32)
  int32_t inverse;  // 0: raster -> voxel order, 1: back
};
cudaError_t launch_voxel_permute(const VoxArgs& a, int num_sms, cudaStream_t stream);

// Rolling KV window append of one chunk to caches of S slots.
struct KvArgs {
  uint4* ck;
  uint4* cv;
  const uint4* nk;
  const uint4* nv;
  int64_t BH, L16;  // heads; 16-byte pieces per chunk per head
  int32_t S;        // slots (>= 2)
  int32_t slot;     // slot to fill, or -1: roll (sink stays) and fill the last
};
cudaError_t launch_kv_window(const KvArgs& a, int num_sms, cudaStream_t stream);

// Bit-packed (words) or block (blocks) keep-masks to CSR lists.
struct FmtArgs {
  const uint32_t* words;   // [rows, W] or null
  const uint8_t* blocks;   // [rows, W] or null
  int64_t* row_ptr;
  int32_t* col_idx;
  int64_t rows, capacity;
  int32_t W, Nk, block_k;
};
cudaError_t launch_index_from_mask(const FmtArgs& a, int num_sms, cudaStream_t stream);

// Which keys a query row sees (sa_mask.cuh has the rule).
struct MaskDev {
  const int32_t* dq;   // [B, nd + 1] first query row of each document, or null
  const int32_t* dk;   // [B, nd + 1] first key of each document
  const int32_t* px;   // [B, nd] prefix keys, or null
  const int32_t* len;  // [B] keys of each batch entry, or null
  int32_t nd;          // documents (0: one, the whole rows)
  int32_t causal;      // 0: none, else tokens per frame
  int32_t Nq, Nk;
};

// SMs of a GB300.  Plans that decide the order of a sum go by this and not by the device's count, so that the same inputs
// give the same bits on any part.
constexpr int kSms = 152;

// Masked forward and cache weights.
struct MaskedArgs {
  const uint16_t* q;   // bf16 views, element strides, d contiguous
  const uint16_t* k;
  const uint16_t* v;
  void* o;
  sa_strides qs, ks, vs, os;
  float* lse;          // [B, Hq, Nq] or null
  const float* slopes; // [Hq] or null
  int32_t* status;
  MaskDev mask;
  int32_t B, Hq, Hkv, R, Nq, Nk, d;
  int32_t out_fp32, neg_scale;
  float scale_log2;    // |scale| log2(e)
  float cap_log2;      // cap log2(e), 0: no cap
  float cap_k1;        // 2 |scale| log2(e) / cap
  // tanh's polynomial on raw products: x (scale_log2 + w (p1 + w (p2 + w p3))), w = x^2 <= cap_limit
  float cap_p1, cap_p2, cap_p3, cap_limit;
  int64_t total_rows;  // B * Hq * Nq
  // masked_plan: a Q tile holds qn queries of R heads each, a unit one or two tiles, a key
  // head row_blocks units, `group` heads are worked on at a time; the first full_units run
  // whole, the other split_units in `splits` runs of keys.  A run's partial result has
  // unit_rows rows (128 a tile; quads: four times the
  // rows of the tile).  slots > 0: the runs are shared out on the device instead, so that
  // all are about as long (quads with at most a unit an SM; slots: partial results)
  int32_t qn, tiles, quads, unit_rows, row_blocks, group, splits, slots;
  int64_t full_units, split_units;
  float* part_o;       // [partial results, unit_rows, d]
  float* part_lse;     // [partial results, unit_rows]
  int32_t* part_first; // slots: first partial result of each batch entry's first head [B],
                       // then how many each head has [B]
};
void masked_plan(MaskedArgs* a);
// Unit number -> key head of the batch and row block.
struct MaskedPlace {
  int bh, rb;
};
__host__ __device__ __forceinline__ MaskedPlace masked_place(const MaskedArgs& a, int u) {
  const int per = a.group * a.row_blocks, grp = u / per, r = u - grp * per;
  const int heads = a.B * a.Hkv - grp * a.group < a.group ? a.B * a.Hkv - grp * a.group : a.group;
  const int k = r / heads;
  return {grp * a.group + (r - k * heads), a.row_blocks - 1 - k};
}
// Joins the partial results of the split units (not those of quads).
cudaError_t launch_masked_join(const MaskedArgs& a, cudaStream_t stream);
cudaError_t launch_masked(const MaskedArgs& a, cudaStream_t stream);

struct WeightArgs {
  MaskedArgs m;        // q, k, mask, scale, cap, slopes
  const float* lse;    // [B, Hq, Nq]
  const float* w_in;   // [B, Hkv, Nk], or null (decay 0)
  float* w_out;        // may be w_in
  float decay;
};
cudaError_t launch_cache_weights(const WeightArgs& a, int num_sms, cudaStream_t stream);

struct EvictArgs {
  const float* w;      // [B, Hkv, Nk]
  const uint16_t* k;
  const uint16_t* v;
  uint16_t* k_out;
  uint16_t* v_out;
  float* w_out;        // [B, Hkv, budget] or null
  int32_t* kept;       // [B, Hkv, budget]
  const int32_t* len;  // [B] or null
  sa_strides ks, vs, kos, vos;
  int32_t B, Hkv, Nk, d, budget, sink, recent;
};
cudaError_t launch_cache_evict(const EvictArgs& a, int num_sms, cudaStream_t stream);

struct RopeArgs {
  const void* x[2];
  void* y[2];
  sa_strides xs[2], ys[2];
  int32_t H[2];
  int32_t B, N, d, half, fp32, inverse;
  int32_t rot;             // rotated elements (the first of a row)
  int32_t axes, first[4];  // pairs first[a] .. first[a + 1] - 1 turn with axis a
  const int32_t* pos;      // [N, axes] positions (batch stride pos_b), or null: grid
  int64_t pos_b;
  int32_t offset[3];
  VoxArgs vox;             // grid and voxel shape (only these fields)
  int32_t voxel_order;
  uint64_t turn[64];       // turns per position of each pair, in units of 2^-64
};
cudaError_t launch_rope(const RopeArgs& a, int num_sms, cudaStream_t stream);
// Everything of a rotation but its tensors: checks, and `args` filled but for x, y, xs, ys, H.
sa_status check_rope(const sa_rope* p, int32_t H0, int32_t H1, RopeArgs* args);
// The explicit positions lie in device memory (after device_info).
bool rope_positions(const sa_rope* p);

// New tokens into an e4m3 cache (x: bf16 keys and values), or its tokens out (y).
struct Cache8Args {
  const void* x[2];      // keys, values: [B, H, n, d]
  void* y[2];            // the reading call's outputs (either may be null)
  sa_strides xs[2];      // of x or y
  uint8_t* codes[2];     // [B, H, N, d]
  sa_strides cs[2];
  float* scales[2];      // [B, H, ceil(N / block)]
  sa_strides ss[2];      // (n unused: blocks follow one another)
  const int32_t* start;  // [B] first token, or null: start0
  const int32_t* counts; // [B] tokens of each entry (at most n), or null
  int64_t start0;
  int32_t B, H, N, d, block, n;
  int32_t blocks;        // set by the launch: blocks of a head that n tokens can touch
  int64_t items;         // set by the launch
};
cudaError_t launch_cache8_append(Cache8Args a, cudaStream_t stream);
cudaError_t launch_cache8_read(Cache8Args a, bool wide, cudaStream_t stream);

// Attention over an e4m3 cache.  m: q, o, lse, mask, sizes, partial results (ks, vs: the codes' strides).
constexpr int kMostEntries = 1024;  // batch entries that the few-row kernel shares out
struct Attend8Args {
  MaskedArgs m;
  const uint8_t* k8;
  const uint8_t* v8;
  const float* k_scale;      // [B, Hkv, ceil(Nk / block)]
  const float* v_scale;
  sa_strides k_scales, v_scales;
  int32_t block_log2;
  float scale_log2;          // scale log2(e), with its sign
};
// Up to 16 rows a key head, and batch entries that its table holds: the few-row kernel.  (Its work goes with the rows, the
// other's with tiles of 128 of them: 24 key heads of 28160 keys, d = 128: 39 us for 4 rows, 42 for 8, 61 for 16, 119 for
// 32; the other 76 for 17 to 64.  1024 entries of 2 key heads of 1000 tokens 157 us, 1025 of them in the other form 272.)
inline bool attend8_few(const Attend8Args& a) { return int64_t(a.m.R) * a.m.Nq <= 16 && a.m.B <= kMostEntries; }
// Short heads are not cut: every block takes whole ones (12 heads of 880 keys: a second kernel and its workspace less).
inline bool attend8_whole(const Attend8Args& a) { return a.m.Nk <= 8 * 128; }
int attend8_few_grid(const Attend8Args& a);
cudaError_t launch_attend8_few(const Attend8Args& a, cudaStream_t stream);
void attend8_many_plan(Attend8Args* a);
cudaError_t launch_attend8_many(const Attend8Args& a, cudaStream_t stream);

// sparse_attn_layer_from_host splits a layer into at most this many chunks.
constexpr int kMaxPipelineChunks = 64;

// ------------------------------------------------------------ host checks
// Shared by every entry point (sa_api.cu defines them).
struct Dims {
  int64_t G, rows;
};
// Shapes, scale, head dim, group size, output dtype and the 32-bit limits
// (rows of the per-row kernels, TMA row coordinates).
sa_status check_problem(const sa_problem* p, Dims* dims);
// The selection rule of a builder call; `stat` < 0 for mean-query scores,
// else the column statistic (its THRESHOLD range differs).
sa_status check_select(const sa_problem* p, const sa_select* sel, int32_t stat);
// Checks that the current device is an sm_103 GPU and gives its SM count;
// also resolves the driver's address-range query used by in_device_allocation.
sa_status device_info(int* num_sms);
// [p, p + bytes) lies inside one device allocation of the current context.
bool in_device_allocation(const void* p, uint64_t bytes);
inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Every argument rule of a builder call except those on the scratch pointer
// itself: `scratch_bytes` below the problem's workspace size returns
// `scratch_short`.  Fills `a` (a->ws left null) and the SM count.
sa_status prepare_build(const sa_problem* p, const sa_select* sel, int32_t stat, const void* q,
                        const void* k, const float* lse, int64_t* row_ptr, int32_t* col_idx,
                        int64_t col_capacity, int64_t* nnz_out_host, size_t scratch_bytes,
                        sa_status scratch_short, BuildArgs* a, int* num_sms);
// Launches the builder on a.ws; with nnz_out_host, synchronises the stream
// and reports nnz and the device status.
sa_status run_build(const BuildArgs& a, int num_sms, int64_t* nnz_out_host, cudaStream_t s);

// Device address of a __device__ variable (`symbol`, its host-side name) in
// the current context, looked up once per (device, context) and cached under
// `id` (0: the builder's fixed scratch, 1: the forward's unit counters).
sa_status symbol_address(const void* symbol, int id, void** addr);

// A named NVTX range around a host call (shows the entry point's launches
// in a profiler's timeline; costs nothing measurable without one).
struct NvtxRange {
  explicit NvtxRange(const char* name);
  ~NvtxRange();
  NvtxRange(const NvtxRange&) = delete;
  NvtxRange& operator=(const NvtxRange&) = delete;
};

// Launches a kernel that may start while the one ahead of it on the stream still
// runs, from that one's end on or from its let_next_kernel_start(); it calls
// wait_for_earlier_kernel() before it touches what that one writes, and at least one
// block calls it in any case, so that its end means the other's end.
template <class... P, class... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t stream,
                         const A&... args) {
  cudaLaunchConfig_t c = {};
  c.gridDim = grid;
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = smem;
  c.stream = stream;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &attr;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, args...);
}

cudaError_t launch_validate(const int64_t* row_ptr, const int32_t* col_idx, int64_t rows,
                            int64_t nnz, int32_t Nk, int32_t* status, cudaStream_t stream);

}  // namespace sa
