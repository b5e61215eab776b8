// Internal interface between the host front end (validation, dispatch) and
// the HIP kernels.  Plain C++; no HIP types, so the front end is host code.
#pragma once

#include <cstddef>
#include <cstdint>

#include "bsmm.h"

namespace bsmm {

constexpr int kBlockK = 128;   // K extent of one scale block and one k-step

// One GEMM problem after validation, in a single strided form that covers
// all three entry points.  Element (g, m, k) of A is at
// a + g*a_sg + m*lda + k; element (g, n, k) of B at b + g*b_sg + n*ldb + k.
// Output (g, m, n) at out + (g*o_sg + m*ldo + n) * sizeof(out element).
struct Problem {
  bsmm_op op;
  bsmm_dtype out_dtype;
  int G, M, N, K;
  const uint8_t* a; int64_t a_sg, lda;
  const uint8_t* b; int64_t b_sg, ldb;
  // scales, strides in elements (float for int8 / blockwise, byte for mx)
  //   int8:      sa[m*sa_m], sb[n*sb_n]                       (sb_kb unused)
  //   blockwise: sa[m*sa_m + kb*sa_kb], sb[kb*sb_kb + nb*sb_n]
  //   mx:        sa[g*sa_sg + m*sa_m + kb], sb[g*sb_sg + nb*sb_n + kb]
  //   mx32:      sa[m*sa_m + c], sb[n*sb_n + c] for 32-long K chunk c (bytes)
  //   scaled_mm: sa[m*sa_m], sb[n*sb_n] (fp32; stride 0 for one scalar)
  //   groupwise: sa[m*sa_m + kb*sa_kb], sb[kb*sb_kb + n*sb_n]
  const void* sa; int64_t sa_sg, sa_m, sa_kb;
  const void* sb; int64_t sb_sg, sb_n, sb_kb;
  void* out; int64_t o_sg, ldo;
  // fp8 scaled_mm epilogue: bias [N] (fp32, or bf16 when bias_bf16), result
  // scale (one fp32); null when absent
  const void* bias; int bias_bf16;
  const float* sr;
};

// Operations whose K loop can read its scales from the packed layouts of
// the pre-pass.
inline bool packable_scales(bsmm_op op) {
  return op == BSMM_OP_FP8_BLOCKWISE || op == BSMM_OP_FP8_MX_BMM || op == BSMM_OP_FP8_MX32_MM ||
         op == BSMM_OP_FP8_GROUPWISE;
}

struct Variant;

struct Plan {
  const Variant* v = nullptr;      // main launch
  int split = 1;                   // K slices of the main launch
  const Variant* tail = nullptr;   // second launch for rows [m_split, M)
  int m_split = 0;                 // 0: one launch covers all of M
  int tail_split = 1;              // K slices of the tail launch
  size_t workspace = 0;            // bytes used
  int source = 2;                  // bsmm_plan_info::source
};

// One kernel launch over rows [row_begin, row_end) of a problem.
struct Launch {
  int row_begin, row_end;
  int split;             // K slices (split-K partials in ws)
  void* ws;              // split-K partials / stream-K slots
  size_t ws_bytes;
  const void* psa;       // packed scale_a, already written (packed variants)
  void* stream;
  int sk_grid = 0;       // stream-K grid (0: the device's co-resident capacity)
};

// Kernel variants compiled into the library.
using LaunchFn = int (*)(const Problem& p, const Launch& l);
struct Variant {
  const char* name;
  int tile_m, tile_n;
  unsigned op_mask;     // bit i set: usable for bsmm_op i
  bool masked_tail;     // safe for rows past M (every variant is)
  bool persistent;      // stream-K: one workgroup per slot of the device
  bool packed_scales;   // fp8: repacks scale_a into the workspace first
  int wg_per_cu;        // workgroups one CU holds (LDS / registers)
  const char* unpacked; // the same kernel without packed scales (or null)
  int max_m;            // largest M the kernel takes in one launch (0: any)
  int kind;             // 0 tile, 1 wide-wave tile, 2 skinny, 3 / 4 narrow (32 / 64 columns)
  LaunchFn launch;
};

// Workspace of a narrow-kernel launch split into S K ranges: S partial
// 128 x tile_n tiles (4-byte elements) per output tile, then one 64-bit
// counter per output tile.  It also covers the split-K partials of the tile
// kernel the narrow launch falls back to (at most 128 rows).
inline size_t narrow_workspace(int G, int N, int tile_n, int split) {
  if (split <= 1) return 0;
  const size_t tiles = (size_t)G * (size_t)((N + tile_n - 1) / tile_n);
  return (size_t)split * tiles * 128u * (size_t)tile_n * 4u + tiles * 8u;
}

// Packed scale_a for the fp8 kernels: K block major, rows padded to a
// multiple of 256, and within every 64 rows the element of row
// 64q + 16i + f stored at position 64q + 4f + i, so that one 16-byte
// (fp32) or 4-byte (e8m0) load gives a lane the scales of its four rows
// f, f+16, f+32, f+48.  Layout [G][KB][Mp] (G = 1 for blockwise).
//
// mx32 (32-element K chunks, both operands): a_scale packed as above with
// the chunk c = K/32 index in place of the K block, [KC][Mp] bytes; then
// (at the next 256-byte boundary) b_scale with column 128g + 16j + f at
// position 128g + 8f + j, [KC][Np] bytes (Np = N rounded up to 256), so
// that one 8-byte load gives a lane the scales of its eight columns f,
// f+16, .., f+112 of a 128-column wave tile.
//
// groupwise (1 x 128 groups on both operands): scale_a packed as for
// blockwise, [KB][Mp] fp32; then (at the next 256-byte boundary) scale_b
// in plain column order, [KB][Np] fp32, columns past N repeating column
// N-1.  The K loop stages each K block's slices of both through LDS.
inline int packed_rows(int M) { return (M + 255) / 256 * 256; }
inline size_t packed_gw_a_bytes(int M, int K) {
  return ((size_t)(K / kBlockK) * (size_t)packed_rows(M) * 4u + 255) / 256 * 256;
}
inline size_t packed_mx32_a_bytes(int M, int K) {
  return ((size_t)(K / 32) * (size_t)packed_rows(M) + 255) / 256 * 256;
}
inline size_t packed_scale_bytes(bsmm_op op, int G, int M, int K, int N = 0) {
  if (!packable_scales(op)) return 0;
  if (op == BSMM_OP_FP8_MX32_MM)
    return packed_mx32_a_bytes(M, K) + ((size_t)(K / 32) * (size_t)packed_rows(N) + 255) / 256 * 256;
  if (op == BSMM_OP_FP8_GROUPWISE)
    return packed_gw_a_bytes(M, K) + packed_gw_a_bytes(N, K);
  const size_t elem = op == BSMM_OP_FP8_BLOCKWISE ? 4u : 1u;
  const size_t n = (size_t)(op == BSMM_OP_FP8_MX_BMM ? G : 1) * (size_t)(K / kBlockK) *
                   (size_t)packed_rows(M) * elem;
  return (n + 255) / 256 * 256;
}

// Workspace a persistent (stream-K) variant wants: two partial tiles and
// two 64-bit counters per workgroup, for a device of kPlanCUs compute units.
constexpr int kPlanCUs = 256;
size_t persistent_workspace(const Variant* v, bsmm_op op);

const Variant* variants(int* count);

// One kernel configuration for one (operation, output type); defined in the
// HIP translation units, one per (OP, OUT) pair, for every configuration in
// bsmm_variants.inc.  PK: the fp8 main loop reads packed scale_a, which the
// launch first writes to the start of the workspace.
template <int OP, int OUT, int WM, int WN, int RING, bool SK, bool PK, int KIND>
int launch_kernel(const Problem& p, const Launch& l);

// Write packed scale_a (layout above) for an fp8 problem to dst, which holds
// packed_scale_bytes(...) bytes and is 16-byte aligned.  Returns 0 on success.
int pack_scale_a(const Problem& p, void* dst, void* stream);
const Variant* find_variant(const char* name);

// Bytes of split-K workspace a variant needs for `split` slices.
size_t splitk_workspace(const Problem& p, int rows, int split);

// Benchmark timing of the main launch of each call (bsmm_timing.cpp).
bool timing_on();
void timing_mark(void* stream, const char* name, bool begin);

// Dynamic quantisation of bf16 / fp32 rows (bsmm_quant.hip).  Arguments are
// validated by the entry points before this is called.
//
// kFp8Columns: groups of 128 rows down each column of x [M, K]; codes only
// transposed, qt [K, M] (row stride ldqt); scale (g, c) at scale[g*s_m +
// c*s_kb] for g < M/128.  kFp8Weight: 128 x 128 blocks; codes in q [M, K]
// and / or qt [K, M] (either may be null); scale (g, cb) at scale[g*s_m +
// cb*s_kb].  kFp8RowsColumns: kFp8Columns plus the 1 x 128 row blocks of the
// same input, codes in q [M, K], scale (m, kb) at scale2[m*s2_m + kb*s2_kb].
struct QuantArgs {
  enum Kind { kInt8Rows = 0, kFp8Blocks = 1, kFp8Mx = 2, kFp8Mx32 = 3, kFp8Columns = 4,
              kFp8Weight = 5, kFp8RowsColumns = 6 };
  Kind kind;
  const void* x;        // [M, K] bf16 or fp32, row stride ldx elements
  int64_t ldx;
  bsmm_dtype x_dtype;   // BSMM_BF16 or BSMM_F32
  void* q;              // [M, K] 1-byte codes, row stride ldq
  int64_t ldq;
  void* scale;          // fp32 (kInt8Rows, kFp8Blocks) or e8m0 bytes (kFp8Mx)
  int64_t s_m, s_kb;    // scale strides in elements (s_kb unused for kInt8Rows)
  int64_t M, K;
  void* qt = nullptr;   // transposed codes [K, M] (kFp8Columns, kFp8Weight)
  int64_t ldqt = 0;
  void* scale2 = nullptr;   // row-block scales (kFp8RowsColumns)
  int64_t s2_m = 0, s2_kb = 0;
};
int launch_quant(const QuantArgs& a, void* stream);

// 4-bit group quantisation of w [R, K] (bsmm_quant.hip): codes q [R, K/2]
// (row stride ldq bytes), scale (r, g) at scale[r*s_r + g], zero (r, g) at
// zero[r*z_r + g] (null: symmetric), values [R, K] of w's type or null.
// Validated by the entry point; R * K / group in [1, 2^30).
struct QuantW4Args {
  const void* w; int64_t ldw; bsmm_dtype w_dtype;
  uint8_t* q; int64_t ldq;
  void* scale; int64_t s_r; bsmm_dtype scale_dtype;
  uint8_t* zero; int64_t z_r;
  void* values; int64_t ldv;
  int group;
  int64_t R, K;
};
int launch_quant_w4(const QuantW4Args& a, void* stream);

// A product with 4-bit weights (bsmm_w4.hip), dense (offsets null: E = 1, S
// rows of x and out) or routed: positions [offsets[e], offsets[e + 1]) of
// order[S] name the output rows ("slots") of expert e, slot s reads row s /
// x_div of x (R rows) and is multiplied by row_scale[s] (null: 1); slots at
// positions from offsets[E] on get zero rows.  K % group == 0 and all sizes
// are positive; validated by the entry points except for the contents of
// order and offsets, which the kernels clamp.
struct W4Args {
  const void* x; int64_t ldx; bsmm_dtype x_dtype;
  const uint8_t* w; int64_t w_se, ldw;
  const void* scale; int64_t s_se, s_n; int s_bf16;
  const uint8_t* zero; int64_t z_se, z_n;
  int group;
  const int32_t* order;
  const int32_t* offsets;
  const float* row_scale;
  int x_div;
  void* out; int64_t ldo; bsmm_dtype out_dtype;
  int E, R, S, N, K;
};
// The kernel for a call: 4, 16 or 32 rows a workgroup (any call), or tiles of
// 128 or 256 rows by 128 columns.  On tiles an fp32 x is cut into three bf16
// planes in the workspace (w4_plane_bytes), and x is addressed by 32-bit
// offsets.
enum class W4Plan { Rows, Tile128, Tile256 };
inline size_t w4_plane_bytes(const W4Args& a) {
  return a.x_dtype == BSMM_F32 ? (size_t)3 * (size_t)a.R * (size_t)a.K * 2u : 0;
}
W4Plan w4_plan(const W4Args& a);
// Rows of a workgroup of W4Plan::Rows, by the rows of the call, routed by an
// expert's average: rows above that take several workgroups, which read the
// codes again, so that 4 rows are for averages of at most 2 (2048 x 4096, 8 of
// 32 experts, fp32: 12 tokens 92 us with 4 rows, 80 with 16; 8 tokens, average
// 2, 67 and 80; bf16 48 and 45, 35 and 45).  Dense, 5 rows of 5120 x 8192 bf16
// take 19.5 us with 4 and 14.5 with 16, 24 rows 22.8 with 16 and 17.6 with 32.
// 8 rows were never better than 16 (8 x 5120 x 8192 bf16 14.7 and 14.9, 32
// tokens x 8 of 32 experts 68 and 55).
inline int w4_item_rows(const W4Args& a) {
  const int64_t rows = a.offsets ? ((int64_t)a.S + a.E - 1) / a.E : a.S;
  return rows <= (a.offsets ? 2 : 4) ? 4 : rows <= 16 || a.x_dtype == BSMM_F32 ? 16 : 32;
}
// ws: w4_plane_bytes bytes for an fp32 x on tiles, else not used
int launch_w4(const W4Args& a, W4Plan plan, void* ws, void* stream);

// A product of routed rows with their experts' bf16 or fp32 weights
// (bsmm_expert.hip).  Slots, order, offsets and row_scale as in W4Args (order
// null: slot p at position p).  Element (n, k) of expert e's weight is at e *
// w_se + n * ldw + k, or with w_across at e * w_se + k * ldw + n.
struct ExpertArgs {
  const void* x; int64_t ldx; bsmm_dtype dtype;      // of x and w
  const void* w; int64_t w_se, ldw; int w_across;
  const int32_t* order;
  const int32_t* offsets;
  const float* row_scale;
  int x_div;
  void* out; int64_t ldo; bsmm_dtype out_dtype;
  int E, R, S, N, K;
};
// Its kernels and the weight gradient's: items of 16 or 32 rows (aligned), tiles
// of up to `rows` x 256 (bf16; rows 128, 192 or 256), 128 x 128 (the gradient's)
// or 64 x 64.  splits > 1: ranges of the contraction, their sums in ws (splits
// * S * N fp32).
enum class ExpertPlan { Rows, Wide, Tiles128, Tiles64 };
// A launch counts its threads in 32 bits, and one of more runs as many as the
// low 32 bits say, without an error: its caller refuses it.
constexpr uint64_t kMaxThreads = (uint64_t)1 << 32;
// The threads of a plan's largest launch
uint64_t expert_mm_threads(const ExpertArgs& a, ExpertPlan plan, int rows, int splits);
int launch_expert_mm(const ExpertArgs& a, ExpertPlan plan, int rows, int splits, void* ws,
                     void* stream);

// The weights' gradient: dw[e] (row stride ldw) sums dy[s / y_div]^T x[s /
// x_div] over the slots of e.  A slot outside [0, S) makes its expert's sums
// undefined, but leads to no access outside the operands.  x_scale null: x of
// dy's type; else x is int8 codes with e8m0 bytes x_scale[row * s_r + k / 32].
struct WgradArgs {
  const void* dy; int64_t ldy; bsmm_dtype dtype; int y_div;
  const void* x; int64_t ldx; int x_div;
  const uint8_t* x_scale; int64_t s_r;
  const int32_t* order;
  const int32_t* offsets;
  void* dw; int64_t w_se, ldw; bsmm_dtype out_dtype;
  int E, Rx, S, N, K;
};
uint64_t expert_wgrad_threads(const WgradArgs& a, ExpertPlan plan, int splits);
// splits > 1: parts of every run, their sums in ws (splits * E * N * K fp32)
int launch_expert_wgrad(const WgradArgs& a, ExpertPlan plan, int splits, void* ws, void* stream);
// A checkpoint's values in bf16, rows of K (0 on success)
int launch_restore_bf16(const void* q, int64_t ldq, const uint8_t* scale, int64_t s_r, void* out,
                        int64_t R, int64_t K, void* stream);

// 8-bit checkpoints (bsmm_ckpt.hip): int8 codes q [R, K] and a byte per 32
// elements of a row, scale[r * s_r + k / 32]; code * 2^(byte - 133).
struct QuantI8MxArgs {
  const void* x; int64_t ldx; bsmm_dtype x_dtype;
  int8_t* q; int64_t ldq;
  uint8_t* scale; int64_t s_r;
  void* values; int64_t ldv;             // null, or what the codes stand for, x's type
  int64_t R, K;
};
int launch_quant_int8_mx(const QuantI8MxArgs& a, void* stream);

// a[r, f] = silu(h[r, f]) * h[r, F + f]; with q the codes of h's rows too.
struct SwigluArgs {
  const void* h; int64_t ldh; bsmm_dtype dtype;      // of h and a
  void* a; int64_t lda;
  int8_t* q; int64_t ldq;                // null: no checkpoint
  uint8_t* scale; int64_t s_r;
  int64_t R, F;
};
int launch_swiglu(const SwigluArgs& a, void* stream);

// Its gradient from the codes of h, for da of row_scale * a (null: 1): dh [R,
// 2F], act = row_scale * a (null: not wanted), drow = sum of da * a (null
// without row_scale).
struct SwigluBackArgs {
  const void* da; int64_t ldda; bsmm_dtype dtype;    // of da, dh and act
  const int8_t* q; int64_t ldq;
  const uint8_t* scale; int64_t s_r;
  const float* row_scale;
  void* dh; int64_t lddh;
  void* act; int64_t ldact;
  float* drow;
  int64_t R, F;
};
int launch_swiglu_backward(const SwigluBackArgs& a, void* stream);

// The expert router (bsmm_route.hip).  logits [T, E], row stride ldl; index,
// weight [T, k] and order [T * k] contiguous; counts [E], offsets [E + 1].
// loss, live and prob_sum are null together.  Tokens go to workgroups in
// blocks of `block` (16 or a multiple of 64, at most 65535); with more than
// one block, hist [blocks][hist_ld] holds each block's counts and, in column
// E, its live tokens (hist_ld a multiple of 8 above E), prob [blocks][E] its
// sums of probabilities, before [blocks][E] the slots of the blocks before it.
constexpr int kRouteMaxE = 1024, kRouteMaxK = 32, kRouteMaxBlocks = 256;
struct RouteArgs {
  const void* logits; int64_t ldl; bsmm_dtype dtype;
  const uint8_t* mask;
  int k, renorm;
  float alpha;
  int32_t* index; float* weight; int32_t* counts; int32_t* offsets; int32_t* order;
  int32_t* live; float* prob_sum; float* loss;
  int T, E, block;
  uint16_t* hist; int hist_ld;
  float* prob; int32_t* before;
};
int launch_route(const RouteArgs& a, int blocks, void* stream);

// Gradient of the logits; dweight and dloss may each be null.
struct RouteBackArgs {
  const void* logits; int64_t ldl; bsmm_dtype dtype;
  const uint8_t* mask;
  const int32_t* index; const float* weight; const int32_t* counts; const int32_t* live;
  int k, renorm;
  float alpha;
  const float* dweight; const float* dloss;
  void* dlogits; int64_t ldd;
  int T, E;
};
int launch_route_backward(const RouteBackArgs& a, void* stream);

// The static device scratch of the allocation-free entry point
// (bsmm_scratch.hip): its size, and the current device's copy's address
// (null, with *err the HIP error, on failure).
constexpr size_t kScratchBytes = (size_t)64 << 20;
void* scratch_device_ptr(int* err);

// Plan selection (host only).
Plan make_plan(bsmm_op op, int G, int M, int N, int K, bsmm_dtype dt,
               size_t workspace_bytes);
Plan make_plan_heuristic(bsmm_op op, int G, int M, int N, int K, bsmm_dtype dt);

}  // namespace bsmm
