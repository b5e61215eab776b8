// Host front end of the 4-bit weight operations: argument validation and the
// C entry points bsmm_quant_w4, bsmm_w4_mm and bsmm_w4_expert_mm of
// include/bsmm.h.  Everything here runs on the host before any HIP call.

#include <cstdint>

#include "bsmm.h"
#include "bsmm_check.h"
#include "bsmm_internal.h"

using namespace bsmm;

namespace {

bool float_dtype(bsmm_dtype d) { return d == BSMM_F32 || d == BSMM_BF16; }
size_t dtype_bytes(bsmm_dtype d) { return d == BSMM_BF16 ? 2 : 4; }

bsmm_status check_group(int group, int64_t K) {
  CHECK(group == 32 || group == 64 || group == 128, BSMM_ERR_ARG,
        "group=%d (32, 64 or 128 elements)", group);
  CHECK(K % group == 0, BSMM_ERR_UNSUPPORTED, "K=%lld is not a multiple of the group of %d",
        (long long)K, group);
  return BSMM_OK;
}

// Checks of the operands both products share; sizes are non-negative and
// below 2^31.  `experts` weights at strides w_se, s_se, z_se.
bsmm_status check_operands(const W4Args& a) {
  const int64_t KG = a.K / a.group;
  CHECK(a.out != nullptr, BSMM_ERR_NULL, "out is NULL");
  CHECK(a.ldo >= a.N, BSMM_ERR_SHAPE, "ldo=%lld below N", (long long)a.ldo);
  CHECK(aligned(a.out, 4), BSMM_ERR_ALIGN, "out not 4-byte aligned");
  // the grid's workgroups, at least 16 rows by 16 columns each
  CHECK(((int64_t)a.S / 16 + a.E + 1) * ((int64_t)a.N / 16 + 1) < kMaxDim, BSMM_ERR_UNSUPPORTED,
        "rows * N beyond the largest grid");
  if (a.K == 0) return BSMM_OK;      // zeros are written, nothing is read
  CHECK(a.x != nullptr && a.w != nullptr && a.scale != nullptr, BSMM_ERR_NULL,
        "x, w or scale is NULL");
  CHECK(a.ldx >= a.K && a.ldw >= a.K / 2, BSMM_ERR_SHAPE,
        "row strides ldx=%lld ldw=%lld below the rows", (long long)a.ldx, (long long)a.ldw);
  CHECK(a.w_se >= 0, BSMM_ERR_LAYOUT, "negative expert stride");
  CHECK((a.s_n == 0 || a.s_n >= KG) && a.s_se >= 0, BSMM_ERR_SCALE_SHAPE,
        "scale strides: a row holds %lld groups (0 repeats one row)", (long long)KG);
  CHECK(a.zero == nullptr || ((a.z_n == 0 || a.z_n >= KG) && a.z_se >= 0), BSMM_ERR_SCALE_SHAPE,
        "zero strides: a row holds %lld groups (0 repeats one row)", (long long)KG);
  CHECK(aligned(a.x, 16) && a.ldx % 8 == 0, BSMM_ERR_ALIGN,
        "x not 16-byte aligned or ldx=%lld not a multiple of 8", (long long)a.ldx);
  CHECK(aligned(a.w, 16) && a.ldw % 16 == 0 && a.w_se % 16 == 0, BSMM_ERR_ALIGN,
        "w, its row stride or its expert stride not 16-byte aligned");
  CHECK(aligned(a.scale, a.s_bf16 ? 2 : 4), BSMM_ERR_ALIGN, "scale not aligned to its type");
  return BSMM_OK;
}

bsmm_status run(const W4Args& a, void* workspace, size_t workspace_bytes, void* stream) {
  const bsmm_status st = check_operands(a);
  if (st != BSMM_OK) return st;
  W4Plan plan = w4_plan(a);
  if (a.x_dtype == BSMM_F32 &&
      (workspace == nullptr || workspace_bytes < w4_plane_bytes(a) || !aligned(workspace, 16)))
    plan = W4Plan::Rows;
  if (launch_w4(a, plan, workspace, stream) != 0) return fail(BSMM_ERR_HIP, "kernel launch failed (w4)");
  return BSMM_OK;
}

}  // namespace

// The times of the three kernels in us, fitted to device times of calls of
// 24 to 4096 rows (weights 800 x 1472 to 5120 x 8192; the groups of 128 in
// bf16 unless said otherwise); the least is taken.
//
// Rows: 5 plus the operations of the padded rows at the rate its matrix
// instructions and folds reach (bf16 260 / 155 / 150 Tflop/s for groups of
// 128 / 64 / 32, fp32 85).
// Tiles: one K step after another (128 rows: 0.8 / 1.0 / 1.2 us, 256 rows:
// 0.95 / 1.02 / 1.55; fp32 walks three planes), in rounds of the tiles that
// the 256 CUs hold: one of 256 rows (a full round 15 % longer), two of 128
// (then 1.65 times as long as one).  Routed, the number of tiles is a guess
// and their codes come from HBM: 1.5 rounds, and one more for every 300 tiles
// beyond 256.
//
//   rows x N x K              Rows   Tile128   Tile256   (us)
//     130 x 5120 x 8192         55        93       123
//     260 x 5120 x 8192         99        99       125
//     520 x 5120 x 8192        151        95       123
//    1040 x 5120 x 8192        276       146       128
//    1040 x 2048 x 4096         72        51        66
//    2047 x 4096 x 4096        212        87        76
//    2047 x 5120 x 8192        486       232       258
//     260 x 2048 x 4096 fp32    72       147       206   (groups of 64)
//     800 x 5120 x 8192 fp32   608       432       403   (groups of 64)
//    1021 tokens x 8, 32 experts of 2048 x 4096:   477       233       274
//     256 tokens x 8, the same                     141       123
//     128 tokens x 8, the same                      86       118
//     512 tokens x 4, 16 experts of 2048 x 2048:    74        48        76
//     300 tokens x 4, the same                      52        45
//     200 tokens x 4, the same                      46        45
//
// Routed calls therefore never take 256 rows: an expert's last tile is half
// empty on average.
W4Plan bsmm::w4_plan(const W4Args& a) {
  const bool f32 = a.x_dtype == BSMM_F32;
  const size_t x = f32 ? w4_plane_bytes(a) : (size_t)a.R * (size_t)a.ldx * 2u;
  const int64_t act = a.E < a.S ? a.E : a.S;
  // at most 32 rows (an expert): a tile would be three quarters empty
  if (a.K == 0 || a.S <= 32 * act || x >= (size_t)0xFFFF0000u) return W4Plan::Rows;
  // blocks of bm rows: dense all of them, routed with half a block to spare
  // for each expert
  auto blocks = [&](int64_t bm) {
    return a.offsets ? ((int64_t)a.S + act * (bm / 2)) / bm + 1 : ((int64_t)a.S + bm - 1) / bm;
  };
  const int64_t tile_cols = ((int64_t)a.N + 127) / 128;
  const double steps = (double)((a.K + 63) / 64) * (f32 ? 3 : 1);
  const int g = a.group == 128 ? 0 : a.group == 64 ? 1 : 2;
  static const double kRate[3] = {260e6, 155e6, 150e6};      // flop per us
  static const double kStep128[3] = {0.8, 1.0, 1.2}, kStep256[3] = {0.95, 1.02, 1.55};

  const int64_t bm = f32 ? 16 : 32;
  const double rows = 5.0 + 2.0 * (double)(blocks(bm) * bm) * a.N * a.K / (f32 ? 85e6 : kRate[g]);
  const int64_t n128 = blocks(128) * tile_cols, rest = n128 % 512;
  const double rounds128 =
      a.offsets ? 1.5 + (n128 > 256 ? (double)(n128 - 256) / 300.0 : 0.0)
                : 1.65 * (double)(n128 / 512) + (rest == 0 ? 0.0 : rest <= 256 ? 1.0 : 1.55);
  const double t128 = 4.0 + rounds128 * steps * kStep128[g];
  if (a.offsets) return rows <= t128 ? W4Plan::Rows : W4Plan::Tile128;
  const double rounds256 = 1.15 * (double)((blocks(256) * tile_cols + 255) / 256);
  const double t256 = 4.0 + rounds256 * steps * kStep256[g];
  if (rows <= t128 && rows <= t256) return W4Plan::Rows;
  return t128 <= t256 ? W4Plan::Tile128 : W4Plan::Tile256;
}

extern "C" {

bsmm_status bsmm_quant_w4(const void* w, int64_t ldw, bsmm_dtype w_dtype, uint8_t* q,
                          int64_t ldq, void* scale, int64_t s_r, bsmm_dtype scale_dtype,
                          uint8_t* zero, int64_t z_r, void* values, int64_t ldv, int group,
                          int64_t R, int64_t K, void* stream) {
  CHECK(float_dtype(w_dtype) && float_dtype(scale_dtype), BSMM_ERR_DTYPE,
        "w and scale must be fp32 or bf16 (got %d, %d)", (int)w_dtype, (int)scale_dtype);
  CHECK(R >= 0 && K >= 0, BSMM_ERR_SHAPE, "negative size R=%lld K=%lld", (long long)R,
        (long long)K);
  CHECK(R < kMaxDim && K < kMaxDim, BSMM_ERR_UNSUPPORTED, "size beyond 2^31");
  bsmm_status st = check_group(group, K);
  if (st != BSMM_OK || R == 0 || K == 0) return st;
  const int64_t KG = K / group;
  CHECK(R * KG < ((int64_t)1 << 30), BSMM_ERR_UNSUPPORTED, "R * K / group = %lld beyond 2^30",
        (long long)(R * KG));
  CHECK(w != nullptr && q != nullptr && scale != nullptr, BSMM_ERR_NULL,
        "w, q or scale is NULL");
  CHECK(ldw >= K && ldq >= K / 2, BSMM_ERR_SHAPE, "row strides ldw=%lld ldq=%lld below the row",
        (long long)ldw, (long long)ldq);
  CHECK(values == nullptr || ldv >= K, BSMM_ERR_SHAPE, "ldv=%lld below K", (long long)ldv);
  CHECK(s_r >= (R > 1 ? KG : 0), BSMM_ERR_SCALE_SHAPE,
        "scale row stride %lld below the %lld groups of a row", (long long)s_r, (long long)KG);
  CHECK(zero == nullptr || z_r >= (R > 1 ? KG : 0), BSMM_ERR_SCALE_SHAPE,
        "zero row stride %lld below the %lld groups of a row", (long long)z_r, (long long)KG);
  CHECK(aligned(w, 16) && ldw % 8 == 0, BSMM_ERR_ALIGN,
        "w not 16-byte aligned or ldw=%lld not a multiple of 8", (long long)ldw);
  CHECK(aligned(q, 16) && ldq % 16 == 0, BSMM_ERR_ALIGN, "q or ldq not 16-byte aligned");
  CHECK(values == nullptr || (aligned(values, 16) && ldv % 8 == 0), BSMM_ERR_ALIGN,
        "values not 16-byte aligned or ldv=%lld not a multiple of 8", (long long)ldv);
  CHECK(aligned(scale, dtype_bytes(scale_dtype)), BSMM_ERR_ALIGN,
        "scale not aligned to its type");
  QuantW4Args a{w, ldw, w_dtype, q, ldq, scale, s_r, scale_dtype, zero, z_r, values, ldv, group,
                R, K};
  if (launch_quant_w4(a, stream) != 0) return fail(BSMM_ERR_HIP, "quantiser launch failed");
  return BSMM_OK;
}

size_t bsmm_w4_workspace_bytes(bsmm_dtype x_dtype, int64_t E, int64_t R, int64_t S, int64_t N,
                               int64_t K, int group) {
  if (E <= 0 || R <= 0 || S <= 0 || N <= 0 || K <= 0 || E > 1024 || R >= kMaxDim ||
      S >= kMaxDim || N >= kMaxDim || K >= kMaxDim || x_dtype != BSMM_F32)
    return 0;
  W4Args a{};
  a.x_dtype = x_dtype;
  a.group = group;
  a.E = (int)E; a.R = (int)R; a.S = (int)S; a.N = (int)N; a.K = (int)K;
  a.ldx = K;
  // a routed call that could pass for a dense one (one expert, R = S) may
  // take a tile where the other does not: enough for both
  static const int32_t routed = 0;
  a.offsets = &routed;
  bool tiled = w4_plan(a) != W4Plan::Rows;
  a.offsets = nullptr;
  if (E == 1 && R == S) tiled = tiled || w4_plan(a) != W4Plan::Rows;
  return tiled ? w4_plane_bytes(a) : 0;
}

const char* bsmm_w4_plan_name(bsmm_dtype x_dtype, int routed, int64_t E, int64_t R, int64_t S,
                              int64_t N, int64_t K, int group) {
  if (E <= 0 || R <= 0 || S <= 0 || N <= 0 || K <= 0 || E > 1024 || R >= kMaxDim ||
      S >= kMaxDim || N >= kMaxDim || K >= kMaxDim || !float_dtype(x_dtype) ||
      (group != 32 && group != 64 && group != 128) || K % group != 0)
    return nullptr;
  static const int32_t some = 0;
  W4Args a{};
  a.x_dtype = x_dtype;
  a.group = group;
  a.E = (int)E; a.R = (int)R; a.S = (int)S; a.N = (int)N; a.K = (int)K;
  a.ldx = K;
  a.offsets = routed ? &some : nullptr;
  switch (w4_plan(a)) {
    case W4Plan::Tile128: return "tile128";
    case W4Plan::Tile256: return "tile256";
    case W4Plan::Rows: break;
  }
  const int rows = w4_item_rows(a);
  return rows == 4 ? "rows4" : rows == 16 ? "rows16" : "rows32";
}

bsmm_status bsmm_w4_mm(const void* x, int64_t ldx, bsmm_dtype x_dtype, const uint8_t* w,
                       int64_t ldw, const void* scale, int64_t s_n, bsmm_dtype scale_dtype,
                       const uint8_t* zero, int64_t z_n, int group, void* out, int64_t ldo,
                       bsmm_dtype out_dtype, int64_t M, int64_t N, int64_t K, void* workspace,
                       size_t workspace_bytes, void* stream) {
  CHECK(float_dtype(x_dtype) && float_dtype(scale_dtype) && float_dtype(out_dtype),
        BSMM_ERR_DTYPE, "x, scale and out must be fp32 or bf16 (got %d, %d, %d)", (int)x_dtype,
        (int)scale_dtype, (int)out_dtype);
  CHECK(M >= 0 && N >= 0 && K >= 0, BSMM_ERR_SHAPE, "negative size M=%lld N=%lld K=%lld",
        (long long)M, (long long)N, (long long)K);
  CHECK(M < kMaxDim && N < kMaxDim && K < kMaxDim, BSMM_ERR_UNSUPPORTED, "size beyond 2^31");
  bsmm_status st = check_group(group, K);
  if (st != BSMM_OK || M == 0 || N == 0) return st;
  W4Args a{};
  a.x = x; a.ldx = ldx; a.x_dtype = x_dtype;
  a.w = w; a.ldw = ldw;
  a.scale = scale; a.s_n = s_n; a.s_bf16 = scale_dtype == BSMM_BF16;
  a.zero = zero; a.z_n = z_n;
  a.group = group;
  a.x_div = 1;
  a.out = out; a.ldo = ldo; a.out_dtype = out_dtype;
  a.E = 1; a.R = (int)M; a.S = (int)M; a.N = (int)N; a.K = (int)K;
  return run(a, workspace, workspace_bytes, stream);
}

bsmm_status bsmm_w4_expert_mm(const void* x, int64_t ldx, bsmm_dtype x_dtype, const uint8_t* w,
                              int64_t w_se, int64_t ldw, const void* scale, int64_t s_se,
                              int64_t s_n, bsmm_dtype scale_dtype, const uint8_t* zero,
                              int64_t z_se, int64_t z_n, int group, const int32_t* order,
                              const int32_t* offsets, int slots_per_row, const float* row_scale,
                              void* out, int64_t ldo, bsmm_dtype out_dtype, int64_t E, int64_t R,
                              int64_t S, int64_t N, int64_t K, void* workspace,
                              size_t workspace_bytes, void* stream) {
  CHECK(float_dtype(x_dtype) && float_dtype(scale_dtype) && float_dtype(out_dtype),
        BSMM_ERR_DTYPE, "x, scale and out must be fp32 or bf16 (got %d, %d, %d)", (int)x_dtype,
        (int)scale_dtype, (int)out_dtype);
  CHECK(E >= 0 && R >= 0 && S >= 0 && N >= 0 && K >= 0, BSMM_ERR_SHAPE,
        "negative size E=%lld R=%lld S=%lld N=%lld K=%lld", (long long)E, (long long)R,
        (long long)S, (long long)N, (long long)K);
  CHECK(R < kMaxDim && S < kMaxDim && N < kMaxDim && K < kMaxDim, BSMM_ERR_UNSUPPORTED,
        "size beyond 2^31");
  CHECK(E <= 1024, BSMM_ERR_UNSUPPORTED, "E=%lld beyond 1024 experts", (long long)E);
  CHECK(slots_per_row >= 1, BSMM_ERR_ARG, "slots_per_row=%d", slots_per_row);
  CHECK(S <= R * slots_per_row, BSMM_ERR_SHAPE, "S=%lld slots beyond R * slots_per_row = %lld",
        (long long)S, (long long)(R * slots_per_row));
  bsmm_status st = check_group(group, K);
  if (st != BSMM_OK || S == 0 || N == 0) return st;
  CHECK(E > 0, BSMM_ERR_SHAPE, "slots but no experts");
  CHECK(order != nullptr && offsets != nullptr, BSMM_ERR_NULL, "order or offsets is NULL");
  CHECK(aligned(order, 4) && aligned(offsets, 4) && aligned(row_scale, 4), BSMM_ERR_ALIGN,
        "order, offsets or row_scale not 4-byte aligned");
  W4Args a{};
  a.x = x; a.ldx = ldx; a.x_dtype = x_dtype;
  a.w = w; a.w_se = w_se; a.ldw = ldw;
  a.scale = scale; a.s_se = s_se; a.s_n = s_n; a.s_bf16 = scale_dtype == BSMM_BF16;
  a.zero = zero; a.z_se = z_se; a.z_n = z_n;
  a.group = group;
  a.order = order; a.offsets = offsets; a.row_scale = row_scale;
  a.x_div = slots_per_row;
  a.out = out; a.ldo = ldo; a.out_dtype = out_dtype;
  a.E = (int)E; a.R = (int)R; a.S = (int)S; a.N = (int)N; a.K = (int)K;
  return run(a, workspace, workspace_bytes, stream);
}

}  // extern "C"
