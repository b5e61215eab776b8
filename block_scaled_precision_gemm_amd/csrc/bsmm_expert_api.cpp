// Host front end of the experts' bf16 and fp32 products: argument validation
// and the C entry points bsmm_expert_mm and bsmm_expert_wgrad of
// include/bsmm.h.  Everything here runs on the host before any HIP call.

#include <cstdint>

#include "bsmm.h"
#include "bsmm_check.h"
#include "bsmm_internal.h"

using namespace bsmm;

namespace {

bool float_dtype(bsmm_dtype d) { return d == BSMM_F32 || d == BSMM_BF16; }
uintptr_t dtype_bytes(bsmm_dtype d) { return d == BSMM_BF16 ? 2 : 4; }
constexpr int64_t kMaxExperts = 1024;
constexpr int64_t kRowTile = 128;

}  // namespace

extern "C" {

bsmm_status bsmm_expert_mm(const void* x, int64_t ldx, const void* w, int64_t w_se, int64_t w_sn,
                           int64_t w_sk, bsmm_dtype dtype, const int32_t* order,
                           const int32_t* offsets, int slots_per_row, const float* row_scale,
                           void* out, int64_t ldo, bsmm_dtype out_dtype, int64_t E, int64_t R,
                           int64_t S, int64_t N, int64_t K, void* workspace,
                           size_t workspace_bytes, void* stream) {
  CHECK(float_dtype(dtype) && float_dtype(out_dtype), BSMM_ERR_DTYPE,
        "operands and out must be fp32 or bf16 (got %d, %d)", (int)dtype, (int)out_dtype);
  CHECK(E >= 0 && R >= 0 && S >= 0 && N >= 0 && K >= 0, BSMM_ERR_SHAPE,
        "negative size E=%lld R=%lld S=%lld N=%lld K=%lld", (long long)E, (long long)R,
        (long long)S, (long long)N, (long long)K);
  CHECK(R < kMaxDim && S < kMaxDim && N < kMaxDim && K < kMaxDim, BSMM_ERR_UNSUPPORTED,
        "size beyond 2^31");
  CHECK(E <= kMaxExperts, BSMM_ERR_UNSUPPORTED, "E=%lld beyond %lld experts", (long long)E,
        (long long)kMaxExperts);
  CHECK(slots_per_row >= 1, BSMM_ERR_ARG, "slots_per_row=%d", slots_per_row);
  CHECK(S <= R * slots_per_row, BSMM_ERR_SHAPE, "S=%lld slots beyond R * slots_per_row = %lld",
        (long long)S, (long long)(R * slots_per_row));
  if (S == 0 || N == 0) return BSMM_OK;
  CHECK(E > 0, BSMM_ERR_SHAPE, "slots but no experts");
  CHECK(offsets != nullptr && out != nullptr, BSMM_ERR_NULL, "offsets or out is NULL");
  CHECK(aligned(order, 4) && aligned(offsets, 4) && aligned(row_scale, 4), BSMM_ERR_ALIGN,
        "order, offsets or row_scale not 4-byte aligned");
  CHECK(ldo >= N, BSMM_ERR_SHAPE, "ldo=%lld below N", (long long)ldo);
  CHECK(aligned(out, dtype_bytes(out_dtype)), BSMM_ERR_ALIGN, "out not aligned to its type");
  // the grid's tiles, at least 16 rows by 16 columns each
  CHECK((S / 16 + E + 1) * (N / 16 + 1) < kMaxDim, BSMM_ERR_UNSUPPORTED,
        "S * N beyond the largest grid");
  ExpertArgs a{};
  if (K > 0) {
    CHECK(x != nullptr && w != nullptr, BSMM_ERR_NULL, "x or w is NULL");
    CHECK(ldx >= K, BSMM_ERR_SHAPE, "ldx=%lld below K", (long long)ldx);
    CHECK(w_se >= 0, BSMM_ERR_LAYOUT, "negative expert stride");
    // along K, or across it; where both strides are 1 one of the sizes is
    const bool along = w_sk == 1 && (w_sn >= K || N == 1);
    CHECK(along || (w_sn == 1 && (w_sk >= N || K == 1)), BSMM_ERR_LAYOUT,
          "w strides n=%lld k=%lld: one must be 1 and the other at least the row",
          (long long)w_sn, (long long)w_sk);
    CHECK(aligned(x, dtype_bytes(dtype)) && aligned(w, dtype_bytes(dtype)), BSMM_ERR_ALIGN,
          "x or w not aligned to its type");
    a.w_across = along ? 0 : 1;
    a.ldw = along ? w_sn : w_sk;
  }
  a.x = x; a.ldx = ldx; a.dtype = dtype;
  a.w = w; a.w_se = w_se;
  a.order = order; a.offsets = offsets; a.row_scale = row_scale;
  a.x_div = slots_per_row;
  a.out = out; a.ldo = ldo; a.out_dtype = out_dtype;
  a.E = (int)E; a.R = (int)R; a.S = (int)S; a.N = (int)N; a.K = (int)K;
  (void)workspace;
  (void)workspace_bytes;
  if (launch_expert_mm(a, stream) != 0)
    return fail(BSMM_ERR_HIP, "kernel launch failed (expert product)");
  return BSMM_OK;
}

size_t bsmm_expert_wgrad_workspace_bytes(bsmm_dtype dtype, int checkpoint, int64_t Rx, int64_t K) {
  if (dtype != BSMM_BF16 || !checkpoint || Rx <= 0 || K <= 0 || Rx >= kMaxDim || K >= kMaxDim)
    return 0;
  return (size_t)Rx * (size_t)K * 2u;
}

bsmm_status bsmm_expert_wgrad(const void* dy, int64_t ldy, bsmm_dtype dtype, int dy_slots_per_row,
                              const void* x, int64_t ldx, int x_slots_per_row,
                              const uint8_t* x_scale, int64_t s_r, const int32_t* order,
                              const int32_t* offsets, void* dw, int64_t w_se, int64_t ldw,
                              bsmm_dtype out_dtype, int64_t E, int64_t Ry, int64_t Rx, int64_t S,
                              int64_t N, int64_t K, void* workspace, size_t workspace_bytes,
                              void* stream) {
  CHECK(float_dtype(dtype) && float_dtype(out_dtype), BSMM_ERR_DTYPE,
        "operands and dw must be fp32 or bf16 (got %d, %d)", (int)dtype, (int)out_dtype);
  CHECK(E >= 0 && Ry >= 0 && Rx >= 0 && S >= 0 && N >= 0 && K >= 0, BSMM_ERR_SHAPE,
        "negative size E=%lld Ry=%lld Rx=%lld S=%lld N=%lld K=%lld", (long long)E, (long long)Ry,
        (long long)Rx, (long long)S, (long long)N, (long long)K);
  CHECK(Ry < kMaxDim && Rx < kMaxDim && S < kMaxDim && N < kMaxDim && K < kMaxDim,
        BSMM_ERR_UNSUPPORTED, "size beyond 2^31");
  CHECK(E <= kMaxExperts, BSMM_ERR_UNSUPPORTED, "E=%lld beyond %lld experts", (long long)E,
        (long long)kMaxExperts);
  CHECK(dy_slots_per_row >= 1 && x_slots_per_row >= 1, BSMM_ERR_ARG, "slots per row %d and %d",
        dy_slots_per_row, x_slots_per_row);
  CHECK(S <= Ry * dy_slots_per_row && S <= Rx * x_slots_per_row, BSMM_ERR_SHAPE,
        "S=%lld slots beyond the rows of dy (%lld) or x (%lld)", (long long)S,
        (long long)(Ry * dy_slots_per_row), (long long)(Rx * x_slots_per_row));
  CHECK(x_scale == nullptr || K % 32 == 0, BSMM_ERR_UNSUPPORTED,
        "K=%lld of a checkpoint is not a multiple of 32", (long long)K);
  if (E == 0 || N == 0 || K == 0) return BSMM_OK;
  CHECK(offsets != nullptr && dw != nullptr, BSMM_ERR_NULL, "offsets or dw is NULL");
  CHECK(aligned(order, 4) && aligned(offsets, 4), BSMM_ERR_ALIGN,
        "order or offsets not 4-byte aligned");
  CHECK(ldw >= K, BSMM_ERR_SHAPE, "ldw=%lld below K", (long long)ldw);
  CHECK(w_se >= (E > 1 ? (N - 1) * ldw + K : 0), BSMM_ERR_LAYOUT,
        "expert stride %lld below a weight's extent", (long long)w_se);
  CHECK(aligned(dw, dtype_bytes(out_dtype)), BSMM_ERR_ALIGN, "dw not aligned to its type");
  CHECK(E * (N / kRowTile + 1) * (K / kRowTile + 1) < kMaxDim, BSMM_ERR_UNSUPPORTED,
        "E * N * K beyond the largest grid");
  if (S > 0) {
    CHECK(dy != nullptr && x != nullptr, BSMM_ERR_NULL, "dy or x is NULL");
    CHECK(ldy >= N && ldx >= K, BSMM_ERR_SHAPE, "row strides ldy=%lld ldx=%lld below the rows",
          (long long)ldy, (long long)ldx);
    CHECK(x_scale == nullptr || s_r >= K / 32, BSMM_ERR_SCALE_SHAPE,
          "scale row stride %lld below the %lld blocks of a row", (long long)s_r,
          (long long)(K / 32));
    CHECK(aligned(dy, dtype_bytes(dtype)) && (x_scale != nullptr || aligned(x, dtype_bytes(dtype))),
          BSMM_ERR_ALIGN, "dy or x not aligned to its type");
  }
  WgradArgs a{};
  a.dy = dy; a.ldy = ldy; a.dtype = dtype; a.y_div = dy_slots_per_row;
  a.x = x; a.ldx = ldx; a.x_div = x_slots_per_row;
  a.x_scale = x_scale; a.s_r = s_r;
  a.order = order; a.offsets = offsets;
  a.dw = dw; a.w_se = w_se; a.ldw = ldw; a.out_dtype = out_dtype;
  a.E = (int)E; a.Rx = (int)Rx; a.S = (int)S; a.N = (int)N; a.K = (int)K;
  const size_t need = bsmm_expert_wgrad_workspace_bytes(dtype, x_scale != nullptr, Rx, K);
  void* ws = need > 0 && S > 0 && workspace_bytes >= need && aligned(workspace, 16) &&
                     aligned(x, 8) && ldx % 8 == 0 ? workspace : nullptr;
  if (launch_expert_wgrad(a, ws, stream) != 0)
    return fail(BSMM_ERR_HIP, "kernel launch failed (expert weight gradient)");
  return BSMM_OK;
}

}  // extern "C"
