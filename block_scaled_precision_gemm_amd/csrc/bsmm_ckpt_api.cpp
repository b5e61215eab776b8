// Host front end of the 8-bit checkpoints and the gate: argument validation
// and the C entry points bsmm_quant_int8_mx, bsmm_swiglu and
// bsmm_swiglu_backward of include/bsmm.h.  Everything here runs on the host
// before any HIP call.

#include <cstdint>

#include "bsmm.h"
#include "bsmm_check.h"
#include "bsmm_internal.h"

using namespace bsmm;

namespace {

bool float_dtype(bsmm_dtype d) { return d == BSMM_F32 || d == BSMM_BF16; }

bsmm_status check_sizes(bsmm_dtype dtype, int64_t R, int64_t K, const char* name) {
  CHECK(float_dtype(dtype), BSMM_ERR_DTYPE, "tensors must be fp32 or bf16 (got %d)", (int)dtype);
  CHECK(R >= 0 && K >= 0, BSMM_ERR_SHAPE, "negative size R=%lld %s=%lld", (long long)R, name,
        (long long)K);
  CHECK(R < kMaxDim && K < kMaxDim / 2, BSMM_ERR_UNSUPPORTED, "size beyond 2^31");
  CHECK(K % 32 == 0, BSMM_ERR_UNSUPPORTED, "%s=%lld is not a multiple of 32", name, (long long)K);
  CHECK(R * (K / 32) < ((int64_t)1 << 29), BSMM_ERR_UNSUPPORTED, "R * %s / 32 beyond 2^29", name);
  return BSMM_OK;
}

// A float tensor of rows of `cols`, and a checkpoint's codes and bytes.
bsmm_status check_rows(const void* p, int64_t ld, int64_t cols, const char* name) {
  CHECK(p != nullptr, BSMM_ERR_NULL, "%s is NULL", name);
  CHECK(ld >= cols, BSMM_ERR_SHAPE, "row stride %lld of %s below the row", (long long)ld, name);
  CHECK(aligned(p, 16) && ld % 8 == 0, BSMM_ERR_ALIGN,
        "%s not 16-byte aligned or its row stride %lld not a multiple of 8", name, (long long)ld);
  return BSMM_OK;
}
bsmm_status check_codes(const int8_t* q, int64_t ldq, const uint8_t* scale, int64_t s_r,
                        int64_t cols) {
  CHECK(q != nullptr && scale != nullptr, BSMM_ERR_NULL, "q or scale is NULL");
  CHECK(ldq >= cols, BSMM_ERR_SHAPE, "row stride ldq=%lld below the row", (long long)ldq);
  CHECK(aligned(q, 8) && ldq % 8 == 0, BSMM_ERR_ALIGN, "q or ldq=%lld not 8-byte aligned",
        (long long)ldq);
  CHECK(s_r >= cols / 32, BSMM_ERR_SCALE_SHAPE,
        "scale row stride %lld below the %lld blocks of a row", (long long)s_r,
        (long long)(cols / 32));
  return BSMM_OK;
}

#define TRY(call) \
  do { const bsmm_status st_ = (call); if (st_ != BSMM_OK) return st_; } while (0)

}  // namespace

extern "C" {

bsmm_status bsmm_quant_int8_mx(const void* x, int64_t ldx, bsmm_dtype x_dtype, int8_t* q,
                               int64_t ldq, uint8_t* scale, int64_t s_r, void* values,
                               int64_t ldv, int64_t R, int64_t K, void* stream) {
  TRY(check_sizes(x_dtype, R, K, "K"));
  if (R == 0 || K == 0) return BSMM_OK;
  TRY(check_rows(x, ldx, K, "x"));
  TRY(check_codes(q, ldq, scale, s_r, K));
  if (values != nullptr) TRY(check_rows(values, ldv, K, "values"));
  const QuantI8MxArgs a{x, ldx, x_dtype, q, ldq, scale, s_r, values, ldv, R, K};
  if (launch_quant_int8_mx(a, stream) != 0) return fail(BSMM_ERR_HIP, "quantiser launch failed");
  return BSMM_OK;
}

bsmm_status bsmm_swiglu(const void* h, int64_t ldh, bsmm_dtype dtype, void* a, int64_t lda,
                        int8_t* q, int64_t ldq, uint8_t* scale, int64_t s_r, int64_t R, int64_t F,
                        void* stream) {
  TRY(check_sizes(dtype, R, F, "F"));
  CHECK((q == nullptr) == (scale == nullptr), BSMM_ERR_NULL,
        "q and scale are given together or not at all");
  if (R == 0 || F == 0) return BSMM_OK;
  TRY(check_rows(h, ldh, 2 * F, "h"));
  TRY(check_rows(a, lda, F, "a"));
  if (q != nullptr) TRY(check_codes(q, ldq, scale, s_r, 2 * F));
  const SwigluArgs args{h, ldh, dtype, a, lda, q, ldq, scale, s_r, R, F};
  if (launch_swiglu(args, stream) != 0) return fail(BSMM_ERR_HIP, "kernel launch failed (gate)");
  return BSMM_OK;
}

bsmm_status bsmm_swiglu_backward(const void* da, int64_t ldda, bsmm_dtype dtype, const int8_t* q,
                                 int64_t ldq, const uint8_t* scale, int64_t s_r,
                                 const float* row_scale, void* dh, int64_t lddh, void* act,
                                 int64_t ldact, float* drow, int64_t R, int64_t F, void* stream) {
  TRY(check_sizes(dtype, R, F, "F"));
  CHECK(drow == nullptr || row_scale != nullptr, BSMM_ERR_ARG, "drow without row_scale");
  if (R == 0) return BSMM_OK;
  CHECK(aligned(row_scale, 4) && aligned(drow, 4), BSMM_ERR_ALIGN,
        "row_scale or drow not 4-byte aligned");
  if (F > 0) {
    TRY(check_rows(da, ldda, F, "da"));
    TRY(check_codes(q, ldq, scale, s_r, 2 * F));
    TRY(check_rows(dh, lddh, 2 * F, "dh"));
    if (act != nullptr) TRY(check_rows(act, ldact, F, "act"));
  }
  const SwigluBackArgs a{da, ldda, dtype, q, ldq, scale, s_r, row_scale, dh, lddh, act, ldact,
                         drow, R, F};
  if (launch_swiglu_backward(a, stream) != 0)
    return fail(BSMM_ERR_HIP, "kernel launch failed (gate gradient)");
  return BSMM_OK;
}

}  // extern "C"
