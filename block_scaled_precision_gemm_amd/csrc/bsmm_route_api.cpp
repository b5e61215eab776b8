// Host front end of the router: argument validation and the C entry points
// bsmm_route_topk and bsmm_route_topk_backward of include/bsmm.h.

#include <cstdint>

#include "bsmm.h"
#include "bsmm_check.h"
#include "bsmm_internal.h"

using namespace bsmm;

namespace {

constexpr int64_t kMaxT = (int64_t)1 << 23;

bsmm_status check_logits(const void* logits, int64_t ld, bsmm_dtype dtype, int64_t T, int64_t E,
                         int k, const char* name) {
  CHECK(dtype == BSMM_F32 || dtype == BSMM_BF16, BSMM_ERR_DTYPE,
        "%s must be fp32 or bf16 (got %d)", name, (int)dtype);
  CHECK(T >= 0 && E >= 0, BSMM_ERR_SHAPE, "negative size T=%lld E=%lld", (long long)T,
        (long long)E);
  CHECK(E >= 1 && E <= kRouteMaxE, BSMM_ERR_UNSUPPORTED, "E=%lld (1 to %d experts)",
        (long long)E, kRouteMaxE);
  CHECK(k >= 1 && k <= kRouteMaxK && k <= E, BSMM_ERR_ARG, "k=%d (1 to %d, at most E=%lld)", k,
        kRouteMaxK, (long long)E);
  CHECK(T <= kMaxT, BSMM_ERR_UNSUPPORTED, "T=%lld beyond 2^23 tokens", (long long)T);
  if (T == 0) return BSMM_OK;
  CHECK(logits != nullptr, BSMM_ERR_NULL, "%s is NULL", name);
  CHECK(ld >= E, BSMM_ERR_SHAPE, "row stride %lld of %s below E", (long long)ld, name);
  CHECK(aligned(logits, dtype == BSMM_BF16 ? 2 : 4), BSMM_ERR_ALIGN,
        "%s not aligned to its type", name);
  return BSMM_OK;
}

// One block up to 64 tokens; then at most one per compute unit, of 16 tokens
// while that is enough (4096 tokens: small workgroups on all of the chip), of
// multiples of 64 beyond.
int tokens_per_block(int64_t T) {
  if (T > 64 && T <= 16 * (int64_t)kRouteMaxBlocks) return 16;
  const int64_t per = 64 * (int64_t)kRouteMaxBlocks;
  return (int)(64 * (T > per ? (T + per - 1) / per : 1));
}
int block_count(int64_t T) {
  const int b = tokens_per_block(T);
  const int n = (int)((T + b - 1) / b);
  return n > 1 ? n : 1;
}
int hist_stride(int64_t E) { return (int)((E + 1 + 7) / 8 * 8); }
size_t hist_bytes(int blocks, int64_t E) {
  return ((size_t)blocks * (size_t)hist_stride(E) * 2u + 255) / 256 * 256;
}

}  // namespace

extern "C" {

size_t bsmm_route_workspace_bytes(int64_t T, int64_t E) {
  if (T <= 0 || T > kMaxT || E <= 0 || E > kRouteMaxE) return 0;
  const int blocks = block_count(T);
  return blocks > 1 ? hist_bytes(blocks, E) + (size_t)blocks * (size_t)E * 8u : 0;
}

bsmm_status bsmm_route_topk(const void* logits, int64_t ldl, bsmm_dtype dtype,
                            const uint8_t* mask, int k, int renorm, float alpha, int32_t* index,
                            float* weight, int32_t* counts, int32_t* offsets, int32_t* order,
                            int32_t* live, float* prob_sum, float* loss, int64_t T, int64_t E,
                            void* workspace, size_t workspace_bytes, void* stream) {
  bsmm_status st = check_logits(logits, ldl, dtype, T, E, k, "logits");
  if (st != BSMM_OK) return st;
  CHECK(counts != nullptr && offsets != nullptr, BSMM_ERR_NULL, "counts or offsets is NULL");
  CHECK(T == 0 || (index != nullptr && weight != nullptr && order != nullptr), BSMM_ERR_NULL,
        "index, weight or order is NULL");
  CHECK((live != nullptr) == (loss != nullptr) && (prob_sum != nullptr) == (loss != nullptr),
        BSMM_ERR_NULL, "live, prob_sum and loss go together");
  CHECK(aligned(index, 4) && aligned(weight, 4) && aligned(counts, 4) && aligned(offsets, 4) &&
            aligned(order, 4) && aligned(live, 4) && aligned(prob_sum, 4) && aligned(loss, 4),
        BSMM_ERR_ALIGN, "an output is not 4-byte aligned");
  const int blocks = block_count(T);
  const size_t need = bsmm_route_workspace_bytes(T, E);
  CHECK(need == 0 || (workspace != nullptr && workspace_bytes >= need), BSMM_ERR_ARG,
        "the workspace must hold %zu bytes (bsmm_route_workspace_bytes)", need);
  CHECK(need == 0 || aligned(workspace, 16), BSMM_ERR_ALIGN, "workspace not 16-byte aligned");
  RouteArgs a{};
  a.logits = logits; a.ldl = ldl; a.dtype = dtype;
  a.mask = mask;
  a.k = k; a.renorm = renorm != 0; a.alpha = alpha;
  a.index = index; a.weight = weight; a.counts = counts; a.offsets = offsets; a.order = order;
  a.live = live; a.prob_sum = prob_sum; a.loss = loss;
  a.T = (int)T; a.E = (int)E;
  a.block = tokens_per_block(T);
  a.hist = static_cast<uint16_t*>(workspace);
  a.hist_ld = hist_stride(E);
  a.prob = need ? reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) +
                                           hist_bytes(blocks, E))
                : nullptr;
  a.before = reinterpret_cast<int32_t*>(a.prob + (need ? (size_t)blocks * (size_t)E : 0));
  if (launch_route(a, blocks, stream) != 0)
    return fail(BSMM_ERR_HIP, "kernel launch failed (route)");
  return BSMM_OK;
}

bsmm_status bsmm_route_topk_backward(const void* logits, int64_t ldl, bsmm_dtype dtype,
                                     const uint8_t* mask, const int32_t* index,
                                     const float* weight, const int32_t* counts,
                                     const int32_t* live, int k, int renorm, float alpha,
                                     const float* dweight, const float* dloss, void* dlogits,
                                     int64_t ldd, int64_t T, int64_t E, void* stream) {
  bsmm_status st = check_logits(logits, ldl, dtype, T, E, k, "logits");
  if (st != BSMM_OK) return st;
  st = check_logits(dlogits, ldd, dtype, T, E, k, "dlogits");
  if (st != BSMM_OK || T == 0) return st;
  CHECK(index != nullptr, BSMM_ERR_NULL, "index is NULL");
  CHECK(dweight == nullptr || weight != nullptr, BSMM_ERR_NULL, "dweight without weight");
  CHECK(dloss == nullptr || (counts != nullptr && live != nullptr), BSMM_ERR_NULL,
        "dloss without counts or live");
  CHECK(aligned(index, 4) && aligned(weight, 4) && aligned(counts, 4) && aligned(live, 4) &&
            aligned(dweight, 4) && aligned(dloss, 4),
        BSMM_ERR_ALIGN, "an input is not 4-byte aligned");
  RouteBackArgs a{};
  a.logits = logits; a.ldl = ldl; a.dtype = dtype;
  a.mask = mask;
  a.index = index; a.weight = weight; a.counts = counts; a.live = live;
  a.k = k; a.renorm = renorm != 0; a.alpha = alpha;
  a.dweight = dweight; a.dloss = dloss;
  a.dlogits = dlogits; a.ldd = ldd;
  a.T = (int)T; a.E = (int)E;
  if (launch_route_backward(a, stream) != 0)
    return fail(BSMM_ERR_HIP, "kernel launch failed (route backward)");
  return BSMM_OK;
}

}  // extern "C"
