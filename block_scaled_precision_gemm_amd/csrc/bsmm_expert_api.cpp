// Host front end of the experts' bf16 and fp32 products: argument validation
// and the C entry points bsmm_expert_mm and bsmm_expert_wgrad of
// include/bsmm.h.  Everything here runs on the host before any HIP call.

#include <cmath>
#include <cstdint>

#include "bsmm.h"
#include "bsmm_check.h"
#include "bsmm_internal.h"

using namespace bsmm;

namespace {

bool float_dtype(bsmm_dtype d) { return d == BSMM_F32 || d == BSMM_BF16; }
uintptr_t dtype_bytes(bsmm_dtype d) { return d == BSMM_BF16 ? 2 : 4; }
constexpr int64_t kMaxExperts = 1024;
// of slots, columns and the contraction: all are counted up to a tile and a few
// steps past the last one, in 32 bits
constexpr int64_t kMaxSize = kMaxDim - 1024;

// A kernel and the ranges of the contraction it is cut into.
struct Choice { ExpertPlan plan; int splits; double us; int rows; };

// The time of a plan in us: `tiles` workgroups (times splits) of `steps`
// contraction steps, `outs` elements of output.  A step of a workgroup takes
// step_us, or each_us for every workgroup on its CU if that is more; a tile
// `fixed` besides.  More ranges fill the chip, but write and read their fp32
// sums, at 4 TB/s and in another launch; they are taken where that is to save
// a seventh (300 tokens x 4 of 16 experts of 2048 x 2048 bf16: 43 us in one
// range, 60 in two; 4000 x 2 of 4 of 300 x 200, weight gradient: 62 us in one,
// 29 in eight).
Choice best_split(ExpertPlan plan, int64_t tiles, int64_t steps, double outs, double step_us,
                  double each_us, double fixed, size_t room) {
  Choice best{plan, 1, 1e30, 0};
  for (int s = 1; s <= 16 && (s == 1 || steps >= 4 * s); ++s) {
    if (s > 1 && (outs * 4 * s > (double)room || tiles * s > (int64_t)1 << 20)) break;
    const double t = (double)(tiles * s) / 256.0, whole = std::floor(t), rest = t - whole;
    const double on_cu = whole + (rest > 0.0 ? 1.0 : 0.0);
    const double step = each_us * on_cu > step_us ? each_us * on_cu : step_us;
    const double us = (double)((steps + s - 1) / s) * step + fixed * on_cu +
                      (s > 1 ? 8.0 + outs * 8 * s / 4e6 : 0.0);
    if (us * (s > 1 && best.splits == 1 ? 1.17 : 1.0) < best.us) best = Choice{plan, s, us, 0};
  }
  return best;
}

// The time of the wide tiles in us, in items of at most bm rows and `parts`
// ranges of `steps` steps.  The experts' loads are not known on the host: a
// third of them each with 0.6, 1 and 1.4 of the average.  A step of 64, 128,
// 192 or 256 rows takes 0.62, 0.95, 1.25 or 1.55 us, a tile 6 besides; CUs take
// tiles as they get free, so that all end within a fifth of a tile of each
// other.  The constants are fitted to the times of 33 shapes, in full grids with
// the experts' weights from HBM; a step and a tile by themselves take what the
// kernel's comment says.  (Of those shapes' best heights of item the model finds
// heights that cost 1.6 % more on average, and 18 % at most.)
double wide_us(const ExpertArgs& a, int64_t act, int bm, int64_t steps, int parts) {
  static const double kStep[4] = {0.62, 0.95, 1.25, 1.55};
  static const double kLoad[3] = {0.6, 1.0, 1.4};
  const double each = (double)act / 3 * parts * (double)(((int64_t)a.N + 255) / 256);
  double work = 0.0, longest = 0.0;
  for (double part : kLoad) {
    const int64_t load = (int64_t)((double)a.S / (double)act * (act > 1 ? part : 1.0)) + 1;
    auto add = [&](int64_t rows, int64_t n) {
      if (rows == 0 || n == 0) return;
      const double us = (double)steps * kStep[(rows + 63) / 64 - 1] + 6;
      work += (double)n * us * each;
      if (us > longest) longest = us;
    };
    add(bm, load / bm);
    add(load % bm, 1);
  }
  const double us = work / 256 + 0.2 * longest;
  return us > longest ? us : longest;
}

// Measured (us; the average is of rows to an expert):
//                                            Rows  Wide  Tiles64
//   1 token x 8 of 64, 2048 x 4096 bf16        33    32           (64 tiles of 256;
//     Wide in four ranges, with a workspace and a second launch, for 3 %)
//   64 x 2 of 8, 1024 x 2048 bf16              14    17           (32)
//   32 x 2 of 8, 4096 x 8192 bf16             117   122           (128)
//   16 x 4 of 16, 4096 x 4096 bf16            111   105           (256)
//   8 x 8 of 32, 2048 x 4096 bf16             105    87           (256)
//   64 x 8 of 32, the same                    134    92           (256)
//   2000 x 4 of 16, 1001 x 2051 bf16                  65    122  (unaligned)
//   64 x 4 of 16, 4096 x 1024 fp32             78            96   (average 16)
//   128 x 4 of 16, the same                   108            97   (32)
//   128 x 4 of 16, input gradient fp32        102           118   (32)
Choice mm_plan(const ExpertArgs& a, size_t room) {
  const bool bf16 = a.dtype == BSMM_BF16;
  const int unit = bf16 ? 8 : 4;
  const int64_t act = a.E < a.S ? a.E : a.S;
  const bool rows = aligned_rows(a.x, a.ldx, a.dtype) && aligned_rows(a.w, a.ldw, a.dtype) &&
                    a.w_se % unit == 0 && a.K % unit == 0 && (!a.w_across || a.N % unit == 0);
  // items of bm rows: an expert's last one is half empty on average
  auto items = [&](int64_t bm) {
    if (act == 1) return ((int64_t)a.S + bm - 1) / bm;
    const int64_t n = ((int64_t)a.S + act * (bm / 2)) / bm;
    return n > act ? n : act;
  };
  auto tiles = [&](int64_t bm, int64_t bn) { return items(bm) * (((int64_t)a.N + bn - 1) / bn); };
  const int64_t few = bf16 ? tiles(256, 256) < 256 ? 16 : 0 : a.w_across ? 32 : 24;
  if (rows && a.S <= few * act) return Choice{ExpertPlan::Rows, 1, 0, 0};
  const double outs = (double)a.S * a.N;
  const int64_t steps = ((int64_t)a.K + 63) / 64;
  // (of any alignment, but 4 columns at least where they are transposed)
  if (bf16 && (!a.w_across || a.N >= 4)) {
    // Items of at most 256, 192 or 128 rows: fewer weights are read again, or
    // the chip is fuller (1021 tokens x 8 of 32, 2048 x 4096: 194, 182, 198 us;
    // 1500 x 4 of 16, 2048 x 2048: 57, 75, 67; 512 x 4 of 16, the same: 46, 41,
    // 38).
    Choice best{ExpertPlan::Wide, 1, 1e30, 0};
    for (int bm = 256; bm >= 128; bm -= 64)
      for (int p = 1; p <= 16 && (p == 1 || steps >= 4 * p); ++p) {
        if (p > 1 && (outs * 4 * p > (double)room || tiles(bm, 256) * p > (int64_t)1 << 20)) break;
        double us = wide_us(a, act, bm, (steps + p - 1) / p, p);
        if (p > 1) us += 8.0 + outs * 8 * p / 4e6;
        // rather one range, and larger items
        const double worth = (p > 1 && best.splits == 1 ? 1.17 : 1.0) *
                             (bm < best.rows ? 1.03 : 1.0);
        if (us * worth < best.us) best = Choice{ExpertPlan::Wide, p, us, bm};
      }
    if (rows) return best;           // else through registers, a tenth slower
    const Choice small = best_split(ExpertPlan::Tiles64, tiles(64, 64), steps, outs, 0.7, 0.5, 1,
                                    room);
    return 1.1 * best.us < small.us ? best : small;
  }
  return best_split(ExpertPlan::Tiles64, tiles(64, 64), bf16 ? steps : 2 * steps, outs, 0.7,
                    bf16 ? 0.5 : 0.55, 1, room);
}

//                                              Wide  Tiles64  Tiles128   (us)
//   333 tokens x 2 of 6, 1001 x 515 fp32                  22        26
//   1000 x 4 of 16, 1024 x 2048 fp32                     196       193
//   4000 x 2 of 4, 300 x 200 bf16                         62       119
//   2121 x 8 of 17, 448 x 480 bf16               44       28        39
//   1832 x 8 of 8, 96 x 2037 bf16                60       51        85
//   484 x 2 of 21, 448 x 2880 bf16               23       32        36
//   1818 x 1 of 2, 1824 x 1568, checkpoint       42       41        34    (Wide: restored)
//   3692 x 2 of 2, 381 x 2592, checkpoint        65      107       100
Choice wgrad_plan(const WgradArgs& a, bool codes, size_t room) {
  const bool bf16 = a.dtype == BSMM_BF16;
  const int64_t act = a.E < a.S ? a.E : a.S > 0 ? a.S : 1;
  const int64_t run = ((int64_t)a.S + act - 1) / act;
  const double outs = (double)a.E * a.N * a.K;
  auto tiles = [&](int64_t t) {
    return a.E * (((int64_t)a.N + t - 1) / t) * (((int64_t)a.K + t - 1) / t);
  };
  const int64_t steps = (run + (bf16 ? 63 : 31)) / (bf16 ? 64 : 32);
  // pieces of rows that are not aligned are in one line more
  const bool odd = bf16 && (a.ldy % 4 != 0 || (!codes && a.ldx % 4 != 0));
  Choice c = best_split(ExpertPlan::Tiles64, tiles(64), steps, outs, odd ? 1.0 : 0.7,
                        !bf16 || odd ? 0.8 : 0.5, 1, room);
  const Choice d = best_split(ExpertPlan::Tiles128, tiles(128), steps, outs,
                              odd ? 2.6 : bf16 ? 2.0 : 2.2, !bf16 || odd ? 2.0 : 1.25,
                              bf16 ? 4 : 9, room);
  if (d.us < c.us) c = d;
  // loads of 4 columns
  if (bf16 && !codes && a.N >= 4 && a.K >= 4) {
    const Choice w = best_split(ExpertPlan::Wide, tiles(256), steps, outs, 1.7, 1.7,
                                a.out_dtype == BSMM_F32 ? 14 : 9, room);
    if (w.us < c.us) c = w;
  }
  return c;
}

// A checkpoint's values in bf16, before the parts.
size_t restored_bytes(bsmm_dtype dtype, int checkpoint, int64_t Rx, int64_t K) {
  return dtype == BSMM_BF16 && checkpoint ? ((size_t)Rx * (size_t)K * 2u + 15u) / 16u * 16u : 0;
}

constexpr size_t kEnough = (size_t)256 << 20;       // no plan's parts are larger

// The kernel of a call with `room` bytes of workspace.  First without a look at
// the room, so that the order of the sums does not follow from what a buffer
// happens to hold beyond the bytes that the query gives; with fewer than that
// plan needs, the best that they allow.
size_t parts_bytes(const ExpertArgs& a, const Choice& c) {
  return c.splits > 1 ? (size_t)c.splits * (size_t)a.S * (size_t)a.N * 4u : 0;
}
Choice mm_choice(const ExpertArgs& a, size_t room) {
  const Choice c = mm_plan(a, kEnough);
  return parts_bytes(a, c) <= room ? c : mm_plan(a, room);
}

// The same for the weight gradient, and whether it multiplies a checkpoint's
// values, restored to bf16 at the workspace's start (whole: the codes' rows
// allow it).
struct WgradChoice { Choice c; bool restored; };
size_t parts_bytes(const WgradArgs& a, const Choice& c) {
  return c.splits > 1 ? (size_t)c.splits * (size_t)a.E * (size_t)a.N * (size_t)a.K * 4u : 0;
}
WgradChoice wgrad_choice(const WgradArgs& a, bool whole, size_t room) {
  const bool codes = a.x_scale != nullptr;
  const size_t values = restored_bytes(a.dtype, codes, a.Rx, a.K);
  // `parts` bytes for sums, and room for the values or none
  auto best = [&](size_t parts, size_t parts_behind_values, bool fits) {
    WgradChoice w{wgrad_plan(a, codes, parts), false};
    if (values > 0 && a.S > 0 && whole && fits) {
      WgradArgs b = a;
      b.ldx = a.K;
      const Choice r = wgrad_plan(b, false, parts_behind_values);
      // where the wide tiles take them then: 3 bytes an element and a launch
      if (r.plan == ExpertPlan::Wide &&
          r.us + 4.0 + (double)a.Rx * (double)a.K * 3 / 4e6 < w.c.us)
        w = WgradChoice{r, true};
    }
    return w;
  };
  const WgradChoice w = best(kEnough, kEnough, true);
  if (parts_bytes(a, w.c) + (w.restored ? values : 0) <= room) return w;
  return best(room, room - values, room >= values);
}

// Any non-null scales, for the queries: plans do not read them.
constexpr uint8_t kSome = 0;

// Arguments of those sizes, rows aligned or not (false: no such call).
bool mm_sizes(bsmm_dtype dtype, int transposed, bool rows, int64_t E, int64_t S, int64_t N,
              int64_t K, ExpertArgs& a) {
  if (!float_dtype(dtype) || E <= 0 || S <= 0 || N <= 0 || K <= 0 || E > kMaxExperts ||
      S >= kMaxSize || N >= kMaxSize || K >= kMaxSize)
    return false;
  a = ExpertArgs{};
  a.dtype = dtype;
  a.w_across = transposed;
  a.ldx = rows ? 0 : 1;
  a.E = (int)E; a.S = (int)S; a.N = (int)N; a.K = (int)K;
  return true;
}
bool wgrad_sizes(bsmm_dtype dtype, int checkpoint, bool dy_rows, bool x_rows, int64_t E,
                 int64_t Rx, int64_t S, int64_t N, int64_t K, WgradArgs& a) {
  if (!float_dtype(dtype) || E <= 0 || Rx <= 0 || S <= 0 || N <= 0 || K <= 0 || E > kMaxExperts ||
      Rx >= kMaxDim || S >= kMaxSize || N >= kMaxSize || K >= kMaxSize)
    return false;
  a = WgradArgs{};
  a.dtype = dtype;
  a.x_scale = checkpoint ? &kSome : nullptr;
  a.ldy = dy_rows ? 0 : 1;
  a.ldx = x_rows ? 0 : 1;
  a.E = (int)E; a.Rx = (int)Rx; a.S = (int)S; a.N = (int)N; a.K = (int)K;
  return true;
}

}  // namespace

extern "C" {

size_t bsmm_expert_mm_workspace_bytes(bsmm_dtype dtype, int transposed, int64_t E, int64_t S,
                                      int64_t N, int64_t K) {
  size_t need = 0;
  ExpertArgs a;
  for (int rows = 0; rows < 2; ++rows) {
    if (!mm_sizes(dtype, transposed, rows, E, S, N, K, a)) return 0;
    const size_t bytes = parts_bytes(a, mm_plan(a, kEnough));
    if (bytes > need) need = bytes;
  }
  return need;
}

const char* bsmm_expert_mm_plan_name(bsmm_dtype dtype, int transposed, int aligned, int64_t E,
                                     int64_t S, int64_t N, int64_t K, size_t workspace_bytes,
                                     int* parts) {
  ExpertArgs a;
  if (!mm_sizes(dtype, transposed, aligned != 0, E, S, N, K, a)) return nullptr;
  const Choice c = mm_choice(a, workspace_bytes);
  if (parts != nullptr) *parts = c.splits;
  if (c.plan == ExpertPlan::Rows) return "rows";
  if (c.plan == ExpertPlan::Tiles64) return "tile64";
  return c.rows == 256 ? "wide256" : c.rows == 192 ? "wide192" : "wide128";
}

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
  CHECK(R < kMaxDim && S < kMaxSize && N < kMaxSize && K < kMaxSize, BSMM_ERR_UNSUPPORTED,
        "R beyond 2^31, or S, N or K beyond 2^31 - 1024");
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
  // tiles are counted in 31 bits, of at least 16 rows by 16 columns each
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
  a.order = order; a.offsets = offsets;
  a.row_scale = K > 0 ? row_scale : nullptr;       // zeros, whatever the scale
  a.x_div = slots_per_row;
  a.out = out; a.ldo = ldo; a.out_dtype = out_dtype;
  a.E = (int)E; a.R = (int)R; a.S = (int)S; a.N = (int)N; a.K = (int)K;
  const Choice c =
      mm_choice(a, workspace != nullptr && aligned(workspace, 16) ? workspace_bytes : 0);
  CHECK(expert_mm_threads(a, c.plan, c.rows, c.splits) < kMaxThreads, BSMM_ERR_UNSUPPORTED,
        "S * N beyond the largest grid");
  if (launch_expert_mm(a, c.plan, c.rows, c.splits, workspace, stream) != 0)
    return fail(BSMM_ERR_HIP, "kernel launch failed (expert product)");
  return BSMM_OK;
}

size_t bsmm_expert_wgrad_workspace_bytes(bsmm_dtype dtype, int checkpoint, int64_t E, int64_t Rx,
                                         int64_t S, int64_t N, int64_t K) {
  size_t need = 0;
  WgradArgs a;
  for (int rows = 0; rows < 2; ++rows) {
    if (!wgrad_sizes(dtype, 0, rows, true, E, Rx, S, N, K, a)) return 0;
    // codes as they are or restored, fp32 or bf16 output
    for (int codes = 0; codes <= (checkpoint != 0); ++codes)
      for (int bf = 0; bf < 2; ++bf) {
        a.out_dtype = bf ? BSMM_BF16 : BSMM_F32;
        const size_t bytes = parts_bytes(a, wgrad_plan(a, codes != 0, kEnough));
        if (bytes > need) need = bytes;
      }
  }
  return need + restored_bytes(dtype, checkpoint, Rx, K);
}

const char* bsmm_expert_wgrad_plan_name(bsmm_dtype dtype, int checkpoint, bsmm_dtype out_dtype,
                                        int dy_aligned, int x_aligned, int64_t E, int64_t Rx,
                                        int64_t S, int64_t N, int64_t K, size_t workspace_bytes,
                                        int* parts) {
  WgradArgs a;
  if (!float_dtype(out_dtype) || (checkpoint && K % 32 != 0) ||
      !wgrad_sizes(dtype, checkpoint, dy_aligned != 0, x_aligned != 0, E, Rx, S, N, K, a))
    return nullptr;
  a.out_dtype = out_dtype;
  const WgradChoice w = wgrad_choice(a, x_aligned != 0, workspace_bytes);
  if (parts != nullptr) *parts = w.c.splits;
  if (w.restored) return "restored";
  return w.c.plan == ExpertPlan::Wide ? "wide256"
         : w.c.plan == ExpertPlan::Tiles128 ? "tile128" : "tile64";
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
  CHECK(Ry < kMaxDim && Rx < kMaxDim && S < kMaxSize && N < kMaxSize && K < kMaxSize,
        BSMM_ERR_UNSUPPORTED, "Ry or Rx beyond 2^31, or S, N or K beyond 2^31 - 1024");
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
  CHECK(E * (N / 64 + 1) * (K / 64 + 1) < kMaxDim, BSMM_ERR_UNSUPPORTED,
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
  uint8_t* ws = aligned(workspace, 16) ? static_cast<uint8_t*>(workspace) : nullptr;
  const WgradChoice w = wgrad_choice(a, aligned(x, 8) && ldx % 8 == 0,
                                     ws != nullptr ? workspace_bytes : 0);
  CHECK(expert_wgrad_threads(a, w.c.plan, w.c.splits) < kMaxThreads, BSMM_ERR_UNSUPPORTED,
        "E * N * K beyond the largest grid");
  if (w.restored) {
    if (launch_restore_bf16(x, ldx, x_scale, s_r, ws, Rx, K, stream) != 0)
      return fail(BSMM_ERR_HIP, "kernel launch failed (checkpoint values)");
    a.x = ws;
    a.ldx = K;
    a.x_scale = nullptr;
    ws += restored_bytes(dtype, 1, Rx, K);
  }
  if (launch_expert_wgrad(a, w.c.plan, w.c.splits, ws, stream) != 0)
    return fail(BSMM_ERR_HIP, "kernel launch failed (expert weight gradient)");
  return BSMM_OK;
}

}  // extern "C"
