// The router of a mixture-of-experts layer (gfx950): top-k choice, per-expert
// counts, the slots sorted by expert, the balance loss and its gradient.
//
//   p = softmax(logits[t]);  index[t, j] = the j-th largest logit's expert
//   weight[t, j] = p[index], or p[index] / sum_j p[index]
//   loss = alpha * E / (k L^2) * sum_e counts[e] * prob_sum[e]
//
// A wave holds one token's logits in registers, PER neighbouring experts a
// lane.  The k rounds of the choice are integer maxima over order-preserving
// keys; of equal keys the lowest lane's, and in a lane the lowest expert's,
// is taken.  A lane's keys are sorted once, so that a round looks at its
// first one only.
//
// The order of the slots is a stable counting sort.  A token's choices are
// distinct experts, so 64 tokens make one 64-bit mask per expert, and a
// slot's rank among them is the number of mask bits below its token: no
// atomic's order can change a result.  Blocks of tokens write their counts, a
// second launch sums them over the blocks before each, and a third places the
// slots.  At most one block per compute unit keeps that table small; more
// tokens make larger blocks.  Up to 64 tokens are one block and one launch.
//
// 16384 x 256 fp32, top-8 with the loss: choice 17 us (eight dependent wave
// maxima a token), counts 4.9, slots 6.8; its gradient 10.6, 3.3 TB/s.  One
// token of 64 experts: 5 us.

#include <hip/hip_runtime.h>

#include <cstdint>

#include "bsmm_internal.h"

namespace bsmm {
namespace {

constexpr int kWaves = 16;              // waves of a workgroup
constexpr uint32_t kNoKey = 0x007FFFFFu;   // the key of -inf; nothing at or below it is chosen

typedef unsigned long long u64;

__device__ __forceinline__ float load_logit(const uint16_t* p) {
  return __uint_as_float((uint32_t)*p << 16);
}
__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ void store_grad(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_grad(uint16_t* p, float v) {
  uint32_t b = __float_as_uint(v);
  b = v != v ? b | 0x400000u : b + 0x7FFFu + ((b >> 16) & 1u);
  *p = (uint16_t)(b >> 16);
}

// Integers in the order of the floats; -0 as +0; a NaN below everything.
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  return v != v ? 0u : b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// Wave reductions by row shifts and row broadcasts; the total is lane 63's.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
  // lanes without a source take 0, the identity: one fused instruction
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true));
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = dpp_max<0x111>(v);
  v = dpp_max<0x112>(v);
  v = dpp_max<0x114>(v);
  v = dpp_max<0x118>(v);
  v = dpp_max<0x142>(v);
  v = dpp_max<0x143>(v);
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
// the same of several values, their chains interleaved
template <int N>
__device__ __forceinline__ void wave_max_all(uint32_t (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = dpp_max<0x111>(v[i]);
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = dpp_max<0x112>(v[i]);
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = dpp_max<0x114>(v[i]);
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = dpp_max<0x118>(v[i]);
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = dpp_max<0x142>(v[i]);
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = dpp_max<0x143>(v[i]);
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = (uint32_t)__builtin_amdgcn_readlane((int)v[i], 63);
}
template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __int_as_float(
                 __builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, false));
}
__device__ __forceinline__ float wave_sum(float v) {
  v = dpp_add<0x111>(v);
  v = dpp_add<0x112>(v);
  v = dpp_add<0x114>(v);
  v = dpp_add<0x118>(v);
  v = dpp_add<0x142>(v);
  v = dpp_add<0x143>(v);
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}
__device__ __forceinline__ int wave_scan(int v) {      // inclusive
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int t = __shfl_up(v, d);
    if (lane >= d) v += t;
  }
  return v;
}

// e^d for d <= 0 (0 below -200, NaN kept): 2^(d log2 e) with the product's
// rounding error and the constant's low part put back, so the error stays
// that of the hardware's 2^x instead of growing with |d|.
__device__ __forceinline__ float exp_neg(float d) {
  constexpr float kL = 0x1.715476p+0f, kLo = 0x1.4ae0c0p-26f, kLn2 = 0x1.62e430p-1f;
  d = d < -200.0f ? -200.0f : d;
  const float t = d * kL;
  const float r = __builtin_fmaf(d, kLo, __builtin_fmaf(d, kL, -t));
  const float e = __builtin_amdgcn_exp2f(t);
  return __builtin_fmaf(e, r * kLn2, e);
}

// A wave's LDS accesses run in order; this keeps the compiler from moving
// them past each other.
__device__ __forceinline__ void order_lds() { asm volatile("" ::: "memory"); }

struct Shared {
  u64 mask[kRouteMaxE];
  int hist[kRouteMaxE];
  int total[kRouteMaxE];
  int base[kRouteMaxE];
  int index[64 * kRouteMaxK];     // the choices of 64 tokens
  int unused[64];
  int scan[kWaves];
  int live, used, unused_base;
  float sum[kWaves];
};

// Tokens [t0, t1): choice and weights, counts into sh.hist, live tokens into
// sh.live, and each wave's sums of probabilities into prob[wave][E] (loss
// only).  sh.hist and sh.live are zero before, complete after a barrier.  A
// wave takes U tokens at a time: the rounds of one token are a chain of
// dependent wave reductions, and U chains fill each other's gaps (16384 x 256
// top-8: 19 us with one, see the launch for U).  `keep`: the choices also go
// to sh.index (64 tokens at most).
template <typename T, int PER, int U, int W>
__device__ void choose(const RouteArgs& a, Shared& sh, float* prob, int t0, int t1, bool keep) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int E = a.E, k = a.k;
  float psum[PER] = {};
  for (int tb = t0 + wave * U; tb < t1; tb += W * U) {
    // all loads before their first use; lane u has token u's mask
    const int tu = tb + (lane & (U - 1));
    const int open = tu < t1 && (a.mask == nullptr || a.mask[min(tu, t1 - 1)] != 0);
    float v[U][PER];
    uint32_t key[U][PER];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const T* row = static_cast<const T*>(a.logits) + (int64_t)min(tb + u, t1 - 1) * a.ldl;
#pragma unroll
      for (int i = 0; i < PER; ++i) v[u][i] = load_logit(row + min(lane * PER + i, E - 1));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool on = __builtin_amdgcn_readlane(open, u) != 0;
#pragma unroll
      for (int i = 0; i < PER; ++i)
        v[u][i] = on && lane * PER + i < E ? v[u][i] : -__builtin_inff();
    }
    // stable insertion sort of a lane's keys, largest first; id: their places
    uint32_t id[U][PER];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        key[u][i] = key_of(v[u][i]);
        id[u][i] = i;
#pragma unroll
        for (int j = i; j > 0; --j) {
          const bool up = key[u][j] > key[u][j - 1];
          const uint32_t k0 = key[u][j - 1], k1 = key[u][j], i0 = id[u][j - 1], i1 = id[u][j];
          key[u][j - 1] = up ? k1 : k0;
          key[u][j] = up ? k0 : k1;
          id[u][j - 1] = up ? i1 : i0;
          id[u][j] = up ? i0 : i1;
        }
      }
    int idx[U];                   // lane j: the j-th choice
    uint32_t chosen[U], top[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      idx[u] = -1;
      chosen[u] = 0;
      top[u] = 0;
    }
    for (int j = 0; j < k; ++j) {
      uint32_t m[U], any = 0;
#pragma unroll
      for (int u = 0; u < U; ++u) m[u] = key[u][0];
      wave_max_all(m);
#pragma unroll
      for (int u = 0; u < U; ++u) any = max(any, m[u]);
      if (any <= kNoKey) break;   // uniform
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (m[u] <= kNoKey) continue;       // uniform: this token has none left
        const int from = __ffsll((u64)__ballot(key[u][0] == m[u])) - 1;
        const int found = from * PER + __builtin_amdgcn_readlane((int)id[u][0], from);
        if (lane == from) {
#pragma unroll
          for (int i = 0; i + 1 < PER; ++i) {
            key[u][i] = key[u][i + 1];
            id[u][i] = id[u][i + 1];
          }
          key[u][PER - 1] = 0;
        }
        if (j == 0) top[u] = m[u];
        if (lane == j) {
          idx[u] = found;
          chosen[u] = m[u];
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = tb + u;
      if (t >= t1) break;         // uniform
      const bool live = top[u] != 0;
      // -inf stands in all places without a logit: its exponential is 0
      const float mx = live ? of_key(top[u]) : 0.0f;
      float ex[PER], s = 0.0f;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        ex[i] = exp_neg(v[u][i] - mx);
        s += ex[i];
      }
      s = wave_sum(s);
      const float we = exp_neg(of_key(chosen[u]) - mx);
      const float w = idx[u] >= 0 ? we : 0.0f;
      const float den = a.renorm ? wave_sum(w) + (s - s) : s;     // s - s: a NaN in the row stays
      if (lane < k) {
        a.index[(int64_t)t * k + lane] = idx[u];
        a.weight[(int64_t)t * k + lane] = idx[u] >= 0 ? w / den : 0.0f;
        if (idx[u] >= 0) atomicAdd(&sh.hist[idx[u]], 1);
        if (keep) sh.index[(t - t0) * k + lane] = idx[u];
      }
      if (live && lane == 0) atomicAdd(&sh.live, 1);
      if (a.loss != nullptr && live) {
        const float r = 1.0f / s;
#pragma unroll
        for (int i = 0; i < PER; ++i) psum[i] += ex[i] * r;
      }
    }
  }
  if (a.loss != nullptr) {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (lane * PER + i < E) prob[wave * E + lane * PER + i] = psum[i];
  }
}

// Sum of the wave rows of prob for expert e.
template <int W>
__device__ __forceinline__ float prob_of(const float* prob, int E, int e) {
  float p = 0.0f;
#pragma unroll
  for (int w = 0; w < W; ++w) p += prob[w * E + e];
  return p;
}

// From sh.total: the experts' offsets into sh.base, the number of chosen
// slots into sh.used, counts and offsets to memory.
__device__ void expert_offsets(const RouteArgs& a, Shared& sh) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int e = threadIdx.x;
  const int n = e < a.E ? sh.total[e] : 0;
  const int incl = wave_scan(n);
  if (lane == 63) sh.scan[wave] = incl;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    if (w < wave) before += sh.scan[w];
    all += sh.scan[w];
  }
  const int off = before + incl - n;
  if (e < a.E) {
    sh.base[e] = off;
    a.counts[e] = n;
    a.offsets[e] = off;
  }
  if (e == 0) {
    sh.used = all;
    a.offsets[a.E] = all;
  }
  __syncthreads();
}

// loss, prob_sum and live from sh.total, the live tokens and the
// probabilities' sums (p: thread e's expert).
__device__ void write_loss(const RouteArgs& a, Shared& sh, float p, int live) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int e = threadIdx.x;
  const float n = (float)max(live, 1);
  float c = 0.0f;
  if (e < a.E) {
    a.prob_sum[e] = p;
    c = ((float)sh.total[e] / n) * (p / n);
  }
  c = wave_sum(c);
  if (lane == 0) sh.sum[wave] = c;
  __syncthreads();
  if (e == 0) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) s += sh.sum[w];
    a.loss[0] = a.alpha * (float)a.E / (float)a.k * s;
    a.live[0] = live;
  }
}

// Order of the slots of tokens [t0, t1): sh.base holds the position of each
// expert's next slot, sh.unused_base that of the next slot without one.  They
// come from the workspace: should a caller have let something else write it
// between the launches, positions outside the order are not written.
// `kept`: sh.index already has the choices (64 tokens at most).
__device__ void place(const RouteArgs& a, Shared& sh, int t0, int t1, bool kept) {
  const int k = a.k;
  // s / k for s < 64 * 32: the multiplier's error stays below 1 / k
  const uint32_t inv = (65536u + k - 1) / k;
  for (int tb = t0; tb < t1; tb += 64) {
    const int nt = min(t1 - tb, 64);
    const int slots = nt * k;
    for (int e = threadIdx.x; e < a.E; e += (int)blockDim.x) sh.mask[e] = 0;
    if (!kept)
      for (int s = threadIdx.x; s < slots; s += (int)blockDim.x)
        sh.index[s] = a.index[(int64_t)tb * k + s];
    __syncthreads();
    for (int s = threadIdx.x; s < slots; s += (int)blockDim.x) {
      const int e = sh.index[s];
      if (e >= 0) atomicOr(&sh.mask[e], 1ull << (s * inv >> 16));
    }
    if (threadIdx.x < 64) {
      // slots without an expert before each token: its last ones
      int n = 0;
      if ((int)threadIdx.x < nt)
        for (int j = k - 1; j >= 0 && sh.index[threadIdx.x * k + j] < 0; --j) ++n;
      const int incl = wave_scan(n);
      sh.unused[threadIdx.x] = sh.unused_base + incl - n;
      __builtin_amdgcn_wave_barrier();
      if (threadIdx.x == 63) sh.unused_base += incl;
    }
    __syncthreads();
    for (int s = threadIdx.x; s < slots; s += (int)blockDim.x) {
      const int t = s * inv >> 16, e = sh.index[s];
      int at;
      if (e >= 0) {
        at = sh.base[e] + __popcll(sh.mask[e] & ((1ull << t) - 1));
      } else {
        at = sh.unused[t];
        for (int j = s - 1; j >= t * k && sh.index[j] < 0; --j) ++at;
      }
      if ((unsigned)at < (unsigned)(a.T * k)) a.order[at] = tb * k + s;
    }
    if (tb + 64 >= t1) break;
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += (int)blockDim.x) sh.base[e] += __popcll(sh.mask[e]);
    __syncthreads();
  }
}

// First launch: one block of tokens per workgroup of W waves.  ONE: one block
// in all (W = 16, a thread per expert), which also writes the rest.
template <typename T, int PER, int U, int W, bool ONE>
__global__ void __launch_bounds__(W * 64) route_choose(RouteArgs a) {
  static_assert(!ONE || W == kWaves, "a thread per expert");
  __shared__ Shared sh;
  extern __shared__ float prob[];       // [W][E], loss only
  for (int e = threadIdx.x; e < a.E; e += W * 64) {
    sh.hist[e] = 0;
    sh.base[e] = 0;
  }
  if (threadIdx.x == 0) sh.live = 0;
  __syncthreads();
  const int t0 = blockIdx.x * a.block, t1 = min(a.T, t0 + a.block);
  choose<T, PER, U, W>(a, sh, prob, t0, t1, ONE);
  __syncthreads();
  if constexpr (!ONE) {
    for (int e = threadIdx.x; e < a.E; e += W * 64) {
      a.hist[(int64_t)blockIdx.x * a.hist_ld + e] = (uint16_t)sh.hist[e];
      if (a.loss != nullptr) a.prob[(int64_t)blockIdx.x * a.E + e] = prob_of<W>(prob, a.E, e);
    }
    if (threadIdx.x == 0) a.hist[(int64_t)blockIdx.x * a.hist_ld + a.E] = (uint16_t)sh.live;
  } else {
    const int e = threadIdx.x;
    if (e < a.E) sh.total[e] = sh.hist[e];
    __syncthreads();
    expert_offsets(a, sh);
    if (a.loss != nullptr)
      write_loss(a, sh, e < a.E ? prob_of<W>(prob, a.E, e) : 0.0f, sh.live);
    if (e == 0) sh.unused_base = sh.used;
    __syncthreads();
    place(a, sh, t0, t1, true);
  }
}

// Second launch, a wave per expert (and one for the live tokens): the slots
// of the expert in the blocks before each block, in all, and the sum of the
// blocks' probabilities.
__global__ void __launch_bounds__(256) route_scan(RouteArgs a, int blocks) {
  constexpr int Q = kRouteMaxBlocks / 64;
  const int lane = threadIdx.x & 63;
  const int e = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (e > a.E) return;
  int n[Q];
  float p[Q];
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    const int b = min(lane * Q + q, blocks - 1);
    n[q] = a.hist[(int64_t)b * a.hist_ld + e];
    p[q] = a.loss != nullptr && e < a.E ? a.prob[(int64_t)b * a.E + e] : 0.0f;
  }
  int sum = 0;
  float ps = 0.0f;
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    if (lane * Q + q >= blocks) n[q] = 0, p[q] = 0.0f;
    sum += n[q];
    ps += p[q];
  }
  const int incl = wave_scan(sum);
  ps = wave_sum(ps);
  const int total = __builtin_amdgcn_readlane(incl, 63);
  if (e == a.E) {
    if (lane == 0 && a.loss != nullptr) a.live[0] = total;
    return;
  }
  int before = incl - sum;
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    const int b = lane * Q + q;
    if (b < blocks) a.before[(int64_t)b * a.E + e] = before;
    before += n[q];
  }
  if (lane == 0) {
    a.counts[e] = total;
    if (a.loss != nullptr) a.prob_sum[e] = ps;
  }
}

// Third launch: a workgroup places one block's slots; the first one also
// writes the offsets and the loss.
__global__ void __launch_bounds__(256) route_place(RouteArgs a) {
  __shared__ Shared sh;
  constexpr int PT = kRouteMaxE / 256;       // experts of a thread
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int me = blockIdx.x, E = a.E;
  const int e0 = threadIdx.x * PT;
  int n[PT], before[PT], all = 0, prev = 0;
#pragma unroll
  for (int i = 0; i < PT; ++i) {
    const int e = min(e0 + i, E - 1);
    n[i] = a.counts[e];
    before[i] = a.before[(int64_t)me * E + e];
  }
#pragma unroll
  for (int i = 0; i < PT; ++i) {
    if (e0 + i >= E) n[i] = before[i] = 0;
    all += n[i];
    prev += before[i];
  }
  const int incl = wave_scan(all), pincl = wave_scan(prev);
  if (lane == 63) {
    sh.scan[wave] = incl;
    sh.scan[4 + wave] = pincl;
  }
  __syncthreads();
  int off = incl - all, used = 0, used_before = 0;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    if (w < wave) off += sh.scan[w];
    used += sh.scan[w];
    used_before += sh.scan[4 + w];
  }
#pragma unroll
  for (int i = 0; i < PT; ++i) {
    if (e0 + i >= E) break;
    sh.base[e0 + i] = off + before[i];
    if (me == 0) a.offsets[e0 + i] = off;
    off += n[i];
  }
  const int t0 = me * a.block, t1 = min(a.T, t0 + a.block);
  if (threadIdx.x == 0) {
    sh.unused_base = used + t0 * a.k - used_before;
    if (me == 0) a.offsets[E] = used;
  }
  if (me == 0 && a.loss != nullptr) {
    const float live = (float)max(a.live[0], 1);
    float c = 0.0f;
#pragma unroll
    for (int i = 0; i < PT; ++i) {
      const float p = a.prob_sum[min(e0 + i, E - 1)];
      if (e0 + i < E) c += ((float)n[i] / live) * (p / live);
    }
    c = wave_sum(c);
    if (lane == 0) sh.sum[wave] = c;
    __syncthreads();
    if (threadIdx.x == 0)
      a.loss[0] = a.alpha * (float)E / (float)a.k * (sh.sum[0] + sh.sum[1] + sh.sum[2] + sh.sum[3]);
  }
  __syncthreads();
  place(a, sh, t0, t1, false);
}

// Gradient of the logits, one wave per token:
//   d_e = p_e (c_e - sum p c) + [plain] p_e (g_e - sum_j w_j dw_j)
//       + [renormalised] w_j (dw_j - sum w dw) at e = index[j],
// c_e = dloss * alpha * E * counts_e / (k L^2), g_e = dw_j at e = index[j].
// A wave takes U tokens at a time, all their loads first; the chosen experts'
// part goes through a row of LDS of the wave's own.
template <typename T, int PER, int U>
__global__ void __launch_bounds__(256) route_backward(RouteBackArgs a) {
  extern __shared__ float dyn[];          // [4][E]
  const int lane = threadIdx.x & 63;
  const int E = a.E, k = a.k;
  float* const add_row = dyn + (threadIdx.x >> 6) * E;
  const int waves = gridDim.x * 4;
  for (int tb = (blockIdx.x * 4 + (threadIdx.x >> 6)) * U; tb < a.T; tb += waves * U) {
    float v[U][PER], w[U], dw[U];
    int idx[U];
    bool on[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = min(tb + u, a.T - 1);
      const T* row = static_cast<const T*>(a.logits) + (int64_t)t * a.ldl;
#pragma unroll
      for (int i = 0; i < PER; ++i) v[u][i] = load_logit(row + min(i * 64 + lane, E - 1));
      const int64_t at = (int64_t)t * k + min(lane, k - 1);
      idx[u] = a.index[at];
      w[u] = dw[u] = 0.0f;
      if (a.dweight != nullptr) {
        w[u] = a.weight[at];
        dw[u] = a.dweight[at];
      }
      on[u] = a.mask == nullptr || a.mask[t] != 0;
    }
    float c[PER], f = 0.0f;
    if (a.dloss != nullptr) {
      const float n = (float)max(a.live[0], 1);
      f = a.dloss[0] * (a.alpha * (float)E / (float)k) / n / n;
#pragma unroll
      for (int i = 0; i < PER; ++i) c[i] = f * (float)a.counts[min(i * 64 + lane, E - 1)];
    } else {
#pragma unroll
      for (int i = 0; i < PER; ++i) c[i] = 0.0f;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = tb + u;
      if (t >= a.T) break;        // uniform
      T* out = static_cast<T*>(a.dlogits) + (int64_t)t * a.ldd;
      if (lane >= k || idx[u] >= E) idx[u] = -1;
      if (idx[u] < 0) w[u] = dw[u] = 0.0f;
      const bool live = on[u] && __builtin_amdgcn_readlane(idx[u], 0) >= 0;
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        if (i * 64 + lane >= E) v[u][i] = -__builtin_inff();
        m = max(m, key_of(v[u][i]));
      }
      const float top = of_key(wave_max(m));
      float s = 0.0f, pc = 0.0f;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        v[u][i] = i * 64 + lane < E ? exp_neg(v[u][i] - top) : 0.0f;
        s += v[u][i];
        pc += v[u][i] * c[i];
      }
      s = wave_sum(s);
      const float r = 1.0f / s;
      const float dot = wave_sum(w[u] * dw[u]);
      const float sub = wave_sum(pc) * r + (a.renorm ? 0.0f : dot);
      if (a.dweight != nullptr) {
#pragma unroll
        for (int i = 0; i < PER; ++i)
          if (i * 64 + lane < E) add_row[i * 64 + lane] = 0.0f;
        order_lds();
        if (idx[u] >= 0) add_row[idx[u]] = w[u] * (a.renorm ? dw[u] - dot : dw[u]);
        order_lds();
      }
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        if (i * 64 + lane >= E) continue;
        float d = v[u][i] * r * (c[i] - sub);
        if (a.dweight != nullptr) d += add_row[i * 64 + lane];
        store_grad(out + i * 64 + lane, live ? d : 0.0f);
      }
      order_lds();
    }
  }
}

// Tokens a wave takes at a time: as many chains as registers allow.
template <int PER> constexpr int kTokens = PER <= 4 ? 4 : PER <= 8 ? 2 : 1;

template <typename T, int PER, int U, int W, bool ONE>
void launch_choose_as(const RouteArgs& a, int blocks, hipStream_t st) {
  const size_t lds = a.loss != nullptr ? (size_t)W * a.E * 4 : 0;
  hipLaunchKernelGGL((route_choose<T, PER, U, W, ONE>), dim3(blocks), dim3(W * 64), lds, st, a);
}

template <typename T, int PER>
void launch_choose_per(const RouteArgs& a, int blocks, hipStream_t st) {
  constexpr int U = kTokens<PER>;
  // with few tokens every wave takes one; blocks of 16 tokens are 4 waves
  if (blocks == 1 && a.T <= kWaves) launch_choose_as<T, PER, 1, kWaves, true>(a, blocks, st);
  else if (blocks == 1) launch_choose_as<T, PER, U, kWaves, true>(a, blocks, st);
  else if (a.block == 16) launch_choose_as<T, PER, U, 4, false>(a, blocks, st);
  else launch_choose_as<T, PER, U, kWaves, false>(a, blocks, st);
}

template <typename T, int PER>
void launch_backward_per(const RouteBackArgs& a, hipStream_t st) {
  // two tokens a wave where that still leaves 4 waves to a SIMD
  constexpr int U = PER <= 8 ? 2 : 1;
  const size_t lds = a.dweight != nullptr ? (size_t)4 * a.E * 4 : 0;
  if (a.T <= 4096 || U == 1)
    hipLaunchKernelGGL((route_backward<T, PER, 1>), dim3((a.T + 3) / 4), dim3(256), lds, st, a);
  else
    hipLaunchKernelGGL((route_backward<T, PER, U>), dim3((a.T + 4 * U - 1) / (4 * U)), dim3(256),
                       lds, st, a);
}

template <typename T>
void launch_choose(const RouteArgs& a, int blocks, hipStream_t st) {
  if (a.E <= 64) launch_choose_per<T, 1>(a, blocks, st);
  else if (a.E <= 128) launch_choose_per<T, 2>(a, blocks, st);
  else if (a.E <= 256) launch_choose_per<T, 4>(a, blocks, st);
  else if (a.E <= 512) launch_choose_per<T, 8>(a, blocks, st);
  else launch_choose_per<T, 16>(a, blocks, st);
}

template <typename T>
void launch_backward(const RouteBackArgs& a, hipStream_t st) {
  if (a.E <= 64) launch_backward_per<T, 1>(a, st);
  else if (a.E <= 128) launch_backward_per<T, 2>(a, st);
  else if (a.E <= 256) launch_backward_per<T, 4>(a, st);
  else if (a.E <= 512) launch_backward_per<T, 8>(a, st);
  else launch_backward_per<T, 16>(a, st);
}

}  // namespace

int launch_route(const RouteArgs& a, int blocks, void* stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (a.dtype == BSMM_BF16) launch_choose<uint16_t>(a, blocks, st);
  else launch_choose<float>(a, blocks, st);
  if (blocks > 1) {
    hipLaunchKernelGGL(route_scan, dim3(a.E / 4 + 1), dim3(256), 0, st, a, blocks);
    hipLaunchKernelGGL(route_place, dim3(blocks), dim3(256), 0, st, a);
  }
  return hipGetLastError() == hipSuccess ? 0 : 1;
}

int launch_route_backward(const RouteBackArgs& a, void* stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (a.dtype == BSMM_BF16) launch_backward<uint16_t>(a, st);
  else launch_backward<float>(a, st);
  return hipGetLastError() == hipSuccess ? 0 : 1;
}

}  // namespace bsmm
