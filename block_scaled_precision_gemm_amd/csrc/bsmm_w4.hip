// Products of bf16 / fp32 activations with 4-bit weights (gfx950).
//
//   out[p, n] = sum_g scale[n, g] * sum_{k in g} (code[n, k] - zero[n, g]) * x[p, k]
//
// A code enters the matrix instruction as the bf16 number 16 + code, which
// is the bit pattern 0x4180 | code << 3: two codes of a dword become a
// packed pair with one shift and one and-or.  With d = sum (16 + code) x and
// e = sum x over a group (e by the same instruction against ones), the
// group's contribution is scale * (d - (16 + zero) * e): every product is
// exact, the sums are fp32, and nothing is rounded to fewer bits before the
// output.  fp32 activations are cut into three bf16 numbers that add up to
// them exactly (8 + 8 + 8 bits), one matrix instruction each.
//
// The pair of codes in a dword's half words are 4 apart, so the activations'
// 8 consecutive elements are paired alike (k, k + 4): the order of k inside
// one matrix instruction is free as long as both operands share it.

#include <hip/hip_runtime.h>

#include <cstdint>

#include "bsmm_internal.h"

namespace bsmm {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

__device__ __forceinline__ uint32_t bf16_bits(float v) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t{v, v}), bf16x2_t)) &
         0xFFFFu;
}

// 8 codes of a dword -> 16 + code as bf16, in the order 0 4 1 5 2 6 3 7
__device__ __forceinline__ u32x4 unpack(uint32_t w) {
  constexpr uint32_t kMask = 0x00780078u, kBias = 0x41804180u;
  return u32x4{((w << 3) & kMask) | kBias, ((w >> 1) & kMask) | kBias,
               ((w >> 5) & kMask) | kBias, ((w >> 9) & kMask) | kBias};
}

// low / high halves of (a, b) as a pair
__device__ __forceinline__ uint32_t lo2(uint32_t a, uint32_t b) {
  return __builtin_amdgcn_perm(b, a, 0x05040100u);
}
__device__ __forceinline__ uint32_t hi2(uint32_t a, uint32_t b) {
  return __builtin_amdgcn_perm(b, a, 0x07060302u);
}

// 8 consecutive activations of one row
template <bool XF32> struct X8;
template <> struct X8<false> { u32x4 v; };
template <> struct X8<true> { u32x4 a, b; };

template <bool XF32>
__device__ __forceinline__ X8<XF32> load_x(const void* x, int64_t at) {
  X8<XF32> r;
  if constexpr (XF32) {
    const u32x4* p = reinterpret_cast<const u32x4*>(static_cast<const float*>(x) + at);
    r.a = p[0];
    r.b = p[1];
  } else {
    r.v = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(x) + at);
  }
  return r;
}

// the bf16 operands of 8 activations (1, or the 3 parts of fp32 values), in
// the order 0 4 1 5 2 6 3 7
template <bool XF32> struct Parts { u32x4 p[XF32 ? 3 : 1]; };

__device__ __forceinline__ Parts<false> parts(const X8<false>& x) {
  Parts<false> r;
  r.p[0] = u32x4{lo2(x.v.x, x.v.z), hi2(x.v.x, x.v.z), lo2(x.v.y, x.v.w), hi2(x.v.y, x.v.w)};
  return r;
}
// the part of v below its top 16 bits (exact)
__device__ __forceinline__ uint32_t below(uint32_t v) {
  return __float_as_uint(__uint_as_float(v) - __uint_as_float(v & 0xFFFF0000u));
}
__device__ __forceinline__ Parts<true> parts(const X8<true>& x) {
  Parts<true> r;
  u32x4 a = x.a, b = x.b;
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    r.p[i] = u32x4{hi2(a.x, b.x), hi2(a.y, b.y), hi2(a.z, b.z), hi2(a.w, b.w)};
    if (i < 2) {
      a = u32x4{below(a.x), below(a.y), below(a.z), below(a.w)};
      b = u32x4{below(b.x), below(b.y), below(b.z), below(b.w)};
    }
  }
  return r;
}

struct Item { int e, p0, rows; };

// Work item `item` of a routed product: every expert's run of positions is
// cut into blocks of bm, in expert order.  Runs in every wave alike: each
// lane counts the blocks of its share of the experts, a scan over the lanes
// finds the one that holds the item.  Offsets are clamped into [0, S], so
// that no array content can lead outside the buffers.
__device__ Item find_item(const int32_t* __restrict__ offsets, int E, int S, int bm, int item) {
  const int lane = threadIdx.x & 63;
  const int per = (E + 63) / 64;
  const int e0 = min(lane * per, E), e1 = min(e0 + per, E);
  int n = 0;
  for (int e = e0; e < e1; ++e) {
    const int lo = min(max(offsets[e], 0), S), hi = min(max(offsets[e + 1], lo), S);
    n += (hi - lo + bm - 1) / bm;
  }
  int incl = n;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int t = __shfl_up(incl, d);
    if (lane >= d) incl += t;
  }
  const unsigned long long past = __ballot(incl > item);
  if (past == 0) return Item{0, 0, 0};
  const int src = __ffsll(past) - 1;
  int rest = item - (incl - n);
  Item r{0, 0, 0};
  if (lane == src) {
    for (int e = e0; e < e1; ++e) {
      const int lo = min(max(offsets[e], 0), S), hi = min(max(offsets[e + 1], lo), S);
      const int b = (hi - lo + bm - 1) / bm;
      if (rest < b) {
        r = Item{e, lo + rest * bm, min(hi - lo - rest * bm, bm)};
        break;
      }
      rest -= b;
    }
  }
  r.e = __builtin_amdgcn_readlane(r.e, src);
  r.p0 = __builtin_amdgcn_readlane(r.p0, src);
  r.rows = __builtin_amdgcn_readlane(r.rows, src);
  return r;
}

__device__ __forceinline__ void store_out(const W4Args& a, int64_t at, float v) {
  if (a.out_dtype == BSMM_BF16) static_cast<uint16_t*>(a.out)[at] = (uint16_t)bf16_bits(v);
  else static_cast<float*>(a.out)[at] = v;
}

// One workgroup: 16 * MT rows by 16 * NT columns, NW waves that split K in
// chunks of 128 and are added through LDS in wave order.
template <bool XF32, int G, int MT, int NT, int NW, bool ROUTED>
__global__ void __launch_bounds__(NW * 64) w4_rows_kernel(W4Args a, int ntn) {
  constexpr int BM = 16 * MT, BN = 16 * NT;
  extern __shared__ float red[];        // [NW][MT * NT][4][64]
  const int tn = blockIdx.x % ntn, item = blockIdx.x / ntn;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int c16 = lane & 15, quad = lane >> 4;
  Item it;
  if (ROUTED) {
    it = find_item(a.offsets, a.E, a.S, BM, item);
    // slots of no expert: zero rows, shared out over the items
    const int used = min(max(a.offsets[a.E], 0), a.S);
    const int items = gridDim.x / ntn;
    for (int p = used + item; p < a.S; p += items) {
      const int slot = a.order[p];
      if (slot < 0 || slot >= a.S) continue;
      for (int i = threadIdx.x; i < BN; i += NW * 64)
        if (tn * BN + i < a.N) store_out(a, slot * a.ldo + tn * BN + i, 0.0f);
    }
    if (it.rows == 0) return;
  } else {
    it = Item{0, item * BM, min(a.S - item * BM, BM)};
  }
  // rows past the item's end repeat its first row: their results are not
  // stored, and a row of the product depends on its own row of x alone
  int64_t xoff[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int m = 16 * i + c16;
    int64_t row = it.p0 + (m < it.rows ? m : 0);
    if (ROUTED) row = min(max(a.order[row] / a.x_div, 0), a.R - 1);
    xoff[i] = row * a.ldx;
  }
  const uint8_t* wp[NT];
  int64_t sp[NT];
  const uint8_t* zp[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int64_t n = min(tn * BN + 16 * j + c16, a.N - 1);
    wp[j] = a.w + it.e * a.w_se + n * a.ldw;
    sp[j] = it.e * a.s_se + n * a.s_n;
    zp[j] = a.zero ? a.zero + it.e * a.z_se + n * a.z_n : nullptr;
  }
  const int K = a.K, KG = K / G;
  const int chunks = (K + 127) / 128;
  f32x4 acc[MT][NT] = {};

  struct Chunk {
    u32x4 w[NT];
    X8<XF32> x[MT][4];
    float s[NT], z[NT];
  };
  // chunk of this wave's step: pairs of chunks (one 128-byte line of codes)
  auto chunk_of = [&](int s) { return ((s >> 1) * NW + wave) * 2 + (s & 1); };
  auto load = [&](Chunk& b, int c) {
    const int kc = c * 128;
    const int wo = kc / 2 + quad * 16 < K / 2 ? kc / 2 + quad * 16 : 0;
    // the group whose scale this lane brings: its own for G = 128, else
    // the one of its quad's 32-element block
    int g = G == 128 ? c : G == 64 ? 2 * c + (quad >> 1) : 4 * c + quad;
    g = min(g, KG - 1);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      b.w[j] = *reinterpret_cast<const u32x4*>(wp[j] + wo);
      b.s[j] = a.s_bf16 ? __uint_as_float(
                              (uint32_t)static_cast<const uint16_t*>(a.scale)[sp[j] + g] << 16)
                        : static_cast<const float*>(a.scale)[sp[j] + g];
      b.z[j] = 16.0f + (zp[j] ? (float)zp[j][g] : 8.0f);
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        // G = 128: a lane's 16 code bytes are 32 consecutive k; else step t
        // takes the 32-element block t, 8 elements to a quad
        int k = G == 128 ? kc + quad * 32 + t * 8 : kc + t * 32 + quad * 8;
        if (k >= K) k = quad * 8;
        b.x[i][t] = load_x<XF32>(a.x, xoff[i] + k);
      }
  };
  auto compute = [&](Chunk& b, int c) {
    const u32x4 ones = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
    f32x4 d[MT][NT], e[MT];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      if (G != 128 && c * 128 + t * 32 >= K) break;      // uniform
      if (t * 32 % G == 0) {
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          e[i] = f32x4{};
#pragma unroll
          for (int j = 0; j < NT; ++j) d[i][j] = f32x4{};
        }
      }
      u32x4 wb[NT];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        uint32_t w = b.w[j][t];
        if (G != 128) {
          // dword `quad` of block t, which quad t loaded
          const int src = (t << 4) | c16;
          const uint32_t w0 = __shfl(b.w[j].x, src), w1 = __shfl(b.w[j].y, src);
          const uint32_t w2 = __shfl(b.w[j].z, src), w3 = __shfl(b.w[j].w, src);
          w = quad == 0 ? w0 : quad == 1 ? w1 : quad == 2 ? w2 : w3;
        }
        wb[j] = unpack(w);
      }
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const Parts<XF32> p = parts(b.x[i][t]);
#pragma unroll
        for (int h = (XF32 ? 3 : 1) - 1; h >= 0; --h) {
          e[i] = mfma(p.p[h], ones, e[i]);
#pragma unroll
          for (int j = 0; j < NT; ++j) d[i][j] = mfma(p.p[h], wb[j], d[i][j]);
        }
      }
      if ((t + 1) * 32 % G == 0) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          float s = b.s[j], z = b.z[j];
          if (G != 128) {
            const int src = (G == 64 ? (t >> 1) << 5 : t << 4) | c16;
            s = __shfl(s, src);
            z = __shfl(z, src);
          }
#pragma unroll
          for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r)
              acc[i][j][r] = __builtin_fmaf(s, __builtin_fmaf(-z, e[i][r], d[i][j][r]),
                                            acc[i][j][r]);
        }
      }
    }
  };

  Chunk b0, b1;
  int s = 0;
  if (chunk_of(0) < chunks) load(b0, chunk_of(0));
  while (chunk_of(s) < chunks) {
    if (chunk_of(s + 1) < chunks) load(b1, chunk_of(s + 1));
    compute(b0, chunk_of(s));
    if (chunk_of(s + 1) >= chunks) break;
    if (chunk_of(s + 2) < chunks) load(b0, chunk_of(s + 2));
    compute(b1, chunk_of(s + 1));
    s += 2;
  }

#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        red[((wave * MT * NT + i * NT + j) * 4 + r) * 64 + lane] = acc[i][j][r];
  __syncthreads();
  for (int i = threadIdx.x; i < BM * BN; i += NW * 64) {
    const int m = i / BN, n = i % BN;
    if (m >= it.rows || tn * BN + n >= a.N) continue;
    const int at = (((m >> 4) * NT + (n >> 4)) * 4 + (m & 3)) * 64 + ((m & 15) >> 2) * 16 + (n & 15);
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; ++w) v += red[w * MT * NT * 256 + at];
    int64_t row = it.p0 + m;
    if (ROUTED) {
      row = a.order[row];
      if (row < 0 || row >= a.S) continue;
      if (a.row_scale) v *= a.row_scale[row];
    }
    store_out(a, row * a.ldo + tn * BN + n, v);
  }
}

template <bool XF32, int G, int MT, int NT, int NW>
void launch_rows(const W4Args& a, hipStream_t st) {
  constexpr int BM = 16 * MT, BN = 16 * NT;
  const int ntn = (a.N + BN - 1) / BN;
  const size_t lds = (size_t)NW * MT * NT * 1024;
  if (a.offsets) {
    const int64_t items = ((int64_t)a.S + (int64_t)(a.E < a.S ? a.E : a.S) * (BM - 1)) / BM;
    hipLaunchKernelGGL((w4_rows_kernel<XF32, G, MT, NT, NW, true>), dim3((unsigned)(items * ntn)),
                       dim3(NW * 64), lds, st, a, ntn);
  } else {
    const int64_t items = ((int64_t)a.S + BM - 1) / BM;
    hipLaunchKernelGGL((w4_rows_kernel<XF32, G, MT, NT, NW, false>),
                       dim3((unsigned)(items * ntn)), dim3(NW * 64), lds, st, a, ntn);
  }
}

template <bool XF32, int G>
void launch_group(const W4Args& a, hipStream_t st) {
  const int64_t rows = a.offsets ? (a.S + a.E - 1) / a.E : a.S;
  if (rows <= 16) launch_rows<XF32, G, 1, 1, 8>(a, st);
  else launch_rows<XF32, G, 2, 1, 8>(a, st);
}

template <bool XF32>
void launch_x(const W4Args& a, hipStream_t st) {
  if (a.group == 32) launch_group<XF32, 32>(a, st);
  else if (a.group == 64) launch_group<XF32, 64>(a, st);
  else launch_group<XF32, 128>(a, st);
}

}  // namespace

int launch_w4(const W4Args& a, void* stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (a.x_dtype == BSMM_F32) launch_x<true>(a, st);
  else launch_x<false>(a, st);
  return hipGetLastError() == hipSuccess ? 0 : 1;
}

}  // namespace bsmm
