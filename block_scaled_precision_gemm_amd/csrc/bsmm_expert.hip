// Products of routed rows with their experts' bf16 or fp32 weights, and the
// weights' gradient (gfx950).
//
//   mm      out[s, n]   = r[s] * sum_k x[s / d, k] * w[e, n, k]     slots s of expert e
//   wgrad   dw[e, n, k] = sum_s dy[s / dy_d, n] * x[s / x_d, k]     over those slots
//
// The products of bf16 are exact in the matrix instruction, those of fp32 run
// on the fp32 one; sums are fp32 and rounded once, at the output.  The int8
// codes of a checkpoint times their power of two have at most 7 bits and so
// are exact in bf16 as in fp32.

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "bsmm_internal.h"
#include "bsmm_routed.h"

namespace bsmm {
namespace {

// A tile of an operand in LDS is 128 bytes of the contraction (kStep
// elements) for 128 rows or columns of the output.  Two layouts, as the
// operand lies in memory:
//   along   rows of 128 bytes, the contraction inside a row
//   across  a row for every element of the contraction, 128 elements long
// The 16-byte units of a row are exchanged by XOR so that a fragment's reads
// spread over the banks.
template <typename T> struct Elem;
template <> struct Elem<uint16_t> {       // bf16 bits
  static constexpr int U = 8, STEP = 64;
};
template <> struct Elem<float> {
  static constexpr int U = 4, STEP = 32;
};
constexpr int kTile = 128;                      // rows and columns of a tile
constexpr int kTileBytes = kTile * 128;

template <typename T>
__device__ __forceinline__ int across_off(int k, int u) {
  if constexpr (sizeof(T) == 2) return k * 256 + ((u ^ ((k & 3) << 2 | ((k >> 3) & 1) << 1)) << 4);
  else return k * 512 + ((u ^ ((k >> 2) & 1) << 3) << 4);
}

// A unit's worth of elements at p, `left` of them inside the operand (the
// others 0).  VEC: p is 16-byte aligned.
template <typename T, bool VEC>
__device__ __forceinline__ u32x4 fetch(const T* p, int left) {
  constexpr int U = Elem<T>::U;
  if (VEC && left >= U) return *reinterpret_cast<const u32x4*>(p);
  T e[U];
#pragma unroll
  for (int i = 0; i < U; ++i) e[i] = i < left ? p[i] : T(0);
  u32x4 v;
  __builtin_memcpy(&v, e, 16);
  return v;
}

// The same from 8-bit codes and their block's exponent byte.
template <typename T>
__device__ __forceinline__ u32x4 fetch_codes(const int8_t* p, const uint8_t* scale, int left) {
  constexpr int U = Elem<T>::U;
  if (left <= 0) return u32x4{0, 0, 0, 0};          // whole blocks: all or nothing
  uint32_t c[2];
  __builtin_memcpy(c, p, U);
  // 2^(byte - 133), 255 a NaN
  const int b = *scale;
  const float s = b == 255 ? __builtin_nanf("") : __builtin_ldexpf(1.0f, b - 133);
  u32x4 v;
  if constexpr (U == 8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = c[i >> 1] >> (16 * (i & 1));
      const float lo = (float)(int8_t)(w & 0xFF) * s, hi = (float)(int8_t)((w >> 8) & 0xFF) * s;
      v[i] = __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __float_as_uint((float)(int8_t)((c[0] >> (8 * i)) & 0xFF) * s);
  }
  return v;
}

// Fragments of turn t (a quarter of the tile's 128 bytes) for 32 rows or
// columns from c0.  A lane holds 16 bytes of one row: of bf16 the 8 elements
// 16 t + 8 half .. of the contraction, of fp32 the 4 elements 8 t + 4 half ..
__device__ __forceinline__ u32x4 frag_along(const uint8_t* tile, int c0, int t) {
  const int lane = threadIdx.x & 63;
  return *reinterpret_cast<const u32x4*>(tile + lds_off(c0 + (lane & 31), 2 * t + (lane >> 5)));
}
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) i16x4* lds_i16x4_t;
// 4 x 16 elements of 16 lanes' 8 bytes each (a row to 4 lanes), transposed:
// the lane gets its column
__device__ __forceinline__ uint2 read_transposed(const uint8_t* p) {
  return __builtin_bit_cast(
      uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t)(uintptr_t)(uint32_t)(uintptr_t)p));
}
template <typename T>
__device__ __forceinline__ u32x4 frag_across(const uint8_t* tile, int c0, int t) {
  const int lane = threadIdx.x & 63, half = lane >> 5;
  if constexpr (sizeof(T) == 2) {
    const int c = c0 + (lane & 16) + (lane & 3) * 4, k = 16 * t + 8 * half + ((lane >> 2) & 3);
    const uint2 a = read_transposed(tile + across_off<T>(k, c >> 3) + (c & 7) * 2);
    const uint2 b = read_transposed(tile + across_off<T>(k + 4, c >> 3) + (c & 7) * 2);
    return u32x4{a.x, a.y, b.x, b.y};
  } else {
    const int c = c0 + (lane & 31), k = 8 * t + 4 * half;
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = *reinterpret_cast<const uint32_t*>(tile + across_off<T>(k + i, c >> 2) + (c & 3) * 4);
    return v;
  }
}

template <typename T>
__device__ __forceinline__ f32x16 product(u32x4 a, u32x4 b, f32x16 c) {
  if constexpr (sizeof(T) == 2) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a[i]), __uint_as_float(b[i]), c, 0,
                                               0, 0);
    return c;
  }
}

// A wave's 64 x 64 of the tile's products over `steps` steps of the
// contraction; load(s) brings step s to the thread's registers, store(buffer)
// takes them to LDS.
template <typename T, bool A_ACROSS, bool B_ACROSS, typename Load, typename Store>
__device__ __forceinline__ void tile_products(uint8_t* smem, int steps, f32x16 (&acc)[2][2],
                                              const Load& load, const Store& store) {
  const int wave = threadIdx.x >> 6, wm = (wave >> 1) * 64, wn = (wave & 1) * 64;
  if (steps > 0) {
    load(0);
    store(smem);
  }
  __syncthreads();
  for (int s = 0; s < steps; ++s) {
    const uint8_t* at = smem + (s & 1) * 2 * kTileBytes;
    const uint8_t* bt = at + kTileBytes;
    if (s + 1 < steps) load(s + 1);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      u32x4 a[2], b[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        a[i] = A_ACROSS ? frag_across<T>(at, wm + 32 * i, t) : frag_along(at, wm + 32 * i, t);
        b[i] = B_ACROSS ? frag_across<T>(bt, wn + 32 * i, t) : frag_along(bt, wn + 32 * i, t);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = product<T>(a[i], b[j], acc[i][j]);
    }
    if (s + 1 < steps) store(smem + ((s + 1) & 1) * 2 * kTileBytes);
    __syncthreads();
  }
}

__device__ __forceinline__ void put(void* out, bsmm_dtype dt, int64_t at, float v) {
  if (dt == BSMM_BF16) static_cast<uint16_t*>(out)[at] = (uint16_t)bf16_bits(v);
  else static_cast<float*>(out)[at] = v;
}

// Row of the wave's block i that register r of a lane holds.
__device__ __forceinline__ int row_of(int i, int r) {
  return 32 * i + (r >> 2) * 8 + ((threadIdx.x >> 5) & 1) * 4 + (r & 3);
}

__device__ __forceinline__ int slot_at(const int32_t* order, int p) { return order ? order[p] : p; }

template <typename T, bool W_ACROSS, bool VEC>
__global__ void __launch_bounds__(256, 2) expert_mm_kernel(ExpertArgs a, int items, int ntn) {
  constexpr int U = Elem<T>::U, STEP = Elem<T>::STEP, UPR = kTile / U;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[4 * kTileBytes];
  int item, tn;
  tile_of(items, ntn, item, tn);
  const Item it = find_item(a.offsets, a.E, a.S, kTile, item);
  const int n0 = tn * kTile;
  // zero rows for the slots of no expert, shared out over the items
  const unsigned used = min(max(a.offsets[a.E], 0), a.S);
  for (unsigned p = used + item; p < (unsigned)a.S; p += items) {    // both below 2^31
    const int slot = slot_at(a.order, p);
    if (slot >= 0 && slot < a.S && (int)threadIdx.x < min(kTile, a.N - n0))
      put(a.out, a.out_dtype, slot * a.ldo + n0 + threadIdx.x, 0.0f);
  }
  if (it.rows == 0) return;

  const T* const x = static_cast<const T*>(a.x);
  const T* const w = static_cast<const T*>(a.w) + it.e * a.w_se;
  // the thread's four units of each tile
  const int u8 = threadIdx.x & 7;
  const T* xr[4];
  const T* wr[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = i * 32 + (threadIdx.x >> 3);
    const int s = slot_at(a.order, it.p0 + min(r, it.rows - 1));
    xr[i] = x + (int64_t)min(max(s / a.x_div, 0), a.R - 1) * a.ldx + u8 * U;
    if (!W_ACROSS) {
      wr[i] = w + (int64_t)min(n0 + r, a.N - 1) * a.ldw + u8 * U;
    } else {
      const int q = i * 256 + threadIdx.x;
      wr[i] = w + (int64_t)(q / UPR) * a.ldw + n0 + q % UPR * U;
    }
  }
  u32x4 va[4], vb[4];
  auto load = [&](int s) {
    const int k = s * STEP;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      va[i] = fetch<T, VEC>(xr[i] + k, a.K - k - u8 * U);
      if (!W_ACROSS) {
        vb[i] = fetch<T, VEC>(wr[i] + k, a.K - k - u8 * U);
      } else {
        const int q = i * 256 + threadIdx.x;
        vb[i] = fetch<T, VEC>(wr[i] + (int64_t)k * a.ldw,
                              k + q / UPR < a.K ? a.N - n0 - q % UPR * U : 0);
      }
    }
  };
  auto store = [&](uint8_t* to) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int q = i * 256 + threadIdx.x;
      *reinterpret_cast<u32x4*>(to + lds_off(q >> 3, q & 7)) = va[i];
      *reinterpret_cast<u32x4*>(to + kTileBytes + (W_ACROSS ? across_off<T>(q / UPR, q % UPR)
                                                            : lds_off(q >> 3, q & 7))) = vb[i];
    }
  };
  f32x16 acc[2][2] = {};
  tile_products<T, false, W_ACROSS>(smem, (int)(((unsigned)a.K + STEP - 1) / STEP), acc, load,
                                    store);

  const int wave = threadIdx.x >> 6, wm = (wave >> 1) * 64;
  const int col = n0 + (wave & 1) * 64 + (threadIdx.x & 31);
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int m = wm + row_of(i, r);
      if (m >= it.rows) continue;
      const int slot = slot_at(a.order, it.p0 + m);
      if (slot < 0 || slot >= a.S) continue;
      const float f = a.row_scale ? a.row_scale[slot] : 1.0f;
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (col + 32 * j < a.N)
          put(a.out, a.out_dtype, slot * a.ldo + col + 32 * j, acc[i][j][r] * f);
    }
}

// CODES: x is an 8-bit checkpoint.
template <typename T, bool CODES, bool VEC>
__global__ void __launch_bounds__(256, 2) expert_wgrad_kernel(WgradArgs a, int ntn, int ntk) {
  constexpr int U = Elem<T>::U, STEP = Elem<T>::STEP, UPR = kTile / U;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[4 * kTileBytes];
  int item, tk;
  tile_of(a.E * ntn, ntk, item, tk);
  const int e = item / ntn, n0 = item % ntn * kTile, k0 = tk * kTile;
  const int lo = min(max(a.offsets[e], 0), a.S), hi = min(max(a.offsets[e + 1], lo), a.S);

  u32x4 va[4], vb[4];
  auto load = [&](int s) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int q = i * 256 + threadIdx.x, u = q % UPR, p = lo + s * STEP + q / UPR;
      const int slot = p < hi ? slot_at(a.order, p) : -1;
      const bool in = slot >= 0 && slot < a.S;
      const int64_t ry = in ? slot / a.y_div : 0, rx = in ? slot / a.x_div : 0;
      va[i] = fetch<T, VEC>(static_cast<const T*>(a.dy) + ry * a.ldy + n0 + u * U,
                            in ? a.N - n0 - u * U : 0);
      const int c = k0 + u * U, left = in ? a.K - c : 0;
      if constexpr (CODES)
        vb[i] = fetch_codes<T>(static_cast<const int8_t*>(a.x) + rx * a.ldx + c,
                               a.x_scale + rx * a.s_r + c / 32, left);
      else
        vb[i] = fetch<T, VEC>(static_cast<const T*>(a.x) + rx * a.ldx + c, left);
    }
  };
  auto store = [&](uint8_t* to) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int q = i * 256 + threadIdx.x, at = across_off<T>(q / UPR, q % UPR);
      *reinterpret_cast<u32x4*>(to + at) = va[i];
      *reinterpret_cast<u32x4*>(to + kTileBytes + at) = vb[i];
    }
  };
  f32x16 acc[2][2] = {};
  tile_products<T, true, true>(smem, (int)(((unsigned)(hi - lo) + STEP - 1) / STEP), acc, load,
                               store);

  const int wave = threadIdx.x >> 6;
  const int row0 = n0 + (wave >> 1) * 64, col = k0 + (wave & 1) * 64 + (threadIdx.x & 31);
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int n = row0 + row_of(i, r);
      if (n >= a.N) continue;
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (col + 32 * j < a.K)
          put(a.dw, a.out_dtype, e * a.w_se + n * a.ldw + col + 32 * j, acc[i][j][r]);
    }
}

template <typename T>
bool vec_ok(const void* p, int64_t ld) {
  return (uintptr_t)p % 16 == 0 && ld % Elem<T>::U == 0;
}

template <typename T>
void launch_mm(const ExpertArgs& a, hipStream_t st) {
  const int64_t act = a.E < a.S ? a.E : a.S;
  const int items = (int)((a.S + act * (kTile - 1)) / kTile), ntn = (a.N + kTile - 1) / kTile;
  const dim3 grid((unsigned)(items * ntn)), block(256);
  const bool vec = vec_ok<T>(a.x, a.ldx) && vec_ok<T>(a.w, a.ldw) && a.w_se % Elem<T>::U == 0;
  if (a.w_across) {
    if (vec) hipLaunchKernelGGL((expert_mm_kernel<T, true, true>), grid, block, 0, st, a, items, ntn);
    else hipLaunchKernelGGL((expert_mm_kernel<T, true, false>), grid, block, 0, st, a, items, ntn);
  } else {
    if (vec) hipLaunchKernelGGL((expert_mm_kernel<T, false, true>), grid, block, 0, st, a, items, ntn);
    else hipLaunchKernelGGL((expert_mm_kernel<T, false, false>), grid, block, 0, st, a, items, ntn);
  }
}

template <typename T>
void launch_wgrad(const WgradArgs& a, hipStream_t st) {
  const int ntn = (a.N + kTile - 1) / kTile, ntk = (a.K + kTile - 1) / kTile;
  const dim3 grid((unsigned)((int64_t)a.E * ntn * ntk)), block(256);
  const bool yv = vec_ok<T>(a.dy, a.ldy);
  if (a.x_scale) {
    if (yv) hipLaunchKernelGGL((expert_wgrad_kernel<T, true, true>), grid, block, 0, st, a, ntn, ntk);
    else hipLaunchKernelGGL((expert_wgrad_kernel<T, true, false>), grid, block, 0, st, a, ntn, ntk);
  } else {
    if (yv && vec_ok<T>(a.x, a.ldx))
      hipLaunchKernelGGL((expert_wgrad_kernel<T, false, true>), grid, block, 0, st, a, ntn, ntk);
    else
      hipLaunchKernelGGL((expert_wgrad_kernel<T, false, false>), grid, block, 0, st, a, ntn, ntk);
  }
}

}  // namespace

int launch_expert_mm(const ExpertArgs& a, void* stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (a.dtype == BSMM_BF16) launch_mm<uint16_t>(a, st);
  else launch_mm<float>(a, st);
  return hipGetLastError() == hipSuccess ? 0 : 1;
}

int launch_expert_wgrad(const WgradArgs& a, void* stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (a.dtype == BSMM_BF16) launch_wgrad<uint16_t>(a, st);
  else launch_wgrad<float>(a, st);
  return hipGetLastError() == hipSuccess ? 0 : 1;
}

}  // namespace bsmm
