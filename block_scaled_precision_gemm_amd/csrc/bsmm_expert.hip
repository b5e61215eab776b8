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

#include "bsmm_check.h"
#include "bsmm_internal.h"
#include "bsmm_routed.h"

namespace bsmm {
namespace {

// A tile of an operand in LDS is 128 bytes of the contraction (STEP elements)
// for 64 MB rows or columns of the output.  Two layouts, as the operand lies
// in memory:
//   along   rows of 128 bytes, the contraction inside a row
//   across  a row for every element of the contraction, 64 MB elements long
// The 16-byte units of a row are exchanged by XOR so that a fragment's reads
// spread over the banks.
template <typename T> struct Elem;
template <> struct Elem<uint16_t> {       // bf16 bits
  static constexpr int U = 8, STEP = 64;
};
template <> struct Elem<float> {
  static constexpr int U = 4, STEP = 32;
};

// Byte offset of unit u of row k in an `across` tile.
template <typename T, int MB>
__device__ __forceinline__ int across_off(int k, int u) {
  constexpr int ROW = 64 * MB * sizeof(T), UNITS = ROW / 16;
  if constexpr (sizeof(T) == 2)
    return k * ROW + (((u ^ ((k & 3) << 2 | ((k >> 3) & 1) << 1)) & (UNITS - 1)) << 4);
  else
    return k * ROW + ((u ^ (((k >> 2) & 1) << 3)) << 4);
}

// A unit's worth of elements at p, `left` of them inside the operand (the
// others 0).  One load whatever the address: the hardware takes any that is
// aligned to the element.
template <typename T>
__device__ __forceinline__ u32x4 fetch(const T* p, int left) {
  constexpr int U = Elem<T>::U;
  u32x4 v = {0, 0, 0, 0};
  if (left >= U) {
    __builtin_memcpy(&v, p, 16);
  } else if (left > 0) {
    T e[U];
#pragma unroll
    for (int i = 0; i < U; ++i) e[i] = i < left ? p[i] : T(0);
    __builtin_memcpy(&v, e, 16);
  }
  return v;
}

// The same from 8-bit codes and their block's exponent byte, in two halves, so
// that nothing waits for the load before the values are wanted.
struct Codes {
  uint32_t c[2];
  int byte;
};
template <typename T>
__device__ __forceinline__ Codes fetch_codes(const int8_t* p, const uint8_t* scale, int left) {
  Codes v{{0, 0}, 127};
  if (left > 0) {                                   // whole blocks: all or nothing
    __builtin_memcpy(v.c, p, Elem<T>::U);
    v.byte = *scale;
  }
  return v;
}
template <typename T>
__device__ __forceinline__ u32x4 value_of(const Codes& q) {
  // 2^(byte - 133), 255 a NaN
  const float s = q.byte == 255 ? __builtin_nanf("") : __builtin_ldexpf(1.0f, q.byte - 133);
  u32x4 v;
  if constexpr (Elem<T>::U == 8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = q.c[i >> 1] >> (16 * (i & 1));
      const float lo = (float)(int8_t)(w & 0xFF) * s, hi = (float)(int8_t)((w >> 8) & 0xFF) * s;
      v[i] = __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = __float_as_uint((float)(int8_t)((q.c[0] >> (8 * i)) & 0xFF) * s);
  }
  return v;
}
template <typename T> __device__ __forceinline__ u32x4 value_of(u32x4 v) { return v; }

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
      uint2,
      __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t)(uintptr_t)(uint32_t)(uintptr_t)p));
}
template <typename T, int MB>
__device__ __forceinline__ u32x4 frag_across(const uint8_t* tile, int c0, int t) {
  const int lane = threadIdx.x & 63, half = lane >> 5;
  if constexpr (sizeof(T) == 2) {
    const int c = c0 + (lane & 16) + (lane & 3) * 4, k = 16 * t + 8 * half + ((lane >> 2) & 3);
    const uint2 a = read_transposed(tile + across_off<T, MB>(k, c >> 3) + (c & 7) * 2);
    const uint2 b = read_transposed(tile + across_off<T, MB>(k + 4, c >> 3) + (c & 7) * 2);
    return u32x4{a.x, a.y, b.x, b.y};
  } else {
    const int c = c0 + (lane & 31), k = 8 * t + 4 * half;
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = *reinterpret_cast<const uint32_t*>(tile + across_off<T, MB>(k + i, c >> 2) +
                                                (c & 3) * 4);
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

// Steps that are on their way in registers while one is multiplied (1000 tokens
// x 4 of 32 experts of 1024 x 1024 fp32: 128 us with one, 116 with two, 118
// with three; 4000 x 2 of 8 of 1001 x 2051 bf16: 101, 97, 94, but its weight
// gradient 124, 120, 127)
constexpr int kAhead = 2;

// A wave's 32 MB x 32 MB of the tile's products over `steps` steps of the
// contraction; load(d, s) brings step s to the thread's registers of set d,
// store(d, buffer) takes them to LDS.
template <typename T, int MB, bool A_ACROSS, bool B_ACROSS, typename Load, typename Store>
__device__ __forceinline__ void tile_products(uint8_t* smem, int steps, f32x16 (&acc)[MB][MB],
                                              const Load& load, const Store& store) {
  constexpr int BYTES = 64 * MB * 128, D = kAhead;
  const int wave = threadIdx.x >> 6, wm = (wave >> 1) * 32 * MB, wn = (wave & 1) * 32 * MB;
#pragma unroll
  for (int d = 0; d < D; ++d)
    if (d < steps) load(d, d);
  if (steps > 0) store(0, smem);
  if (D < steps) load(0, D);
  __syncthreads();
  for (int s0 = 0; s0 < steps; s0 += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      const int s = s0 + d;
      if (s >= steps) break;
      const uint8_t* at = smem + (s & 1) * 2 * BYTES;
      const uint8_t* bt = at + BYTES;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        u32x4 a[MB], b[MB];
#pragma unroll
        for (int i = 0; i < MB; ++i) {
          a[i] = A_ACROSS ? frag_across<T, MB>(at, wm + 32 * i, t) : frag_along(at, wm + 32 * i, t);
          b[i] = B_ACROSS ? frag_across<T, MB>(bt, wn + 32 * i, t) : frag_along(bt, wn + 32 * i, t);
        }
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
          for (int j = 0; j < MB; ++j) acc[i][j] = product<T>(a[i], b[j], acc[i][j]);
      }
      const int e = d + 1 == D ? 0 : d + 1;          // step s + 1's set
      if (s + 1 < steps) store(e, smem + ((s + 1) & 1) * 2 * BYTES);
      if (s + 1 + D < steps) load(e, s + 1 + D);
      __syncthreads();
    }
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

// n / d for 0 <= n < 2^31 (Granlund and Montgomery, "Division by invariant
// integers using multiplication", 1994): (mulhi(m, n) + n) >> l
struct Divisor { uint32_t m; int l; };
__device__ __forceinline__ uint32_t divide(uint32_t n, Divisor d) {
  return (__umulhi(d.m, n) + n) >> d.l;
}

// The slots (-1: not stored) and scales of an item's rows.
__device__ __forceinline__ void item_slots(const ExpertArgs& a, const Item& it, int rows,
                                           int* slots, float* scales) {
  const int r = threadIdx.x;
  if (r >= rows) return;
  const int s = r < it.rows ? slot_at(a.order, it.p0 + r) : -1;
  const bool in = s >= 0 && s < a.S;
  slots[r] = in ? s : -1;
  scales[r] = in && a.row_scale ? a.row_scale[s] : 1.0f;
}

// Zero rows for the slots of no expert in columns [n0, n0 + cols), shared out
// over the items, a wave to a row.
__device__ __forceinline__ void zero_rows(const ExpertArgs& a, int n0, int cols, int item,
                                          int items) {
  const int waves = blockDim.x >> 6;
  const unsigned used = min(max(a.offsets[a.E], 0), a.S);
  for (unsigned p = used + item * waves + (threadIdx.x >> 6); p < (unsigned)a.S;
       p += items * waves) {                                         // all below 2^31
    const int slot = slot_at(a.order, p);
    if (slot < 0 || slot >= a.S) continue;
    for (int c = threadIdx.x & 63; c < cols; c += 64)
      if (n0 + c < a.N) put(a.out, a.out_dtype, slot * a.ldo + n0 + c, 0.0f);
  }
}

// A workgroup's tile of `rows` x cols of them (false: none).  Tiles are ordered
// in groups of `group` rows by all columns, and runs of `run` of them dealt out
// to the XCDs (hardware ids go round robin over 8): the workgroups that an XCD
// holds at a time share operands in its L2, and experts that have many rows,
// or items that do not exist, fall to all XCDs alike.
__device__ __forceinline__ bool deal_tile(int rows, int cols, int run, int group, int& row,
                                          int& col) {
  const int xcd = blockIdx.x & 7, local = blockIdx.x >> 3, turn = local / run;
  const int id = (turn * 8 + xcd) * run + (local - turn * run);
  if ((unsigned)id >= (unsigned)(rows * cols)) return false;
  const int width = group * cols, g = id / width, first = group * g, n = min(rows - first, group);
  const int in = id - g * width;
  row = first + in % n;
  col = in / n;
  return true;
}

// A call whose tiles are few is cut along the contraction too: `splits` parts,
// fp32, one behind the other in the workspace (the launch's out), which
// reduce_parts adds in order.  These find the part of an item and its range,
// and point the output at it.
__device__ __forceinline__ void part_of(ExpertArgs& a, int items, int splits, int step, int& item,
                                        int& s0, int& s1) {
  const int steps = (int)(((unsigned)a.K + step - 1) / step);
  const int part = splits > 1 ? item / items : 0, per = (steps + splits - 1) / splits;
  item -= part * items;
  s0 = min(part * per, steps);
  s1 = min(s0 + per, steps);
  if (splits > 1) a.out = static_cast<float*>(a.out) + (int64_t)part * a.S * a.N;
}
__device__ __forceinline__ int run_of(WgradArgs& a, int ntn, int splits, int step, int& item,
                                      int& lo, int& hi) {
  const int part = splits > 1 ? item / (a.E * ntn) : 0;
  item -= part * a.E * ntn;
  const int e = item / ntn;
  lo = min(max(a.offsets[e], 0), a.S);
  hi = min(max(a.offsets[e + 1], lo), a.S);
  if (splits > 1) {
    const int per = ((hi - lo + step - 1) / step + splits - 1) / splits;    // steps of a part
    lo = (int)min((int64_t)lo + (int64_t)part * per * step, (int64_t)hi);
    hi = (int)min((int64_t)lo + (int64_t)per * step, (int64_t)hi);
    a.dw = static_cast<float*>(a.dw) + (int64_t)part * a.E * a.N * a.K;
  }
  return e;
}

// out(r, c) at out[(r / inner) * outer_ld + (r % inner) * ld + c] = the sum of
// the parts' [rows, cols].  Bound by its launch and the parts' bytes, which the
// plans count (bsmm_expert_api.cpp, best_split).
__global__ void __launch_bounds__(256) reduce_parts(const float* __restrict__ parts, int splits,
                                                    void* out, bsmm_dtype dt, int64_t rows,
                                                    int cols, int64_t inner, int64_t outer_ld,
                                                    int64_t ld) {
  const int64_t n = rows * cols;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int64_t r = n <= 0x7FFFFFFF ? (unsigned)i / (unsigned)cols : i / cols;
    const int64_t o = n <= 0x7FFFFFFF ? (unsigned)r / (unsigned)inner : r / inner;
    float v = 0.0f;
    for (int s = 0; s < splits; ++s) v += parts[s * n + i];
    put(out, dt, o * outer_ld + (r - o * inner) * ld + (i - r * cols), v);
  }
}

// ---------------------------------------------------------------------------
// Any type, alignment and size: tiles of 64 x 64 (four waves of 32 x 32; 128 x
// 128 and 64 x 64 in gradients of many tiles, MB = 2), both operands through
// registers into two slots of LDS, in the layout they have in memory; bf16 that
// lies across is transposed by the LDS read.  fp32 runs at the fp32 matrix
// instruction's rate, a sixteenth of bf16's, which bounds it where there are
// enough tiles (900 tokens x 4 of 16 experts of 1024 x 2048: 165 us, 92 of the
// 151 TFLOP/s of a large product).  Few tiles are bound by latency (333 x 2 of 6
// of 1001 x 515: 22 us, its weight gradient 17).
// ---------------------------------------------------------------------------
template <typename T, bool W_ACROSS>
__global__ void __launch_bounds__(256, 2) expert_mm_kernel(ExpertArgs a, int items, int ntn,
                                                           int splits, int run) {
  constexpr int U = Elem<T>::U, STEP = Elem<T>::STEP, TILE = 64, BYTES = TILE * 128;
  constexpr int UPR = TILE / U, NU = 2;               // units of an across row, of a thread
  __shared__ __attribute__((aligned(1024))) uint8_t smem[4 * BYTES];
  __shared__ int slots[TILE];
  __shared__ float scales[TILE];
  int item, tn, s0, s1;
  if (!deal_tile(items * splits, ntn, run, 4, item, tn)) return;
  part_of(a, items, splits, STEP, item, s0, s1);
  const Item it = find_item(a.offsets, a.E, a.S, TILE, item);
  const int n0 = tn * TILE;
  zero_rows(a, n0, TILE, item, items);
  if (it.rows == 0) return;
  item_slots(a, it, TILE, slots, scales);
  __syncthreads();

  const T* const x = static_cast<const T*>(a.x);
  const T* const w = static_cast<const T*>(a.w) + it.e * a.w_se;
  // the thread's units of each tile
  const int u8 = threadIdx.x & 7;
  const T* xr[NU];
  const T* wr[NU];
#pragma unroll
  for (int i = 0; i < NU; ++i) {
    const int r = i * 32 + (threadIdx.x >> 3);
    const int s = max(slots[min(r, it.rows - 1)], 0);
    xr[i] = x + (int64_t)min(s / a.x_div, a.R - 1) * a.ldx + u8 * U;
    if (!W_ACROSS) {
      wr[i] = w + (int64_t)min(n0 + r, a.N - 1) * a.ldw + u8 * U;
    } else {
      const int q = i * 256 + threadIdx.x;
      wr[i] = w + (int64_t)(q / UPR) * a.ldw + n0 + q % UPR * U;
    }
  }
  u32x4 va[kAhead][NU], vb[kAhead][NU];
  auto load = [&](int d, int s) {
    const int k = (s0 + s) * STEP;
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      va[d][i] = fetch<T>(xr[i] + k, a.K - k - u8 * U);
      if (!W_ACROSS) {
        vb[d][i] = fetch<T>(wr[i] + k, a.K - k - u8 * U);
      } else {
        const int q = i * 256 + threadIdx.x;
        vb[d][i] = fetch<T>(wr[i] + (int64_t)k * a.ldw,
                            k + q / UPR < a.K ? a.N - n0 - q % UPR * U : 0);
      }
    }
  };
  auto store = [&](int d, uint8_t* to) {
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      const int q = i * 256 + threadIdx.x;
      *reinterpret_cast<u32x4*>(to + lds_off(q >> 3, q & 7)) = va[d][i];
      *reinterpret_cast<u32x4*>(to + BYTES + (W_ACROSS ? across_off<T, 1>(q / UPR, q % UPR)
                                                       : lds_off(q >> 3, q & 7))) = vb[d][i];
    }
  };
  f32x16 acc[1][1] = {};
  tile_products<T, 1, false, W_ACROSS>(smem, s1 - s0, acc, load, store);

  const int wave = threadIdx.x >> 6, wm = (wave >> 1) * 32;
  const int col = n0 + (wave & 1) * 32 + (threadIdx.x & 31);
  if (col >= a.N) return;
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const int m = wm + row_of(0, r), slot = slots[m];
    if (slot >= 0) put(a.out, a.out_dtype, slot * a.ldo + col, acc[0][0][r] * scales[m]);
  }
}

// CODES: x is an 8-bit checkpoint.
template <typename T, int MB, bool CODES>
__global__ void __launch_bounds__(256, 2) expert_wgrad_kernel(WgradArgs a, int ntn, int ntk,
                                                              int splits, int run, Divisor yd,
                                                              Divisor xd) {
  constexpr int U = Elem<T>::U, STEP = Elem<T>::STEP, TILE = 64 * MB, BYTES = TILE * 128;
  constexpr int UPR = TILE / U, NU = 2 * MB;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[4 * BYTES];
  int item, tk, lo, hi;
  if (!deal_tile(splits * a.E * ntn, ntk, run, 1, item, tk)) return;
  const int e = run_of(a, ntn, splits, STEP, item, lo, hi);
  const int n0 = item % ntn * TILE, k0 = tk * TILE;

  // the thread's units are the same columns of rows 256 / UPR apart
  const int u = threadIdx.x % UPR, row = threadIdx.x / UPR;
  const int cy = n0 + u * U, cx = k0 + u * U;
  constexpr int D = kAhead;
  u32x4 va[D][NU];
  std::conditional_t<CODES, Codes, u32x4> vb[D][NU];
  int next[D][NU];                      // the slots of a set's next rows
  auto slots_of = [&](int d, int s) {
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      const int64_t p = lo + (int64_t)s * STEP + i * (256 / UPR) + row;
      next[d][i] = p < hi ? slot_at(a.order, (int)p) : -1;
    }
  };
#pragma unroll
  for (int d = 0; d < D; ++d) slots_of(d, d);
  auto load = [&](int d, int s) {
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      const int slot = next[d][i];
      const bool in = slot >= 0 && slot < a.S;
      const int64_t ry = in ? divide(slot, yd) : 0, rx = in ? divide(slot, xd) : 0;
      va[d][i] = fetch<T>(static_cast<const T*>(a.dy) + ry * a.ldy + cy, in ? a.N - cy : 0);
      if constexpr (CODES)
        vb[d][i] = fetch_codes<T>(static_cast<const int8_t*>(a.x) + rx * a.ldx + cx,
                                  a.x_scale + rx * a.s_r + cx / 32, in ? a.K - cx : 0);
      else
        vb[d][i] = fetch<T>(static_cast<const T*>(a.x) + rx * a.ldx + cx, in ? a.K - cx : 0);
    }
    slots_of(d, s + D);
  };
  auto store = [&](int d, uint8_t* to) {
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      const int at = across_off<T, MB>(i * (256 / UPR) + row, u);
      *reinterpret_cast<u32x4*>(to + at) = va[d][i];
      *reinterpret_cast<u32x4*>(to + BYTES + at) = value_of<T>(vb[d][i]);
    }
  };
  f32x16 acc[MB][MB] = {};
  tile_products<T, MB, true, true>(smem, (int)(((unsigned)(hi - lo) + STEP - 1) / STEP), acc, load,
                                   store);

  const int wave = threadIdx.x >> 6;
  const int row0 = n0 + (wave >> 1) * 32 * MB;
  const int col = k0 + (wave & 1) * 32 * MB + (threadIdx.x & 31);
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int n = row0 + row_of(i, r);
      if (n >= a.N) continue;
#pragma unroll
      for (int j = 0; j < MB; ++j)
        if (col + 32 * j < a.K)
          put(a.dw, a.out_dtype, e * a.w_se + n * a.ldw + col + 32 * j, acc[i][j][r]);
    }
}

// ---------------------------------------------------------------------------
// bf16: tiles of BM = 64 MI rows by 256 columns, eight waves
// of 32 MI x 64 (MI x 2 blocks of 32 x 32 x 16 instructions), the contraction
// in steps of 64.
//
// Both tiles stand in LDS as rows of 128 bytes with the contraction inside.
// Operands that lie in memory that way go global -> LDS directly, two or three
// steps ahead: the slots take all 160 KB.  (Not with rows that are not 16-byte
// aligned: 1000 tokens x 2 of 8 experts of 2048 x 2000 take 36 us, x 2001,
// through registers, 46.)  The other kind goes through registers: a wave has 8
// neighbouring elements of the contraction (rows in memory) and a lane 4
// columns, which it transposes with 16 byte permutations and writes as 4 x 16
// bytes, the loads a step ahead.  (The transposing LDS read would spare that,
// but the compiler waits for every direct load in flight before one, and before
// an LDS write, so that a tile that needs one takes the other operand through
// registers too.)
//
// The source order is the schedule: a turn's fragments are read during the
// turn before, and the barrier stands before the last turn, whose products
// then cover the first fragments of the next step.  After it nobody reads the
// step's slot any more, and the direct loads of the step that gets it go out.
//
// The matrix cores bound long products: 8192^3 812 us (1354 TFLOP/s; the
// library's rate for it is 1384), the input's gradient 957 us (1149: the
// transposition takes turns of the vector unit and of LDS), the weights'
// gradient 1010 us (1089).  A step of 256 rows takes 1.48, 1.68 and 1.7 us; a
// tile 9.5 us besides, its first loads and its stores, 18 with fp32 results.
// Experts' weights from HBM bound few rows (64 tokens x 8 of 32 of 2048 x 4096,
// 537 MB: 92 us), and between the two the tiles that experts leave partly empty
// (4096 x 8 of 64: 568 us, 968 TFLOP/s).  Slower: four waves of 128 x 128, two
// workgroups a CU of 128 x 256 and steps of 32, groups of waves a turn apart,
// workgroups that take tile after tile, full items first.
// ---------------------------------------------------------------------------
constexpr int kWide = 256;                      // columns of a tile
__device__ const uint32_t kZeros[128] = {};     // a row of zeros
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
// in memory, aligned to its elements alone: the instructions take any such
// address, and at the same rate
typedef unsigned u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef unsigned u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
// a load from global memory, whatever the pointer was chosen from
template <typename V>
__device__ __forceinline__ V load_global(const void* p) {
  return *(const __attribute__((address_space(1))) V*)(uintptr_t)p;
}

// Unit c of row r of a tile that is written transposed: a write's 64 rows r =
// 4 lane + j and a read's 32 neighbouring rows both spread over the 8 units.
__device__ __forceinline__ int turned_off(int r, int c) {
  return (r << 7) + ((c ^ ((r >> 2) & 7) ^ ((r & 3) << 1)) << 4);
}

template <int MI> struct Wide {
  static constexpr int BM = 64 * MI, ROWS = 32 * MI;   // of the tile, of a wave
  static constexpr int A = BM * 128, B = kWide * 128;  // bytes of a step's tiles
  // slots of the rows' and the columns' tiles where loads are direct (through
  // registers 2 each): the weights come from HBM, so they get three
  static constexpr int DA = MI > 2 ? 2 : 3, DB = 3;
};
constexpr int kWideBytes = 2 * Wide<4>::A + 3 * Wide<4>::B;      // all of the CU's 160 KB
constexpr int kWidePitch = 64 * 4 + 16;         // of a row of results in LDS
constexpr int kWideStage = 8 * 32 * kWidePitch; // the waves' results; the rows' slots follow

__device__ __forceinline__ void lds_done() {
  __builtin_amdgcn_s_waitcnt(0xC07F);           // lgkmcnt(0), in the compiler's count too
}

// 8 rows x 4 columns on their way to an operand's tile
struct Turn { u32x2 row[8]; };
// A lane's 4 columns are columns 4 lane .. of a tile that begins at column c0
// of n (>= 4), and are loaded 8 bytes at a time from the last 4 of n at most:
// where n % 4 != 0 the lane that reaches past the end moves its columns back
// down.  (Those of the lanes behind it are not stored.)
struct Columns {
  int first;                             // of the lanes' offsets `at`, in bytes
  uint32_t at;
  int down;                              // bits, 0 in most lanes
  bool odd;                              // whether any lane of the tile has some
  __device__ __forceinline__ Columns(int c0, int n, int lane)
      : first(min(c0, n - 4)), at((uint32_t)min(4 * lane, n - 4 - first) * 2),
        odd(n % 4 != 0 && c0 + 256 > n) {
    down = 16 * min(max(c0 + 4 * lane - first - (int)at / 2, 0), 3);
  }
  __device__ __forceinline__ void place(Turn& v) const {
    if (!odd) return;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v.row[i] = __builtin_bit_cast(u32x2, __builtin_bit_cast(uint64_t, v.row[i]) >> down);
  }
};
// column c of them
__device__ __forceinline__ void put_turned(const Turn& v, uint8_t* tile, int octet, int c) {
  u32x4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o[i] = __builtin_amdgcn_perm(v.row[2 * i + 1][c >> 1], v.row[2 * i][c >> 1],
                                 c & 1 ? 0x07060302u : 0x05040100u);
  *reinterpret_cast<u32x4*>(tile + turned_off(4 * (threadIdx.x & 63) + c, octet)) = o;
}

// The products of one tile.  DIRECT: ops.direct_a(last, s, slot, i) and
// direct_b issue load i of a wave's MI and 4 direct loads of step s.  Else
// ops.fetch(last, s, i) issues load i of NR to registers (ops.begin(last, s)
// before the first), ops.put(a, b, i) writes part i of NP of them.  last:
// whether s may be the last step, which may end early.
//
// The fragments enter the instruction exchanged: a lane's 16 results of a
// block are 4 x 4 neighbouring columns of one row.
template <int MI, bool DIRECT, bool A_TURNED, bool B_TURNED, int NR, int NP, typename Ops>
__device__ __forceinline__ void wide_products(uint8_t* smem, int steps, f32x16 (&acc)[MI][2],
                                              Ops& ops) {
  using W = Wide<MI>;
  constexpr int DA = DIRECT ? W::DA : 2, DB = DIRECT ? W::DB : 2, M = 2 * MI;
  uint8_t* const bs = smem + DA * W::A;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int wm = (wave >> 2) * W::ROWS, wn = (wave & 3) * 64;
  struct Frag { u32x4 a[MI], b[2]; };
  // fragment x of turn t: the two of the columns, then those of the rows
  auto read = [&](Frag& f, const uint8_t* at, const uint8_t* bt, int t, int x) {
    const int c = 2 * t + (lane >> 5), r = lane & 31;
    if (x < 2)
      f.b[x] = *reinterpret_cast<const u32x4*>(
          bt + (wn + 32 * x) * 128 + (B_TURNED ? turned_off(r, c) : lds_off(r, c)));
    else
      f.a[x - 2] = *reinterpret_cast<const u32x4*>(
          at + (wm + 32 * (x - 2)) * 128 + (A_TURNED ? turned_off(r, c) : lds_off(r, c)));
  };
  if (steps == 0) return;
  constexpr std::true_type last{};
  if constexpr (DIRECT) {
    // in the order of the loop: the rows' tile of a step before the columns'
#pragma unroll
    for (int s = 0; s < DA; ++s) {
      if (s >= steps) break;
#pragma unroll
      for (int i = 0; i < MI; ++i) ops.direct_a(last, s, smem + s * W::A, i);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (s < 2) ops.direct_b(last, s, bs + s * W::B, i);
    }
    if (DA == 3 && steps > 2) wait_vmcnt<2 * MI + 4>();
    else if (steps > 1) wait_vmcnt<MI + 4>();
    else wait_vmcnt<0>();
  } else {
    ops.begin(last, 0);
#pragma unroll
    for (int i = 0; i < NR; ++i) ops.fetch(last, 0, i);
#pragma unroll
    for (int i = 0; i < NP; ++i) ops.put(smem, bs, i);
    if (steps > 1) {
      ops.begin(last, 1);
#pragma unroll
      for (int i = 0; i < NR; ++i) ops.fetch(last, 1, i);
    }
  }
  lds_done();
  barrier();
  Frag f[2];
#pragma unroll
  for (int x = 0; x < MI + 2; ++x) read(f[0], smem, bs, 0, x);
  // this step's slots, and the columns' one of the step before
  uint8_t* at = smem;
  uint8_t* bt = bs;
  uint8_t* old = bs + (DB - 1) * W::B;
  // HOT: enough steps follow, so the body has no branch
  auto step = [&](auto end, int s) {
    constexpr bool HOT = !decltype(end)::value;
    uint8_t* const an = at == smem + (DA - 1) * W::A ? smem : at + W::A;
    uint8_t* const bn = bt == bs + (DB - 1) * W::B ? bs : bt + W::B;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      if (t == 3) {
        // this wave's direct loads of the next step have landed, its tiles are
        // written and it has read this step's fragments; then everyone
        if (DIRECT) {
          if (HOT || s + 2 < steps) wait_vmcnt<DA == 3 ? MI + 4 : 4>(); else wait_vmcnt<0>();
        }
        lds_done();
        barrier();
      }
      if (!DIRECT && t == 2 && (HOT || s + 2 < steps)) ops.begin(end, s + 2);
      __builtin_amdgcn_sched_barrier(0);
      // between the products, so that no queue fills up and stops them: the
      // next fragments, and the loads and writes
#pragma unroll
      for (int m = 0; m < M; ++m) {
        const int i = m >> 1, j = m & 1;
        acc[i][j] = product<uint16_t>(f[t & 1].b[j], f[t & 1].a[i], acc[i][j]);
        auto share = [&](int n, auto one) {
#pragma unroll
          for (int x = n * m / M; x < n * (m + 1) / M; ++x) one(x);
        };
        if (t < 3) share(MI + 2, [&](int x) { read(f[(t + 1) & 1], at, bt, t + 1, x); });
        else if (HOT || s + 1 < steps) share(MI + 2, [&](int x) { read(f[0], an, bn, 0, x); });
        if (DIRECT) {
          if (t == 0 && (HOT || s + 2 < steps))
            share(4, [&](int x) { ops.direct_b(end, s + 2, old, x); });
          if (t == 3 && (HOT || s + DA < steps))
            share(MI, [&](int x) { ops.direct_a(end, s + DA, at, x); });
        } else {
          if (t == 1 && (HOT || s + 1 < steps)) share(NP, [&](int x) { ops.put(an, bn, x); });
          if (t == 2 && (HOT || s + 2 < steps))
            share(NR, [&](int x) { ops.fetch(end, s + 2, x); });
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    old = bt;
    at = an;
    bt = bn;
  };
  int s = 0;
#pragma unroll 1
  for (; s + 4 < steps; ++s) step(std::false_type{}, s);
#pragma unroll 1
  for (; s < steps; ++s) step(last, s);
}

// A wave's 32 MI x 64 results to memory, a block of 32 rows at a time through
// LDS, so that a store covers whole runs of a row.  row(m): the address of
// column 0 of the wave's row m (null: not stored), scale(m) its factor; cols:
// the columns from there to the end.  The stores pass the caches by: they would
// push out what the next tiles read (4096 tokens x 8 of 32 experts, fp32
// gradients of 2048 x 4096: 810 -> 767 us).
template <int MI, typename Row, typename Scale>
__device__ __forceinline__ void wide_store(uint8_t* smem, const f32x16 (&acc)[MI][2],
                                           bsmm_dtype dt, int cols, const Row& row,
                                           const Scale& scale) {
  constexpr int PITCH = kWidePitch;                    // reads and writes without conflicts
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  uint8_t* const part = smem + wave * (32 * PITCH);
#pragma unroll
  for (int i = 0; i < MI; ++i) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        *reinterpret_cast<f32x4*>(part + (lane & 31) * PITCH +
                                  (32 * j + 8 * g + 4 * (lane >> 5)) * 4) =
            f32x4{acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2],
                  acc[i][j][4 * g + 3]};
    if (dt == BSMM_BF16) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int m = 8 * q + (lane >> 3), c = (lane & 7) * 8;
        const f32x4* const p = reinterpret_cast<const f32x4*>(part + m * PITCH + c * 4);
        const float f = scale(32 * i + m);
        const f32x4 v = p[0] * f, w = p[1] * f;
        uint8_t* const to = static_cast<uint8_t*>(row(32 * i + m));
        if (to == nullptr) continue;
        if (c + 8 <= cols) {
          u32x4 o;
          o[0] = bf16_pair(v[0], v[1]);
          o[1] = bf16_pair(v[2], v[3]);
          o[2] = bf16_pair(w[0], w[1]);
          o[3] = bf16_pair(w[2], w[3]);
          __builtin_nontemporal_store(o, reinterpret_cast<u32x4_any*>(to + c * 2));
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (c + k < cols)
              reinterpret_cast<uint16_t*>(to)[c + k] = (uint16_t)bf16_bits(k < 4 ? v[k & 3]
                                                                                 : w[k & 3]);
        }
      }
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const int m = 4 * q + (lane >> 4), c = (lane & 15) * 4;
        const f32x4 v = *reinterpret_cast<const f32x4*>(part + m * PITCH + c * 4) *
                        scale(32 * i + m);
        uint8_t* const to = static_cast<uint8_t*>(row(32 * i + m));
        if (to == nullptr) continue;
        if (c + 4 <= cols) {
          __builtin_nontemporal_store(v, reinterpret_cast<f32x4_any*>(to + c * 4));
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (c + k < cols) reinterpret_cast<float*>(to)[c + k] = v[k];
        }
      }
    }
  }
}

// An item of at most 64 MI rows from column n0.
template <int MI, bool W_ACROSS, bool DIRECT>
__device__ __forceinline__ void expert_mm_item(const ExpertArgs& a, const Item& it, int n0,
                                               int s0, int s1, uint8_t* smem) {
  using W = Wide<MI>;
  int* const slots = reinterpret_cast<int*>(smem + kWideStage);
  float* const scales = reinterpret_cast<float*>(slots + 256);
  item_slots(a, it, 64 * MI, slots, scales);
  __syncthreads();
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // load t of an operand brings rows 64 t + 8 wave + lane / 8 of its tile;
  // rows and columns past the end repeat others (not stored)
  struct {
    const ExpertArgs& a;
    int wave, lane, xk;
    Columns cols;
    const uint16_t* w;
    int s0, n, turn;
    // Step s of the walk, which an expert starts `turn` steps in.  All tiles
    // walk at a time, and experts a power of two of bytes apart would take the
    // same memory channels (64 rows x 32 experts of 2048 x 4096: 127 us, 99
    // with the turn, 98 without it at 2048 x 4160).  It follows from the expert
    // alone, and so does the order of the sums.
    __device__ __forceinline__ int step(int s) const {
      s += turn;
      return s0 + (s < n ? s : s - n);
    }
    const uint16_t* xp[MI];
    const uint16_t* wp[4];
    u32x4 xv[MI], wv[4];
    Turn v;
    // the lane's unit of a row that lies along
    __device__ __forceinline__ u32x4 unit(bool last, const uint16_t* p, int s) const {
      if (!last || a.K % 8 == 0) return load_global<u32x4_any>(along(last, p, s));
      s = step(s);
      return bsmm::fetch<uint16_t>(p + s * 64, a.K - xk - s * 64);
    }
    __device__ __forceinline__ const uint16_t* along(bool last, const uint16_t* p, int s) const {
      s = step(s);
      return !last || s * 64 + xk < a.K ? p + s * 64 : reinterpret_cast<const uint16_t*>(kZeros);
    }
    __device__ __forceinline__ void direct_a(bool last, int s, uint8_t* slot, int i) {
      to_lds<16>(along(last, xp[i], s), slot + (i * 8 + wave) * 1024);
    }
    __device__ __forceinline__ void direct_b(bool last, int s, uint8_t* slot, int i) {
      to_lds<16>(along(last, wp[i], s), slot + (i * 8 + wave) * 1024);
    }
    __device__ __forceinline__ void begin(bool, int) {}
    __device__ __forceinline__ void fetch(bool last, int s, int i) {
      if (i < MI) {
        xv[i] = unit(last, xp[i], s);
      } else if (!W_ACROSS) {
        wv[i - MI] = unit(last, wp[i - MI], s);
      } else {
        const int k = step(s) * 64 + wave * 8 + i - MI;
        const uint16_t* row = w + (int64_t)k * a.ldw + cols.first;
        if (last) row = k < a.K ? row : reinterpret_cast<const uint16_t*>(kZeros);
        v.row[i - MI] =
            load_global<u32x2_any>(reinterpret_cast<const uint8_t*>(row) + cols.at);
      }
    }
    __device__ __forceinline__ void put(uint8_t* at, uint8_t* bt, int i) {
      if (i < MI) {
        *reinterpret_cast<u32x4*>(at + (i * 8 + wave) * 1024 + lane * 16) = xv[i];
      } else if (!W_ACROSS) {
        *reinterpret_cast<u32x4*>(bt + ((i - MI) * 8 + wave) * 1024 + lane * 16) = wv[i - MI];
      } else {
        if (i == MI) cols.place(v);
        put_turned(v, bt, wave, i - MI);
      }
    }
  } ops{a, wave, lane, ((lane & 7) ^ swz(8 * wave + (lane >> 3))) * 8,
        Columns(n0, W_ACROSS ? a.N : 4, lane),
        static_cast<const uint16_t*>(a.w) + it.e * a.w_se, s0, s1 - s0,
        a.K % 64 == 0 && s1 > s0 ? it.e % (s1 - s0) : 0, {}, {}, {}, {}, {}};
#pragma unroll
  for (int t = 0; t < MI; ++t) {
    const int s = max(slots[64 * t + 8 * wave + (lane >> 3)], 0);
    ops.xp[t] = static_cast<const uint16_t*>(a.x) + (int64_t)min(s / a.x_div, a.R - 1) * a.ldx +
                ops.xk;
  }
  if constexpr (!W_ACROSS) {
#pragma unroll
    for (int t = 0; t < 4; ++t)
      ops.wp[t] = ops.w + (int64_t)min(n0 + 64 * t + 8 * wave + (lane >> 3), a.N - 1) * a.ldw +
                  ops.xk;
  }
  __syncthreads();                      // the slots have been read
  f32x16 acc[MI][2] = {};
  wide_products<MI, DIRECT, false, W_ACROSS, MI + (W_ACROSS ? 8 : 4), MI + 4>(
      smem, s1 - s0, acc, ops);
  barrier();                            // nobody reads the tiles any more
  item_slots(a, it, 64 * MI, slots, scales);
  __syncthreads();
  const int wm = (wave >> 2) * W::ROWS, col = n0 + (wave & 3) * 64;
  const int size = a.out_dtype == BSMM_BF16 ? 2 : 4;
  uint8_t* const out = static_cast<uint8_t*>(a.out) + (int64_t)col * size;
  wide_store<MI>(
      smem, acc, a.out_dtype, a.N - col,
      [&](int m) -> void* {
        const int slot = slots[wm + m];
        return slot < 0 ? nullptr : out + slot * a.ldo * size;
      },
      [&](int m) { return scales[wm + m]; });
}

// DIRECT: rows along, 16-byte aligned, whole units.
template <bool W_ACROSS, bool DIRECT>
__global__ void __launch_bounds__(512, 2) expert_mm_wide(ExpertArgs a, int rows, int items,
                                                         int ntn, int splits, int run) {
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  // groups of 4 items (1, 2 and 8 were within 2 %; one expert of 8192^3: 8 the
  // same, 2 and 1 took 2 and 7 % more)
  int item, tn, s0, s1;
  if (!deal_tile(items * splits, ntn, run, 4, item, tn)) return;
  part_of(a, items, splits, 64, item, s0, s1);
  const Item it = find_item(a.offsets, a.E, a.S, rows, item);
  const int n0 = tn * kWide;
  zero_rows(a, n0, kWide, item, items);
  if (it.rows == 0) return;
  // only as many rows as there are, to 64: an expert's last item would
  // multiply 128 empty rows on average
  const int mi = (it.rows + 63) / 64;
  if (mi == 4) expert_mm_item<4, W_ACROSS, DIRECT>(a, it, n0, s0, s1, smem);
  else if (mi == 3) expert_mm_item<3, W_ACROSS, DIRECT>(a, it, n0, s0, s1, smem);
  else if (mi == 2) expert_mm_item<2, W_ACROSS, DIRECT>(a, it, n0, s0, s1, smem);
  else expert_mm_item<1, W_ACROSS, DIRECT>(a, it, n0, s0, s1, smem);
}

__global__ void __launch_bounds__(512, 2) expert_wgrad_wide(WgradArgs a, int ntn, int ntk,
                                                            int splits, int run, Divisor yd,
                                                            Divisor xd) {
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  int item, tk, lo, hi;
  if (!deal_tile(splits * a.E * ntn, ntk, run, 1, item, tk)) return;
  const int e = run_of(a, ntn, splits, 64, item, lo, hi);
  const int n0 = item % ntn * 256, k0 = tk * kWide, lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // the wave's 8 positions of a step; lane i < 8 has the slot of the i-th
  struct {
    const WgradArgs& a;
    Divisor yd, xd;
    int wave, lane, lo, hi;
    const uint8_t* dy;
    const uint8_t* x;
    Columns cy, cx;
    int mine;
    int64_t oy, ox;
    int rows;
    Turn vy, vx;
    __device__ __forceinline__ int slot_of(int s) const {
      return lo < hi ? slot_at(a.order, min(lo + s * 64 + wave * 8 + (lane & 7), hi - 1)) : 0;
    }
    __device__ __forceinline__ void direct_a(bool, int, uint8_t*, int) {}
    __device__ __forceinline__ void direct_b(bool, int, uint8_t*, int) {}
    __device__ __forceinline__ void begin(bool last, int s) {
      const uint32_t slot = min(max(mine, 0), a.S - 1);
      oy = (int64_t)divide(slot, yd) * a.ldy * 2;
      ox = (int64_t)divide(slot, xd) * a.ldx * 2;
      rows = last ? hi - lo - s * 64 - wave * 8 : 8;
      mine = slot_of(s + 1);
    }
    static __device__ __forceinline__ int64_t lane_of(int64_t v, int i) {
      const uint32_t l = __builtin_amdgcn_readlane((int)v, i);
      return (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(v >> 32), i) << 32 | l);
    }
    // dy's rows, then x's
    __device__ __forceinline__ void fetch(bool last, int, int i) {
      const bool second = i >= 8;
      const int r = i & 7;
      const uint8_t* p = second ? x + lane_of(ox, r) : dy + lane_of(oy, r);
      if (last) p = r < rows ? p : reinterpret_cast<const uint8_t*>(kZeros);
      (second ? vx : vy).row[r] = load_global<u32x2_any>(p + (second ? cx.at : cy.at));
    }
    __device__ __forceinline__ void put(uint8_t* at, uint8_t* bt, int i) {
      if (i == 0) cy.place(vy);
      if (i == 4) cx.place(vx);
      if (i < 4) put_turned(vy, at, wave, i);
      else put_turned(vx, bt, wave, i - 4);
    }
  } ops{a, yd, xd, wave, lane, lo, hi, static_cast<const uint8_t*>(a.dy),
        static_cast<const uint8_t*>(a.x), Columns(n0, a.N, lane), Columns(k0, a.K, lane),
        0, 0, 0, 0, {}, {}};
  ops.dy += (int64_t)ops.cy.first * 2;
  ops.x += (int64_t)ops.cx.first * 2;
  ops.mine = ops.slot_of(0);
  f32x16 acc[4][2] = {};
  wide_products<4, false, true, true, 16, 8>(smem, (int)(((unsigned)(hi - lo) + 63) / 64), acc,
                                             ops);
  barrier();                            // nobody reads the tiles any more
  const int row0 = n0 + (wave >> 2) * 128, col = k0 + (wave & 3) * 64;
  const int size = a.out_dtype == BSMM_BF16 ? 2 : 4;
  uint8_t* const out = static_cast<uint8_t*>(a.dw) + (e * a.w_se + col) * size;
  wide_store<4>(
      smem, acc, a.out_dtype, a.K - col,
      [&](int m) -> void* {
        return row0 + m < a.N ? out + (row0 + m) * a.ldw * size : nullptr;
      },
      [](int) { return 1.0f; });
}

// ---------------------------------------------------------------------------
// Few rows: items of 16 or, along, 32 rows by 64 columns, 16 x 16 instructions
// with the weight as the first operand.  The eight waves of a workgroup share
// out cn = 8 / ks column groups and ks ranges of the contraction; partial sums
// are added through LDS in order.
//
// Everything goes straight to registers, kDepth chunks of 64 bytes (32 bf16 or
// 16 fp32 of the contraction) ahead: no barrier, each weight byte is used by
// one wave.  Bound by the weights' bytes (1 token x 8 of 64 experts of 2048 x
// 4096 bf16, 134 MB: 33 us, 4.1 TB/s; 33 x 4 of 16 of 4099 x 1024 fp32, 268 MB:
// 76 us, 3.5 TB/s, a few workgroups in a second round).  Items of 32 rows have
// three chunks ahead, for their registers (64 x 4 of 16 of 4096 x 1024 fp32: 90
// us in items of 16, 78 of 32); across, they spill.  Along, a lane's 16 bytes
// are one column's.  Across, a lane has 4 neighbouring columns: of bf16 8 rows,
// transposed by byte permutations, of fp32 4 rows, each lane's 4 values then
// belonging to 4 column blocks.
// ---------------------------------------------------------------------------
constexpr int kRowsWaves = 8;

// A chunk of one wave: x's fragments and those of its 4 column blocks
template <typename T, bool ACROSS, int MB> struct Chunk {
  u32x4 x[MB];
  std::conditional_t<ACROSS && sizeof(T) == 2, u32x2, u32x4>
      w[ACROSS && sizeof(T) == 2 ? 8 : 4];
};

// An item of at most 16 MB rows; column group blockIdx.x * cn + cw.
template <typename T, bool W_ACROSS, int MB>
__device__ __forceinline__ void expert_rows_item(const ExpertArgs& a, const Item& it, int log_ks,
                                                 float (&part)[kRowsWaves][16][68]) {
  constexpr int U = Elem<T>::U, CHUNK = 4 * U, kDepth = MB == 1 ? 4 : 3;
  const int lane = threadIdx.x & 63, c16 = lane & 15, quad = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ks = 1 << log_ks, cn = kRowsWaves >> log_ks;
  const int kw = wave & (ks - 1), cw = wave >> log_ks;
  const int n0 = (blockIdx.x * cn + cw) * 64, cols = cn * 64;

  const T* x[MB];
#pragma unroll
  for (int b = 0; b < MB; ++b) {
    const int slot = slot_at(a.order, it.p0 + min(16 * b + c16, it.rows - 1));
    const int64_t row = min(max(slot / a.x_div, 0), a.R - 1);
    x[b] = static_cast<const T*>(a.x) + row * a.ldx + quad * U;
  }
  const T* const w = static_cast<const T*>(a.w) + it.e * a.w_se;
  const T* wp[4];
  if constexpr (W_ACROSS) {
    wp[0] = w + (int64_t)(quad * U) * a.ldw + min(n0 + 4 * c16, a.N - 4);
  } else {
#pragma unroll
    for (int t = 0; t < 4; ++t)
      wp[t] = w + (int64_t)min(n0 + 16 * t + c16, a.N - 1) * a.ldw + quad * U;
  }
  const T* const zero = reinterpret_cast<const T*>(kZeros);
  using C = Chunk<T, W_ACROSS, MB>;
  const int chunks = (int)(((unsigned)a.K + CHUNK - 1) / CHUNK), per = (chunks + ks - 1) >> log_ks;
  int c = min(kw * per, chunks);
  const int end = n0 < a.N ? min(c + per, chunks) : c;
  auto load = [&](C& v, int c) {
    const int k = c * CHUNK;
    const bool in = k + quad * U < a.K;                // K % U == 0
#pragma unroll
    for (int b = 0; b < MB; ++b) v.x[b] = load_global<u32x4>(in ? x[b] + k : zero);
    if constexpr (W_ACROSS) {
      const T* const p = wp[0] + k * a.ldw;
#pragma unroll
      for (int i = 0; i < U; ++i)
        v.w[i] = load_global<std::remove_reference_t<decltype(v.w[0])>>(in ? p + i * a.ldw : zero);
    } else {
#pragma unroll
      for (int t = 0; t < 4; ++t) v.w[t] = load_global<u32x4>(in ? wp[t] + k : zero);
    }
  };
  f32x4 acc[MB][4] = {};
  auto consume = [&](const C& v) {
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      if constexpr (sizeof(T) == 2) {
        u32x4 f;
        if constexpr (W_ACROSS) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            f[i] = __builtin_amdgcn_perm(v.w[2 * i + 1][t >> 1], v.w[2 * i][t >> 1],
                                         t & 1 ? 0x07060302u : 0x05040100u);
        } else {
          f = v.w[t];
        }
#pragma unroll
        for (int b = 0; b < MB; ++b)
          acc[b][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, f),
                                                              __builtin_bit_cast(bf16x8, v.x[b]),
                                                              acc[b][t], 0, 0, 0);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int b = 0; b < MB; ++b)
            acc[b][t] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                __uint_as_float(W_ACROSS ? v.w[j][t] : v.w[t][j]), __uint_as_float(v.x[b][j]),
                acc[b][t], 0, 0, 0);
      }
    }
  };
  C v[kDepth];
#pragma unroll
  for (int d = 0; d < kDepth; ++d)
    if (c + d < end) load(v[d], c + d);
#pragma unroll 1
  for (; c + 2 * kDepth <= end; c += kDepth) {
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      consume(v[d]);
      load(v[d], c + kDepth + d);
    }
  }
#pragma unroll
  for (int d = 0; d < kDepth; ++d)
    if (c + d < end) {
      consume(v[d]);
      if (c + kDepth + d < end) load(v[d], c + kDepth + d);
    }
#pragma unroll
  for (int d = 0; d < kDepth; ++d)
    if (c + kDepth + d < end) consume(v[d]);

#pragma unroll
  for (int b = 0; b < MB; ++b) {
    if (b > 0) __syncthreads();
    // a lane has row c16 and of column block t the columns 4 quad + r
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        part[wave][c16][W_ACROSS ? 16 * quad + 4 * r + t : 16 * t + 4 * quad + r] = acc[b][t][r];
    __syncthreads();
    // row m of the block to threads m, m + 16 ..: neighbouring threads have
    // neighbouring columns
    const int rows = min(it.rows - 16 * b, 16);
    for (int i = threadIdx.x; i < rows * cols; i += kRowsWaves * 64) {
      const int m = i / cols, n = i - m * cols, at = blockIdx.x * cols + n;
      const int s = slot_at(a.order, it.p0 + 16 * b + m);
      if (at >= a.N || s < 0 || s >= a.S) continue;
      float sum = 0.0f;
      for (int j = 0; j < ks; ++j) sum += part[((n >> 6) << log_ks) + j][m][n & 63];
      put(a.out, a.out_dtype, s * a.ldo + at, a.row_scale ? sum * a.row_scale[s] : sum);
    }
  }
}

template <typename T, bool W_ACROSS>
__global__ void __launch_bounds__(kRowsWaves * 64, 4) expert_mm_rows(ExpertArgs a, int bm,
                                                                     int log_ks) {
  __shared__ __attribute__((aligned(16))) float part[kRowsWaves][16][68];
  const int item = blockIdx.y, cols = (kRowsWaves >> log_ks) * 64;
  const Item it = find_item(a.offsets, a.E, a.S, bm, item);
  zero_rows(a, blockIdx.x * cols, cols, item, gridDim.y);
  if (it.rows == 0) return;
  if constexpr (!W_ACROSS) {
    if (it.rows > 16) return expert_rows_item<T, W_ACROSS, 2>(a, it, log_ks, part);
  }
  expert_rows_item<T, W_ACROSS, 1>(a, it, log_ks, part);
}

Divisor divisor(uint32_t d) {
  int l = 0;
  while (((uint64_t)1 << l) < d) ++l;
  return Divisor{(uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << l) - d)) / d + 1), l};
}

// The launch of items of few rows: at most bm of them, by cn = 8 >> log_ks
// groups of 64 columns.
struct RowsGrid {
  int bm, log_ks;
  int64_t items, ntn;
  explicit RowsGrid(const ExpertArgs& a) {
    const int64_t act = a.E < a.S ? a.E : a.S, groups = ((int64_t)a.N + 63) / 64;
    // (64 x 2 of 8 of 1024 x 2048: 14.3 us in items of 16, 16.3 of 32; others below)
    bm = a.w_across || act * groups < 256 ? 16 : 32;
    items = ((int64_t)a.S + act * (bm - 1)) / bm;
    // Waves that fill the chip, in workgroups of even cost.  Along: 1024 groups
    // in 1, 2, 4 or 8 ranges take 176, 126, 106, 112 us (8 tokens x 8 of 32
    // experts of 2048 x 4096); where experts have items of either kind, 150,
    // 129, 125, 108 (128 x 4 of 16 of 4096 x 1024 fp32).  Across, an expert's
    // second item reads the weights again: better while the first does, so all
    // waves take the same columns then (64 x 4 of 16 of 4096 x 1024 fp32: 266,
    // 141, 81, 78 us; 32 x 8 of 32 of 2048 x 4096: 124, 109, 106, 111; 16 x 8:
    // 92, 94, 95, 103).
    int64_t busy, target;
    if (a.w_across) {
      busy = (a.S + act * 8) / 16 + 1;
      target = a.S <= 6 * act ? 2048 : 8192;
    } else {
      busy = a.S <= 16 * act ? act : (a.S + act * 16) / 32;
      target = a.S <= 16 * act ? 4096 : 32768;
    }
    log_ks = 0;
    while (log_ks < 3 && (busy * groups << log_ks) < target) ++log_ks;
    ntn = (groups + (8 >> log_ks) - 1) / (8 >> log_ks);
  }
};

template <typename T, bool W_ACROSS>
void launch_rows(const ExpertArgs& a, hipStream_t st) {
  const RowsGrid g(a);                              // some thousand items at most
  hipLaunchKernelGGL((expert_mm_rows<T, W_ACROSS>), dim3((unsigned)g.ntn, (unsigned)g.items),
                     dim3(kRowsWaves * 64), 0, st, a, g.bm, g.log_ks);
}

void launch_reduce(const float* parts, int splits, void* out, bsmm_dtype dt, int64_t rows,
                   int cols, int64_t inner, int64_t outer_ld, int64_t ld, hipStream_t st) {
  const int64_t blocks = (rows * cols + 255) / 256;
  hipLaunchKernelGGL(reduce_parts, dim3((unsigned)(blocks < 16384 ? blocks : 16384)), dim3(256), 0,
                     st, parts, splits, out, dt, rows, cols, inner, outer_ld, ld);
}

// Runs of tiles for deal_tile, and the grid.  Runs of 8, so that the XCDs' work
// is even: with an eighth of the grid to each, most of the items that do not
// exist fell to the last XCDs, and an expert's tiles to one (300 tokens x 8 of
// 32 experts of 2048 x 4096: 128 us in runs of 8, 162 in eighths; 4096 x 8 of
// 64, input gradient: 699 and 793; 4096 x 8 of 32, weight gradient: 682 and
// 784; runs of 16, 32, 64 there: 701, 744, 754).  One expert's tiles are even,
// and neighbours share more operands in eighths (2048 x 4096 x 4096: 62 us,
// 65 in runs of 8).
struct Deal {
  int run;
  int64_t grid;
  Deal(int64_t tiles, int64_t real, bool one) {
    const int64_t eighth = (real + 7) / 8;
    run = (int)(one || eighth < 8 ? eighth : 8);
    grid = (tiles + 8 * run - 1) / (8 * run) * (8 * run);
  }
};

// Items, columns of tiles and the dealing of a product's tiles, and of the
// weight gradient's.
struct MmGrid {
  int items, ntn, threads;
  Deal deal;
  MmGrid(const ExpertArgs& a, ExpertPlan plan, int rows, int splits)
      : MmGrid(a, plan == ExpertPlan::Wide ? rows : 64, plan == ExpertPlan::Wide ? kWide : 64,
               splits) {
    threads = plan == ExpertPlan::Wide ? 512 : 256;
  }

 private:
  static int items_of(const ExpertArgs& a, int bm) {
    const int64_t act = a.E < a.S ? a.E : a.S;
    return (int)(((int64_t)a.S + act * (bm - 1)) / bm);
  }
  static int64_t real_of(const ExpertArgs& a, int bm) {
    const int64_t act = a.E < a.S ? a.E : a.S;
    const int64_t real = ((int64_t)a.S + act * (bm / 2)) / bm, items = items_of(a, bm);
    return real < act ? act : real < items ? real : items;
  }
  MmGrid(const ExpertArgs& a, int bm, int bn, int splits)
      : items(items_of(a, bm)), ntn((a.N + bn - 1) / bn), threads(0),
        deal((int64_t)items * splits * ntn, real_of(a, bm) * splits * ntn,
             (a.E < a.S ? a.E : a.S) == 1) {}
};
struct WgradGrid {
  int ntn, ntk, threads;
  Deal deal;
  WgradGrid(const WgradArgs& a, ExpertPlan plan, int splits)
      : WgradGrid(a, plan == ExpertPlan::Wide ? 256 : plan == ExpertPlan::Tiles128 ? 128 : 64,
                  splits) {
    threads = plan == ExpertPlan::Wide ? 512 : 256;
  }

 private:
  WgradGrid(const WgradArgs& a, int tile, int splits)
      : ntn((a.N + tile - 1) / tile), ntk((a.K + tile - 1) / tile), threads(0),
        deal((int64_t)splits * a.E * ntn * ntk, (int64_t)splits * a.E * ntn * ntk, false) {}
};

template <typename T, bool W_ACROSS>
void launch_mm(ExpertArgs a, ExpertPlan plan, int rows, int splits, void* ws, hipStream_t st) {
  if (plan == ExpertPlan::Rows) return launch_rows<T, W_ACROSS>(a, st);
  void* const out = a.out;
  const int64_t ldo = a.ldo;
  const bsmm_dtype dt = a.out_dtype;
  if (splits > 1) {
    a.out = ws;
    a.ldo = a.N;
    a.out_dtype = BSMM_F32;
  }
  const MmGrid g(a, plan, rows, splits);
  const dim3 grid((unsigned)g.deal.grid), block(g.threads);
  if (plan == ExpertPlan::Wide) {
    if constexpr (sizeof(T) == 2) {
      const bool direct = !W_ACROSS && a.K % 8 == 0 && aligned_rows(a.x, a.ldx, a.dtype) &&
                          aligned_rows(a.w, a.ldw, a.dtype) && a.w_se % 8 == 0;
      if (direct)
        hipLaunchKernelGGL((expert_mm_wide<W_ACROSS, !W_ACROSS>), grid, block, kWideBytes, st, a,
                           rows, g.items, g.ntn, splits, g.deal.run);
      else
        hipLaunchKernelGGL((expert_mm_wide<W_ACROSS, false>), grid, block, kWideBytes, st, a, rows,
                           g.items, g.ntn, splits, g.deal.run);
    }
  } else {
    hipLaunchKernelGGL((expert_mm_kernel<T, W_ACROSS>), grid, block, 0, st, a, g.items, g.ntn,
                       splits, g.deal.run);
  }
  if (splits > 1)
    launch_reduce(static_cast<const float*>(ws), splits, out, dt, a.S, a.N, a.S, 0, ldo, st);
}

template <typename T, int MB>
void launch_wgrad_tiles(const WgradArgs& a, const WgradGrid& g, int splits, hipStream_t st) {
  const dim3 grid((unsigned)g.deal.grid), block(g.threads);
  const Divisor yd = divisor(a.y_div), xd = divisor(a.x_div);
  if (a.x_scale)
    hipLaunchKernelGGL((expert_wgrad_kernel<T, MB, true>), grid, block, 0, st, a, g.ntn, g.ntk,
                       splits, g.deal.run, yd, xd);
  else
    hipLaunchKernelGGL((expert_wgrad_kernel<T, MB, false>), grid, block, 0, st, a, g.ntn, g.ntk,
                       splits, g.deal.run, yd, xd);
}

template <typename T>
void launch_wgrad(WgradArgs a, ExpertPlan plan, int splits, void* ws, hipStream_t st) {
  void* const dw = a.dw;
  const int64_t w_se = a.w_se, ldw = a.ldw;
  const bsmm_dtype dt = a.out_dtype;
  if (splits > 1) {
    a.dw = ws;
    a.ldw = a.K;
    a.w_se = (int64_t)a.N * a.K;
    a.out_dtype = BSMM_F32;
  }
  const WgradGrid g(a, plan, splits);
  if (plan == ExpertPlan::Wide) {
    if constexpr (sizeof(T) == 2)
      hipLaunchKernelGGL(expert_wgrad_wide, dim3((unsigned)g.deal.grid), dim3(g.threads),
                         kWideBytes, st, a, g.ntn, g.ntk, splits, g.deal.run, divisor(a.y_div),
                         divisor(a.x_div));
  } else if (plan == ExpertPlan::Tiles128) {
    launch_wgrad_tiles<T, 2>(a, g, splits, st);
  } else {
    launch_wgrad_tiles<T, 1>(a, g, splits, st);
  }
  if (splits > 1)
    launch_reduce(static_cast<const float*>(ws), splits, dw, dt, (int64_t)a.E * a.N, a.K, a.N, w_se,
                  ldw, st);
}

}  // namespace

uint64_t expert_mm_threads(const ExpertArgs& a, ExpertPlan plan, int rows, int splits) {
  if (plan == ExpertPlan::Rows) return (uint64_t)RowsGrid(a).ntn * (kRowsWaves * 64);   // in x
  const MmGrid g(a, plan, rows, splits);
  return (uint64_t)g.deal.grid * (uint64_t)g.threads;
}

uint64_t expert_wgrad_threads(const WgradArgs& a, ExpertPlan plan, int splits) {
  const WgradGrid g(a, plan, splits);
  return (uint64_t)g.deal.grid * (uint64_t)g.threads;
}

int launch_expert_mm(const ExpertArgs& a, ExpertPlan plan, int rows, int splits, void* ws,
                     void* stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (a.dtype == BSMM_BF16) {
    if (a.w_across) launch_mm<uint16_t, true>(a, plan, rows, splits, ws, st);
    else launch_mm<uint16_t, false>(a, plan, rows, splits, ws, st);
  } else {
    if (a.w_across) launch_mm<float, true>(a, plan, rows, splits, ws, st);
    else launch_mm<float, false>(a, plan, rows, splits, ws, st);
  }
  return hipGetLastError() == hipSuccess ? 0 : 1;
}

int launch_expert_wgrad(const WgradArgs& a, ExpertPlan plan, int splits, void* ws, void* stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (a.dtype == BSMM_BF16) launch_wgrad<uint16_t>(a, plan, splits, ws, st);
  else launch_wgrad<float>(a, plan, splits, ws, st);
  return hipGetLastError() == hipSuccess ? 0 : 1;
}

}  // namespace bsmm
