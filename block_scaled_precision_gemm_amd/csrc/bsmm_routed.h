// Device pieces shared by the products of routed rows (gfx950): register
// types, work items, direct loads to LDS, tile order.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace bsmm {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) void* lds_ptr_t;

__device__ __forceinline__ uint32_t bf16_bits(float v) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t{v, v}), bf16x2_t)) &
         0xFFFFu;
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t{lo, hi}), bf16x2_t));
}

struct Item { int e, p0, rows; };

// Work item `item` of a routed product: every expert's run of positions is
// cut into blocks of bm, in expert order.  Runs in every wave alike: each
// lane counts the blocks of its share of the experts, a scan over the lanes
// finds the one that holds the item.  Offsets are clamped into [0, S], so
// that no array content can lead outside the buffers; offsets that do not
// rise may count to more than 32 bits hold, and the sums then wrap, but an
// item is taken only from within a run.
__device__ Item find_item(const int32_t* __restrict__ offsets, int E, int S, unsigned bm,
                          unsigned item) {
  const int lane = threadIdx.x & 63;
  const int per = (E + 63) / 64;
  const int e0 = min(lane * per, E), e1 = min(e0 + per, E);
  unsigned n = 0;
  for (int e = e0; e < e1; ++e) {
    const int lo = min(max(offsets[e], 0), S), hi = min(max(offsets[e + 1], lo), S);
    n += ((unsigned)(hi - lo) + bm - 1) / bm;
  }
  unsigned incl = n;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const unsigned t = __shfl_up(incl, d);
    if (lane >= d) incl += t;
  }
  const unsigned long long past = __ballot(incl > item);
  if (past == 0) return Item{0, 0, 0};
  const int src = __ffsll(past) - 1;
  unsigned rest = item - (incl - n);
  Item r{0, 0, 0};
  if (lane == src) {
    for (int e = e0; e < e1; ++e) {
      const int lo = min(max(offsets[e], 0), S), hi = min(max(offsets[e + 1], lo), S);
      const unsigned b = ((unsigned)(hi - lo) + bm - 1) / bm;
      if (rest < b) {
        const int at = (int)(rest * bm);
        r = Item{e, lo + at, min(hi - lo - at, (int)bm)};
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

template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void wait_lgkm0() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
}

// A lane's SIZE bytes at src to dst + 16 * lane (SIZE 16) or dst + 4 * lane
// (SIZE 4, or 1 and 2, widened with zeros); dst is the wave's.
template <int SIZE>
__device__ __forceinline__ void to_lds(const void* src, uint8_t* dst) {
  auto* const from = (__attribute__((address_space(1))) void*)(uintptr_t)src;
  auto* const to = (__attribute__((address_space(3))) void*)(uintptr_t)(uint32_t)(uintptr_t)dst;
  if constexpr (SIZE == 1) __builtin_amdgcn_global_load_lds(from, to, 1, 0, 0);
  else if constexpr (SIZE == 2) __builtin_amdgcn_global_load_lds(from, to, 2, 0, 0);
  else if constexpr (SIZE == 4) __builtin_amdgcn_global_load_lds(from, to, 4, 0, 0);
  else __builtin_amdgcn_global_load_lds(from, to, 16, 0, 0);
}

// The same from base + voff + soff, 31 bits together: soff is the wave's, and
// the load needs no vector instruction for its address.
typedef __amdgpu_buffer_rsrc_t rsrc_t;
__device__ __forceinline__ rsrc_t buffer_at(const void* base) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, 0x7FFFFFFF,
                                           0x00020000);
}
template <int SIZE>
__device__ __forceinline__ void to_lds(rsrc_t rs, uint32_t voff, uint32_t soff, uint8_t* dst) {
  auto* const to = (__attribute__((address_space(3))) void*)(uintptr_t)(uint32_t)(uintptr_t)dst;
  const int v = (int)voff, s = (int)soff;
  if constexpr (SIZE == 1) __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, to, 1, v, s, 0, 0);
  else if constexpr (SIZE == 2) __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, to, 2, v, s, 0, 0);
  else if constexpr (SIZE == 4) __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, to, 4, v, s, 0, 0);
  else __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, to, 16, v, s, 0, 0);
}

__device__ __forceinline__ int swz(int r) { return (r & 7) ^ ((r >> 3) & 1); }
__device__ __forceinline__ int lds_off(int r, int c) { return (r << 7) + ((c ^ swz(r)) << 4); }

__device__ __forceinline__ void barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Logical workgroup ids: contiguous runs per XCD (hardware ids go round robin
// over 8), then groups of 8 row blocks by all column blocks, so that the
// workgroups an XCD holds at a time share x rows and weight columns in its L2.
__device__ __forceinline__ void tile_of(int items, int ntn, int& item, int& tn) {
  const int total = gridDim.x, hw = blockIdx.x;
  const int per = total >> 3, rem = total & 7, xcd = hw & 7, local = hw >> 3;
  const int id = xcd < rem ? xcd * (per + 1) + local : rem * (per + 1) + (xcd - rem) * per + local;
  const int width = 8 * ntn, g = id / width, first = 8 * g, n = min(items - first, 8);
  const int in = id - g * width;
  item = first + in % n;
  tn = in / n;
}

}  // namespace
}  // namespace bsmm
