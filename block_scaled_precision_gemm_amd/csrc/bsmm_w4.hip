// Products of bf16 / fp32 activations with 4-bit weights (gfx950).
//
//   out[p, n] = sum_g scale[n, g] * sum_{k in g} (code[n, k] - zero[n, g]) * x[p, k]
//
// The matrix instructions take code - zero, an integer of at most 8 bits and a
// sign and so exact in bf16: every product is exact, the sums are fp32 and
// hold nothing but the result's own terms, and nothing is rounded to fewer
// bits before the output.  Sums of 16 + code less 16 + zero times the sum of x
// take half the instructions to unpack, but both are larger than the result
// wherever x has a mean, and fp32 loses by it: K = 8192 in groups of 128,
// fp32 x of one sign 1e-5 of the result, one channel of 3000 that meets
// weights of 0 1e-4; as it is 1.3e-7 for both.  fp32 activations are cut into
// three bf16 numbers that add up to them exactly (8 + 8 + 8 bits), one matrix
// instruction each.

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

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

// high halves of (a, b) as a pair
__device__ __forceinline__ uint32_t hi2(uint32_t a, uint32_t b) {
  return __builtin_amdgcn_perm(b, a, 0x07060302u);
}

// Codes 2q and 2q + 1 of a dword -> code - z as a pair of bf16 (integers of 8
// bits and a sign: the upper halves of their fp32 forms)
__device__ __forceinline__ uint32_t unpack_pair(uint32_t w, int q, float z) {
  uint32_t e = w & 0x0F0F0F0Fu, o = (w >> 4) & 0x0F0F0F0Fu;
  // opaque: keeps the byte conversions from being split into shift and convert
  asm("" : "+v"(e), "+v"(o));
  const float a = (float)((e >> (8 * q)) & 0xFFu) - z, b = (float)((o >> (8 * q)) & 0xFFu) - z;
  return hi2(__float_as_uint(a), __float_as_uint(b));
}

// All 8, in order
__device__ __forceinline__ u32x4 unpack(uint32_t w, float z) {
  return u32x4{unpack_pair(w, 0, z), unpack_pair(w, 1, z), unpack_pair(w, 2, z),
               unpack_pair(w, 3, z)};
}

// 8 consecutive activations of one row
template <bool XF32> struct X8;
template <> struct X8<false> { u32x4 v; };
template <> struct X8<true> { u32x4 a, b; };

// the bf16 operands of 8 activations (1, or the 3 parts of fp32 values)
template <bool XF32> struct Parts { u32x4 p[XF32 ? 3 : 1]; };

__device__ __forceinline__ Parts<false> parts(const X8<false>& x) {
  return Parts<false>{{x.v}};
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
    r.p[i] = u32x4{hi2(a.x, a.y), hi2(a.z, a.w), hi2(b.x, b.y), hi2(b.z, b.w)};
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

__device__ __forceinline__ void store_out(const W4Args& a, int64_t at, float v) {
  if (a.out_dtype == BSMM_BF16) static_cast<uint16_t*>(a.out)[at] = (uint16_t)bf16_bits(v);
  else static_cast<float*>(a.out)[at] = v;
}

// Routed: zero rows for the slots of no expert, columns [col, col + cols),
// shared out over the items.
__device__ __forceinline__ void zero_unused(const W4Args& a, int col, int cols, int item,
                                            int items, int threads) {
  const unsigned used = min(max(a.offsets[a.E], 0), a.S);
  for (unsigned p = used + item; p < (unsigned)a.S; p += items) {    // both below 2^31
    const int slot = a.order[p];
    if (slot < 0 || slot >= a.S) continue;
    for (int i = threadIdx.x; i < cols; i += threads)
      if (col + i < a.N) store_out(a, slot * a.ldo + col + i, 0.0f);
  }
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

// ---------------------------------------------------------------------------
// Few rows: items of BM rows (4, 16 or 32); each of the W waves of a workgroup
// has 16 columns and one of ks ranges of K (W / ks column groups a
// workgroup), and the ks partial sums are added through LDS in order.  A
// wave's share is cut so that enough waves are in flight whatever the sizes.
//
// Codes, scales, zero points and x of a chunk of 128 k go global -> LDS
// directly, into a ring of D slots of the wave's own: no barrier, D - 1 chunks
// in flight and one loop body.  The body's size matters more than its work:
// a decode call runs each wave through a handful of chunks, and straight-line
// code for them was slower by the instruction fetches (1 x 1024 x 4096: 8.7 us
// with four chunks unrolled).  LDS also does the cross-lane part: with G = 128
// a lane's 16 bytes of codes are 32 consecutive k; with smaller groups a lane
// reads one dword of each 32-element block, so that one product stays inside
// one group, and every lane reads the scale of the block's own lanes.
//
// One row is bound by the start of the waves and the latency of their loads
// (1 x 5120 x 8192 bf16: 22 MB in 10.7 us, 11.7 with weights that are in no
// cache; reading the same bytes in this layout and nothing else takes 6),
// several rows by the instructions issued (13 x 4099 x 7168 fp32: 23 us, 460
// instructions a chunk and wave; 33 tokens x 4 of 16 experts of 4096 x 1024,
// fp32: 30 to 35 us, by the experts' loads).
// ---------------------------------------------------------------------------
// Waves that fill the chip: 8 a CU (1024 or 4096 were no faster anywhere).
constexpr int64_t kRowTarget = 2048;

// A wave's LDS: the ring, and two regions of scales and zero points, which
// come for SG groups at a time (a segment): loads of 4 groups, a group to a
// quad.  A workgroup's is at most half of a CU's 160 KB: two workgroups a CU,
// so that a grid a little above the number of CUs does not take two rounds.
template <bool XF32, int BM>
struct RowRing {
  static constexpr int W = BM <= 4 ? 8 : 4;                     // waves of a workgroup
  static constexpr int XL = BM * (XF32 ? 512 : 256) / 1024;     // x loads of a chunk
  static constexpr int PER = XL + 1;                            // loads of a chunk
  static constexpr int SLOT = PER * 1024;
  static constexpr int SG = PER > 8 ? 8 : 16;
  static constexpr int SEG_BYTES = SG * 16 * 4;
  static constexpr int SCALES = 4 * SEG_BYTES;
  static constexpr int D = (80 * 1024 / W - SCALES) / SLOT;     // as many as fit
  static constexpr int WAVE = D * SLOT + SCALES;
  static constexpr int BYTES = W * WAVE;
  static_assert((D == 2 || D == 3) && (D - 1) * PER < 64, "ring depth");
  // a segment is loaded before the last chunk that precedes its own
  static_assert(SG * 32 / 128 >= D, "segment length");
};

template <bool XF32, int G, int BM, bool ROUTED>
__global__ void __launch_bounds__((RowRing<XF32, BM>::W * 64), 2)
w4_rows_kernel(W4Args a, int item0, int log_ks, int wide) {
  using Ring = RowRing<XF32, BM>;
  constexpr int MT = (BM + 15) / 16, ES = XF32 ? 4 : 2;
  constexpr int UNITS = 128 * ES / 16;  // 16-byte units of a row's chunk
  constexpr int D = Ring::D;
  // no division on the way to the first load: it is a microsecond of a call
  const int ks = 1 << log_ks, cn = Ring::W >> log_ks, BN = 16 * cn;
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  const int tn = blockIdx.x, item = item0 + blockIdx.y;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int kw = wave & (ks - 1), cw = wave >> log_ks;
  const int c16 = lane & 15, quad = lane >> 4;
  Item it;
  if (ROUTED) {
    it = find_item(a.offsets, a.E, a.S, BM, item);
    zero_unused(a, tn * BN, BN, item, gridDim.y, Ring::W * 64);
    if (it.rows == 0) return;
  } else {
    it = Item{0, item * BM, min(a.S - item * BM, BM)};
  }
  const int K = a.K, KG = (int)((unsigned)K / G);
  const int chunks = (int)(((unsigned)K + 127) / 128), per = (chunks + ks - 1) >> log_ks;
  const int c0 = kw * per, c1 = min(c0 + per, chunks);
  const int n = tn * BN + cw * 16 + c16;       // the lane's column

  // Sources: a base that is the wave's plus 32-bit offsets of the lanes, so
  // that a load needs no vector instruction: calls of several rows are bound
  // by the instructions issued (a wave of 13 fp32 rows spends 61 % of its time
  // on them).  `wide`: rows so far apart that the offsets do not fit; then,
  // and where a chunk or segment reaches past the end of the row, every lane
  // makes its address.
  //
  // x: load t brings units 64 t + lane of the slot's x, unit p of row r at p ^
  // (r % 16) so that 16 rows' reads of one unit spread over the banks; rows
  // past the end repeat the first (a row of the product depends on its own
  // row of x alone, and theirs are not stored).
  const int row0 = ROUTED ? 0 : it.p0;
  const uint8_t* const xb = static_cast<const uint8_t*>(a.x) + row0 * a.ldx * ES;
  int xr[Ring::XL], xk[Ring::XL];
  uint32_t xo[Ring::XL];
#pragma unroll
  for (int t = 0; t < Ring::XL; ++t) {
    const int r = (64 * t + lane) / UNITS, u = ((lane % UNITS) ^ (r & 15));
    int64_t row = it.p0 + (r < it.rows ? r : 0);
    if (ROUTED) row = min(max(a.order[row] / a.x_div, 0), a.R - 1);
    xr[t] = (int)row - row0;
    xk[t] = u * (16 / ES);
    xo[t] = (uint32_t)(((int64_t)xr[t] * a.ldx + xk[t]) * ES);
  }
  const bool s16 = a.s_bf16 != 0, has_zero = a.zero != nullptr;
  const int ss = s16 ? 2 : 4;
  const int col0 = min(tn * BN + cw * 16, a.N - 1);
  const int64_t nc = min(n, a.N - 1) - col0;
  const uint8_t* const wb = a.w + it.e * a.w_se + col0 * a.ldw;
  const uint8_t* const sb =
      static_cast<const uint8_t*>(a.scale) + (it.e * a.s_se + col0 * a.s_n) * ss;
  const uint8_t* const zb = has_zero ? a.zero + it.e * a.z_se + col0 * a.z_n : nullptr;
  const uint32_t wo = (uint32_t)(nc * a.ldw + quad * 16);
  const uint32_t so = (uint32_t)((nc * a.s_n + quad) * ss), zo = (uint32_t)(nc * a.z_n + quad);
  const rsrc_t xrs = buffer_at(xb), wrs = buffer_at(wb), srs = buffer_at(sb), zrs = buffer_at(zb);
  uint8_t* const ring = smem + wave * Ring::WAVE;
  uint8_t* const scl = ring + D * Ring::SLOT;
  auto load = [&](int c, uint8_t* slot) {
    const int kc = c * 128;
    if (!wide && (G == 128 || kc + 128 <= K)) {
#pragma unroll
      for (int t = 0; t < Ring::XL; ++t) to_lds<16>(xrs, xo[t], kc * ES, slot + t * 1024);
      to_lds<16>(wrs, wo, kc / 2, slot + Ring::XL * 1024);
    } else {
      // past the end of the row: its start again, in products that are left out
#pragma unroll
      for (int t = 0; t < Ring::XL; ++t) {
        const int k = kc + xk[t];
        to_lds<16>(xb + (xr[t] * a.ldx + (G == 128 || k < K ? k : xk[t] % 32)) * ES,
                   slot + t * 1024);
      }
      const int k = kc + quad * 32;
      to_lds<16>(wb + nc * a.ldw + (G == 128 || k < K ? k : 0) / 2, slot + Ring::XL * 1024);
    }
  };
  // segment i of the wave's groups, to region i % 2
  constexpr int SEG = Ring::SG * G / 128;        // chunks of a segment
  const int g0 = c0 * 128 / G;
  auto load_segment = [&](int i) {
    uint8_t* const dst = scl + (i & 1) * (2 * Ring::SEG_BYTES);
    const int g = g0 + i * Ring::SG;
    const int left = (c1 - c0) * (128 / G) - i * Ring::SG;     // groups the wave has left
    auto each = [&](auto one) {
#pragma unroll
      for (int h = 0; h < Ring::SG / 4; ++h) {
        if (4 * h >= left) break;
        one(g + 4 * h, dst + h * 256);
      }
    };
    if (!wide && g + Ring::SG <= KG) {
      if (s16) each([&](int gg, uint8_t* to) { to_lds<2>(srs, so, 2 * gg, to); });
      else each([&](int gg, uint8_t* to) { to_lds<4>(srs, so, 4 * gg, to); });
      if (has_zero)
        each([&](int gg, uint8_t* to) { to_lds<1>(zrs, zo, gg, to + Ring::SEG_BYTES); });
    } else {
      auto at = [&](int gg, int64_t ld) { return nc * ld + min(gg + quad, KG - 1); };
      if (s16) each([&](int gg, uint8_t* to) { to_lds<2>(sb + 2 * at(gg, a.s_n), to); });
      else each([&](int gg, uint8_t* to) { to_lds<4>(sb + 4 * at(gg, a.s_n), to); });
      if (has_zero)
        each([&](int gg, uint8_t* to) { to_lds<1>(zb + at(gg, a.z_n), to + Ring::SEG_BYTES); });
    }
  };

  f32x4 acc[MT] = {};
  // Without zero points both regions hold 8 for good: the groups' products
  // then have no branch between them and overlap.  This, the scale 0 for
  // groups past the row, sums in ordinary registers (the launch bound's 2) and
  // addresses without vector instructions took 70 x 5120 x 8192 fp32 from 102
  // to 87 us, 13 x 4099 x 7168 fp32 from 29.4 to 26.7, 64 routed tokens x 8
  // from 80 to 75.
  if (!has_zero) {
#pragma unroll
    for (int i = 0; i < 2 * Ring::SEG_BYTES / 256; ++i)
      *reinterpret_cast<uint32_t*>(scl + (i & 1 ? 3 : 1) * Ring::SEG_BYTES + (i >> 1) * 256 +
                                   lane * 4) = 8;
  }
  if (c0 < c1) {
    load(c0, ring);
    load_segment(0);
#pragma unroll 1
    for (int u = 1; u < D && c0 + u < c1; ++u) load(c0 + u, ring + u * Ring::SLOT);
  }
  // the lane's output slots, on their way during the products
  int to[MT][4];
  if constexpr (ROUTED) {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        to[i][r] = a.order[it.p0 + min(16 * i + 4 * quad + r, it.rows - 1)];
  }
  uint8_t* slot = ring;
#pragma unroll 1
  for (int c = c0; c < c1; ++c) {
    // This chunk's loads have landed, and those of the chunks after it may be
    // in flight: the newest ones, whatever scales were loaded among them.
    const int newer = c1 - 1 - c;
    if (newer >= D - 1) wait_vmcnt<(D - 1) * Ring::PER>();
    else if (D == 3 && newer == 1) wait_vmcnt<Ring::PER>();
    else wait_vmcnt<0>();
    // a segment's first chunk fetches the next segment; its own one landed
    // before this chunk did, or with it (the first)
    const int in = (c - c0) & (SEG - 1), seg = (unsigned)(c - c0) / SEG;
    if (in == 0 && c + SEG < c1) load_segment(seg + 1);
    const uint8_t* const sc = scl + (seg & 1) * (2 * Ring::SEG_BYTES) + in * (128 / G) * 64;
    const uint8_t* const codes = slot + Ring::XL * 1024;
    f32x4 d[MT];
    float z = 0.0f;
    u32x4 wv;
    if (G == 128) wv = *reinterpret_cast<const u32x4*>(codes + lane * 16);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const uint8_t* const sl = sc + (t * 32 / G * 16 + c16) * 4;
      if (t * 32 % G == 0) {
#pragma unroll
        for (int i = 0; i < MT; ++i) d[i] = f32x4{};
        z = (float)*reinterpret_cast<const uint32_t*>(sl + Ring::SEG_BYTES);
      }
      const u32x4 wq = unpack(G == 128 ? wv[t]
                                       : *reinterpret_cast<const uint32_t*>(
                                             codes + (16 * t + c16) * 16 + quad * 4),
                              z);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const int r = BM < 16 ? c16 % BM : 16 * i + c16;
        const int k = G == 128 ? quad * 32 + t * 8 : t * 32 + quad * 8;
        const uint8_t* xs = slot + r * (UNITS * 16);
        X8<XF32> x;
        if constexpr (XF32) {
          x.a = *reinterpret_cast<const u32x4*>(xs + ((k / 4) ^ (r & 15)) * 16);
          x.b = *reinterpret_cast<const u32x4*>(xs + ((k / 4 + 1) ^ (r & 15)) * 16);
        } else {
          x.v = *reinterpret_cast<const u32x4*>(xs + ((k / 8) ^ (r & 15)) * 16);
        }
        const Parts<XF32> p = parts(x);
#pragma unroll
        for (int h = (XF32 ? 3 : 1) - 1; h >= 0; --h) d[i] = mfma(p.p[h], wq, d[i]);
      }
      if ((t + 1) * 32 % G == 0) {
        const uint32_t sv = *reinterpret_cast<const uint32_t*>(sl);
        // groups past the end of the row: scale 0
        const bool in_row = G == 128 || c * 128 + t * 32 < K;
        const float sf = in_row ? __uint_as_float(s16 ? sv << 16 : sv) : 0.0f;
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            acc[i][r] = __builtin_fmaf(sf, d[i][r], acc[i][r]);
      }
    }
    wait_lgkm0();             // the slot has been read
    if (c + D < c1) load(c + D, slot);
    slot = slot == ring + (D - 1) * Ring::SLOT ? ring : slot + Ring::SLOT;
  }

  // partial sums of K ranges 1 .. ks - 1 to LDS (over the rings, whose loads
  // have all landed), added in order by range 0
  if (ks > 1) {
    float* const red = reinterpret_cast<float*>(smem);
    __syncthreads();
    if (kw > 0) {
      float* r0 = red + ((kw - 1) * cn + cw) * (MT * 256);
#pragma unroll
      for (int i = 0; i < MT; ++i) *reinterpret_cast<f32x4*>(r0 + i * 256 + lane * 4) = acc[i];
    }
    __syncthreads();
    if (kw > 0) return;
#pragma unroll 1
    for (int w = 0; w < ks - 1; ++w) {
      const float* r0 = red + (w * cn + cw) * (MT * 256);
#pragma unroll
      for (int i = 0; i < MT; ++i)
        acc[i] += *reinterpret_cast<const f32x4*>(r0 + i * 256 + lane * 4);
    }
  }
  if constexpr (ROUTED) {
    if (a.row_scale) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i][r] *= a.row_scale[min(max(to[i][r], 0), a.S - 1)];
    }
  }
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int m = 16 * i + 4 * quad + r;
      int64_t row = it.p0 + m;
      if constexpr (ROUTED) row = to[i][r];
      if (m >= it.rows || (ROUTED && (row < 0 || row >= a.S))) continue;
      if (n < a.N) store_out(a, row * a.ldo + n, acc[i][r]);
    }
}

// ---------------------------------------------------------------------------
// Many rows: tiles of BM = 64 * WM rows by BN = 64 * WN columns, a wave to
// each 64 x 64 (2 x 2 blocks of 32 x 32 x 16 instructions), K in steps of 64.
//
// The x tile goes global -> LDS directly into a ring of three slots, two
// steps ahead.  The weight tile is held in LDS as bf16 integers code - zero
// (exact), in two slots: each thread keeps the codes of one column's run two
// steps ahead in registers and unpacks the next step's while this step's
// matrix instructions run, so that a code is unpacked once per workgroup and
// not once per wave.  A group's sum is then folded into the accumulator with
// one multiply-add by the lane's column scale.
//
// LDS rows are 128 bytes (64 bf16) with the 16-byte chunks XOR-swizzled, so
// that the 16 consecutive rows of a fragment read hit distinct banks.
//
// A step takes 0.8 (128 rows) to 0.95 us (256), of which the matrix cores
// need 0.54: LDS reads, unpacking and folds hide only in part.  2047 x 5120 x
// 8192 bf16 takes 236 us, 727 Tflop/s; 1021 tokens x 8 of 32 experts of 2048 x
// 4096 235 us, 584 Tflop/s.
// ---------------------------------------------------------------------------
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) void* lds_ptr_t;

constexpr int kStepK = 64;

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

struct TileArgs {
  const uint16_t* x;      // bf16 planes [planes][R][ldx]
  int64_t ldx;
  uint32_t plane;         // bytes from one plane to the next
  int planes;
  uint32_t x_bytes;       // of all planes, below 2^32
  int items, ntn;
};

template <int G, bool S16, int WM, int WN, bool ROUTED>
__global__ void __launch_bounds__(WM * WN * 64, 2) w4_tile_kernel(W4Args a, TileArgs ta) {
  constexpr int NW = WM * WN, NT = NW * 64;
  constexpr int BM = 64 * WM, BN = 64 * WN;
  constexpr int XS = BM * 128, BS = BN * 128;       // bytes of a slot
  constexpr int LA = BM / 8 / NW;                   // x loads per wave and step
  constexpr int CB = BN * 32 / NT;                  // code bytes per thread and step (8 or 16)
  constexpr int CW = CB / 4;
  constexpr int NG = G < 64 ? 64 / G : 1;           // scale groups in a step
  static_assert(CB == 8 || CB == 16, "one wide load of codes per thread");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[3 * XS + 2 * BS];
  uint8_t* const xs = smem;
  uint8_t* const bs = smem + 3 * XS;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int wm = wave / WN, wn = wave % WN;
  const int c32 = lane & 31, half = lane >> 5;
  int item, tn;
  tile_of(ta.items, ta.ntn, item, tn);
  Item it;
  if (ROUTED) {
    it = find_item(a.offsets, a.E, a.S, BM, item);
    zero_unused(a, tn * BN, BN, item, ta.items, NT);
    if (it.rows == 0) return;
  } else {
    it = Item{0, item * BM, min(a.S - item * BM, BM)};
  }

  // x: wave instruction t brings rows 8 (t NW + wave) + lane / 8 of the tile;
  // rows past the end repeat the first
  uint32_t xo[LA];
#pragma unroll
  for (int t = 0; t < LA; ++t) {
    const int r = (t * NW + wave) * 8 + (lane >> 3);
    int64_t row = it.p0 + (r < it.rows ? r : 0);
    if (ROUTED) row = min(max(a.order[row] / a.x_div, 0), a.R - 1);
    xo[t] = (uint32_t)(row * ta.ldx * 2) + (((lane & 7) ^ swz(r)) << 4);
  }
  const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint16_t*>(ta.x), (short)0, (int)ta.x_bytes, 0x00020000);

  // codes: this thread's column and its run of CB bytes of every step
  const int bc = threadIdx.x / (32 / CB), part = threadIdx.x % (32 / CB);
  const int64_t bn = min(tn * BN + bc, a.N - 1);
  const uint8_t* wp = a.w + it.e * a.w_se + bn * a.ldw + part * CB;
  // without zero points the byte that is read (a scale's) is not used
  const uint8_t* zp = (a.zero ? a.zero + it.e * a.z_se + bn * a.z_n
                              : static_cast<const uint8_t*>(a.scale)) + part * CB * 2 / G;
  const bool has_zero = a.zero != nullptr;
  using scale_t = std::conditional_t<S16, uint16_t, uint32_t>;
  const scale_t* sp[2];
#pragma unroll
  for (int j = 0; j < 2; ++j)
    sp[j] = static_cast<const scale_t*>(a.scale) + it.e * a.s_se +
            (int64_t)min(tn * BN + wn * 64 + j * 32 + c32, a.N - 1) * a.s_n;

  const int K = a.K;
  const int steps1 = (K + kStepK - 1) / kStepK;       // per plane
  const int steps = steps1 * ta.planes;
  // the last step of a plane has only its first group (G = 32)
  auto half_step = [&](int ks) { return G == 32 && (ks + 1) * kStepK > K; };
  struct Codes { uint32_t w[CW]; uint8_t z; };
  struct Scales { scale_t s[NG][2]; };
  // A step: its K step within the plane, its byte offset in x
  struct Pos {
    int ks;
    uint32_t off;
  };
  auto next_pos = [&](Pos p) {
    const bool wrap = p.ks + 1 == steps1;
    return Pos{wrap ? 0 : p.ks + 1,
               p.off + (wrap ? ta.plane - (uint32_t)(steps1 - 1) * (kStepK * 2) : kStepK * 2)};
  };

  auto load_x = [&](Pos p, uint32_t slot) {
    // the missing half of a half step repeats the first (never read): no
    // load reaches past its row
    const uint32_t back = half_step(p.ks) && (((lane & 7) ^ (lane >> 3)) & 4) ? 64u : 0u;
#pragma unroll
    for (int t = 0; t < LA; ++t) {
      const lds_ptr_t l =
          (lds_ptr_t)(uintptr_t)(uint32_t)(uintptr_t)(xs + slot + (t * NW + wave) * 1024);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, l, 16, (int)(xo[t] - back), (int)p.off, 0, 0);
    }
  };
  auto load_codes = [&](Codes& c, Pos p) {
    // past a half step: the row's start again, not used
    const bool past = half_step(p.ks) && part * CB >= 16;
    const int at = past ? -part * CB : p.ks * 32;
    if constexpr (CB == 16) {
      const u32x4 v = *reinterpret_cast<const u32x4*>(wp + at);
#pragma unroll
      for (int i = 0; i < 4; ++i) c.w[i] = v[i];
    } else {
      const uint2 v = *reinterpret_cast<const uint2*>(wp + at);
      c.w[0] = v.x;
      c.w[1] = v.y;
    }
    c.z = zp[past ? -(part * CB * 2 / G) : p.ks * kStepK / G];
  };
  auto load_scales = [&](Scales& c, int ks) {
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const int i = g == 1 && half_step(ks) ? 0 : ks * kStepK / G + g;
#pragma unroll
      for (int j = 0; j < 2; ++j) c.s[g][j] = sp[j][i];
    }
  };
  uint32_t wo[CW];      // where this thread's unpacked codes go in a weight slot
#pragma unroll
  for (int i = 0; i < CW; ++i) wo[i] = lds_off(bc, part * CW + i);
  auto zero_of = [&](const Codes& c) { return has_zero ? (float)c.z : 8.0f; };
  auto write_code = [&](u32x4 v, int i, uint32_t slot) {
    *reinterpret_cast<u32x4*>(bs + slot + wo[i]) = v;
  };

  // d: the open group's sums; pend: the scales of the group that d holds
  // until its next group's first product replaces it
  f32x16 acc[2][2] = {}, d[2][2] = {};
  float pend[2] = {0.0f, 0.0f};
  auto fold = [&](int i, int j) {
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[i][j][r] = __builtin_fmaf(pend[j], d[i][j][r], acc[i][j][r]);
  };
  struct Frag { u32x4 a[2], b[2]; };
  uint32_t fo[4];       // a lane's fragment offsets in either tile, rows c32
#pragma unroll
  for (int t = 0; t < 4; ++t) fo[t] = lds_off(c32, 2 * t + half);
  auto frags = [&](Frag& f, int t, const uint8_t* xt, const uint8_t* bt) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      f.a[i] = *reinterpret_cast<const u32x4*>(xt + fo[t] + i * 4096);
      f.b[i] = *reinterpret_cast<const u32x4*>(bt + fo[t] + i * 4096);
    }
  };

  // prologue: codes of steps 0 and 1, x of 0 and 1, scales of 0
  Codes c0, c1;
  Scales s0, s1;
  Pos p0{0, 0};
  Pos p1 = next_pos(p0), p2 = next_pos(p1);
  uint32_t x0 = 0, x1 = XS, x2 = 2 * XS;     // x slots of this step, the next, the one after
  load_codes(c0, p0);
  load_scales(s0, 0);
  load_x(p0, x0);
  c1 = c0;
  if (steps > 1) {
    load_codes(c1, p1);
    load_x(p1, x1);
  }
#pragma unroll
  for (int i = 0; i < CW; ++i) {
    u32x4 v;
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = unpack_pair(c0.w[i], q, zero_of(c0));
    write_code(v, i, 0);
  }
  // One step: the products of 64 k, in four turns of 16 k by four blocks.
  // ODD: its parity (weight slot; for G = 128 the group's half).  HOT: two
  // more steps follow, so the body has no branch.
  //
  // The source order is the schedule.  A turn's fragments are read during the
  // turn before; the barrier stands before the last turn, whose products then
  // cover the first fragments of the next step.  Unpacking and folds are
  // shared out between the products, which leave the VALU about four
  // instructions each.  A group's blocks (0, 0) and (0, 1) are folded in its
  // last turn, the other two in the next group's first.
  Frag f[2];
  // the pairs of codes unpacked before product n: 8 in turns 1 and 2, or 16
  // in turns 0 to 2
  auto first_pair = [](int n) {
    return CW == 4 ? (n < 12 ? n * 4 / 3 : 16) : n < 4 ? 0 : n < 12 ? n - 4 : 8;
  };
  auto step = [&](auto odd, auto hot, int s, const Codes& next, Codes& after, const Scales& now,
                  Scales& later) {
    constexpr int ODD = decltype(odd)::value;
    constexpr bool HOT = decltype(hot)::value;
    const uint8_t* xt = xs + x0 + wm * 64 * 128;
    const uint8_t* bt = bs + ODD * BS + wn * 64 * 128;
    const float z = zero_of(next);
    // the second group of a half step is not there: its x and codes repeat
    // finite values, its scale is 0
    const bool cut = half_step(p0.ks);
    u32x4 v;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const bool first = G == 128 ? ODD == 0 && t == 0 : t * 16 % G == 0;
      const bool last = G == 128 ? ODD == 1 && t == 3 : (t + 1) * 16 % G == 0;
      if (t == 3) {
        // this wave's x loads of the next step have landed (newer: this
        // step's codes, zero point and x), its fragments and weights too;
        // then everyone's
        if (HOT || s + 2 < steps) wait_vmcnt<LA + 2>(); else wait_vmcnt<0>();
        wait_lgkm0();
        barrier();
        if (HOT || s + 1 < steps)
          frags(f[0], 0, xs + x1 + wm * 64 * 128, bs + (1 - ODD) * BS + wn * 64 * 128);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int i = q >> 1, j = q & 1;
        d[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
            __builtin_bit_cast(bf16x8, f[t & 1].a[i]), __builtin_bit_cast(bf16x8, f[t & 1].b[j]),
            first ? f32x16{} : d[i][j], 0, 0, 0);
        if (q == 0 && t < 3) frags(f[(t + 1) & 1], t + 1, xt, bt);
        if (first && q < 2) fold(1, q);
        if (last && q == 0) {
          const int g = G < 64 ? t * 16 / G : 0;
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            pend[n] = __uint_as_float(S16 ? (uint32_t)now.s[g][n] << 16 : now.s[g][n]);
            if (g == 1 && cut) pend[n] = 0.0f;
          }
        }
        if (last && q >= 2) fold(0, q - 2);
        if (q == 1 && t == 0) {
          if (HOT || s + 1 < steps) load_scales(later, p1.ks);
          if (HOT || s + 2 < steps) load_codes(after, p2);
        }
        if (q == 3 && t == 0 && (HOT || s + 2 < steps)) load_x(p2, x2);
        // the next step's weights (after the last step: to a slot nobody
        // reads), all written before the barrier of turn 3
#pragma unroll
        for (int p = first_pair(4 * t + q); p < first_pair(4 * t + q + 1); ++p) {
          v[p & 3] = unpack_pair(next.w[p >> 2], p & 3, z);
          if ((p & 3) == 3) write_code(v, p >> 2, (1 - ODD) * BS);
        }
        if (HOT) __builtin_amdgcn_sched_barrier(0);
      }
    }
    p0 = p1;
    p1 = p2;
    p2 = next_pos(p2);
    const uint32_t x = x0;
    x0 = x1;
    x1 = x2;
    x2 = x;
  };
  if (steps > 1) wait_vmcnt<LA>(); else wait_vmcnt<0>();      // x of step 0
  wait_lgkm0();
  barrier();
  frags(f[0], 0, xs + x0 + wm * 64 * 128, bs + wn * 64 * 128);
  constexpr std::integral_constant<int, 0> even{};
  constexpr std::integral_constant<int, 1> odd{};
  int s = 0;
  for (; s + 3 < steps; s += 2) {
    step(even, std::true_type{}, s, c1, c0, s0, s1);
    step(odd, std::true_type{}, s + 1, c0, c1, s1, s0);
  }
  for (; s < steps; s += 2) {
    step(even, std::false_type{}, s, c1, c0, s0, s1);
    if (s + 1 >= steps) break;
    step(odd, std::false_type{}, s + 1, c0, c1, s1, s0);
  }

#pragma unroll
  for (int j = 0; j < 2; ++j) fold(1, j);
  // Out: the slots and scales of a lane's 32 rows are loaded together (one
  // after another, between the stores: 1021 tokens x 8 of 32 experts, 2048 x
  // 4096, took 281 us instead of 256, 512 x 4 of 16, 2048 x 2048, 59 for 50).
  const int n0 = tn * BN + wn * 64 + c32;
  auto row_of = [&](int i, int r) {
    return wm * 64 + i * 32 + (r >> 2) * 8 + half * 4 + (r & 3);
  };
  int slot[2][16];
  if constexpr (ROUTED) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r)
        slot[i][r] = a.order[it.p0 + min(row_of(i, r), it.rows - 1)];
    if (a.row_scale) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const float rsc = a.row_scale[min(max(slot[i][r], 0), a.S - 1)];
          acc[i][0][r] *= rsc;
          acc[i][1][r] *= rsc;
        }
    }
  }
  auto out = [&](auto put) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int m = row_of(i, r);
        int64_t row = it.p0 + m;
        if constexpr (ROUTED) row = slot[i][r];
        if (m >= it.rows || (ROUTED && (row < 0 || row >= a.S))) continue;
#pragma unroll
        for (int j = 0; j < 2; ++j)
          if (n0 + 32 * j < a.N) put(row * a.ldo + n0 + 32 * j, acc[i][j][r]);
      }
  };
  if (a.out_dtype == BSMM_BF16)
    out([&](int64_t at, float v) { static_cast<uint16_t*>(a.out)[at] = (uint16_t)bf16_bits(v); });
  else
    out([&](int64_t at, float v) { static_cast<float*>(a.out)[at] = v; });
}

// fp32 activations as three bf16 planes that add up to them exactly
__global__ void __launch_bounds__(256) split_planes(const float* __restrict__ x, int64_t ldx,
                                                    uint16_t* __restrict__ planes, int64_t plane,
                                                    int K, int64_t chunks) {
  const int per_row = K / 8;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < chunks;
       i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / per_row;
    const int k = (int)(i - row * per_row) * 8;
    const u32x4* src = reinterpret_cast<const u32x4*>(x + row * ldx + k);
    u32x4 u = src[0], v = src[1];
#pragma unroll
    for (int p = 0; p < 3; ++p) {
      *reinterpret_cast<u32x4*>(planes + p * plane + row * K + k) =
          u32x4{hi2(u.x, u.y), hi2(u.z, u.w), hi2(v.x, v.y), hi2(v.z, v.w)};
      if (p < 2) {
        u = u32x4{below(u.x), below(u.y), below(u.z), below(u.w)};
        v = u32x4{below(v.x), below(v.y), below(v.z), below(v.w)};
      }
    }
  }
}

template <int G, bool S16, int WM, int WN, bool ROUTED>
void launch_tiles(const W4Args& a, void* ws, hipStream_t st) {
  constexpr int BM = 64 * WM, BN = 64 * WN;
  TileArgs t{};
  t.ntn = (a.N + BN - 1) / BN;
  if (a.x_dtype == BSMM_F32) {
    uint16_t* planes = static_cast<uint16_t*>(ws);
    const int64_t chunks = (int64_t)a.R * (a.K / 8);
    const int64_t blocks = (chunks + 255) / 256;
    hipLaunchKernelGGL(split_planes, dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(256),
                       0, st, static_cast<const float*>(a.x), a.ldx, planes,
                       (int64_t)a.R * a.K, a.K, chunks);
    t.x = planes;
    t.ldx = a.K;
    t.planes = 3;
    t.plane = (uint32_t)((int64_t)a.R * a.K * 2);
    t.x_bytes = 3 * t.plane;
  } else {
    t.x = static_cast<const uint16_t*>(a.x);
    t.ldx = a.ldx;
    t.planes = 1;
    t.x_bytes = (uint32_t)(((int64_t)(a.R - 1) * a.ldx + a.K) * 2);
  }
  t.items = ROUTED ? (int)(((int64_t)a.S + (int64_t)(a.E < a.S ? a.E : a.S) * (BM - 1)) / BM)
                   : (int)(((int64_t)a.S + BM - 1) / BM);
  hipLaunchKernelGGL((w4_tile_kernel<G, S16, WM, WN, ROUTED>), dim3((unsigned)(t.items * t.ntn)),
                     dim3(WM * WN * 64), 0, st, a, t);
}

// As many K ranges as leave about 8 waves to a CU, at most one per chunk.
template <bool XF32, int G, int BM>
void launch_rows(const W4Args& a, hipStream_t st) {
  const int64_t act = a.E < a.S ? a.E : a.S;
  const int64_t items = a.offsets ? (a.S + act * (BM - 1)) / BM : ((int64_t)a.S + BM - 1) / BM;
  // routed: about half of a block is missing from an expert's last one
  const int64_t busy = a.offsets ? (a.S + act * (BM / 2)) / BM + 1 : items;
  const int64_t tiles = busy * ((a.N + 15) / 16);
  const int chunks = (a.K + 127) / 128;
  constexpr int W = RowRing<XF32, BM>::W;
  int log_ks = 0;
  while ((1 << log_ks) < W && (tiles << log_ks) < kRowTarget && (2 << log_ks) <= chunks) ++log_ks;
  const int BN = 16 * (W >> log_ks);
  const dim3 block(W * 64);
  // the lanes' 32-bit offsets: from the item's first row (routed: from row 0)
  // and from the wave's first column
  const int64_t limit = (int64_t)1 << 31;
  const int64_t x_rows = a.offsets ? a.R : BM;
  const int wide = x_rows * a.ldx * (XF32 ? 4 : 2) >= limit || 16 * a.ldw >= limit ||
                   64 * a.s_n >= limit || 16 * a.z_n >= limit;
  constexpr int lds = RowRing<XF32, BM>::BYTES;
  // at most 65535 items a launch
  for (int64_t i = 0; i < items; i += 65535) {
    const dim3 grid((unsigned)((a.N + BN - 1) / BN),
                    (unsigned)(items - i < 65535 ? items - i : 65535));
    if (a.offsets)
      hipLaunchKernelGGL((w4_rows_kernel<XF32, G, BM, true>), grid, block, lds, st, a, (int)i,
                         log_ks, wide);
    else
      hipLaunchKernelGGL((w4_rows_kernel<XF32, G, BM, false>), grid, block, lds, st, a, (int)i,
                         log_ks, wide);
  }
}

template <bool XF32, int G>
void launch_few(const W4Args& a, hipStream_t st) {
  const int rows = w4_item_rows(a);
  if (rows == 4) launch_rows<XF32, G, 4>(a, st);
  else if (rows == 16) launch_rows<XF32, G, 16>(a, st);
  else launch_rows<XF32, G, XF32 ? 16 : 32>(a, st);        // fp32 never gets here
}

template <int G, bool S16>
void launch_plan(const W4Args& a, W4Plan plan, void* ws, hipStream_t st) {
  if (plan == W4Plan::Tile256) launch_tiles<G, S16, 4, 2, false>(a, ws, st);
  else if (a.offsets) launch_tiles<G, S16, 2, 2, true>(a, ws, st);
  else launch_tiles<G, S16, 2, 2, false>(a, ws, st);
}

template <int G>
void launch_group(const W4Args& a, W4Plan plan, void* ws, hipStream_t st) {
  if (plan != W4Plan::Rows) {
    if (a.s_bf16) launch_plan<G, true>(a, plan, ws, st);
    else launch_plan<G, false>(a, plan, ws, st);
    return;
  }
  if (a.x_dtype == BSMM_F32) launch_few<true, G>(a, st);
  else launch_few<false, G>(a, st);
}

}  // namespace

int launch_w4(const W4Args& a, W4Plan plan, void* ws, void* stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (a.group == 32) launch_group<32>(a, plan, ws, st);
  else if (a.group == 64) launch_group<64>(a, plan, ws, st);
  else launch_group<128>(a, plan, ws, st);
  return hipGetLastError() == hipSuccess ? 0 : 1;
}

}  // namespace bsmm
