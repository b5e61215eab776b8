// 8-bit checkpoints of activations, and the gate silu(g) * u of a feed-forward
// layer with its gradient from one (gfx950).
//
// A checkpoint holds int8 codes and, per 32 elements of a row, a power of two
// as an e8m0 byte (the OCP microscaling format MXINT8): with amax = m 2^p, m
// in [1, 2),
//   byte = p + 127 (0 below 2^-127, 127 for amax 0),  code = rne(x 2^(6-p))
//   within +-127,  value = code 2^(byte - 133)
// A block that holds an infinity or a NaN gets byte 255, codes 0, and stands
// for NaNs.  Integers and not e4m3: an activation kept for the backward pass
// wants precision near its block's maximum, not range (largest error 2^-7 of
// amax where e4m3 has 2^-4 of the element), and a value has at most 7 bits, so
// that it is exact in bf16 and the products that read it need no rounding.
//
// All kernels read and write each byte once: bound by HBM.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "bsmm.h"
#include "bsmm_internal.h"
#include "bsmm_routed.h"

namespace bsmm {
namespace {

// ---- 8 consecutive elements of a row, as fp32 --------------------------------

__device__ __forceinline__ void load8(const uint16_t* p, float (&f)[8]) {
  const u32x4 v = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(v[i] << 16);
    f[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
  const f32x4 a = reinterpret_cast<const f32x4*>(p)[0], b = reinterpret_cast<const f32x4*>(p)[1];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[i] = a[i];
    f[4 + i] = b[i];
  }
}
__device__ __forceinline__ void store8(uint16_t* p, const float (&f)[8]) {
  u32x4 v;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t{f[2 * i], f[2 * i + 1]}),
                                                                bf16x2_t));
  *reinterpret_cast<u32x4*>(p) = v;
}
__device__ __forceinline__ void store8(float* p, const float (&f)[8]) {
  reinterpret_cast<f32x4*>(p)[0] = f32x4{f[0], f[1], f[2], f[3]};
  reinterpret_cast<f32x4*>(p)[1] = f32x4{f[4], f[5], f[6], f[7]};
}

// ---- codes ---------------------------------------------------------------------

// The byte of the 32 elements that a quad of lanes holds, 8 each.
__device__ __forceinline__ int block_byte(const float (&f)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(f[i]) & 0x7FFFFFFFu);
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xF, 0xF, false));
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xF, 0xF, false));
  // the exponent field is p + 127, 0 for subnormals and 255 for inf and NaN
  return m == 0 ? 127 : (int)(m >> 23);
}

// Codes (as integers in f) and their packed form.
__device__ __forceinline__ uint2 encode(float (&f)[8], int byte) {
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float t = __builtin_rintf(__builtin_ldexpf(f[i], 133 - byte));
    f[i] = byte == 255 ? 0.0f : __builtin_amdgcn_fmed3f(t, -127.0f, 127.0f);
    c[i] = (uint32_t)(int)f[i];
  }
  auto four = [](uint32_t p, uint32_t q, uint32_t r, uint32_t s) {
    const uint32_t lo = __builtin_amdgcn_perm(q, p, 0x0C0C0400u);
    const uint32_t hi = __builtin_amdgcn_perm(s, r, 0x0C0C0400u);
    return __builtin_amdgcn_perm(hi, lo, 0x05040100u);
  };
  return make_uint2(four(c[0], c[1], c[2], c[3]), four(c[4], c[5], c[6], c[7]));
}

// What 8 codes stand for.
__device__ __forceinline__ void decode(uint2 c, int byte, float (&f)[8]) {
  const float s = byte == 255 ? __builtin_nanf("") : __builtin_ldexpf(1.0f, byte - 133);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    f[i] = (float)(int8_t)(((i < 4 ? c.x : c.y) >> (8 * (i & 3))) & 0xFFu) * s;
}

// The codes of the lane's 8 elements, and their byte by a quad's first lane.
__device__ __forceinline__ void save8(float (&f)[8], int8_t* q, uint8_t* scale, int k, int byte) {
  const uint2 c = encode(f, byte);
  *reinterpret_cast<uint2*>(q + k) = c;
  if ((k & 31) == 0) scale[k >> 5] = (uint8_t)byte;
}

// 8 elements a thread: 16-byte loads, 4 lanes to a block.  16384 x 5120 bf16
// with the values: 72 us, 5.8 TB/s.
template <typename T>
__global__ void __launch_bounds__(256) quant_int8_mx(QuantI8MxArgs a, unsigned chunks) {
  const unsigned per_row = (unsigned)a.K / 8;
  for (unsigned i = blockIdx.x * 256 + threadIdx.x; i < chunks; i += gridDim.x * 256) {
    const int64_t row = i / per_row;
    const int k = (int)(i - (unsigned)row * per_row) * 8;
    float f[8];
    load8(static_cast<const T*>(a.x) + row * a.ldx + k, f);
    const int byte = block_byte(f);
    save8(f, a.q + row * a.ldq, a.scale + row * a.s_r, k, byte);
    if (a.values) {
      const float s = byte == 255 ? __builtin_nanf("") : __builtin_ldexpf(1.0f, byte - 133);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] *= s;
      store8(static_cast<T*>(a.values) + row * a.ldv + k, f);
    }
  }
}

// A checkpoint's values in bf16, rows of K.  4096 x 4096: 15 us with nothing in
// the caches, 3.3 TB/s.
__global__ void __launch_bounds__(256) restore_bf16(const int8_t* q, int64_t ldq,
                                                    const uint8_t* scale, int64_t s_r,
                                                    uint16_t* out, unsigned K, int64_t chunks) {
  const unsigned per_row = K / 8;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < chunks;
       i += (int64_t)gridDim.x * 256) {
    const int64_t row = chunks <= 0x7FFFFFFF ? (unsigned)i / per_row : i / per_row;
    const int k = (int)(i - row * per_row) * 8;
    float f[8];
    decode(*reinterpret_cast<const uint2*>(q + row * ldq + k), scale[row * s_r + (k >> 5)], f);
    store8(out + row * K + k, f);
  }
}

// ---- gate ----------------------------------------------------------------------

// log2(e) and what is missing of it, negative
constexpr float kLog2e = -1.44269502162933349609375f, kLog2eRest = -1.925963033500011079e-8f;

// sigma(g) = 1 / (1 + e^-g) = 2^-25 / (2^-25 + e) with e = 2^-25 e^-g, which
// stays in fp32 down to g = -104, below which sigma is 0 (e^-104 < 2^-150); and
// the sum stays below 2^126, from where on its reciprocal would be flushed.
// Above 30 sigma is 1.  e^-g = 2^n 2^f, the exponent's whole part n - 25 read
// from the low bits of a sum with 1.5 * 2^23 - 25.  A NaN gate gives a number:
// the caller multiplies by g, which keeps it.
__device__ __forceinline__ float sigma(float g) {
  constexpr float kWhole = 12582912.0f - 25.0f;
  const float x = __builtin_amdgcn_fmed3f(g, -104.0f, 30.0f);
  const float t = __builtin_fmaf(x, kLog2e, kWhole), n = t - kWhole;
  const float f = __builtin_fmaf(x, kLog2eRest, __builtin_fmaf(x, kLog2e, -n));
  const float e = __uint_as_float(__float_as_uint(__builtin_amdgcn_exp2f(f)) +
                                  (__float_as_uint(t) << 23));
  return __builtin_amdgcn_rcpf(e + 0x1p-25f) * 0x1p-25f;
}

// sigma(g) and sigma(-g) = 1 - sigma(g), from p = e^-|g| in [0, 1]: as 1 / (1 +
// p) and p / (1 + p) neither leaves fp32, and the small one falls to 0 where it
// is below 2^-150, on either side, instead of to a power of two that a large g
// would multiply.
struct Sigmas {
  float s, c;
};
__device__ __forceinline__ Sigmas sigmas(float g) {
  const float x = __builtin_fminf(__builtin_fabsf(g), 104.0f);
  const float n = __builtin_rintf(x * kLog2e);
  const float f = __builtin_fmaf(x, kLog2eRest, __builtin_fmaf(x, kLog2e, -n));
  const float p = __builtin_ldexpf(__builtin_amdgcn_exp2f(f), (int)n);
  const float big = __builtin_amdgcn_rcpf(1.0f + p), small = p * big;
  return g < 0.0f ? Sigmas{small, big} : Sigmas{big, small};
}

// 32768 x 2048 bf16 with the checkpoint: 100 us, 5.4 TB/s.
template <typename T, bool CKPT>
__global__ void __launch_bounds__(256) swiglu(SwigluArgs a, unsigned chunks) {
  const unsigned per_row = (unsigned)a.F / 8;
  for (unsigned i = blockIdx.x * 256 + threadIdx.x; i < chunks; i += gridDim.x * 256) {
    const int64_t row = i / per_row;
    const int k = (int)(i - (unsigned)row * per_row) * 8;
    const T* h = static_cast<const T*>(a.h) + row * a.ldh + k;
    float g[8], u[8], v[8];
    load8(h, g);
    load8(h + a.F, u);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = g[j] * sigma(g[j]) * u[j];
    store8(static_cast<T*>(a.a) + row * a.lda + k, v);
    if constexpr (CKPT) {
      int8_t* q = a.q + row * a.ldq;
      uint8_t* s = a.scale + row * a.s_r;
      save8(g, q, s, k, block_byte(g));
      save8(u, q + a.F, s + a.F / 32, k, block_byte(u));
    }
  }
}

// A wave to a row, so that the row's sum needs no other wave.  32768 x 2048
// bf16 with act and the sums: 123 us, 5.5 TB/s.
template <typename T>
__global__ void __launch_bounds__(256) swiglu_backward(SwigluBackArgs a) {
  const int lane = threadIdx.x & 63;
  for (int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); row < a.R;
       row += (int64_t)gridDim.x * 4) {
    const T* da = static_cast<const T*>(a.da) + row * a.ldda;
    const int8_t* q = a.q + row * a.ldq;
    const uint8_t* s = a.scale + row * a.s_r;
    T* dh = static_cast<T*>(a.dh) + row * a.lddh;
    const float r = a.row_scale ? a.row_scale[row] : 1.0f;
    float sum = 0.0f;
    for (int k = lane * 8; k < a.F; k += 512) {
      float d[8], g[8], u[8];
      load8(da + k, d);
      decode(*reinterpret_cast<const uint2*>(q + k), s[k >> 5], g);
      decode(*reinterpret_cast<const uint2*>(q + a.F + k), s[(a.F + k) >> 5], u);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const Sigmas sg = sigmas(g[j]);
        const float silu = g[j] * sg.s, act = silu * u[j];
        sum = __builtin_fmaf(d[j], act, sum);
        const float rd = r * d[j];
        // silu' = sg (1 + g (1 - sg))
        const float slope = __builtin_fmaf(silu, sg.c, sg.s);
        g[j] = rd * (u[j] * slope);              // the slope is at most 1.1
        u[j] = rd * silu;
        d[j] = r * act;
      }
      store8(dh + k, g);
      store8(dh + a.F + k, u);
      if (a.act) store8(static_cast<T*>(a.act) + row * a.ldact + k, d);
    }
    if (a.drow) {
#pragma unroll
      for (int m = 32; m > 0; m >>= 1) sum += __shfl_xor(sum, m);
      if (lane == 0) a.drow[row] = sum;
    }
  }
}

// Workgroups for `threads` of work, 256 each; beyond 65536 of them they loop.
unsigned blocks_for(int64_t threads) {
  const int64_t b = (threads + 255) / 256;
  return (unsigned)(b < 65536 ? b : 65536);
}

}  // namespace

int launch_quant_int8_mx(const QuantI8MxArgs& a, void* stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  const int64_t chunks = a.R * (a.K / 8);
  const dim3 grid(blocks_for(chunks)), block(256);
  if (a.x_dtype == BSMM_BF16)
    hipLaunchKernelGGL(quant_int8_mx<uint16_t>, grid, block, 0, st, a, (unsigned)chunks);
  else
    hipLaunchKernelGGL(quant_int8_mx<float>, grid, block, 0, st, a, (unsigned)chunks);
  return hipGetLastError() == hipSuccess ? 0 : 1;
}

int launch_restore_bf16(const void* q, int64_t ldq, const uint8_t* scale, int64_t s_r, void* out,
                        int64_t R, int64_t K, void* stream) {
  const int64_t chunks = R * (K / 8);
  hipLaunchKernelGGL(restore_bf16, dim3(blocks_for(chunks)), dim3(256), 0,
                     static_cast<hipStream_t>(stream), static_cast<const int8_t*>(q), ldq, scale,
                     s_r, static_cast<uint16_t*>(out), (unsigned)K, chunks);
  return hipGetLastError() == hipSuccess ? 0 : 1;
}

int launch_swiglu(const SwigluArgs& a, void* stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  const int64_t chunks = a.R * (a.F / 8);
  const dim3 grid(blocks_for(chunks)), block(256);
  const unsigned n = (unsigned)chunks;
  if (a.dtype == BSMM_BF16) {
    if (a.q) hipLaunchKernelGGL((swiglu<uint16_t, true>), grid, block, 0, st, a, n);
    else hipLaunchKernelGGL((swiglu<uint16_t, false>), grid, block, 0, st, a, n);
  } else {
    if (a.q) hipLaunchKernelGGL((swiglu<float, true>), grid, block, 0, st, a, n);
    else hipLaunchKernelGGL((swiglu<float, false>), grid, block, 0, st, a, n);
  }
  return hipGetLastError() == hipSuccess ? 0 : 1;
}

int launch_swiglu_backward(const SwigluBackArgs& a, void* stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  const dim3 grid(blocks_for(a.R * 64)), block(256);
  if (a.dtype == BSMM_BF16) hipLaunchKernelGGL(swiglu_backward<uint16_t>, grid, block, 0, st, a);
  else hipLaunchKernelGGL(swiglu_backward<float>, grid, block, 0, st, a);
  return hipGetLastError() == hipSuccess ? 0 : 1;
}

}  // namespace bsmm
