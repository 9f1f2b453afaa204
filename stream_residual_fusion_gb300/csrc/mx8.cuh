// mx8.cuh -- MXFP8 blocks of activation checkpoints: 32 consecutive features of a row as E4M3
// codes with one E8M0 scale (OCP Microscaling formats v1.0), from and to bf16 pairs.
//
// The scale of a block is 2^(floor(log2 amax) - 8), amax the largest finite magnitude of the
// block (code floor(log2 amax) - 8 + 127, at least 0; 0 for a block without a finite nonzero
// value). Elements are x / scale rounded to nearest even, +-448 at most. An infinity or NaN
// becomes the NaN code: a checkpoint never turns a value that is not finite into one that is.
#pragma once
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "ptx.cuh"

namespace mhc {

constexpr int MX_BLOCK = 32;

// The larger 15-bit magnitudes of 8 bf16 values in 4 words, one in each half word. Non-negative bf16
// patterns order like their values; 0x7f80 and above are the infinities and NaNs.
__device__ __forceinline__ uint32_t max_halves8(const uint32_t (&w)[4]) {
  uint32_t m = w[0] & 0x7fff7fffu;
#pragma unroll
  for (int i = 1; i < 4; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
  return m;
}
// The same with infinities and NaNs left out.
__device__ __forceinline__ uint32_t finite_max_halves8(const uint32_t (&w)[4]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = w[i] & 0x7fffu, b = w[i] & 0x7fff0000u;
    m = __vmaxu2(m, (a < 0x7f80u ? a : 0u) | (b < 0x7f800000u ? b : 0u));
  }
  return m;
}
__device__ __forceinline__ uint32_t max_of_halves(uint32_t m) { return max(m & 0xffffu, m >> 16); }

// E8M0 code of a block whose largest finite magnitude has bits m.
__device__ __forceinline__ uint32_t scale_code_of(uint32_t m) {
  const uint32_t e = m >> 7;
  return e > 8 ? e - 8 : 0;
}

// 8 bf16 values (4 words) as E4M3 codes under scale code e. ODD: infinities become NaNs.
template <bool ODD>
__device__ __forceinline__ uint2 encode8(const uint32_t (&w)[4], uint32_t e) {
  const float inv = __uint_as_float((254u - e) << 23);   // 2^(127 - e), exact
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t lo = w[i] << 16, hi = w[i] & 0xffff0000u;
    if (ODD) {
      if ((lo & 0x7f800000u) == 0x7f800000u) lo |= 0x400000u;
      if ((hi & 0x7f800000u) == 0x7f800000u) hi |= 0x400000u;
    }
    c[i] = __nv_cvt_float2_to_fp8x2(make_float2(__uint_as_float(lo) * inv, __uint_as_float(hi) * inv),
                                    __NV_SATFINITE, __NV_E4M3);
  }
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// The float 2^(e - 127) of a scale code (subnormal for 0; NaN for 255, which no encoder writes).
__device__ __forceinline__ float scale_value(uint32_t e) {
  return __uint_as_float((e << 23) | (((e + 1) & 0xffu) <= 1u ? 0x400000u : 0u));
}

// Values of two E4M3 codes (the low half word) times `s`; exact.
__device__ __forceinline__ f2 decode2(uint32_t c, f2 s) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(c & 0xffffu), __NV_E4M3);
  const float2 v = __half22float2(__half2(h));
  return mul2(f2{v.x, v.y}, s);
}

}  // namespace mhc
