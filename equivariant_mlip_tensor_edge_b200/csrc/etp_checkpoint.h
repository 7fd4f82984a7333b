// The 8-bit checkpoint code: 32 consecutive values of a row share a power-of-two scale. Internal to
// libetp; used by the store and restore kernels and by the group norm, which writes and reads codes.
//
//   scale 2^e, e = the smallest integer >= -126 with max|x| <= top 2^e, top = 127 (int8) or 448 (e4m3)
//   code = x / 2^e rounded to the nearest (ties to even) integer or e4m3 number
//
// A power of two divides without rounding, so the code of a value does not depend on the precision
// it is computed in, and a restored value is exact in 32 bits. The scale byte is e + 127; 255 marks
// a block with a NaN or an infinity, whose values all restore as NaN.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "etp_internal.h"

namespace etp {

constexpr int kCkptBlock = 32;
constexpr unsigned kCkptBad = 255u;

// max|x| is kept as the bit pattern of |x|: as integers these order like the values, with infinity
// and then NaN on top, which a floating maximum would drop.
__device__ __forceinline__ unsigned abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// Scale byte of a block whose largest |x| has these bits. top 2^e >= amax: 127 = 1.984375 x 2^6 and
// 448 = 1.75 x 2^8, so the exponent is amax's less 6 (8), one more if its significand is larger.
__device__ __forceinline__ unsigned scale_byte(unsigned amax, bool int8) {
  if (amax >= 0x7f800000u) return kCkptBad;
  const int k = static_cast<int>(amax >> 23);
  const unsigned frac = amax & 0x7fffffu;
  const int e = int8 ? k - 6 + (frac > 0x7e0000u ? 1 : 0) : k - 8 + (frac > 0x600000u ? 1 : 0);
  return static_cast<unsigned>(e < 1 ? 1 : e);
}

// 2^-e, the factor in front of the rounding (bytes up to 249 occur: 4 <= 254 - byte)
__device__ __forceinline__ float inv_scale(unsigned byte) {
  return byte == kCkptBad ? 0.0f : __uint_as_float((254u - byte) << 23);
}
// 2^e, or NaN for a marked block: code x NaN = NaN
__device__ __forceinline__ float scale_of(unsigned byte) {
  return byte == kCkptBad ? __uint_as_float(0x7fc00000u) : __uint_as_float(byte << 23);
}

// code of one value; bad blocks store code 0 (inf * 0 is NaN: the select comes first)
__device__ __forceinline__ unsigned encode(float x, float inv, bool bad, bool int8) {
  const float v = bad ? 0.0f : x * inv;
  if (int8) return static_cast<unsigned>(__float2int_rn(v)) & 0xffu;
  return __nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ unsigned encode4(const float (&x)[4], float inv, bool bad, bool int8) {
  if (int8)
    return encode(x[0], inv, bad, true) | encode(x[1], inv, bad, true) << 8 | encode(x[2], inv, bad, true) << 16 |
           encode(x[3], inv, bad, true) << 24;
  const float2 a = bad ? make_float2(0.f, 0.f) : make_float2(x[0] * inv, x[1] * inv);
  const float2 b = bad ? make_float2(0.f, 0.f) : make_float2(x[2] * inv, x[3] * inv);
  return static_cast<unsigned>(__nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, __NV_E4M3)) |
         static_cast<unsigned>(__nv_cvt_float2_to_fp8x2(b, __NV_SATFINITE, __NV_E4M3)) << 16;
}

__device__ __forceinline__ float decode(unsigned code, float scale, bool int8) {
  if (int8) return static_cast<float>(static_cast<signed char>(code)) * scale;
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(code), __NV_E4M3))) * scale;
}
__device__ __forceinline__ void decode4(unsigned codes, float scale, bool int8, float (&v)[4]) {
  if (int8) {
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = static_cast<float>(static_cast<signed char>(codes >> (8 * k))) * scale;
  } else {
    const float2 a = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes), __NV_E4M3)));
    const float2 b = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes >> 16), __NV_E4M3)));
    v[0] = a.x * scale; v[1] = a.y * scale; v[2] = b.x * scale; v[3] = b.y * scale;
  }
}

// ---------------------------------------------------------------- values of a row in 32 or 16 bits

template <class T> __device__ __forceinline__ float to_f32(T v);
template <> __device__ __forceinline__ float to_f32(float v) { return v; }
template <> __device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <> __device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <class T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f32(float v) { return __float2half_rn(v); }

template <class T> struct Limits;
template <> struct Limits<float> { static constexpr float max = 3.402823466e+38f; };
template <> struct Limits<__nv_bfloat16> { static constexpr float max = 3.38953139e+38f; };
template <> struct Limits<__half> { static constexpr float max = 65504.0f; };

// V values (V = 1 or 4) as floats; 4 of them in one access, whose alignment the caller guarantees
template <class T, int V>
__device__ __forceinline__ void load_v(const T* __restrict__ p, float (&v)[V]) {
  if constexpr (V == 1) {
    v[0] = to_f32<T>(__ldg(p));
  } else if constexpr (sizeof(T) == 4) {
    const float4 t = __ldg(reinterpret_cast<const float4*>(p));
    v[0] = t.x; v[1] = t.y; v[2] = t.z; v[3] = t.w;
  } else {
    union { uint2 u; T h[4]; } t;
    t.u = __ldg(reinterpret_cast<const uint2*>(p));
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = to_f32<T>(t.h[k]);
  }
}

template <class T, int V>
__device__ __forceinline__ void store_v(T* p, const float (&v)[V]) {
  if constexpr (V == 1) {
    *p = from_f32<T>(v[0]);
  } else if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
    union { uint2 u; T h[4]; } t;
#pragma unroll
    for (int k = 0; k < 4; ++k) t.h[k] = from_f32<T>(v[k]);
    *reinterpret_cast<uint2*>(p) = t.u;
  }
}

}  // namespace etp
