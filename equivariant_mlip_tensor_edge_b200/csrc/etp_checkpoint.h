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

// max(|a|, |b|) that keeps a NaN, which fmaxf would drop
__device__ __forceinline__ float max_abs(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
  return r;
}

// Scale byte of a block with largest |x| amax. top 2^e >= amax: 127 = 1.984375 x 2^6 and 448 = 1.75 x
// 2^8, so the exponent is amax's less 6 (8), one more if its significand is larger: the addition
// carries into the exponent then.
__device__ __forceinline__ unsigned scale_byte(float amax, bool int8) {
  const unsigned bits = __float_as_uint(amax);
  const int e = static_cast<int>((bits + (int8 ? 0x1ffffu : 0x1fffffu)) >> 23) - (int8 ? 6 : 8);
  return bits >= 0x7f800000u ? kCkptBad : static_cast<unsigned>(max(e, 1));
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
// four codes. int8: x 2^-e + 1.5 x 2^23 is rounded to an integer, whose low byte is the code
__device__ __forceinline__ unsigned encode4(const float (&x)[4], float inv, bool bad, bool int8) {
  unsigned codes;
  if (int8) {
    unsigned t[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) t[k] = __float_as_uint(fmaf(x[k], inv, 12582912.0f));
    codes = __byte_perm(__byte_perm(t[0], t[1], 0x0040), __byte_perm(t[2], t[3], 0x0040), 0x5410);
  } else {
    codes = static_cast<unsigned>(__nv_cvt_float2_to_fp8x2(make_float2(x[0] * inv, x[1] * inv), __NV_SATFINITE, __NV_E4M3)) |
            static_cast<unsigned>(__nv_cvt_float2_to_fp8x2(make_float2(x[2] * inv, x[3] * inv), __NV_SATFINITE, __NV_E4M3)) << 16;
  }
  return bad ? 0u : codes;
}

__device__ __forceinline__ float decode(unsigned code, float scale, bool int8) {
  if (int8) return static_cast<float>(static_cast<signed char>(code)) * scale;
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(code), __NV_E4M3))) * scale;
}
__device__ __forceinline__ void decode4(unsigned codes, float scale, bool int8, float (&v)[4]) {
  if (int8) {
    // a float 2^23 + b + 128 from byte b with its sign bit flipped, less 2^23 + 128: a permutation and an
    // addition, at four times the rate of a conversion
    const unsigned flipped = codes ^ 0x80808080u;
    v[0] = (__uint_as_float(__byte_perm(flipped, 0x4b000000u, 0x7440)) - 8388736.0f) * scale;
    v[1] = (__uint_as_float(__byte_perm(flipped, 0x4b000000u, 0x7441)) - 8388736.0f) * scale;
    v[2] = (__uint_as_float(__byte_perm(flipped, 0x4b000000u, 0x7442)) - 8388736.0f) * scale;
    v[3] = (__uint_as_float(__byte_perm(flipped, 0x4b000000u, 0x7443)) - 8388736.0f) * scale;
  } else {
    const float2 a = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes), __NV_E4M3)));
    const float2 b = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes >> 16), __NV_E4M3)));
    v[0] = a.x * scale; v[1] = a.y * scale; v[2] = b.x * scale; v[3] = b.y * scale;
  }
}

template <int V>
__device__ __forceinline__ void store_codes(uint8_t* q, const float (&x)[V], float inv, bool bad, bool int8) {
  if constexpr (V == 4) *reinterpret_cast<unsigned*>(q) = encode4(x, inv, bad, int8);
  else if constexpr (V == 2)
    *reinterpret_cast<uint16_t*>(q) = static_cast<uint16_t>(encode(x[0], inv, bad, int8) | encode(x[1], inv, bad, int8) << 8);
  else *q = static_cast<uint8_t>(encode(x[0], inv, bad, int8));
}
template <int V>
__device__ __forceinline__ void load_codes(const uint8_t* q, float scale, bool int8, float (&x)[V]) {
  if constexpr (V == 4) {
    decode4(*reinterpret_cast<const unsigned*>(q), scale, int8, x);
  } else if constexpr (V == 2) {
    const unsigned t = *reinterpret_cast<const uint16_t*>(q);
    x[0] = decode(t & 0xffu, scale, int8);
    x[1] = decode(t >> 8, scale, int8);
  } else {
    x[0] = decode(*q, scale, int8);
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

// a value, and two values of a size, as one word
template <int kBytes> struct Word;
template <> struct Word<2> { using type = unsigned short; };
template <> struct Word<4> { using type = unsigned; };
template <int kBytes> struct Pair;
template <> struct Pair<2> { using type = unsigned; };
template <> struct Pair<4> { using type = uint2; };

// V values (1, 2 or 4) as floats, in one access, whose alignment the caller guarantees
template <class T, int V>
__device__ __forceinline__ void load_v(const T* __restrict__ p, float (&v)[V]) {
  static_assert(V != 2, "pairs are read from shared memory");
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

// Stored to be read by another kernel at the earliest: what is in L2 for this one stays.
__device__ __forceinline__ void store_word(unsigned short* p, unsigned short v) { __stcs(p, v); }
__device__ __forceinline__ void store_word(unsigned* p, unsigned v) { __stcs(p, v); }
__device__ __forceinline__ void store_word(uint2* p, uint2 v) { __stcs(p, v); }

template <class T, int V>
__device__ __forceinline__ void store_v(T* p, const float (&v)[V]) {
  if constexpr (V == 1) {
    union { typename Word<sizeof(T)>::type u; T h; } t{};
    t.h = from_f32<T>(v[0]);
    store_word(reinterpret_cast<typename Word<sizeof(T)>::type*>(p), t.u);
  } else if constexpr (V == 2) {
    union { typename Pair<sizeof(T)>::type u; T h[2]; } t{};
    t.h[0] = from_f32<T>(v[0]);
    t.h[1] = from_f32<T>(v[1]);
    store_word(reinterpret_cast<typename Pair<sizeof(T)>::type*>(p), t.u);
  } else if constexpr (sizeof(T) == 4) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
  } else {
    union { uint2 u; T h[4]; } t;
#pragma unroll
    for (int k = 0; k < 4; ++k) t.h[k] = from_f32<T>(v[k]);
    __stcs(reinterpret_cast<uint2*>(p), t.u);
  }
}

}  // namespace etp
