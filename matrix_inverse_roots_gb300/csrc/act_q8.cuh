// The 8-bit activation format and the element types of the training operators.
//
// A row of `cols` values is cut into groups of 32 columns, the last one padded with
// zeros.  A group holds 32 codes q of 8 bits (int8 or e4m3) and one scale 2^e, stored
// as the byte e + 127; its values are q 2^e.  e is the smallest exponent at which the
// group's largest magnitude does not round past the largest code:
//   int8  e = floor(log2 amax) - 6, plus 1 where amax 2^-e >= 127.5 (it would round
//         to 128);
//   e4m3  e = floor(log2 amax) - 8, plus 1 where amax 2^-e > 464 (the tie below 480
//         goes to the even code, 448).
// Scaling by 2^-e is exact, so a value is rounded once, to the nearest code, ties to
// even.  e is kept in [-124, 121] (int8) or [-124, 119] (e4m3): every value is then a
// finite bf16 number (7 or 4 significant bits, steps of 2^-133 at least), which is what
// lets a tensor-core product take a checkpoint without rounding it again.  A group that
// holds an infinity or a NaN gets the byte 255, and all of it reads back as NaN.
#pragma once

#include <cuda_fp8.h>

#include "dash_common.cuh"
#include "dashroot.h"

namespace dash {

constexpr int Q8_GROUP = 32;
constexpr uint32_t Q8_NAN_SCALE = 255u;

// ---------------------------------------------------------------- element types

template <typename T>
struct Elem;
template <>
struct Elem<float> {
  static constexpr bool is_bf16 = false;
  static __device__ __forceinline__ float to(float x) { return x; }
  static __device__ __forceinline__ float from(float x) { return x; }
};
template <>
struct Elem<__half> {
  static constexpr bool is_bf16 = false;
  static __device__ __forceinline__ float to(__half x) { return __half2float(x); }
  static __device__ __forceinline__ __half from(float x) { return __float2half_rn(x); }
};
template <>
struct Elem<__nv_bfloat16> {
  static constexpr bool is_bf16 = true;
  static __device__ __forceinline__ float to(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ __forceinline__ __nv_bfloat16 from(float x) { return __float2bfloat16_rn(x); }
};

// Element i of a dash_dtype array, for the small per-column vectors whose type is a
// run-time argument.
__device__ __forceinline__ float load_dt(const void* p, int dt, int64_t i) {
  if (dt == DASH_DT_F32) return static_cast<const float*>(p)[i];
  if (dt == DASH_DT_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  return __half2float(static_cast<const __half*>(p)[i]);
}

// ---------------------------------------------------------------- codes

// The scale byte of a group from the bits of its largest magnitude (sign cleared).  The
// bits of non-negative floats order like the floats, infinities and NaN above all.
// Adding to the mantissa carries into the exponent exactly from the amax that rounds past
// the largest code: 127.5 / 64 has mantissa bits 0x7f0000, 464 / 256 has 0x680000.
template <int FMT>
__device__ __forceinline__ uint32_t q8_scale_byte(uint32_t amax_bits) {
  if (amax_bits >= 0x7f800000u) return Q8_NAN_SCALE;
  constexpr uint32_t up = (FMT == DASH_Q8_INT8) ? 0x10000u : 0x17ffffu;
  constexpr int down = (FMT == DASH_Q8_INT8) ? 6 : 8;
  constexpr int hi = (FMT == DASH_Q8_INT8) ? 121 + 127 : 119 + 127;
  const int b = static_cast<int>((amax_bits + up) >> 23) - down;
  return static_cast<uint32_t>(b < 3 ? 3 : (b > hi ? hi : b));
}

// 2^-e of a scale byte (byte 3 .. 248, so the result is a normal float; for the NaN byte
// the codes do not matter).
__device__ __forceinline__ float q8_inv_scale(uint32_t byte) {
  return __uint_as_float((254u - (byte == Q8_NAN_SCALE ? 127u : byte)) << 23);
}

// 2^e, or NaN.
__device__ __forceinline__ float q8_scale(uint32_t byte) {
  return byte == Q8_NAN_SCALE ? __uint_as_float(0x7fc00000u) : __uint_as_float(byte << 23);
}

// The code nearest to v (already scaled), saturating; 0 for NaN in int8.
template <int FMT>
__device__ __forceinline__ uint32_t q8_code(float v) {
  if (FMT == DASH_Q8_INT8) {
    int r = __float2int_rn(v);
    r = r < -127 ? -127 : (r > 127 ? 127 : r);
    return static_cast<uint32_t>(r) & 0xffu;
  }
  return static_cast<uint32_t>(__nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3));
}

// The value of a code before scaling.
template <int FMT>
__device__ __forceinline__ float q8_value(uint32_t code) {
  if (FMT == DASH_Q8_INT8) return static_cast<float>(static_cast<int8_t>(code));
  const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(code), __NV_E4M3);
  return __half2float(__half(h));
}

// ---------------------------------------------------------------- eight at a time
// A thread's unit of work is eight consecutive columns; four neighbouring lanes hold one
// group.

// Eight elements from p, of which `n` (0 .. 8) exist; the others are zero.  VEC: p is
// 16-byte aligned and n is 0 or 8.
template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* p, int n, float (&v)[8]) {
  if constexpr (!VEC) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = k < n ? Elem<T>::to(p[k]) : 0.0f;
  } else {
    if (n <= 0) {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = 0.0f;
      return;
    }
    if constexpr (sizeof(T) == 4) {
      const float4 a = reinterpret_cast<const float4*>(p)[0];
      const float4 b = reinterpret_cast<const float4*>(p)[1];
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
      const uint4 a = *reinterpret_cast<const uint4*>(p);
      const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if constexpr (sizeof(T) == 2 && Elem<T>::is_bf16) {
          v[2 * k] = __uint_as_float(w[k] << 16);
          v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
        } else {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
          v[2 * k] = f.x;
          v[2 * k + 1] = f.y;
        }
      }
    }
  }
}

template <typename T, bool VEC>
__device__ __forceinline__ void store8(T* p, int n, const float (&v)[8]) {
  if constexpr (!VEC) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < n) p[k] = Elem<T>::from(v[k]);
  } else {
    if (n <= 0) return;
    if constexpr (sizeof(T) == 4) {
      reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else if constexpr (Elem<T>::is_bf16) {
      *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf162(v[0], v[1]), pack_bf162(v[2], v[3]),
                                                pack_bf162(v[4], v[5]), pack_bf162(v[6], v[7]));
    } else {
      *reinterpret_cast<uint4*>(p) = make_uint4(pack_half2(v[0], v[1]), pack_half2(v[2], v[3]),
                                                pack_half2(v[4], v[5]), pack_half2(v[6], v[7]));
    }
  }
}

// Eight elements of a per-column vector whose type is a run-time argument.  vec: the
// vector is 16-byte aligned and n is 0 or 8.
__device__ __forceinline__ void load8_dt(const void* p, int dt, bool vec, int64_t i, int n,
                                         float (&v)[8]) {
  if (vec) {
    if (dt == DASH_DT_F32)
      load8<float, true>(static_cast<const float*>(p) + i, n, v);
    else if (dt == DASH_DT_BF16)
      load8<__nv_bfloat16, true>(static_cast<const __nv_bfloat16*>(p) + i, n, v);
    else
      load8<__half, true>(static_cast<const __half*>(p) + i, n, v);
    return;
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = k < n ? load_dt(p, dt, i + k) : 0.0f;
}

// Largest magnitude bits of the group that this lane shares with its three neighbours.
__device__ __forceinline__ uint32_t group_amax(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) m = max(m, __float_as_uint(v[k]) & 0x7fffffffu);
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  return max(m, __shfl_xor_sync(0xffffffffu, m, 2));
}

// Scale byte and codes of eight values from their group's largest magnitude.
__device__ __forceinline__ uint32_t q8_encode8(int fmt, uint32_t amax, const float (&v)[8],
                                               uint2& codes) {
  if (fmt == DASH_Q8_INT8) {
    const uint32_t b = q8_scale_byte<DASH_Q8_INT8>(amax);
    const float inv = q8_inv_scale(b);
    uint32_t c[8];
    if (b == 121u + 127u) {
      // The largest scale does not grow any further: saturate.
#pragma unroll
      for (int k = 0; k < 8; ++k) c[k] = q8_code<DASH_Q8_INT8>(v[k] * inv);
    } else {
      // 1.5 2^23 + x holds x, rounded to nearest even, in its low byte; the product is
      // exact.
#pragma unroll
      for (int k = 0; k < 8; ++k) c[k] = __float_as_uint(fmaf(v[k], inv, 12582912.0f));
    }
    codes.x = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
    codes.y = __byte_perm(__byte_perm(c[4], c[5], 0x0040), __byte_perm(c[6], c[7], 0x0040), 0x5410);
    return b;
  }
  const uint32_t b = q8_scale_byte<DASH_Q8_E4M3>(amax);
  const float inv = q8_inv_scale(b);
  uint32_t h[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    h[k] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * k] * inv, v[2 * k + 1] * inv),
                                    __NV_SATFINITE, __NV_E4M3);
  codes.x = h[0] | (h[1] << 16);
  codes.y = h[2] | (h[3] << 16);
  return b;
}

// The values of eight codes.
__device__ __forceinline__ void q8_decode8(int fmt, const uint2& codes, uint32_t byte,
                                           float (&v)[8]) {
  const float s = q8_scale(byte);
  if (fmt == DASH_Q8_INT8) {
    // 2^23 + (q + 128) from the code's byte, less 2^23 + 128.
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t u = (k < 4 ? codes.x : codes.y) ^ 0x80808080u;
      v[k] = (__uint_as_float(__byte_perm(u, 0x4b000000u, 0x7440 + (k & 3))) - 8388736.0f) * s;
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t w = k < 2 ? codes.x : codes.y;
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
          static_cast<__nv_fp8x2_storage_t>((k & 1) ? w >> 16 : w & 0xffffu), __NV_E4M3);
      const float2 f = __half22float2(__half2(h));
      v[2 * k] = f.x * s;
      v[2 * k + 1] = f.y * s;
    }
  }
}

__device__ __forceinline__ uint32_t warp_max_u32(uint32_t v) {
  return __reduce_max_sync(0xffffffffu, v);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

}  // namespace dash
