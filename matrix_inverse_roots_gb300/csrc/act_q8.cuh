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
  static __device__ __forceinline__ float to(float x) { return x; }
  static __device__ __forceinline__ float from(float x) { return x; }
};
template <>
struct Elem<__half> {
  static __device__ __forceinline__ float to(__half x) { return __half2float(x); }
  static __device__ __forceinline__ __half from(float x) { return __float2half_rn(x); }
};
template <>
struct Elem<__nv_bfloat16> {
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

__device__ __forceinline__ uint32_t warp_max_u32(uint32_t v) {
  return __reduce_max_sync(0xffffffffu, v);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

}  // namespace dash
