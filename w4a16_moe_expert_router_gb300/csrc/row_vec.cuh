// row_vec.cuh -- 16-byte pieces of fp16, bf16 and fp32 rows.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ptx.cuh"

namespace moe {

// 16 bytes of a row as fp32 values and back (one rounding, to nearest even).
template <int kType>
struct Vec;
template <>
struct Vec<0> {
  static constexpr int n = 8;
  static __device__ __forceinline__ void load(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 p = __half22float2(bits_h2(w[i]));
      f[2 * i] = p.x;
      f[2 * i + 1] = p.y;
    }
  }
  static __device__ __forceinline__ uint4 store(const float (&f)[8]) {
    return make_uint4(h2_bits(__floats2half2_rn(f[0], f[1])), h2_bits(__floats2half2_rn(f[2], f[3])),
                      h2_bits(__floats2half2_rn(f[4], f[5])), h2_bits(__floats2half2_rn(f[6], f[7])));
  }
};
template <>
struct Vec<1> {
  static constexpr int n = 8;
  static __device__ __forceinline__ void load(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // a bf16 value is the upper half of an fp32 value
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&p);
  }
  static __device__ __forceinline__ uint4 store(const float (&f)[8]) {
    return make_uint4(pack(f[0], f[1]), pack(f[2], f[3]), pack(f[4], f[5]), pack(f[6], f[7]));
  }
};
template <>
struct Vec<2> {
  static constexpr int n = 4;
  static __device__ __forceinline__ void load(const uint4& v, float (&f)[4]) {
    f[0] = __uint_as_float(v.x);
    f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z);
    f[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ uint4 store(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};

// Single 16-bit values (type 0 fp16, 1 bf16).
template <int kType>
__device__ __forceinline__ uint16_t to16(float f) {
  if constexpr (kType == 0)
    return __half_as_ushort(__float2half_rn(f));
  else
    return __bfloat16_as_ushort(__float2bfloat16_rn(f));
}
template <int kType>
__device__ __forceinline__ float from16(uint16_t v) {
  if constexpr (kType == 0)
    return __half2float(__ushort_as_half(v));
  else
    return __uint_as_float(static_cast<uint32_t>(v) << 16);
}

}  // namespace moe
