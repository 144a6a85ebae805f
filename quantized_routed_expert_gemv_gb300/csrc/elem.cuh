// elem.cuh -- element types of the operators around the layer
// (include/moe_block.h): loads, stores and conversions of bf16, f16 and f32
// values, one at a time or as aligned vectors of eight; scales and codes of
// blocks quantised to e4m3.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "../../include/moe_block.h"

namespace moe {

__host__ __device__ __forceinline__ int elem_size(int type) { return type == MOE_F32 ? 4 : 2; }
__host__ __forceinline__ bool elem_type_ok(int type) { return type == MOE_BF16 || type == MOE_F16 || type == MOE_F32; }

// A 16-bit value's bits to fp32 (exact).
__device__ __forceinline__ float half_bits_to_f32(uint32_t bits, int type) {
  return type == MOE_BF16 ? __uint_as_float(bits << 16) : __half2float(__ushort_as_half(static_cast<uint16_t>(bits)));
}

// fp32 to a 16-bit type's bits, to nearest even (NaN stays NaN).
__device__ __forceinline__ uint32_t f32_to_half_bits(float v, int type) {
  return type == MOE_BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(v)) : __half_as_ushort(__float2half_rn(v));
}

__device__ __forceinline__ float load_elem(const void* p, int type, int64_t i) {
  if (type == MOE_F32) return static_cast<const float*>(p)[i];
  return half_bits_to_f32(static_cast<const uint16_t*>(p)[i], type);
}

__device__ __forceinline__ void store_elem(void* p, int type, int64_t i, float v) {
  if (type == MOE_F32)
    static_cast<float*>(p)[i] = v;
  else
    static_cast<uint16_t*>(p)[i] = static_cast<uint16_t>(f32_to_half_bits(v, type));
}

// Eight 16-bit values in a uint4.
__device__ __forceinline__ void unpack8(uint4 r, int type, float (&v)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
  if (type == MOE_BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __half2float(__ushort_as_half(static_cast<uint16_t>(w[i])));
      v[2 * i + 1] = __half2float(__ushort_as_half(static_cast<uint16_t>(w[i] >> 16)));
    }
  }
}

// Two values to a word of 16-bit ones, the first in the low half.
__device__ __forceinline__ uint32_t pack2(float lo, float hi, int type) {
  if (type == MOE_BF16) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
  }
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8], int type) {
  return make_uint4(pack2(v[0], v[1], type), pack2(v[2], v[3], type), pack2(v[4], v[5], type),
                    pack2(v[6], v[7], type));
}

// Eight values at element i (i a multiple of 8 of a 16-byte aligned row).
__device__ __forceinline__ void load8(const void* p, int type, int64_t i, float (&v)[8]) {
  if (type == MOE_F32) {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    const float4 a = q[0], b = q[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    unpack8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i), type, v);
  }
}

__device__ __forceinline__ void store8(void* p, int type, int64_t i, const float (&v)[8]) {
  if (type == MOE_F32) {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    q[0] = make_float4(v[0], v[1], v[2], v[3]);
    q[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) = pack8(v, type);
  }
}

// 32 bytes at a 32-byte boundary: a whole sector for a lane.
__device__ __forceinline__ void load32(const void* p, uint32_t (&v)[8]) {
  asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
               : "l"(p));
}
__device__ __forceinline__ void store32(void* p, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]),
               "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// The scale of a block whose largest |x| has these bits: the smallest power
// of two s >= 2^-126 with max <= 448 s (448 = 1.75 * 2^8), 1 for zeros, NaN
// if there is an infinity or a NaN.  `inv` is 1 / s (0 for NaN).
__device__ __forceinline__ float block_scale(uint32_t max_bits, float& inv) {
  if (max_bits == 0) return inv = 1.0f;
  if (max_bits >= 0x7F800000u) {
    inv = 0.0f;
    return __uint_as_float(0x7FC00000u);
  }
  int p = static_cast<int>(max_bits >> 23) - 127 - ((max_bits & 0x7FFFFFu) <= 0x600000u ? 8 : 7);
  p = max(p, -126);
  inv = __uint_as_float(static_cast<uint32_t>(127 - p) << 23);
  return __uint_as_float(static_cast<uint32_t>(127 + p) << 23);
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

}  // namespace moe
