// elem.cuh -- element types of the operators around the layer
// (include/moe_block.h): loads, stores and conversions of bf16, f16 and f32
// values, one at a time or as aligned vectors of eight.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
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

}  // namespace moe
