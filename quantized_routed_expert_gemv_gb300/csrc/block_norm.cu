// block_norm.cu -- the block boundary (moe_block_norm): post-norm, gate,
// scaled residual and the next block's pre-norm in one pass over the rows.
//
// Mathematics: r = y * rsqrt(mean(y^2) + eps) * w_post, h' = s h + g r,
// x = h' * rsqrt(mean(h'^2) + eps) * w_pre.  The two means need the whole
// row, so a row's values stay in registers between them: y and h are read
// once, h' and x written once, nothing in between goes to memory.
//
// Bound: memory traffic for many rows (about 11 operations per value against
// 8 to 12 bytes), the latency of one load and two reductions for few.
#include <cstdint>

#include <cuda_runtime.h>

#include "elem.cuh"

namespace moe {
int reportf(int code, const char* fmt, ...);

namespace {

constexpr int kMaxHidden = 16384;

// Sum over the row's threads, the same value in all of them.  A block of 32
// threads per row needs no barrier.  `red` has one slot per warp.
__device__ __forceinline__ float row_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if (blockDim.x == 32) return v;
  const int warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  if ((threadIdx.x & 31) == 0) red[warp] = v;
  __syncthreads();
  float s = static_cast<int>(threadIdx.x & 31) < nw ? red[threadIdx.x & 31] : 0.0f;
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  return s;
}

template <int VEC>
__device__ __forceinline__ void load_chunk(const void* p, int type, int64_t row, int j, int H, float (&v)[VEC]) {
  if constexpr (VEC == 8) {
    if (j + 8 <= H) {
      load8(p, type, row + j, v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = j + i < H ? load_elem(p, type, row + j + i) : 0.0f;
    }
  } else {
    v[0] = j < H ? load_elem(p, type, row + j) : 0.0f;
  }
}

template <int VEC>
__device__ __forceinline__ void store_chunk(void* p, int type, int64_t row, int j, int H, const float (&v)[VEC]) {
  if constexpr (VEC == 8) {
    if (j + 8 <= H) {
      store8(p, type, row + j, v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (j + i < H) store_elem(p, type, row + j + i, v[i]);
    }
  } else {
    if (j < H) store_elem(p, type, row + j, v[0]);
  }
}

// blockDim = (threads per row, rows per block); more than one row per block
// only with 32 threads per row.  A thread holds NC chunks of VEC values.
template <int VEC, int NC>
__global__ void __launch_bounds__(VEC == 8 ? 512 : 1024) block_norm_kernel(const moe_block_norm_args a) {
  __shared__ float red[2][32];
  const int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  if (t >= a.rows) return;
  const int H = a.hidden;
  float v[NC][VEC], h[NC][VEC];
  float ss = 0.0f;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int j = (c * blockDim.x + threadIdx.x) * VEC;
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[c][i] = h[c][i] = 0.0f;
    if (a.y) load_chunk<VEC>(a.y, a.y_type, t * a.ld_y, j, H, v[c]);
    if (a.h) load_chunk<VEC>(a.h, a.h_type, t * a.ld_h, j, H, h[c]);
  }
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int i = 0; i < VEC; ++i) ss = fmaf(v[c][i], v[c][i], ss);
  const float inv_h = 1.0f / static_cast<float>(H);
  float rs = 1.0f;
  if (a.post_norm) rs = rsqrtf(row_sum(ss, red[0]) * inv_h + a.eps);
  ss = 0.0f;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int j = (c * blockDim.x + threadIdx.x) * VEC;
    if (a.y) {
      float w[VEC];
      if (a.post_norm) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) w[i] = 0.0f;
        if (a.w_post) load_chunk<VEC>(a.w_post, a.w_type, 0, j, H, w);
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[c][i] *= rs * (a.w_add + w[i]);
      }
      if (a.gate) {
        if (a.ld_gate_col) {
          load_chunk<VEC>(a.gate, a.gate_type, t * a.ld_gate_row, j, H, w);
        } else {
          const float g = load_elem(a.gate, a.gate_type, t * a.ld_gate_row);
#pragma unroll
          for (int i = 0; i < VEC; ++i) w[i] = g;
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[c][i] *= w[i];
      }
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      if (a.h) v[c][i] = fmaf(a.residual_scale, h[c][i], v[c][i]);
      if (j + i < H) ss = fmaf(v[c][i], v[c][i], ss);
    }
    if (a.h_out) store_chunk<VEC>(a.h_out, a.h_type, t * a.ld_h_out, j, H, v[c]);
  }
  if (!a.x_out) return;
  rs = 1.0f;
  if (a.pre_norm) rs = rsqrtf(row_sum(ss, red[1]) * inv_h + a.eps);
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int j = (c * blockDim.x + threadIdx.x) * VEC;
    if (a.pre_norm) {
      float w[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) w[i] = 0.0f;
      if (a.w_pre) load_chunk<VEC>(a.w_pre, a.w_type, 0, j, H, w);
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[c][i] *= rs * (a.w_add + w[i]);
    }
    store_chunk<VEC>(a.x_out, a.x_type, t * a.ld_x_out, j, H, v[c]);
  }
}

template <int VEC>
cudaError_t launch_vec(const moe_block_norm_args& a, int nc, dim3 grid, dim3 block, cudaStream_t st) {
  switch (nc) {
    case 1: block_norm_kernel<VEC, 1><<<grid, block, 0, st>>>(a); break;
    case 2: block_norm_kernel<VEC, 2><<<grid, block, 0, st>>>(a); break;
    case 4: block_norm_kernel<VEC, 4><<<grid, block, 0, st>>>(a); break;
    default:
      if constexpr (VEC == 1) block_norm_kernel<VEC, 16><<<grid, block, 0, st>>>(a);
  }
  return cudaGetLastError();
}

bool vec_ok(const void* p, int type, int64_t ld) {
  return !p || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * elem_size(type) % 16 == 0);
}

int check_matrix(const char* name, const void* p, int type, int64_t ld, int32_t hidden) {
  if (!elem_type_ok(type)) return reportf(MOE_ERR_ARG, "moe_block_norm: %s has an unknown type %d", name, type);
  if (reinterpret_cast<uintptr_t>(p) % elem_size(type))
    return reportf(MOE_ERR_ALIGN, "moe_block_norm: %s is not aligned to its elements", name);
  if (ld < hidden)
    return reportf(MOE_ERR_ARG, "moe_block_norm: %s has rows of %d values %lld apart", name, hidden,
                   static_cast<long long>(ld));
  return MOE_OK;
}

}  // namespace
}  // namespace moe

extern "C" int moe_block_norm(const moe_block_norm_args* args, void* stream) {
  using namespace moe;
  if (!args) return reportf(MOE_ERR_ARG, "moe_block_norm: args is NULL");
  const moe_block_norm_args a = *args;
  if (a.rows < 0) return reportf(MOE_ERR_ARG, "moe_block_norm: rows=%d is negative", a.rows);
  if (a.rows == 0) return MOE_OK;  // whatever the buffers: empty ones may be NULL
  if (a.hidden < 1 || a.hidden > kMaxHidden)
    return reportf(MOE_ERR_ARG, "moe_block_norm: hidden=%d must be in [1, %d]", a.hidden, kMaxHidden);
  if (!a.y && !a.h) return reportf(MOE_ERR_ARG, "moe_block_norm: y and h are both NULL");
  if (!a.h_out && !a.x_out) return reportf(MOE_ERR_ARG, "moe_block_norm: h_out and x_out are both NULL");
  if ((a.post_norm != 0 && a.post_norm != 1) || (a.pre_norm != 0 && a.pre_norm != 1))
    return reportf(MOE_ERR_ARG, "moe_block_norm: post_norm=%d and pre_norm=%d must be 0 or 1", a.post_norm, a.pre_norm);
  if (!(a.eps > 0.0f)) return reportf(MOE_ERR_ARG, "moe_block_norm: eps must be positive");
  if (a.w_add != 0.0f && a.w_add != 1.0f) return reportf(MOE_ERR_ARG, "moe_block_norm: w_add must be 0 or 1");
  int rc;
  if (a.y && (rc = check_matrix("y", a.y, a.y_type, a.ld_y, a.hidden))) return rc;
  if (a.h && (rc = check_matrix("h", a.h, a.h_type, a.ld_h, a.hidden))) return rc;
  if (a.h_out && (rc = check_matrix("h_out", a.h_out, a.h_type, a.ld_h_out, a.hidden))) return rc;
  if (a.x_out && (rc = check_matrix("x_out", a.x_out, a.x_type, a.ld_x_out, a.hidden))) return rc;
  if (a.w_post && (rc = check_matrix("w_post", a.w_post, a.w_type, a.hidden, a.hidden))) return rc;
  if (a.w_pre && (rc = check_matrix("w_pre", a.w_pre, a.w_type, a.hidden, a.hidden))) return rc;
  if (a.gate) {
    if ((rc = check_matrix("gate", a.gate, a.gate_type, a.hidden, a.hidden))) return rc;
    if ((a.ld_gate_col != 0 && a.ld_gate_col != 1) || a.ld_gate_row < 0)
      return reportf(MOE_ERR_ARG, "moe_block_norm: ld_gate_col=%lld must be 0 or 1, ld_gate_row=%lld not negative",
                     static_cast<long long>(a.ld_gate_col), static_cast<long long>(a.ld_gate_row));
  }

  const bool vec = vec_ok(a.y, a.y_type, a.ld_y) && vec_ok(a.h, a.h_type, a.ld_h) &&
                   vec_ok(a.h_out, a.h_type, a.ld_h_out) && vec_ok(a.x_out, a.x_type, a.ld_x_out) &&
                   vec_ok(a.w_post, a.w_type, 0) && vec_ok(a.w_pre, a.w_type, 0) &&
                   (!a.ld_gate_col || vec_ok(a.gate, a.gate_type, a.ld_gate_row));
  const int chunks = vec ? (a.hidden + 7) / 8 : a.hidden;
  const int max_nc = vec ? 4 : 16;
  int nc = 1;
  dim3 block(32, 1);
  if (chunks <= 32) {
    block.y = 4;
  } else {
    while (nc < max_nc && chunks > 512 * nc) nc = nc == 4 ? 16 : nc * 2;
    block.x = ((chunks + nc - 1) / nc + 31) / 32 * 32;
  }
  const dim3 grid((static_cast<unsigned>(a.rows) + block.y - 1) / block.y);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = vec ? launch_vec<8>(a, nc, grid, block, st) : launch_vec<1>(a, nc, grid, block, st);
  if (e != cudaSuccess) return reportf(MOE_ERR_CUDA, "moe_block_norm: %s (%s)", cudaGetErrorString(e), cudaGetErrorName(e));
  return MOE_OK;
}
