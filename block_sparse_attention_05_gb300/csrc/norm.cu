// norm.cu -- the residual sum and its root-mean-square norm, in front of a
// layer's projections (the index prologue among them), in bf16 or E4M3:
//   h = x + residual,  sum = bf16(h),  y = h / sqrt(mean(h^2) + eps) * gamma.
// The norm is taken from the fp32 h, before its rounding to the residual
// stream.  E4M3 output: one fp32 scale per row, max |y| / 448 (1 when that is
// 0), code = round-to-nearest-even(y / scale), the rule of the other fp8 codes.
//
// Bound by HBM: x and residual are read and sum and y written once (8 bytes an
// element, 7 with codes).  One CTA per row, the row in registers between the
// reductions, so nothing is read twice.
#include <cuda_fp8.h>

#include "common.cuh"
#include "kernels.h"

namespace msa {

namespace {

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

struct AddOp { __device__ static float of(float a, float b) { return a + b; } };
struct MaxOp { __device__ static float of(float a, float b) { return fmaxf(a, b); } };

// The same value in every thread; `red` holds a word per warp and is free again after the call's first barrier of
// the next reduction on the other buffer.
template <typename Op>
__device__ __forceinline__ float block_reduce(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = Op::of(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  const int warps = blockDim.x >> 5;
  if (warps == 1) return v;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = red[0];
  for (int w = 1; w < warps; ++w) t = Op::of(t, red[w]);
  return t;
}

// VEC elements per access (8: 16-byte accesses, for widths that are a multiple
// of 8; 1: any width), CH accesses per thread.
template <int VEC, int CH, bool FP8>
__global__ void __launch_bounds__(1024) add_rms_norm_kernel(NormParams p) {
  __shared__ float red[2][32];
  const long long row = blockIdx.x;
  const int T = blockDim.x, n = p.width / VEC;
  const __nv_bfloat16* x = p.x + row * p.width;
  const __nv_bfloat16* res = p.residual ? p.residual + row * p.width : nullptr;
  float h[CH][VEC];
  float sq = 0.0f;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int i = c * T + threadIdx.x;
#pragma unroll
    for (int j = 0; j < VEC; ++j) h[c][j] = 0.0f;
    if (i < n) {
      if (VEC == 8) {
        const uint4 a = reinterpret_cast<const uint4*>(x)[i];
        const uint32_t wa[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          h[c][2 * j % VEC] = __uint_as_float(wa[j] << 16);
          h[c][(2 * j + 1) % VEC] = __uint_as_float(wa[j] & 0xFFFF0000u);
        }
        if (res) {
          const uint4 b = reinterpret_cast<const uint4*>(res)[i];
          const uint32_t wb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            h[c][2 * j % VEC] += __uint_as_float(wb[j] << 16);
            h[c][(2 * j + 1) % VEC] += __uint_as_float(wb[j] & 0xFFFF0000u);
          }
        }
      } else {
        h[c][0] = __bfloat162float(x[i]);
        if (res) h[c][0] += __bfloat162float(res[i]);
      }
#pragma unroll
      for (int j = 0; j < VEC; ++j) sq = fmaf(h[c][j], h[c][j], sq);
    }
  }
  // every thread has read its elements, so the outputs below may overwrite x or the residual in place
  const float total = block_reduce<AddOp>(sq, red[0]);
  const float r = 1.0f / sqrtf(total / static_cast<float>(p.width) + p.eps);
  float top = 0.0f;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int i = c * T + threadIdx.x;
    if (i >= n) continue;
    if (VEC == 8) {
      if (p.sum)
        reinterpret_cast<uint4*>(p.sum + row * p.width)[i] =
            make_uint4(pack2(h[c][0], h[c][1 % VEC]), pack2(h[c][2 % VEC], h[c][3 % VEC]),
                       pack2(h[c][4 % VEC], h[c][5 % VEC]), pack2(h[c][6 % VEC], h[c][7 % VEC]));
      const uint4 gm = reinterpret_cast<const uint4*>(p.gamma)[i];
      const uint32_t w[4] = {gm.x, gm.y, gm.z, gm.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        h[c][2 * j % VEC] = h[c][2 * j % VEC] * r * __uint_as_float(w[j] << 16);
        h[c][(2 * j + 1) % VEC] = h[c][(2 * j + 1) % VEC] * r * __uint_as_float(w[j] & 0xFFFF0000u);
      }
      if (!FP8)
        reinterpret_cast<uint4*>(p.y + row * p.width)[i] =
            make_uint4(pack2(h[c][0], h[c][1 % VEC]), pack2(h[c][2 % VEC], h[c][3 % VEC]),
                       pack2(h[c][4 % VEC], h[c][5 % VEC]), pack2(h[c][6 % VEC], h[c][7 % VEC]));
    } else {
      if (p.sum) p.sum[row * p.width + i] = __float2bfloat16_rn(h[c][0]);
      h[c][0] = h[c][0] * r * __bfloat162float(p.gamma[i]);
      if (!FP8) p.y[row * p.width + i] = __float2bfloat16_rn(h[c][0]);
    }
    if (FP8)
#pragma unroll
      for (int j = 0; j < VEC; ++j) top = fmaxf(top, fabsf(h[c][j]));
  }
  if (!FP8) return;
  top = block_reduce<MaxOp>(top, red[1]);
  float scale = __fdiv_rn(top, 448.0f);
  if (!(scale > 0.0f)) scale = 1.0f;
  if (threadIdx.x == 0) p.scale[row] = scale;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int i = c * T + threadIdx.x;
    if (i >= n) continue;
    if (VEC == 8) {
      uint32_t q[2] = {0, 0};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = make_float2(__fdiv_rn(h[c][2 * j % VEC], scale), __fdiv_rn(h[c][(2 * j + 1) % VEC], scale));
        q[j >> 1] |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3)) << (16 * (j & 1));
      }
      reinterpret_cast<uint2*>(p.y8 + row * p.width)[i] = make_uint2(q[0], q[1]);
    } else {
      p.y8[row * p.width + i] = __nv_cvt_float_to_fp8(__fdiv_rn(h[c][0], scale), __NV_SATFINITE, __NV_E4M3);
    }
  }
}

template <int VEC, int CH>
cudaError_t launch_norm(const NormParams& p, int threads, cudaStream_t stream) {
  auto* fn = p.y8 ? add_rms_norm_kernel<VEC, CH, true> : add_rms_norm_kernel<VEC, CH, false>;
  fn<<<static_cast<unsigned>(p.rows), threads, 0, stream>>>(p);
  note_launches(1);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_add_rms_norm(const NormParams& p, cudaStream_t stream) {
  const bool vec = p.width % 8 == 0;
  const int n = vec ? p.width / 8 : p.width;
  // as few threads as keep CH at 4 (32 or 4 elements in flight per input), then more accesses per thread
  int threads = ((n + 3) / 4 + 31) / 32 * 32;
  if (threads > 1024) threads = 1024;
  const int ch = (n + threads - 1) / threads;
  if (vec) {
    if (ch <= 4) return launch_norm<8, 4>(p, threads, stream);
    return launch_norm<8, 8>(p, threads, stream);   // up to 65,536 elements
  }
  if (ch <= 4) return launch_norm<1, 4>(p, threads, stream);
  if (ch <= 16) return launch_norm<1, 16>(p, threads, stream);
  return launch_norm<1, 64>(p, threads, stream);    // up to 65,536 elements
}

}  // namespace msa
