// norm.cu -- the residual sum and its root-mean-square norm, in front of a
// layer's projections (the index prologue among them), in bf16 or E4M3:
//   h = x + residual,  sum = bf16(h),  y = h / sqrt(mean(h^2) + eps) * gamma.
// The norm is taken from the fp32 h, before its rounding to the residual
// stream.  E4M3 output: one fp32 scale per row, max |y| / 448 (1 when that is
// below 2^-120), code = round-to-nearest-even(y / scale), as of an fp32 division.
//
// Bound by HBM: x and residual are read and sum and y written once (8 bytes an
// element, 7 with codes).  Rows of up to 32,768 stay in registers between the
// reductions, so nothing is read twice; of wider ones, 72 elements a thread in 64
// registers, 112 to 144 bytes a thread go to local memory.  Measured at 16,384 x
// 8,192: bf16 154 us (7.0 TB/s), codes 142 us (6.6 TB/s); with the warps' sums of a
// row added one after another instead of by shuffles the codes took 210 us (two
// reductions a row).  Wide rows leave an SM one CTA, whose loads and stores take
// turns: 4,096 x 32,768 207 and 203 us, 2,048 x 65,536 245 and 270 us (the same
// elements).
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

// The same value in every thread of the row's: `lanes` neighbours of a warp, or (lanes 0) the CTA; `red` holds a word
// per warp.  Values are >= 0 in both uses, so absent ones count as 0.
template <typename Op, bool WARP>
__device__ __forceinline__ float row_reduce(float v, float* red, int lanes) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (!WARP || o < lanes) v = Op::of(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  const int warps = blockDim.x >> 5;
  if (WARP || warps == 1) return v;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = static_cast<int>(threadIdx.x & 31) < warps ? red[threadIdx.x & 31] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = Op::of(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}

__device__ __forceinline__ void unpack8(const uint4& a, float (&f)[8]) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[2 * j] = __uint_as_float(w[j] << 16);
    f[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}

// A CTA per row, or (WARP) 8, 16 or 32 lanes of a warp per row; CH chunks of 8
// elements per thread.  Chunks are aligned in the tensor as a whole, so every
// access is 16 bytes whatever the width: with ODD (a width that is no multiple
// of 8) a row begins `lead` elements into its first chunk, elements of its
// neighbours in the first and last chunk count as 0 and are not written, and the
// tensor's last, partial chunk is read by element.
constexpr int kWarpThreads = 256;

// a / b, rounded to nearest, from 1 / b, rounded to nearest: the product, and the product's remainder times the reciprocal
// added once (Markstein, "Computation of elementary functions on the IBM RISC System/6000 processor", 1990).  The product
// alone is off by 2^-24 in rows at a time, which moves values that lie between two codes.
__device__ __forceinline__ float2 quotients(float2 a, float b, float inv) {
  const float2 i2 = make_float2(inv, inv), q = fmul2(a, i2);
  return ffma2(ffma2(q, make_float2(-b, -b), a), i2, q);
}

template <int CH, bool FP8, bool ODD, bool WARP>
__global__ void __launch_bounds__(WARP ? kWarpThreads : 1024) add_rms_norm_kernel(NormParams p, int lanes) {
  __shared__ float red[2][32];
  griddep_wait();
  const int T = WARP ? lanes : blockDim.x, t = WARP ? threadIdx.x & (lanes - 1) : threadIdx.x;
  const long long row = WARP ? (blockIdx.x * static_cast<long long>(kWarpThreads) + threadIdx.x) / lanes : blockIdx.x;
  const long long start = row * p.width;
  const int lead = ODD ? static_cast<int>(start & 7) : 0;
  const long long base = start - lead, end = p.rows * p.width;
  const int n = !WARP || row < p.rows ? (lead + p.width + 7) >> 3 : 0;  // no chunk past the last row
  // elements [lo, hi) of chunk i are the row's; all of them but for the first and the last chunk
  auto lo_of = [&](int i) { return ODD && i == 0 ? lead : 0; };
  auto hi_of = [&](int i) { return ODD ? min(8, lead + p.width - 8 * i) : 8; };
  auto inner = [&](int i) { return !ODD || (i > 0 && i < n - 1); };
  float h[CH][8];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int i = c * T + t;
#pragma unroll
    for (int j = 0; j < 8; ++j) h[c][j] = 0.0f;
    if (i >= n) continue;
    const long long at = base + 8ll * i;
    if (!ODD || at + 8 <= end) {
      unpack8(*reinterpret_cast<const uint4*>(p.x + at), h[c]);
      if (p.residual) {
        float r[8];
        unpack8(*reinterpret_cast<const uint4*>(p.residual + at), r);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[c][j] += r[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (at + j < end)
          h[c][j] = __bfloat162float(p.x[at + j]) + (p.residual ? __bfloat162float(p.residual[at + j]) : 0.0f);
    }
  }
  float sq = 0.0f;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int i = c * T + t;
    if (ODD && !inner(i)) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < lo_of(i) || j >= hi_of(i)) h[c][j] = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) sq = fmaf(h[c][j], h[c][j], sq);
  }
  // every thread has read its elements, so the outputs below may overwrite x or the residual in place (in WARP mode the
  // neighbours' elements in a row's first and last chunk may have been written by then: they are not used)
  const float total = row_reduce<AddOp, WARP>(sq, red[0], lanes);
  const float r = 1.0f / sqrtf(total / static_cast<float>(p.width) + p.eps);
  float top = 0.0f;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int i = c * T + t;
    if (i >= n) continue;
    const long long at = base + 8ll * i;
    const bool full = inner(i);
    const int lo = full ? 0 : lo_of(i), hi = full ? 8 : hi_of(i);
    if (p.sum) {
      if (full) {
        *reinterpret_cast<uint4*>(p.sum + at) = pack8(h[c]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j >= lo && j < hi) p.sum[at + j] = __float2bfloat16_rn(h[c][j]);
      }
    }
    if (!ODD) {
      float gm[8];
      unpack8(reinterpret_cast<const uint4*>(p.gamma)[i], gm);
#pragma unroll
      for (int j = 0; j < 8; ++j) h[c][j] = h[c][j] * r * gm[j];
    } else if (full) {  // gamma's eight elements from an address that is only 2-byte aligned
      const __nv_bfloat16* gm = p.gamma + (8 * i - lead);
      if (lead & 1) {
        h[c][0] = h[c][0] * r * __bfloat162float(gm[0]);
        h[c][7] = h[c][7] * r * __bfloat162float(gm[7]);
#pragma unroll
        for (int j = 1; j < 7; j += 2) {
          const uint32_t w = *reinterpret_cast<const uint32_t*>(gm + j);
          h[c][j] = h[c][j] * r * __uint_as_float(w << 16);
          h[c][j + 1] = h[c][j + 1] * r * __uint_as_float(w & 0xFFFF0000u);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          const uint32_t w = *reinterpret_cast<const uint32_t*>(gm + j);
          h[c][j] = h[c][j] * r * __uint_as_float(w << 16);
          h[c][j + 1] = h[c][j + 1] * r * __uint_as_float(w & 0xFFFF0000u);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j >= lo && j < hi) h[c][j] = h[c][j] * r * __bfloat162float(p.gamma[8 * i + j - lead]);
    }
    if (FP8) {
#pragma unroll
      for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(h[c][j]));
    } else if (full) {
      *reinterpret_cast<uint4*>(p.y + at) = pack8(h[c]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j >= lo && j < hi) p.y[at + j] = __float2bfloat16_rn(h[c][j]);
    }
  }
  if (!FP8) return;
  top = row_reduce<MaxOp, WARP>(top, red[1], lanes);
  float scale = __fdiv_rn(top, 448.0f);
  if (!(scale >= 0x1p-120f)) scale = 1.0f;  // a row of (next to) nothing: codes 0
  if (t == 0 && n > 0) p.scale[row] = scale;
  const float inv = __frcp_rn(scale);
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int i = c * T + t;
    if (i >= n) continue;
    const long long at = base + 8ll * i;
    uint32_t q[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = quotients(make_float2(h[c][2 * j], h[c][2 * j + 1]), scale, inv);
      q[j >> 1] |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3)) << (16 * (j & 1));
    }
    if (inner(i)) {
      *reinterpret_cast<uint2*>(p.y8 + at) = make_uint2(q[0], q[1]);
    } else {
      const int lo = lo_of(i), hi = hi_of(i);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j >= lo && j < hi) p.y8[at + j] = static_cast<uint8_t>(q[j >> 2] >> (8 * (j & 3)));
    }
  }
}

template <int CH, bool WARP>
cudaError_t launch_norm(const NormParams& p, int threads, cudaStream_t stream) {  // WARP: threads of a row
  const bool odd = p.width % 8 != 0;
  auto* fn = p.y8 ? (odd ? add_rms_norm_kernel<CH, true, true, WARP> : add_rms_norm_kernel<CH, true, false, WARP>)
                  : (odd ? add_rms_norm_kernel<CH, false, true, WARP> : add_rms_norm_kernel<CH, false, false, WARP>);
  const long long ctas = WARP ? (p.rows * threads + kWarpThreads - 1) / kWarpThreads : p.rows;
  const cudaError_t e = launch_pdl(fn, dim3(static_cast<unsigned>(ctas)), dim3(WARP ? kWarpThreads : threads), 0, stream,
                                   p, threads);
  if (e == cudaSuccess) note_launches(1);
  return e;
}

}  // namespace

cudaError_t launch_add_rms_norm(const NormParams& p, int sms, cudaStream_t stream) {
  const int n = (p.width + (p.width % 8 ? 14 : 7)) / 8;  // chunks of a row at most (8,193)
  auto threads_for = [&](int ch) { return ((n + ch - 1) / ch + 31) / 32 * 32; };
  // narrow rows: several to a CTA (with one each the SMs' 32 CTAs would have too few bytes in flight)
  if (n <= 32) return launch_norm<1, true>(p, n <= 8 ? 8 : n <= 16 ? 16 : 32, stream);
  if (n <= 64) return launch_norm<2, true>(p, 32, stream);
  // few rows: latency, one chunk per thread; else two (16,384 x 8,192: 156 us, 178 with four and half the threads)
  if (n <= 1024 && p.rows <= 4 * sms) return launch_norm<1, false>(p, threads_for(1), stream);
  if (n <= 2 * 1024) return launch_norm<2, false>(p, threads_for(2), stream);
  if (n <= 4 * 1024) return launch_norm<4, false>(p, threads_for(4), stream);
  return launch_norm<9, false>(p, threads_for(9), stream);
}

}  // namespace msa
