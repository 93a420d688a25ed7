// attn.cuh -- device helpers shared by the dense attention kernels (decode; prompts and trees): the softmax in log2 units,
// conversions of weights and codes, and a row of tensor memory multiplied by a factor.
#pragma once

#include "common.cuh"

namespace msa {

namespace {

constexpr float kLn2 = 0.6931471805599453f;
// A weight is 2^(s c - m) of an exact product and a maximum that is rounded, off by half the maximum's last place: 2^-14
// below this size of a logit in log2 units (710 nats), but without bound above it (2^127 from logits of 2^31).  Rows at or
// above it round their logits first: an fp32 softmax of fp32 logits, like that of the weights kernel, which reads them.
constexpr float kRoundLogits = 1024.0f;
// A product's factor with a page's scale in it, kept a normal number: 0 times a masked -inf, or inf times a product of 0,
// would be NaN.  A scale that is NaN stays it.
__device__ __forceinline__ float normal_factor(float c) {
  return c < 1.17549435e-38f ? 1.17549435e-38f : c > 3.40282347e38f ? 3.40282347e38f : c;
}

__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// 2^(a - b) with 0 for a = -inf whatever b (b may be -inf too)
__device__ __forceinline__ float exp2_diff(float a, float b) {
  return a == -INFINITY ? 0.0f : exp2_approx(a - b);
}
// 1 / l of a sum of weights; 0 when every weight is 0 (all logits -inf), as for a row without keys
__device__ __forceinline__ float inverse(float l) { return l == 0.0f ? 0.0f : 1.0f / l; }

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// two E4M3 codes (low 16 bits) -> fp16 pair; exact
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<unsigned short>(codes)));
  return r;
}

// Multiplies this thread's row of O or S (128 TMEM columns) by f.  Rare; out of line to leave the softmax its registers.
__device__ __noinline__ void scale_row(uint32_t addr, float f) {
  for (int c = 0; c < 128; c += 8) {
    uint32_t w[8];
    tmem_ld_8cols(addr + c, w);
    tmem_ld_wait_regs8(w);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(__uint_as_float(w[j]) * f);
    tmem_st_8cols(addr + c, w);
  }
  tmem_st_wait();
}

}  // namespace

}  // namespace msa
