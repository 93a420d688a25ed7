// attn.cuh -- device helpers shared by the dense attention kernels: the softmax in log2 units, conversions of weights and
// codes, and a row of tensor memory multiplied by a factor.
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

// Element i of lane t4 of four goes to element t4 of lane i.
__device__ __forceinline__ void quad_transpose(uint32_t (&x)[4], int t4) {
#pragma unroll
  for (int d = 1; d <= 2; d <<= 1)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i & d) continue;
      const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, t4 & d ? x[i] : x[i | d], d);
      if (t4 & d) x[i] = got;
      else x[i | d] = got;
    }
}

// 16 rows (TMEM lanes, from a multiple of 16) of 32 columns: registers 4 i + {0, 1} hold columns 8 i + 2 (lane % 4) +
// {0, 1} of row lane / 4, registers 4 i + {2, 3} those of row lane / 4 + 8.
__device__ __forceinline__ void tmem_ld_16rows_32cols(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_wait_regs16(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

// 16-byte pieces of a unit's codes (rows of 128 bytes, TMA's 128-byte swizzle) to 16-bit values in the layout in which
// TMA lands bf16 rows: K as bf16 (the queries' type), V as fp16 (the weights' type), both exact.  128 threads; eight
// lanes read a row, and those of its second half write their pieces in the other order, so that eight lanes' stores
// meet all banks.  Rows from `valid` on become zeros (V: 0 * NaN is NaN).
template <bool BF16>
__device__ __forceinline__ void widen(const uint8_t* codes, uint8_t* to, int thread, int valid) {
  const int chunk = thread & 7, half = chunk >> 2;
  const uint32_t flip = half;
#pragma unroll 1  // two or more at once hold up the MMAs' reads of shared memory (2 to 8 % slower)
  for (int row = thread >> 3; row < 128; row += 16) {
    const int x = row & 7;
    uint4 in = *reinterpret_cast<const uint4*>(codes + row * 128 + ((chunk ^ x) << 4));
    if (row >= valid) in = make_uint4(0, 0, 0, 0);
    const uint32_t w[4] = {in.x, in.y, in.z, in.w};
    uint32_t out[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      out[j] = e4m3x2_to_f16x2(j & 1 ? w[j >> 1] >> 16 : w[j >> 1]);
      if (BF16) {  // four significant bits: the upper half of the value in fp32
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&out[j]));
        out[j] = __byte_perm(__float_as_uint(f.x), __float_as_uint(f.y), 0x7632);
      }
    }
    uint4* dst = reinterpret_cast<uint4*>(to + half * 16384 + row * 128);
    const uint4 a = make_uint4(out[0], out[1], out[2], out[3]), b = make_uint4(out[4], out[5], out[6], out[7]);
    const uint32_t at = 2 * (chunk & 3);
    dst[(at + flip) ^ x] = flip ? b : a;
    dst[(at + 1 - flip) ^ x] = flip ? a : b;
  }
}

}  // namespace

}  // namespace msa
