// Device pieces shared by the decode kernels (tq_decode.cu, tq_paged_decode.cu, tq_paged_split.cuh):
// tensor-core instructions, fp16 parts, and the sign operand of the QJL term.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "tq_internal.h"

namespace tq {
namespace {

constexpr int D = kHeadDim;
constexpr int HG = 8;                  // query heads per MMA row block (hi rows 0-7, lo rows 8-15)
constexpr int PART = 4 + D;            // (max, sum, pad, pad, o'[128]) per partial: o' 16-byte aligned
constexpr unsigned FULL = 0xffffffffu;

// ------------------------------------------------------------------------------------------ PTX

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __halves2half2(__float2half_rn(lo), __float2half_rn(hi));
  return *reinterpret_cast<const uint32_t*>(&h);
}

// QJL sign operand: pair P (bits P and P + 16 of the lane's sign word, sketch rows 2t + e of
// k-half P % 2 of k-step P / 2) as a half2 of 1 + b 2^(q - 10), b the sign bit: the word, shifted
// so that the pair lands on mantissa bits q and q + 16 (q = 6 + P % 4), masked and ORed into 1.0.
// The B operand rows of such a pair are pre-scaled by 2^(10 - q), so the MMA yields
// C + sum_l b_l sq_l with the per-head constant C = sum_l 2^(10 - q_l) sq_l.
template <int P>
__device__ __forceinline__ uint32_t sgn(uint32_t w) {
  constexpr int q = 6 + (P & 3);
  uint32_t x;
  if constexpr (P < 4) x = w << 6;
  else if constexpr (P < 8) x = w << 2;
  else if constexpr (P < 12) x = w >> 2;
  else x = w >> 6;
  return (x & (0x00010001u << q)) | 0x3C003C00u;
}
// 2^(10 - q) of pair P: the B-row scale that undoes the mantissa position.
__host__ __device__ constexpr float sgn_scale(int P) { return (float)(16 >> (P & 3)); }

// Transpose an 8x8 matrix of 16-bit elements held one row pair per lane (m8n8 fragment layout).
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
  return y;
}

// x as fp16 hi + lo (about 22 significant bits) packed into one half2 (hi in the low half).
__device__ __forceinline__ uint32_t hilo_half2(float x) {
  const float hi = __half2float(__float2half_rn(x));
  const __half2 h = __floats2half2_rn(hi, x - hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

}  // namespace
}  // namespace tq
