// Device pieces shared by the decode kernels (tq_decode.cu, tq_paged_split.cuh): tensor-core and
// shared-memory instructions, the pair tables that turn packed codes into fp16 operands, and the sign
// operand of the QJL term.
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

// 4-byte async copy (src_bytes = 0: no global read, zero fill).
__device__ __forceinline__ void cp_async4(void* dst, const void* src, int src_bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n" ::"r"(smem_u32(dst)), "l"(src),
               "r"(src_bytes));
}
__device__ __forceinline__ void cp_async8(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;\n" ::"r"(smem_u32(dst)), "l"(src));
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __halves2half2(__float2half_rn(lo), __float2half_rn(hi));
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Split x into fp16 hi + lo with x ~= hi + lo (about 22 significant bits).
__device__ __forceinline__ void split_half(float x, float& hi, float& lo) {
  hi = __half2float(__float2half_rn(x));
  lo = x - hi;
}

// Pair p (0..15) of a thread's key-code chunk: 2*KB bits starting at bit 2*KB*p.
template <int KB, int P>
__device__ __forceinline__ uint32_t k_pair_index(const uint32_t (&c)[KB]) {
  constexpr int off = 2 * KB * P;
  constexpr int w = off / 32, sh = off % 32;
  constexpr uint32_t mask = (1u << (2 * KB)) - 1u;
  if constexpr (KB == 4) {
    return __byte_perm(c[w], 0u, 0x4440u | (uint32_t)(sh / 8));  // byte sh/8, zero-extended
  } else if constexpr (sh + 2 * KB <= 32) {
    return (c[w] >> sh) & mask;
  } else {
    return __funnelshift_r(c[w], c[w + 1], sh) & mask;
  }
}

// Value-code pair indices of tokens a and b (one lane group's 16 codes each): index of code nu is
// code_a(nu) | code_b(nu) << VB.  For 4- and 2-bit codes the two chunks are interleaved field by
// field with a few logic operations, after which every index is one byte / nibble extract.
template <int VB>
struct VPairs {
  uint32_t w[VB == 3 ? 4 : 2 * (VB == 4 ? 2 : 1)];
  __device__ __forceinline__ void build(uint64_t ca, uint64_t cb) {
    if constexpr (VB == 4) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t a = (uint32_t)(h ? ca >> 32 : ca), b = (uint32_t)(h ? cb >> 32 : cb);
        w[2 * h + 0] = (a & 0x0F0F0F0Fu) | ((b << 4) & 0xF0F0F0F0u);   // nu = 8h + 2k
        w[2 * h + 1] = ((a >> 4) & 0x0F0F0F0Fu) | (b & 0xF0F0F0F0u);   // nu = 8h + 2k + 1
      }
    } else if constexpr (VB == 2) {
      const uint32_t a = (uint32_t)ca, b = (uint32_t)cb;
      w[0] = (a & 0x33333333u) | ((b << 2) & 0xCCCCCCCCu);   // nibble k: nu = 2k
      w[1] = ((a >> 2) & 0x33333333u) | (b & 0xCCCCCCCCu);   // nibble k: nu = 2k + 1
    } else {
      w[0] = (uint32_t)ca;
      w[1] = (uint32_t)(ca >> 32);
      w[2] = (uint32_t)cb;
      w[3] = (uint32_t)(cb >> 32);
    }
  }
  template <int NU>
  __device__ __forceinline__ uint32_t index() const {
    if constexpr (VB == 4) {
      return __byte_perm(w[2 * (NU >> 3) + (NU & 1)], 0u, 0x4440u | (uint32_t)((NU & 7) >> 1));
    } else if constexpr (VB == 2) {
      return (w[NU & 1] >> (4 * (NU >> 1))) & 0xFu;
    } else {
      const uint64_t ca = (uint64_t)w[0] | ((uint64_t)w[1] << 32);
      const uint64_t cb = (uint64_t)w[2] | ((uint64_t)w[3] << 32);
      return (uint32_t)((ca >> (3 * NU)) & 7u) | ((uint32_t)((cb >> (3 * NU)) & 7u) << 3);
    }
  }
};

__device__ __forceinline__ void mbar_init_(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;\n" ::"r"(smem_u32(bar)), "r"(count));
}
__device__ __forceinline__ void mbar_arrive_(uint64_t* bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];\n" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void mbar_expect_tx_(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;\n" ::"r"(smem_u32(bar)),
               "r"(bytes)
               : "memory");
}
// The thread's earlier cp.async copies arrive on the mbarrier when they land (counted in its init).
__device__ __forceinline__ void cp_async_arrive_noinc(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];\n" ::"r"(smem_u32(bar)) : "memory");
}
// One bulk copy global -> shared (sizes and addresses multiples of 16), completion in bytes.
__device__ __forceinline__ void bulk_g2s(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(
          smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t addr, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(done)
      : "r"(addr), "r"(parity), "r"(100000u)
      : "memory");
  return done != 0;
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

// Value chunk of one token for this lane group (16 codes of VB bits) as a 64-bit integer.
template <int VB>
__device__ __forceinline__ uint64_t load_v_chunk(const unsigned char* row, int gid) {
  if constexpr (VB == 4) {
    const uint2 w = *reinterpret_cast<const uint2*>(row + 8 * gid);
    return (uint64_t)w.x | ((uint64_t)w.y << 32);
  } else if constexpr (VB == 2) {
    return (uint64_t)*reinterpret_cast<const uint32_t*>(row + 4 * gid);
  } else {  // 6 bytes per lane group: read the aligned 12 bytes of the group pair
    const uint32_t* p = reinterpret_cast<const uint32_t*>(row + 12 * (gid >> 1));
    const uint32_t w0 = p[0], w1 = p[1], w2 = p[2];
    if (gid & 1) return (uint64_t)((w1 >> 16) | (w2 << 16)) | ((uint64_t)(w2 >> 16) << 32);
    return (uint64_t)w0 | ((uint64_t)(w1 & 0xffffu) << 32);
  }
}

// Transpose an 8x8 matrix of 16-bit elements held one row pair per lane (m8n8 fragment layout).
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];\n" : "=r"(v) : "r"(addr));
  return v;
}
// Vector shared loads at addresses the caller guarantees aligned (stage rows are 16-byte aligned).
__device__ __forceinline__ uint4 lds128(const void* p) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];\n" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(smem_u32(p)));
  return v;
}
__device__ __forceinline__ uint2 lds64(const void* p) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];\n" : "=r"(v.x), "=r"(v.y) : "r"(smem_u32(p)));
  return v;
}
// x as fp16 hi + lo (about 22 significant bits) packed into one half2 (hi in the low half).
__device__ __forceinline__ uint32_t hilo_half2(float x) {
  const float hi = __half2float(__float2half_rn(x));
  const __half2 h = __floats2half2_rn(hi, x - hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Pair tables: a pair of codes -> half2 of centroids, replicated per lane (bank = lane).
// 4-bit keys and values: 256 entries of 256 bytes (K replicas at +0, V at +128) starting at a
// 64 KB-aligned address, so one byte permute of the code word and of rk / rv (table address |
// lane offset) is the entry's address.  Other widths: separate K and V tables of 128-byte entries,
// address = (index << 7) + rk / rv.
template <int KB, int VB>
struct PairLut {
  static constexpr bool kPacked = KB == 4 && VB == 4;
  uint32_t rk, rv;
  uint32_t rk2, rv2;  // mixed layout: the 3-bit tables of the non-outlier half
  __device__ __forceinline__ uint32_t k2(uint32_t e) const { return lds32((e << 7) + rk2); }
  __device__ __forceinline__ uint32_t v2(uint32_t e) const { return lds32((e << 7) + rv2); }
  __device__ __forceinline__ uint32_t k(uint32_t e) const { return lds32((e << 7) + rk); }
  __device__ __forceinline__ uint32_t v(uint32_t e) const { return lds32((e << 7) + rv); }
  template <int Bt>
  __device__ __forceinline__ uint32_t k_byte(uint32_t w) const { return lds32(__byte_perm(w, rk, 0x7604u | (Bt << 4))); }
  template <int Bt>
  __device__ __forceinline__ uint32_t v_byte(uint32_t w) const { return lds32(__byte_perm(w, rv, 0x7604u | (Bt << 4))); }
};

// Key pair P (0..15) of a thread's code chunk, as a half2 of centroids.
template <int KB, int VB, int P>
__device__ __forceinline__ uint32_t k_pair(const PairLut<KB, VB>& L, const uint32_t (&c)[KB]) {
  if constexpr (PairLut<KB, VB>::kPacked) return L.template k_byte<P & 3>(c[P >> 2]);
  else return L.k(k_pair_index<KB, P>(c));
}
// Value pair NU of a token pair, as a half2 of centroids.
template <int KB, int VB, int NU>
__device__ __forceinline__ uint32_t v_pair(const PairLut<KB, VB>& L, const VPairs<VB>& p) {
  if constexpr (PairLut<KB, VB>::kPacked) return L.template v_byte<((NU & 7) >> 1)>(p.w[2 * (NU >> 3) + (NU & 1)]);
  else return L.v(p.template index<NU>());
}

}  // namespace
}  // namespace tq
