// tq_paged_decode_attn: single-token attention of a ragged batch over a paged pool.
//
//   est_i = <q', khat'_i> + ||r_i|| sqrt(pi/2)/m <S q', 2 sign_i - 1>,  q' = Pi q,
//   out = Pi^T sum_i softmax(scale est)_i vhat'_i,  lse = log sum_i exp(scale est_i).
//
// Three launches, each a programmatic dependent of the one before:
//   prep    q' and S q' of every head and their tensor-core operands; the running sum of the lengths
//   split   the stream over the pages (tq_paged_split.cuh): one CTA per SM over an even share
//   merge   joins the partials of a head by log-sum-exp and turns o' back with Pi^T
// Prep and merge read Pi and S (64 KB each) once per CTA, not once per head.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "tq_decode_core.h"
#include "tq_paged.h"

namespace tq {
namespace {

// Same bits as the contiguous decode's, and bit 4: a page number or a length out of range.
__device__ unsigned int g_paged_error;

// -------------------------------------------------------------------------- 128 x 128 products
//
// Prep and merge multiply Pi, S and Pi^T with the vectors of up to eight heads.  On the FP32 units such
// a product is bound by reading the vectors from shared memory (16 us for 512 units of eight heads);
// here warp w keeps rows 16w .. 16w + 15 of the matrix as m16n8k16 A fragments, fp16 hi + lo of 2^8 M,
// for all units it meets, and the heads are the 8 columns.  The vectors enter as fp16 hi + lo of x 2^e
// with max |x| 2^e in [2^10, 2^11): M x = 2^-(8+e) (Mhi xhi + Mhi xlo + Mlo xhi), off by about 2^-22.

constexpr int MT = 256;              // threads: eight warps of 16 rows
constexpr int VS = D + 4;            // stride of a head's vector in shared memory (no bank conflicts)
constexpr float M_SCALE = 256.0f;

template <bool LO>
struct AFrag {
  uint32_t hi[8][4], lo[LO ? 8 : 1][4];
  __device__ __forceinline__ void set(int kk, int r, float x, float y) {
    x *= M_SCALE;
    y *= M_SCALE;
    float xh, xl, yh, yl;
    split_half(x, xh, xl);
    split_half(y, yh, yl);
    hi[kk][r] = pack_half2(xh, yh);
    if constexpr (LO) lo[kk][r] = pack_half2(xl, yl);
  }
  // rows 16w + gq (+ 8) of a row-major matrix, columns 16kk + 2t (+ 8), + 1
  __device__ __forceinline__ void load(const float* M, int w, int gq, int t) {
#pragma unroll
    for (int kk = 0; kk < 8; ++kk)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float2 v = __ldg(reinterpret_cast<const float2*>(M + (16 * w + gq + 8 * (r & 1)) * D + 16 * kk + 2 * t + 8 * (r >> 1)));
        set(kk, r, v.x, v.y);
      }
  }
  // the same of its transpose
  __device__ __forceinline__ void load_t(const float* M, int w, int gq, int t) {
#pragma unroll
    for (int kk = 0; kk < 8; ++kk)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float* m = M + (16 * kk + 2 * t + 8 * (r >> 1)) * D + 16 * w + gq + 8 * (r & 1);
        set(kk, r, __ldg(m), __ldg(m + D));
      }
  }
};

// A lane's share of its column's vector: x[4kk + 2r + i] = element 16kk + 8r + 2t + i of head gq.
// Products of the warp's 16 rows with the eight vectors: y[0], y[1]: row gq of heads 2t, 2t + 1, y[2],
// y[3]: row gq + 8.
template <bool LO>
__device__ __forceinline__ void rows_times(const AFrag<LO>& A, const float (&x)[32], float (&y)[4]) {
  float mx = 0.0f;
#pragma unroll
  for (int i = 0; i < 32; ++i) mx = fmaxf(mx, fabsf(x[i]));
  mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 1));
  mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 2));
  int e = ((__float_as_int(mx) >> 23) & 255) - 127;
  e = e < -100 ? -100 : e > 126 ? 126 : e;  // (infinities and NaN stay what they are)
  const float up = __int_as_float((127 + 10 - e) << 23);
  float d[2][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) d[0][i] = d[1][i] = 0.0f;
#pragma unroll
  for (int kk = 0; kk < 8; ++kk) {
    uint32_t bh[2], bl[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float h0, l0, h1, l1;
      split_half(x[4 * kk + 2 * r] * up, h0, l0);
      split_half(x[4 * kk + 2 * r + 1] * up, h1, l1);
      bh[r] = pack_half2(h0, h1);
      bl[r] = pack_half2(l0, l1);
    }
    mma16816(d[0], A.hi[kk], bh[0], bh[1]);
    mma16816(d[1], A.hi[kk], bl[0], bl[1]);
    if constexpr (LO) mma16816(d[1], A.lo[kk], bh[0], bh[1]);
  }
  const float down = __int_as_float((127 + e - 18) << 23);  // of head gq: 2^(e - 10) / 2^8
  const int t = threadIdx.x & 3;
  const float d0 = __shfl_sync(FULL, down, 8 * t), d1 = __shfl_sync(FULL, down, 8 * t + 4);
  y[0] = (d[0][0] + d[1][0]) * d0;
  y[1] = (d[0][1] + d[1][1]) * d1;
  y[2] = (d[0][2] + d[1][2]) * d0;
  y[3] = (d[0][3] + d[1][3]) * d1;
}
__device__ __forceinline__ void lane_share(const float* v, float (&x)[32]) {  // v: the head's vector
  const int t = threadIdx.x & 3;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float2 p = *reinterpret_cast<const float2*>(v + 8 * i + 2 * t);
    x[2 * i] = p.x;
    x[2 * i + 1] = p.y;
  }
}

// ------------------------------------------------------------------------------------------ prep

struct PrepArgs {
  int B, Hq, Hkv, g, hgroups, nb;
  int units, max_tokens, window;
  float sK, sQ;
  const void* q;
  int q_bf16;
  const float* Pi;
  const float* S;
  const int32_t* lens;
  uint32_t* ops;
  int64_t* before;
  unsigned int* err;
};

template <bool QJL>
__global__ void __launch_bounds__(MT, 1) paged_prep(const __grid_constant__ PrepArgs a) {
  __shared__ float qs[HG][VS], ss[HG][VS];
  __shared__ float4 hc[HG];
  __shared__ int64_t wsum[MT / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  if (blockIdx.x == gridDim.x - 1) {
    // the last CTA: groups of the sequences before each one
    if (tid == 0) *a.err = 0u;
    int64_t base = 0;
    bool bad = false;
    for (int b0 = 0; b0 < a.B; b0 += MT) {
      int first, len;
      const int n = b0 + tid < a.B ? a.lens[b0 + tid] : 0;
      bad = bad || n < 0 || n > a.max_tokens;
      int64_t x = seq_groups(n, a.max_tokens, a.window, first, len);
      const int64_t own = x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(FULL, x, o);
        if (lane >= o) x += y;
      }
      __syncthreads();  // the last round's warp sums are read
      if (lane == 31) wsum[warp] = x;
      __syncthreads();
      int64_t low = 0, all = 0;
      for (int w = 0; w < MT / 32; ++w) {
        low += w < warp ? wsum[w] : 0;
        all += wsum[w];
      }
      if (b0 + tid < a.B) a.before[b0 + tid] = base + low + x - own;
      base += all;
    }
    if (tid == 0) a.before[a.B] = base;
    if (bad) atomicOr(a.err, 16u);  // (after the barriers that follow its clearing)
    return;
  }
  const int gq = lane >> 2, t = lane & 3, hgn = 4 * a.nb, ctas = gridDim.x - 1;
  const int seg_words = seg_bytes(a.nb) / 4;
  // this lane's share of head gq of unit u (0 past the unit's heads)
  auto load_q = [&](int u, float (&x)[32]) {
    const int hg = u % a.hgroups, bk = u / a.hgroups;
    const bool live = u < a.units && gq < min(HG, a.g - hg * HG);
    const int64_t at = ((int64_t)bk * a.g + hg * HG + gq) * D + 2 * t;
    if (!live) {
#pragma unroll
      for (int i = 0; i < 32; ++i) x[i] = 0.0f;
    } else if (a.q_bf16) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(reinterpret_cast<const __nv_bfloat16*>(a.q) + at + 8 * i));
        x[2 * i] = __uint_as_float(w << 16);
        x[2 * i + 1] = __uint_as_float(w & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float2 w = __ldg(reinterpret_cast<const float2*>(reinterpret_cast<const float*>(a.q) + at + 8 * i));
        x[2 * i] = w.x;
        x[2 * i + 1] = w.y;
      }
    }
  };
  float next[32];
  load_q(blockIdx.x, next);
  AFrag<true> pi;
  AFrag<false> sk;
  pi.load(a.Pi, warp, gq, t);
  if constexpr (QJL) sk.load(a.S, warp, gq, t);  // (entries exact in fp16)
  for (int u = blockIdx.x; u < a.units; u += ctas) {
    const int hg = u % a.hgroups, nh = min(HG, a.g - hg * HG);
    float x[32], y[4];
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] = next[i];
    load_q(u + ctas, next);
    rows_times(pi, x, y);
    const int row = 16 * warp + gq;
    qs[2 * t][row] = y[0];
    qs[2 * t + 1][row] = y[1];
    qs[2 * t][row + 8] = y[2];
    qs[2 * t + 1][row + 8] = y[3];
    __syncthreads();
    if constexpr (QJL) {
      lane_share(qs[gq], x);
      rows_times(sk, x, y);
      ss[2 * t][row] = y[0];
      ss[2 * t + 1][row] = y[1];
      ss[2 * t][row + 8] = y[2];
      ss[2 * t + 1][row + 8] = y[3];
      __syncthreads();
    }
    // per head: a power of two 2^-e that brings q' and 16 S q' below 2^14 (fp16 range), and the QJL
    // constant Kh = -C - 0.5 sum_l sq_l 2^-e, C the sum of the fp16 parts of the pre-scaled S q':
    // sum_l sq_l (2 b_l - 1) = 2 (D_hi + D_lo + Kh) in the split kernel's product
    if (warp < hgn) {
      const int h = warp;
      if (h >= nh) {
        if (lane == 0) hc[h] = make_float4(a.sK, a.sQ, 0.0f, 1.0f);
      } else {
        float mx = 0.0f;
#pragma unroll
        for (int k = lane; k < D; k += 32) mx = fmaxf(mx, fmaxf(fabsf(qs[h][k]), QJL ? 16.0f * fabsf(ss[h][k]) : 0.0f));
#pragma unroll
        for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, o));
        const int ex = (mx < 16384.0f || !(mx < INFINITY)) ? 0 : ((__float_as_int(mx) >> 23) & 255) - 127 - 13;
        const float dn = __int_as_float((127 - ex) << 23);
        float ch = 0.0f, sh = 0.0f;
        if constexpr (QJL) {
#pragma unroll
          for (int k = lane; k < D; k += 32) {
            const float scl = (float)(16 >> ((k >> 3) & 3));  // sgn_scale of the k-step pair
            const float v = ss[h][k] * dn * scl;
            const float hi = __half2float(__float2half_rn(v));
            const float lo = __half2float(__float2half_rn(v - hi));
            ch += hi + lo;
            sh += (hi + lo) * (1.0f / scl);
          }
#pragma unroll
          for (int o = 16; o; o >>= 1) {
            ch += __shfl_xor_sync(FULL, ch, o);
            sh += __shfl_xor_sync(FULL, sh, o);
          }
        }
        if (lane == 0) {
          const float up = __int_as_float((127 + ex) << 23);
          hc[h] = make_float4(a.sK * up, a.sQ * up, -ch - 0.5f * sh, dn);
        }
      }
    }
    __syncthreads();
    // Fragments: columns as seg_bytes says; k-step kk holds k = 16kk + 2t, + 1 (register 0), + 8, + 9
    // (register 1) of lane (gq, t).  Word 2kk + r of a lane is q', word 16 + 2kk + r is S q'; stored
    // [block][word / 4][lane][word % 4].
    uint4* dst = reinterpret_cast<uint4*>(a.ops + (int64_t)u * seg_words);
    for (int i = tid; i < a.nb * 256; i += MT) {
      const int w4 = (i >> 5) & 7, ln = i & 31, nb = i >> 8, sq = w4 >> 2;
      const int h = a.nb == 1 ? ln >> 3 : ln >> 2;
      const bool lo = a.nb == 1 ? (ln >> 2) & 1 : nb;
      uint32_t v[4] = {0u, 0u, 0u, 0u};
      if (h < nh && (!sq || QJL)) {
        const float* src = (sq ? ss[h] : qs[h]) + 32 * (w4 & 3) + 2 * (ln & 3);
        const float dn = hc[h].w;
#pragma unroll
        for (int j = 0; j < 4; ++j) {  // k-steps 2 (w4 % 4) and + 1, both registers
          const float f = dn * (sq ? sgn_scale(j) : 1.0f);
          float h0, l0, h1, l1;
          split_half(src[8 * j] * f, h0, l0);
          split_half(src[8 * j + 1] * f, h1, l1);
          v[j] = lo ? pack_half2(l0, l1) : pack_half2(h0, h1);
        }
      }
      dst[i] = make_uint4(v[0], v[1], v[2], v[3]);
    }
    if (tid < hgn) reinterpret_cast<float4*>(dst + a.nb * 256)[tid] = hc[tid];
    __syncthreads();  // the next unit reuses the vectors
  }
}

// ------------------------------------------------------------------------------------------ merge
//
// A CTA joins the partials of all heads of a unit (warp h those of head h) or, when there are too few
// units to fill the SMs, of one head (the warps share its partials), and turns the joined o' back:
// o_i = sum_j Pi[j][i] o'_j, with Pi^T loaded before the wait for the split kernel.

constexpr int MW = MT / 32;

struct MergeArgs {
  int B, Hq, Hkv, g, hgroups, hgn, ctas, warps, items;
  const float* part;
  const int64_t* before;
  const float* Pi;
  const unsigned int* err;
  void* out;
  int out_bf16;
  float* lse;
};

template <bool ONE>
__global__ void __launch_bounds__(MT) paged_merge(const __grid_constant__ MergeArgs a) {
  __shared__ float os[HG][VS];              // joined o' of each head
  __shared__ float rm[MW], rl[MW], ro[ONE ? MW : 1][D];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, gq = lane >> 2, t = lane & 3;
  AFrag<true> pt;
  pt.load_t(a.Pi, warp, gq, t);
  for (int i = tid; i < HG * VS; i += MT) (&os[0][0])[i] = 0.0f;  // columns without a head
  __syncthreads();
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  if (blockIdx.x == 0 && tid == 0 && *a.err) atomicOr(&g_paged_error, *a.err);
  const int U = a.Hkv * a.hgroups;
  const int64_t N = __ldcg(a.before + a.B) * U;
  const Cut cut = cut_of(N, a.ctas, a.warps);
  for (int item = blockIdx.x; item < a.items; item += gridDim.x) {
    const int u = ONE ? item / a.hgn : item, h0 = ONE ? item % a.hgn : 0;
    const int b = u / U, uu = u - b * U, hg = uu % a.hgroups, kvh = uu / a.hgroups;
    const int nh = min(HG, a.g - hg * HG);
    if (ONE && h0 >= nh) continue;
    const int64_t orow = (int64_t)b * a.Hq + (int64_t)kvh * a.g + hg * HG;
    const int64_t lo = __ldcg(a.before + b), G = __ldcg(a.before + b + 1) - lo;
    // Partials: the unit's own record (of the warp, or the joint CTA, that opens it), then those of the
    // warps that go on with it: in the CTA where the unit opens, one for each CTA inside the unit, and in
    // the CTA where it ends (one if that CTA ends with it).
    int S = 0, w0 = 0, c0 = 0, c1 = 0, in0 = 0, mid = 0;
    if (G > 0) {
      const int64_t f0 = lo * U + (int64_t)uu * G, f1 = f0 + G;
      w0 = range_of(N, cut, f0);
      const int w1 = range_of(N, cut, f1 - 1);
      c0 = w0 / cut.warps;
      c1 = w1 / cut.warps;
      const bool joint0 = range_start(N, cut, (int64_t)c0 * cut.warps) == f0 && range_start(N, cut, (int64_t)(c0 + 1) * cut.warps) <= f1;
      in0 = joint0 ? 0 : min(w1, (c0 + 1) * cut.warps - 1) - w0;
      mid = max(0, c1 - c0 - 1);
      S = 1 + in0 + mid;
      if (c1 > c0) S += range_start(N, cut, (int64_t)(c1 + 1) * cut.warps) == f1 ? 1 : w1 - c1 * cut.warps + 1;
    }
    auto slot_of = [&](int s) -> int64_t {
      if (s == 0) return u;
      const int W = s <= in0 ? w0 + s : s <= in0 + mid ? (c0 + s - in0) * cut.warps : c1 * cut.warps + s - 1 - in0 - mid;
      return (int64_t)a.B * U + W;
    };
    const int h = ONE ? h0 : warp;
    float M = -1e30f, L = 0.0f;
    float4 O = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (h < nh) {
#pragma unroll 4
      for (int s = ONE ? warp : 0; s < S; s += ONE ? MW : 1) {
        const float* p = a.part + (slot_of(s) * a.hgn + h) * PART;
        const float2 ml = __ldcg(reinterpret_cast<const float2*>(p));
        const float4 o = __ldcg(reinterpret_cast<const float4*>(p + 4) + lane);
        const float Mn = fmaxf(M, ml.x);
        const float w0 = ex2(M - Mn), w1 = ex2(ml.x - Mn);
        L = fmaf(w1, ml.y, L * w0);
        O.x = fmaf(w1, o.x, O.x * w0);
        O.y = fmaf(w1, o.y, O.y * w0);
        O.z = fmaf(w1, o.z, O.z * w0);
        O.w = fmaf(w1, o.w, O.w * w0);
        M = Mn;
      }
    }
    if constexpr (ONE) {
      if (lane == 0) {
        rm[warp] = M;
        rl[warp] = L;
      }
      *reinterpret_cast<float4*>(&ro[warp][4 * lane]) = O;
      __syncthreads();
      if (warp == 0) {
        O = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        L = 0.0f;
#pragma unroll
        for (int k = 0; k < MW; ++k) M = fmaxf(M, rm[k]);
#pragma unroll
        for (int k = 0; k < MW; ++k) {
          const float w = ex2(rm[k] - M);
          const float4 o = *reinterpret_cast<const float4*>(&ro[k][4 * lane]);
          L = fmaf(w, rl[k], L);
          O.x = fmaf(w, o.x, O.x);
          O.y = fmaf(w, o.y, O.y);
          O.z = fmaf(w, o.z, O.z);
          O.w = fmaf(w, o.w, O.w);
        }
      }
    }
    if (h < nh && (!ONE || warp == 0)) {
      const float inv = L != 0.0f ? 1.0f / L : 0.0f;
      *reinterpret_cast<float4*>(&os[ONE ? 0 : h][4 * lane]) = make_float4(O.x * inv, O.y * inv, O.z * inv, O.w * inv);
      if (a.lse && lane == 0) a.lse[orow + h] = S ? M * 0.69314718055994531f + logf(L) : -INFINITY;
    }
    __syncthreads();
    float x[32], y[4];
    lane_share(os[gq], x);
    rows_times(pt, x, y);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int col = 2 * t + (i & 1);
      if (ONE ? col == 0 : col < nh) {
        const int64_t at = (orow + (ONE ? h0 : col)) * D + 16 * warp + gq + 8 * (i >> 1);
        if (a.out_bf16) reinterpret_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(y[i]);
        else reinterpret_cast<float*>(a.out)[at] = y[i];
      }
    }
    __syncthreads();  // the next item reuses the vectors
  }
}

// ------------------------------------------------------------------------------------------ host

int attr_of(cudaDeviceAttr attr, int fallback) {
  int dev = 0, v = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&v, attr, dev) != cudaSuccess || v <= 0) {
    cudaGetLastError();
    return fallback;
  }
  return v;
}

struct WsPlan {
  int hgroups, nb;
  int64_t units;
  size_t ops, part, before, err, bytes;
};
WsPlan ws_plan(int B, int Hq, int Hkv, int ctas) {
  WsPlan w;
  const int g = Hq / Hkv;
  w.hgroups = (g + HG - 1) / HG;
  w.nb = g <= 4 ? 1 : 2;
  w.units = (int64_t)B * Hkv * w.hgroups;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  w.ops = 0;
  w.part = up((size_t)w.units * seg_bytes(w.nb));
  w.before = w.part + up((size_t)(w.units + ctas * paged_warps(w.nb)) * 4 * w.nb * PART * 4);
  w.err = w.before + up((size_t)(B + 1) * 8);
  w.bytes = w.err + 256;
  return w;
}

template <typename A>
tq_status launch_dep(void (*kernel)(const A), int64_t grid, int threads, cudaStream_t s, bool dependent, const char* name,
                     const A& a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = dependent ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
  if (e != cudaSuccess) return fail(TQ_ERR_CUDA, "%s launch: %s", name, cudaGetErrorString(e));
  return TQ_OK;
}

tq_status check_heads(int B, int Hq, const tq_cache* pool) {
  if (B < 1 || B > 65536) return fail(TQ_ERR_INVALID_ARG, "B %d (1..65536)", B);
  if (Hq < 1 || Hq % pool->Hkv) return fail(TQ_ERR_INVALID_ARG, "Hq %d vs Hkv %d", Hq, pool->Hkv);
  if ((int64_t)B * Hq > 1 << 22) return fail(TQ_ERR_INVALID_ARG, "%d x %d query rows", B, Hq);
  return TQ_OK;
}

}  // namespace

unsigned int paged_decode_errors(bool* ok) {
  unsigned int v = 0;
  *ok = cudaMemcpyFromSymbol(&v, g_paged_error, sizeof(v)) == cudaSuccess;
  return v;
}
int paged_reset_errors() {
  const unsigned int z = 0;
  return cudaMemcpyToSymbol(g_paged_error, &z, sizeof(z)) == cudaSuccess ? 0 : -1;
}

}  // namespace tq

extern "C" size_t tq_paged_decode_workspace_size(int B, int Hq, const tq_cache* pool) {
  using namespace tq;
  if (!pool || pool->Hkv < 1 || check_heads(B, Hq, pool) != TQ_OK) return 0;
  return ws_plan(B, Hq, pool->Hkv, attr_of(cudaDevAttrMultiProcessorCount, 148)).bytes;
}

extern "C" tq_status tq_paged_decode_attn(const tq_params* params, const void* q, int q_dtype, int B, int Hq,
                                          const tq_cache* pool, const int32_t* table, int64_t table_stride,
                                          int max_pages, const int32_t* seq_lens, int window, float scale, void* out,
                                          int out_dtype, float* lse, void* workspace, size_t workspace_bytes,
                                          void* stream) {
  using namespace tq;
  const NvtxRange nvtx_range("tq_paged_decode_attn");
  clear_error();
  tq_status st = check_pool(pool);
  if (st == TQ_OK) st = check_params(params, pool);
  if (st == TQ_OK) st = check_heads(B, Hq, pool);
  if (st != TQ_OK) return st;
  if ((q_dtype != TQ_F32 && q_dtype != TQ_BF16) || (out_dtype != TQ_F32 && out_dtype != TQ_BF16))
    return fail(TQ_ERR_UNSUPPORTED, "q_dtype %d / out_dtype %d", q_dtype, out_dtype);
  if (max_pages < 1 || table_stride < max_pages || (int64_t)max_pages * pool->T_cap > 1 << 30)
    return fail(TQ_ERR_INVALID_ARG, "max_pages %d of %d tokens, table_stride %lld", max_pages, pool->T_cap, (long long)table_stride);
  if (window < 0) return fail(TQ_ERR_INVALID_ARG, "window %d", window);
  if (!q || !out || !workspace || !table || !seq_lens) return fail(TQ_ERR_INVALID_ARG, "q / out / workspace / table / seq_lens is NULL");
  if (!aligned16(q) || !aligned16(out) || !aligned16(workspace) || !aligned4(table) || !aligned4(seq_lens) || !aligned4(lse))
    return fail(TQ_ERR_INVALID_ARG, "q / out / workspace must be 16-byte aligned, table / seq_lens / lse 4-byte");
  const int sms = attr_of(cudaDevAttrMultiProcessorCount, 148);
  const WsPlan w = ws_plan(B, Hq, pool->Hkv, sms);
  if (workspace_bytes < w.bytes) return fail(TQ_ERR_WORKSPACE, "workspace %zu bytes, need %zu", workspace_bytes, w.bytes);
  uint8_t* ws = reinterpret_cast<uint8_t*>(workspace);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const double sc = (scale > 0.0f ? (double)scale : 1.0 / sqrt((double)D)) * 1.4426950408889634;  // log2 units

  PagedArgs a;
  a.B = B;
  a.Hq = Hq;
  a.Hkv = pool->Hkv;
  a.g = Hq / pool->Hkv;
  a.hgroups = w.hgroups;
  a.pages = pool->B;
  a.ps = pool->T_cap;
  // exact for every group number below 2^32 / groups per page and far beyond (2^64 / d rounded up is off by
  // less than d / 2^64 relative)
  a.gpp_inv = ~0ull / (uint64_t)(pool->T_cap / kGroup) + 1;
  a.table_stride = table_stride;
  a.max_tokens = max_pages * pool->T_cap;
  a.window = window;
  a.ctas = sms;
  a.table = table;
  a.lens = seq_lens;
  a.k_codes = pool->k_codes;
  a.k_signs = pool->k_signs;
  a.k_norm = pool->k_norm;
  a.k_rnorm = pool->k_rnorm;
  a.v_codes = pool->v_codes;
  a.v_norm = pool->v_norm;
  a.kc = params->k_centroids;
  a.vc = params->v_centroids;
  a.ops = reinterpret_cast<uint32_t*>(ws + w.ops);
  a.part = reinterpret_cast<float*>(ws + w.part);
  a.before = reinterpret_cast<int64_t*>(ws + w.before);
  a.err = reinterpret_cast<unsigned int*>(ws + w.err);

  PrepArgs p;
  p.B = B;
  p.Hq = Hq;
  p.Hkv = pool->Hkv;
  p.g = a.g;
  p.hgroups = w.hgroups;
  p.nb = w.nb;
  const bool qjl = pool->qjl_m != 0;
  p.units = (int)w.units;
  p.max_tokens = a.max_tokens;
  p.window = window;
  p.sK = (float)(sc / sqrt((double)D));
  p.sQ = qjl ? (float)(sc * 2.0 * sqrt(M_PI / 2.0) / pool->qjl_m) : 0.0f;
  p.q = q;
  p.q_bf16 = q_dtype == TQ_BF16;
  p.Pi = params->Pi;
  p.S = params->S;
  p.lens = seq_lens;
  p.ops = a.ops;
  p.before = a.before;
  p.err = a.err;
  st = launch_dep(qjl ? paged_prep<true> : paged_prep<false>, std::min<int64_t>(w.units, sms - 1) + 1, MT, s, false, "paged prep", p);
  if (st != TQ_OK) return st;
  st = pool->k_bits == 2   ? paged_split_k2(a, pool->v_bits, qjl, s)
       : pool->k_bits == 3 ? paged_split_k3(a, pool->v_bits, qjl, s)
                           : paged_split_k4(a, pool->v_bits, qjl, s);
  if (st != TQ_OK) return st;
  MergeArgs m;
  m.B = B;
  m.Hq = Hq;
  m.Hkv = pool->Hkv;
  m.g = a.g;
  m.hgroups = w.hgroups;
  m.hgn = 4 * w.nb;
  m.ctas = sms;
  m.warps = paged_warps(w.nb);
  m.part = a.part;
  m.before = a.before;
  m.Pi = params->Pi;
  m.err = a.err;
  m.out = out;
  m.out_bf16 = out_dtype == TQ_BF16;
  m.lse = lse;
  // one head per CTA while the units alone would leave SMs idle; two CTAs fit an SM
  const bool one = w.units < sms;
  m.items = (int)(one ? w.units * m.hgn : w.units);
  return launch_dep(one ? paged_merge<true> : paged_merge<false>, std::min<int64_t>(m.items, 2 * sms), MT, s, true, "paged merge", m);
}
