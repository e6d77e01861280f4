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
#include "tq_launch.h"
#include "tq_paged.h"

namespace tq {
namespace {

// Same bits as the contiguous decode's, and bit 4: a page number or a length out of range.
__device__ unsigned int g_paged_error;

// -------------------------------------------------------------------------- 128 x 128 products
//
// Prep and merge multiply Pi, S and Pi^T with the vectors of many heads.  On the FP32 units such a
// product is bound by reading the vectors from shared memory (32 us for 512 units of eight heads in
// prep); here warp w keeps rows 16w .. 16w + 15 of the matrix as m16n8k16 A fragments, fp16 hi + lo of
// 2^8 M, for all heads it meets, and a CTA takes 8 or 16 heads at a time as the columns.  The vectors
// enter as fp16 hi + lo of x 2^e with max |x| 2^e in [2^10, 2^11), converted once and shared:
// M x = 2^-(8+e) (Mhi xhi + Mhi xlo + Mlo xhi), off by about 2^-22.  The tensor cores cut their sums off
// instead of rounding them, so the large products of each k-step are summed on the FP32 units (out of a
// 4096-token window in fp32: 1.6e-6 off with the sums kept in the tensor cores, 1.1e-6 so).
// The order of the columns in a k-step is free: k-step kk of lane t is columns 16kk + 4t .. + 3.

constexpr int MT = 256;              // threads: eight warps of 16 rows
constexpr int MW = MT / 32;
constexpr float M_SCALE = 256.0f;

// x and y as pairs of fp16 hi and lo parts.
__device__ __forceinline__ void split_pair(float x, float y, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x, y);
  const float2 f = __half22float2(h);
  const __half2 l = __floats2half2_rn(x - f.x, y - f.y);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = *reinterpret_cast<const uint32_t*>(&l);
}

template <bool LO>
struct AFrag {
  uint32_t hi[8][4], lo[LO ? 8 : 1][4];
  __device__ __forceinline__ void set(int kk, int r, float x, float y) {
    uint32_t l;
    split_pair(x * M_SCALE, y * M_SCALE, hi[kk][r], l);
    if constexpr (LO) lo[kk][r] = l;
  }
  // as laid out by store(): 16 KB of a warp's fragments in 16-byte words
  __device__ __forceinline__ void store(uint4* w, int lane) const {
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) {
      w[64 * kk + lane] = make_uint4(hi[kk][0], hi[kk][1], hi[kk][2], hi[kk][3]);
      w[64 * kk + 32 + lane] = make_uint4(lo[kk][0], lo[kk][1], lo[kk][2], lo[kk][3]);
    }
  }
  __device__ __forceinline__ void fetch(const uint4* w, int lane) {
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) {
      const uint4 h = __ldcg(w + 64 * kk + lane), l = __ldcg(w + 64 * kk + 32 + lane);
      hi[kk][0] = h.x; hi[kk][1] = h.y; hi[kk][2] = h.z; hi[kk][3] = h.w;
      lo[kk][0] = l.x; lo[kk][1] = l.y; lo[kk][2] = l.z; lo[kk][3] = l.w;
    }
  }
  // rows 16w + gq (+ 8) of a row-major matrix
  __device__ __forceinline__ void load(const float* M, int w, int gq, int t) {
#pragma unroll
    for (int kk = 0; kk < 8; ++kk)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(M + (16 * w + gq + 8 * r) * D + 16 * kk + 4 * t));
        set(kk, r, v.x, v.y);
        set(kk, 2 + r, v.z, v.w);
      }
  }
  // the same of its transpose
  __device__ __forceinline__ void load_t(const float* M, int w, int gq, int t) {
#pragma unroll
    for (int kk = 0; kk < 8; ++kk)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float* m = M + (16 * kk + 4 * t + 2 * (r >> 1)) * D + 16 * w + gq + 8 * (r & 1);
        set(kk, r, __ldg(m), __ldg(m + D));
      }
  }
};

// Vectors of R heads as B operands: fp16 pairs of columns 2j, 2j + 1, hi and lo parts, and the factor
// 2^-(8+e) of each.
template <int R>
struct Vecs {
  static constexpr int W = D / 2 + 4;  // words of a row (no bank conflicts)
  uint32_t hi[R][W], lo[R][W];
  float down[R];
  // by one warp: row r, lane l holding elements 4l .. 4l + 3
  __device__ __forceinline__ void put(int r, int lane, const float4& v) {
    float mx = fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
#pragma unroll
    for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, o));
    int e = ((__float_as_int(mx) >> 23) & 255) - 127;
    e = e < -100 ? -100 : e > 126 ? 126 : e;  // (infinities and NaN stay what they are)
    const float up = __int_as_float((127 + 10 - e) << 23);
    uint2 h, l;
    split_pair(v.x * up, v.y * up, h.x, l.x);
    split_pair(v.z * up, v.w * up, h.y, l.y);
    *reinterpret_cast<uint2*>(&hi[r][2 * lane]) = h;
    *reinterpret_cast<uint2*>(&lo[r][2 * lane]) = l;
    if (lane == 0) down[r] = __int_as_float((127 + e - 18) << 23);  // 2^(e - 10) / 2^8
  }
};

// Products of a warp's 16 matrix rows with vectors 8 nb .. 8 nb + 7: y[0], y[1]: row gq of vectors
// 8 nb + 2t, + 1; y[2], y[3]: row gq + 8.
template <bool LO, int R>
__device__ __forceinline__ void rows_times(const AFrag<LO>& A, const Vecs<R>& x, int nb, int gq, int t, float (&y)[4]) {
  float d[2][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) d[0][i] = d[1][i] = 0.0f;
#pragma unroll
  for (int kk = 0; kk < 8; ++kk) {
    const uint2 bh = *reinterpret_cast<const uint2*>(&x.hi[8 * nb + gq][8 * kk + 2 * t]);
    const uint2 bl = *reinterpret_cast<const uint2*>(&x.lo[8 * nb + gq][8 * kk + 2 * t]);
    float p[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    mma16816(p, A.hi[kk], bh.x, bh.y);
    mma16816(d[1], A.hi[kk], bl.x, bl.y);
    if constexpr (LO) mma16816(d[1], A.lo[kk], bh.x, bh.y);
#pragma unroll
    for (int i = 0; i < 4; ++i) d[0][i] += p[i];
  }
  const float d0 = x.down[8 * nb + 2 * t], d1 = x.down[8 * nb + 2 * t + 1];
  y[0] = (d[0][0] + d[1][0]) * d0;
  y[1] = (d[0][1] + d[1][1]) * d1;
  y[2] = (d[0][2] + d[1][2]) * d0;
  y[3] = (d[0][3] + d[1][3]) * d1;
}
// ... of all R vectors, to rows of fp32 results.
constexpr int VS = D + 4;
template <bool LO, int R>
__device__ __forceinline__ void product(const AFrag<LO>& A, const Vecs<R>& x, float (*res)[VS], int warp, int gq, int t) {
#pragma unroll
  for (int nb = 0; nb < R / 8; ++nb) {
    float y[4];
    rows_times(A, x, nb, gq, t, y);
    const int row = 16 * warp + gq;
    res[8 * nb + 2 * t][row] = y[0];
    res[8 * nb + 2 * t + 1][row] = y[1];
    res[8 * nb + 2 * t][row + 8] = y[2];
    res[8 * nb + 2 * t + 1][row + 8] = y[3];
  }
}

// Heads are numbered with the gaps of units that are not full: head p is column p % hgn of unit p / hgn.
struct HeadPlace {
  int unit, col;
  bool live;
  int64_t row;  // of q and out: b Hq + h
};
__device__ __forceinline__ HeadPlace head_place(int p, int hgn, int hgroups, int g, int units) {  // (p < 2^25)
  HeadPlace h;
  h.unit = p >> (hgn == 4 ? 2 : 3);
  h.col = p - h.unit * hgn;
  const int bk = h.unit / hgroups, hg = h.unit - bk * hgroups;
  h.live = h.unit < units && h.col < min(HG, g - hg * HG);
  h.row = (int64_t)bk * g + hg * HG + h.col;
  return h;
}

// ------------------------------------------------------------------------------------------ prep

constexpr int PR = 16;  // heads of a CTA at a time, two per warp

struct PrepArgs {
  int B, g, hgroups, nb;
  int units, max_tokens, window;
  float sK, sQ;
  const void* q;
  int q_bf16;
  const float* Pi;
  const float* S;
  const int32_t* lens;
  uint32_t* ops;
  int64_t* before;
  uint4* pit;  // fragments of Pi^T, for the merge kernel
  unsigned int* err;
};

template <bool QJL>
__global__ void __launch_bounds__(MT, 1) paged_prep(const __grid_constant__ PrepArgs a) {
  __shared__ __align__(16) Vecs<PR> vec;
  __shared__ __align__(16) float qs[PR][VS];
  __shared__ __align__(16) float ss[QJL ? PR : 1][VS];
  __shared__ __align__(16) uint32_t tile[PR * seg_bytes(1) / 16];  // operands of the heads' units
  __shared__ int64_t wsum[MW];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  if (blockIdx.x == gridDim.x - 1) {
    // the last CTA: the fragments of Pi^T (a CTA of the merge kernel that formed them itself spent half its
    // time on it), and the groups of the sequences before each one
    {
      AFrag<true> pt;
      pt.load_t(a.Pi, warp, lane >> 2, lane & 3);
      pt.store(a.pit + 512 * warp, lane);
    }
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
      for (int w = 0; w < MW; ++w) {
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
  const int heads = a.units * hgn;
  auto load_q = [&](int p) -> float4 {
    const HeadPlace h = head_place(p, hgn, a.hgroups, a.g, a.units);
    if (!h.live) return make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (!a.q_bf16) return __ldg(reinterpret_cast<const float4*>(reinterpret_cast<const float*>(a.q) + h.row * D) + lane);
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(reinterpret_cast<const __nv_bfloat16*>(a.q) + h.row * D) + lane);
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                       __uint_as_float(w.y & 0xffff0000u));
  };
  float4 next[2];
  next[0] = load_q(blockIdx.x * PR + 2 * warp);
  next[1] = load_q(blockIdx.x * PR + 2 * warp + 1);
  AFrag<true> pi;
  AFrag<false> sk;
  pi.load(a.Pi, warp, gq, t);
  if constexpr (QJL) sk.load(a.S, warp, gq, t);  // (entries exact in fp16)
  for (int p0 = blockIdx.x * PR; p0 < heads; p0 += ctas * PR) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      vec.put(2 * warp + x, lane, next[x]);
      next[x] = load_q(p0 + ctas * PR + 2 * warp + x);
    }
    __syncthreads();
    product(pi, vec, qs, warp, gq, t);
    __syncthreads();
    float4 q4[2], s4[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      q4[x] = *reinterpret_cast<const float4*>(&qs[2 * warp + x][4 * lane]);
      s4[x] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    if constexpr (QJL) {
#pragma unroll
      for (int x = 0; x < 2; ++x) vec.put(2 * warp + x, lane, q4[x]);
      __syncthreads();
      product(sk, vec, ss, warp, gq, t);
      __syncthreads();
#pragma unroll
      for (int x = 0; x < 2; ++x) s4[x] = *reinterpret_cast<const float4*>(&ss[2 * warp + x][4 * lane]);
    }
    // Per head: a power of two 2^-e that brings the largest of q' and 16 S q' into [2^13, 2^14), and the QJL
    // constant Kh = -C - 0.5 sum_l sq_l 2^-e, C the sum of the fp16 parts of the pre-scaled S q':
    // sum_l sq_l (2 b_l - 1) = 2 (D_hi + D_lo + Kh) in the split kernel's product.
    // Then the head's fragments: k-step kk holds k = 16kk + 2t, + 1 (register 0), + 8, + 9 (register 1)
    // of lane (gq, t); word 2kk + r of a lane is q', word 16 + 2kk + r is S q'; a unit's words are
    // [block][word / 4][lane][word % 4] with columns as seg_bytes says.
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const HeadPlace h = head_place(p0 + 2 * warp + x, hgn, a.hgroups, a.g, a.units);
      const float qv[4] = {q4[x].x, q4[x].y, q4[x].z, q4[x].w}, sv[4] = {s4[x].x, s4[x].y, s4[x].z, s4[x].w};
      float mx = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) mx = fmaxf(mx, fmaxf(fabsf(qv[i]), 16.0f * fabsf(sv[i])));
#pragma unroll
      for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, o));
      const int ex = !(mx < INFINITY) ? 0 : max(((__float_as_int(mx) >> 23) & 255) - 127, -90) - 13;
      const float dn = __int_as_float((127 - ex) << 23);
      const float scl = (float)(16 >> ((lane >> 1) & 3));  // sgn_scale of the lane's k-step pair
      uint32_t qh[2], ql[2], sh[2], sl[2];
      float ch = 0.0f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        split_pair(qv[2 * i] * dn, qv[2 * i + 1] * dn, qh[i], ql[i]);
        split_pair(sv[2 * i] * dn * scl, sv[2 * i + 1] * dn * scl, sh[i], sl[i]);
        const float2 fh = __half22float2(*reinterpret_cast<const __half2*>(&sh[i])), fl = __half22float2(*reinterpret_cast<const __half2*>(&sl[i]));
        ch += (fh.x + fl.x) + (fh.y + fl.y);
      }
      float sum = ch * (1.0f / scl);
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        ch += __shfl_xor_sync(FULL, ch, o);
        sum += __shfl_xor_sync(FULL, sum, o);
      }
      // this head's unit in the tile
      uint32_t* u = tile + (2 * warp + x) / hgn * (seg_bytes(a.nb) / 4);
      const int word = 2 * (lane >> 2) + ((lane & 3) >> 1), t0 = 2 * (lane & 1);
      const int ln = a.nb == 1 ? 8 * h.col : 4 * h.col;                      // lane 4 gq of the hi column
      const int lo = a.nb == 1 ? 16 : 1024;                                  // words from hi to lo
      uint32_t* w = u + (word >> 2) * 128 + (ln + t0) * 4 + (word & 3);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        w[4 * i] = qh[i];
        w[lo + 4 * i] = ql[i];
        if constexpr (QJL) {
          w[512 + 4 * i] = sh[i];
          w[512 + lo + 4 * i] = sl[i];
        }
      }
      if (lane == 0) {
        const float up = __int_as_float((127 + ex) << 23);
        reinterpret_cast<float4*>(u + a.nb * 1024)[h.col] = make_float4(a.sK * up, a.sQ * up, -ch - 0.5f * sum, dn);
      }
    }
    __syncthreads();
    const int u0 = p0 / hgn, n = min(PR / hgn, a.units - u0) * (seg_bytes(a.nb) / 16);
    uint4* dst = reinterpret_cast<uint4*>(a.ops + (int64_t)u0 * (seg_bytes(a.nb) / 4));
    for (int i = tid; i < n; i += MT) dst[i] = reinterpret_cast<const uint4*>(tile)[i];
    // (the tile is written again behind the next round's barriers)
  }
}

// ------------------------------------------------------------------------------------------ merge
//
// A CTA joins the partials of eight heads, one per warp, and turns the joined o' back,
// o_i = sum_j Pi[j][i] o'_j.  ONE, for few heads: one head, whose partials the eight warps share.  Two CTAs
// share an SM (128 registers: ten more cost a batch of 512 heads 4 us).

struct MergeArgs {
  int B, Hkv, g, hgroups, hgn, ctas, warps, units;
  const float* part;
  const int64_t* before;
  const uint4* pit;
  const unsigned int* err;
  void* out;
  int out_bf16;
  float* lse;
};

// Partials of a unit: its own record (of the warp, or the joint CTA, that opens it), then those of the
// warps that go on with it: in the CTA where the unit opens, one for each CTA inside the unit, and in the
// CTA where it ends (one if that CTA ends with it).
struct Records {
  int S, w0, c0, c1, in0, mid, warps;
  int64_t unit, units;
  __device__ __forceinline__ void of(int64_t N, const Cut& cut, int64_t f0, int64_t G, int64_t u, int64_t all) {
    unit = u;
    units = all;
    warps = cut.warps;
    S = w0 = c0 = c1 = in0 = mid = 0;
    if (G == 0) return;
    const int64_t f1 = f0 + G;
    w0 = range_of(N, cut, f0);
    const int w1 = range_of(N, cut, f1 - 1);
    c0 = w0 / warps;
    c1 = w1 / warps;
    const bool joint0 = range_start(N, cut, (int64_t)c0 * warps) == f0 && range_start(N, cut, (int64_t)(c0 + 1) * warps) <= f1;
    in0 = joint0 ? 0 : min(w1, (c0 + 1) * warps - 1) - w0;
    mid = max(0, c1 - c0 - 1);
    S = 1 + in0 + mid;
    if (c1 > c0) S += range_start(N, cut, (int64_t)(c1 + 1) * warps) == f1 ? 1 : w1 - c1 * warps + 1;
  }
  __device__ __forceinline__ int64_t slot(int s) const {
    if (s == 0) return unit;
    return units + (s <= in0 ? w0 + s : s <= in0 + mid ? (c0 + s - in0) * warps : c1 * warps + s - 1 - in0 - mid);
  }
};

template <bool ONE>
__global__ void __launch_bounds__(MT, 2) paged_merge(const __grid_constant__ MergeArgs a) {
  constexpr int R = 8;
  __shared__ __align__(16) Vecs<R> vec;
  __shared__ __align__(16) float res[R][VS];
  __shared__ float rm[MW], rl[MW];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, gq = lane >> 2, t = lane & 3;
  vec.put(warp, lane, make_float4(0.0f, 0.0f, 0.0f, 0.0f));  // (ONE: the columns without a head)
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  AFrag<true> pt;
  pt.fetch(a.pit + 512 * warp, lane);
  if (blockIdx.x == 0 && tid == 0 && *a.err) atomicOr(&g_paged_error, *a.err);
  const int U = a.Hkv * a.hgroups;
  const int64_t N = __ldcg(a.before + a.B) * U;
  const Cut cut = cut_of(N, a.ctas, a.warps);
  const int heads = a.units * a.hgn;
  constexpr int STEP = ONE ? 1 : R;
  for (int p0 = blockIdx.x * STEP; p0 < heads; p0 += gridDim.x * STEP) {
    if (ONE && !head_place(p0, a.hgn, a.hgroups, a.g, a.units).live) continue;
    {
      const HeadPlace h = head_place(ONE ? p0 : p0 + warp, a.hgn, a.hgroups, a.g, a.units);
      float M = kNoScore, L = 0.0f;
      float4 O = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      int S = 0;
      if (h.live) {
        const int b = h.unit / U, uu = h.unit - b * U;
        const int64_t lo = __ldcg(a.before + b), G = __ldcg(a.before + b + 1) - lo;
        Records rec;
        rec.of(N, cut, lo * U + (int64_t)uu * G, G, h.unit, a.units);
        S = rec.S;
        constexpr int BATCH = 4, NEXT = ONE ? MW : 1;  // (loads of a batch together: one at a time they
        for (int s0 = ONE ? warp : 0; s0 < S; s0 += BATCH * NEXT) {  // took 9 us for a unit of 17 partials)
          float2 ml[BATCH];
          float4 o[BATCH];
#pragma unroll
          for (int i = 0; i < BATCH; ++i) {
            const int s = s0 + i * NEXT;
            const float* p = a.part + (rec.slot(s < S ? s : 0) * a.hgn + h.col) * PART;
            ml[i] = __ldcg(reinterpret_cast<const float2*>(p));
            o[i] = __ldcg(reinterpret_cast<const float4*>(p + 4) + lane);
          }
          float top = M;
#pragma unroll
          for (int i = 0; i < BATCH; ++i) {
            if (s0 + i * NEXT >= S) ml[i] = make_float2(kNoScore, 0.0f);
            top = fmaxf(top, ml[i].x);
          }
          const float w0 = ex2(M - top);
          L *= w0;
          O.x *= w0;
          O.y *= w0;
          O.z *= w0;
          O.w *= w0;
#pragma unroll
          for (int i = 0; i < BATCH; ++i) {
            if (s0 + i * NEXT >= S) break;
            const float w = ex2(ml[i].x - top);
            L = fmaf(w, ml[i].y, L);
            O.x = fmaf(w, o[i].x, O.x);
            O.y = fmaf(w, o[i].y, O.y);
            O.z = fmaf(w, o[i].z, O.z);
            O.w = fmaf(w, o[i].w, O.w);
          }
          M = top;
        }
      }
      if constexpr (ONE) {
        if (lane == 0) {
          rm[warp] = M;
          rl[warp] = L;
        }
        *reinterpret_cast<float4*>(&res[warp][4 * lane]) = O;
        __syncthreads();
        if (warp == 0) {
          O = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          L = 0.0f;
#pragma unroll
          for (int k = 0; k < MW; ++k) M = fmaxf(M, rm[k]);
#pragma unroll
          for (int k = 0; k < MW; ++k) {
            const float w = ex2(rm[k] - M);
            const float4 o = *reinterpret_cast<const float4*>(&res[k][4 * lane]);
            L = fmaf(w, rl[k], L);
            O.x = fmaf(w, o.x, O.x);
            O.y = fmaf(w, o.y, O.y);
            O.z = fmaf(w, o.z, O.z);
            O.w = fmaf(w, o.w, O.w);
          }
        }
      }
      if (!ONE || warp == 0) {
        const float inv = L != 0.0f ? 1.0f / L : 0.0f;
        vec.put(ONE ? 0 : warp, lane, make_float4(O.x * inv, O.y * inv, O.z * inv, O.w * inv));
        if (h.live && a.lse && lane == 0) a.lse[h.row] = S ? M * 0.69314718055994531f + logf(L) : -INFINITY;
      }
    }
    __syncthreads();
    product(pt, vec, res, warp, gq, t);
    __syncthreads();
    const int r = ONE ? 0 : warp;
    const HeadPlace h = head_place(p0 + r, a.hgn, a.hgroups, a.g, a.units);
    if (h.live && !(ONE && warp)) {
      const float4 v = *reinterpret_cast<const float4*>(&res[r][4 * lane]);
      if (a.out_bf16) {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
        reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(a.out) + h.row * D)[lane] =
            make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
      } else {
        reinterpret_cast<float4*>(reinterpret_cast<float*>(a.out) + h.row * D)[lane] = v;
      }
    }
    if constexpr (ONE) __syncthreads();  // (res is the warps' partials again)
  }
}

// ------------------------------------------------------------------------------------------ host

struct WsPlan {
  int hgroups, nb;
  int64_t units;
  size_t ops, part, before, pit, err, bytes;
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
  w.pit = w.before + up((size_t)(B + 1) * 8);
  w.err = w.pit + (size_t)MW * 512 * sizeof(uint4);
  w.bytes = w.err + 256;
  return w;
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
  return ws_plan(B, Hq, pool->Hkv, sm_count()).bytes;
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
  const int sms = sm_count();
  const WsPlan w = ws_plan(B, Hq, pool->Hkv, sms);
  if (workspace_bytes < w.bytes) return fail(TQ_ERR_WORKSPACE, "workspace %zu bytes, need %zu", workspace_bytes, w.bytes);
  uint8_t* ws = reinterpret_cast<uint8_t*>(workspace);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const double sc = (scale > 0.0f ? (double)scale : 1.0 / sqrt((double)D)) * 1.4426950408889634;  // log2 units

  PagedArgs a;
  a.B = B;
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
  p.pit = reinterpret_cast<uint4*>(ws + w.pit);
  p.err = a.err;
  st = launch(qjl ? paged_prep<true> : paged_prep<false>, std::min<int64_t>((w.units * 4 * w.nb + PR - 1) / PR, sms - 1) + 1, MT, 0,
              s, false, "paged prep", p);
  if (st != TQ_OK) return st;
  st = pool->k_bits == 2   ? paged_split_k2(a, pool->v_bits, qjl, s)
       : pool->k_bits == 3 ? paged_split_k3(a, pool->v_bits, qjl, s)
                           : paged_split_k4(a, pool->v_bits, qjl, s);
  if (st != TQ_OK) return st;
  MergeArgs m;
  m.B = B;
  m.Hkv = pool->Hkv;
  m.g = a.g;
  m.hgroups = w.hgroups;
  m.hgn = 4 * w.nb;
  m.ctas = sms;
  m.warps = paged_warps(w.nb);
  m.part = a.part;
  m.before = a.before;
  m.pit = p.pit;
  m.err = a.err;
  m.out = out;
  m.out_bf16 = out_dtype == TQ_BF16;
  m.lse = lse;
  m.units = (int)w.units;
  // One head per CTA while all fit at once (two CTAs per SM), else eight: 256 heads of 512 tokens 22 against
  // 25 us, 384 heads 26 against 25.5, 1024 heads 35 against 26, 9600 heads 147 against 61.  (Sixteen at a
  // time were no faster than eight anywhere, and 4 to 6 us slower up to 1200 heads.)
  const int64_t heads = w.units * m.hgn, room = 2 * sms;
  if (heads <= room) return launch(paged_merge<true>, heads, MT, 0, s, true, "paged merge", m);
  return launch(paged_merge<false>, std::min<int64_t>((heads + MW - 1) / MW, room), MT, 0, s, true, "paged merge", m);
}
