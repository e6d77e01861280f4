// tq_rope: rotary positions of queries and keys with one or several position axes.
//
// Pair i of every head of token n turns by t = pos[axis(i)][n] * base^(-2i/128).  Everything a
// token's heads need is 64 angles, so a CTA takes a few tokens at a time: 64 threads per token turn
// positions into (cos, sin) in shared memory while every thread's first loads of q and k are already
// under way, then the heads stream through in 16-byte loads and stores.
//
// The angle is formed in turns, pos * (base^(-2i/128) / 2 pi), in fp64 and reduced to [-1/2, 1/2]
// before it becomes fp32 for sincospi: at position 2^20 an fp32 product would be off by 0.06 rad.
// The rotation itself is fp32, rounded once to the output's type.  Bound by memory: every element is
// read and written once.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "tq_internal.h"

namespace tq {
namespace {

constexpr int D = kHeadDim;
constexpr int PAIRS = D / 2;
constexpr int THREADS = 256;
constexpr int TOK_MAX = 4;   // tokens of a CTA
constexpr int PRE = 4;       // work items a thread has loads in flight for

struct RopeArgs {
  const void* x[2];          // q, k
  void* y[2];
  int64_t sn[2], sh[2];      // input strides (elements)
  int H[2];
  int N, tok, axes;
  const int32_t* pos;
  int64_t pos_stride;
  float sign;                // -1: inverse
  uint8_t axis[PAIRS];
  double turns[PAIRS];       // base^(-2i/128) / (2 pi)
};

// 16 bytes of T as floats and back.
template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(const uint4& r, float (&v)[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(const uint4& r, float (&v)[4]) {
    v[0] = __uint_as_float(r.x);
    v[1] = __uint_as_float(r.y);
    v[2] = __uint_as_float(r.z);
    v[3] = __uint_as_float(r.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&v)[4]) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  }
};

// A work item is two 16-byte vectors of one head: coordinates c N .. and 64 + c N .. (HALF), or
// 2 c N .. in sequence (PAIR); V = items per head.
template <typename T, bool HALF>
__global__ void __launch_bounds__(THREADS) rope_kernel(const __grid_constant__ RopeArgs a) {
  using Vc = Vec<T>;
  constexpr int E = Vc::N, V = PAIRS / E;
  __shared__ float2 cs[TOK_MAX][PAIRS];
  const int tid = threadIdx.x;
  const int n0 = blockIdx.x * a.tok, nt = min(a.tok, a.N - n0);
  const int per_tok = (a.H[0] + a.H[1]) * V, total = nt * per_tok;
  // item -> input and output vectors
  auto where = [&](int item, const uint4*& src, uint4*& dst, int& tok, int& c) {
    tok = item / per_tok;
    int r = item - tok * per_tok;
    c = r % V;
    int h = r / V;
    const int which = h < a.H[0] ? 0 : 1;
    h -= which ? a.H[0] : 0;
    const int64_t n = n0 + tok;
    src = reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(a.x[which]) + n * a.sn[which] + h * a.sh[which]);
    dst = reinterpret_cast<uint4*>(reinterpret_cast<T*>(a.y[which]) + (n * a.H[which] + h) * D);
  };
  constexpr int STEP = HALF ? V : 1;  // vectors between an item's two
  auto first = [](int c) { return HALF ? c : 2 * c; };

  uint4 lo[PRE], hi[PRE];
#pragma unroll
  for (int p = 0; p < PRE; ++p) {
    const int item = tid + p * THREADS;
    if (item < total) {
      const uint4* src;
      uint4* dst;
      int tok, c;
      where(item, src, dst, tok, c);
      lo[p] = src[first(c)];
      hi[p] = src[first(c) + STEP];
    }
  }
  for (int i = tid; i < nt * PAIRS; i += THREADS) {
    const int tok = i / PAIRS, p = i % PAIRS;
    const double t = (double)a.pos[a.axis[p] * a.pos_stride + n0 + tok] * a.turns[p];
    float s, c;
    sincospif(2.0f * (float)(t - rint(t)), &s, &c);
    cs[tok][p] = make_float2(c, a.sign * s);
  }
  __syncthreads();
  for (int base = 0; base < total; base += PRE * THREADS) {
#pragma unroll
    for (int p = 0; p < PRE; ++p) {
      const int item = base + tid + p * THREADS;
      if (item >= total) break;
      const uint4* src;
      uint4* dst;
      int tok, c;
      where(item, src, dst, tok, c);
      float x[E], y[E];
      Vc::unpack(lo[p], x);
      Vc::unpack(hi[p], y);
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const float2 w = cs[tok][c * E + i];
        if constexpr (HALF) {  // (x[i], y[i]) is pair cE + i
          const float u = x[i];
          x[i] = fmaf(u, w.x, -(y[i] * w.y));
          y[i] = fmaf(u, w.y, y[i] * w.x);
        } else {               // the 2E coordinates in sequence are pairs cE ..
          float& u = 2 * i < E ? x[(2 * i) % E] : y[(2 * i) % E];
          float& v = 2 * i < E ? x[(2 * i + 1) % E] : y[(2 * i + 1) % E];
          const float u0 = u;
          u = fmaf(u0, w.x, -(v * w.y));
          v = fmaf(u0, w.y, v * w.x);
        }
      }
      dst[first(c)] = Vc::pack(x);
      dst[first(c) + STEP] = Vc::pack(y);
      // the item this register pair takes next
      const int next = item + PRE * THREADS;
      if (next < total) {
        where(next, src, dst, tok, c);
        lo[p] = src[first(c)];
        hi[p] = src[first(c) + STEP];
      }
    }
  }
}

}  // namespace
}  // namespace tq

extern "C" tq_status tq_rope(const void* q, int64_t q_stride_n, int64_t q_stride_h, int Hq, const void* k,
                             int64_t k_stride_n, int64_t k_stride_h, int Hkv, int dtype, int N, const int32_t* pos,
                             int64_t pos_stride, int axes, const uint8_t* axis_of_pair, double base, int style,
                             int inverse, void* q_out, void* k_out, void* stream) {
  using namespace tq;
  const NvtxRange nvtx_range("tq_rope");
  clear_error();
  if (dtype != TQ_F32 && dtype != TQ_BF16) return fail(TQ_ERR_UNSUPPORTED, "dtype %d", dtype);
  if (style != TQ_ROPE_HALF && style != TQ_ROPE_PAIR) return fail(TQ_ERR_UNSUPPORTED, "style %d", style);
  if (N < 0 || Hq < 0 || Hkv < 0 || Hq > 4096 || Hkv > 4096)
    return fail(TQ_ERR_INVALID_ARG, "sizes N=%d Hq=%d Hkv=%d", N, Hq, Hkv);
  if (axes < 1 || axes > 256 || !axis_of_pair || (N > 0 && !pos) || !aligned4(pos))
    return fail(TQ_ERR_INVALID_ARG, "axes %d / axis_of_pair / pos", axes);
  if (axes > 1 && pos_stride < 0) return fail(TQ_ERR_INVALID_ARG, "pos_stride %lld", (long long)pos_stride);
  if (!(base > 0.0) || !std::isfinite(base)) return fail(TQ_ERR_INVALID_ARG, "base %g", base);
  const int64_t es = dtype == TQ_F32 ? 4 : 2;
  const void* x[2] = {q, k};
  void* y[2] = {q_out, k_out};
  const int64_t sn[2] = {q_stride_n, k_stride_n}, sh[2] = {q_stride_h, k_stride_h};
  const int H[2] = {Hq, Hkv};
  for (int w = 0; w < 2; ++w) {
    if (H[w] == 0 || N == 0) continue;
    if (!x[w] || !y[w] || !aligned16(x[w]) || !aligned16(y[w]))
      return fail(TQ_ERR_INVALID_ARG, "q / k / outputs NULL or not 16-byte aligned");
    if (sn[w] < 0 || sh[w] < 0 || (sn[w] * es) % 16 || (sh[w] * es) % 16)
      return fail(TQ_ERR_INVALID_ARG, "strides (%lld, %lld) invalid", (long long)sn[w], (long long)sh[w]);
    const bool packed = sh[w] == kHeadDim && sn[w] == (int64_t)H[w] * kHeadDim;
    if (x[w] == y[w] && !packed)
      return fail(TQ_ERR_INVALID_ARG, "in place needs a contiguous input");
  }
  RopeArgs a = {};
  for (int i = 0; i < PAIRS; ++i) {
    if (axis_of_pair[i] >= axes) return fail(TQ_ERR_INVALID_ARG, "axis_of_pair[%d] = %d of %d axes", i, axis_of_pair[i], axes);
    a.axis[i] = axis_of_pair[i];
    a.turns[i] = std::pow(base, -2.0 * i / kHeadDim) / (2.0 * M_PI);
  }
  if (N == 0 || Hq + Hkv == 0) return TQ_OK;
  for (int w = 0; w < 2; ++w) {
    a.x[w] = x[w];
    a.y[w] = y[w];
    a.sn[w] = sn[w];
    a.sh[w] = sh[w];
    a.H[w] = H[w];
  }
  a.N = N;
  a.axes = axes;
  a.pos = pos;
  a.pos_stride = pos_stride;
  a.sign = inverse ? -1.0f : 1.0f;
  // one token per CTA while that still fills the SMs' threads once, else TOK_MAX
  a.tok = N <= 1184 ? 1 : TOK_MAX;
  const int grid = (N + a.tok - 1) / a.tok;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == TQ_BF16) {
    if (style == TQ_ROPE_HALF) rope_kernel<__nv_bfloat16, true><<<grid, THREADS, 0, s>>>(a);
    else rope_kernel<__nv_bfloat16, false><<<grid, THREADS, 0, s>>>(a);
  } else {
    if (style == TQ_ROPE_HALF) rope_kernel<float, true><<<grid, THREADS, 0, s>>>(a);
    else rope_kernel<float, false><<<grid, THREADS, 0, s>>>(a);
  }
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(TQ_ERR_CUDA, "rope launch: %s", cudaGetErrorString(e));
  return TQ_OK;
}
