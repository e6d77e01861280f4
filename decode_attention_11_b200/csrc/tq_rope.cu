// tq_rope: rotary positions of queries and keys with one or several position axes.
//
// Pair i of every head of token n turns by t = pos[axis(i)][n] * base^(-2i/128).  A token's heads share
// its 64 angles, so 64 threads take a token: each turns one position into (cos, sin), and, after one
// barrier, keeps those of the pairs it works on in registers for all the heads it passes (every 8th, or
// every 4th in fp32).  All loads of a thread's first heads are under way before the angles are formed.
//
// The angle is formed in turns, pos * (base^(-2i/128) / 2 pi), in fp64 and reduced to [-1/2, 1/2]
// before it becomes fp32 for sincospi: at position 2^20 an fp32 product would be off by 0.06 rad.
// The rotation itself is fp32, rounded once to the output's type.  Bound by memory: every element is
// read and written once.  (Items spread over a CTA's threads by division, each reading its (cos, sin) from
// shared memory, took 67 us for 16384 tokens of 40 bf16 heads, bound by their instructions.)
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "tq_internal.h"

namespace tq {
namespace {

constexpr int D = kHeadDim;
constexpr int PAIRS = D / 2;
constexpr int PRE = 3;       // heads a thread has loads in flight for

struct RopeArgs {
  const void* x[2];          // q, k
  void* y[2];
  int64_t sn[2], sh[2];      // input strides (elements)
  int H[2];
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

// V threads share a head: thread c works on its pairs c E .. c E + E - 1: the 16-byte vectors c and c + V
// (HALF), or 2c and 2c + 1 (PAIR).  A CTA has one token: four to a CTA took 56 us for 16384 tokens of 40 bf16
// heads where this takes 52 us, and loads for five heads in flight 19.0 us for 5003 tokens of 18 fp32 heads
// where those for three take 18.1 us (fewer registers, more CTAs).
template <typename T, bool HALF>
__global__ void __launch_bounds__(PAIRS) rope_kernel(const __grid_constant__ RopeArgs a) {
  using Vc = Vec<T>;
  constexpr int E = Vc::N, V = PAIRS / E, HS = PAIRS / V;  // HS: heads at a time
  __shared__ __align__(16) float2 cs[PAIRS];
  const int i64 = threadIdx.x, c = i64 % V, h0 = i64 / V;
  const int n = blockIdx.x, H = a.H[0] + a.H[1];
  constexpr int STEP = HALF ? V : 1;
  const int first = HALF ? c : 2 * c;
  const T* in[2] = {reinterpret_cast<const T*>(a.x[0]) + (int64_t)n * a.sn[0], reinterpret_cast<const T*>(a.x[1]) + (int64_t)n * a.sn[1]};
  T* out[2] = {reinterpret_cast<T*>(a.y[0]) + (int64_t)n * a.H[0] * D, reinterpret_cast<T*>(a.y[1]) + (int64_t)n * a.H[1] * D};
  uint4 lo[PRE], hi[PRE];
  auto load = [&](int p, int h) {
    const uint4* src = reinterpret_cast<const uint4*>(h < a.H[0] ? in[0] + h * a.sh[0] : in[1] + (h - a.H[0]) * a.sh[1]) + first;
    lo[p] = src[0];
    hi[p] = src[STEP];
  };
#pragma unroll
  for (int p = 0; p < PRE; ++p)
    if (h0 + p * HS < H) load(p, h0 + p * HS);
  const double t = (double)a.pos[a.axis[i64] * a.pos_stride + n] * a.turns[i64];
  float s, co;
  sincospif(2.0f * (float)(t - rint(t)), &s, &co);
  cs[i64] = make_float2(co, a.sign * s);
  __syncthreads();
  float2 w[E];
#pragma unroll
  for (int i = 0; i < E; i += 2) {
    const float4 v = *reinterpret_cast<const float4*>(&cs[c * E + i]);
    w[i] = make_float2(v.x, v.y);
    w[i + 1] = make_float2(v.z, v.w);
  }
  for (int hb = h0; hb < H; hb += PRE * HS) {
#pragma unroll
    for (int p = 0; p < PRE; ++p) {
      const int h = hb + p * HS;
      if (h >= H) break;
      float x[E], y[E];
      Vc::unpack(lo[p], x);
      Vc::unpack(hi[p], y);
#pragma unroll
      for (int i = 0; i < E; ++i) {
        // HALF: (x[i], y[i]) is pair cE + i; PAIR: the 2E coordinates in sequence are pairs cE ..
        float& u = HALF ? x[i] : 2 * i < E ? x[(2 * i) % E] : y[(2 * i) % E];
        float& v = HALF ? y[i] : 2 * i < E ? x[(2 * i + 1) % E] : y[(2 * i + 1) % E];
        const float u0 = u;
        u = fmaf(u0, w[i].x, -(v * w[i].y));
        v = fmaf(u0, w[i].y, v * w[i].x);
      }
      uint4* dst = reinterpret_cast<uint4*>(h < a.H[0] ? out[0] + h * D : out[1] + (h - a.H[0]) * D) + first;
      dst[0] = Vc::pack(x);
      dst[STEP] = Vc::pack(y);
      if (h + PRE * HS < H) load(p, h + PRE * HS);
    }
  }
}

// base^(-2i/128) / (2 pi) for all pairs: six square roots and products of their powers in extended
// precision, rounded once (64 calls of pow would take as long as the launch).
void turns_of(double base, double (&turns)[PAIRS]) {
  long double root[6];  // base^(-2^k / 64)
  root[5] = 1.0L / sqrtl((long double)base);
  for (int k = 4; k >= 0; --k) root[k] = sqrtl(root[k + 1]);
  long double p[PAIRS];
  p[0] = 1.0L;
  for (int i = 1; i < PAIRS; ++i) {
    const int k = 31 - __builtin_clz(i);
    p[i] = p[i - (1 << k)] * root[k];
  }
  for (int i = 0; i < PAIRS; ++i) turns[i] = (double)(p[i] / (2.0L * 3.14159265358979323846264338327950288L));
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
    const bool packed = (H[w] == 1 || sh[w] == kHeadDim) && (N == 1 || sn[w] == (int64_t)H[w] * kHeadDim);
    if (x[w] == y[w] && !packed)
      return fail(TQ_ERR_INVALID_ARG, "in place needs a contiguous input");
  }
  RopeArgs a;
  turns_of(base, a.turns);
  for (int i = 0; i < PAIRS; ++i) {
    if (axis_of_pair[i] >= axes) return fail(TQ_ERR_INVALID_ARG, "axis_of_pair[%d] = %d of %d axes", i, axis_of_pair[i], axes);
    a.axis[i] = axis_of_pair[i];
  }
  if (N == 0 || Hq + Hkv == 0) return TQ_OK;
  for (int w = 0; w < 2; ++w) {
    a.x[w] = x[w];
    a.y[w] = y[w];
    a.sn[w] = sn[w];
    a.sh[w] = sh[w];
    a.H[w] = H[w];
  }
  a.pos = pos;
  a.pos_stride = pos_stride;
  a.sign = inverse ? -1.0f : 1.0f;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == TQ_BF16) {
    if (style == TQ_ROPE_HALF) rope_kernel<__nv_bfloat16, true><<<N, PAIRS, 0, s>>>(a);
    else rope_kernel<__nv_bfloat16, false><<<N, PAIRS, 0, s>>>(a);
  } else {
    if (style == TQ_ROPE_HALF) rope_kernel<float, true><<<N, PAIRS, 0, s>>>(a);
    else rope_kernel<float, false><<<N, PAIRS, 0, s>>>(a);
  }
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(TQ_ERR_CUDA, "rope launch: %s", cudaGetErrorString(e));
  return TQ_OK;
}
