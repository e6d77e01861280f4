// Rows of a paged pool: tq_paged_quantize (rows into pages) and tq_paged_read (rows back as values).
//
// Quantize has two routes.  Many rows go through the tcgen05 pipeline of tq_quantize (or its general
// kernel for fp32), which take a slot per token.  A decode step's few rows would leave that pipeline
// with a tile or two per SM and its full depth of latency, so they have a kernel of their own here:
// a CTA takes up to ROWS (token, kv-head) rows, whose keys and values are the eight columns of fp64
// matrix products with Pi, then S (each warp keeps 16 matrix rows in registers), and does the
// definition's arithmetic directly in fp64:
//   n = ||x||, u = sqrt(128) Pi x / n, idx = #{t_i <= u}, rho = u - c[idx], ||r|| = n ||rho|| / sqrt(128),
//   sign bits of S rho.
// No guard bands and no second pass are needed.  (Plain fp64 dot products, four threads a matrix row, took
// 18 us for 512 rows, bound by reading the vectors from shared memory.)
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "tq_internal.h"

namespace tq {
namespace {

constexpr int D = kHeadDim;
constexpr unsigned FULL = 0xffffffffu;

struct RowArgs {
  const void* k;
  const void* v;
  int64_t sn, sh;
  int in_f32;
  int N, Hkv, rows;  // rows: (token, kv-head) rows of a CTA
  const int32_t* slots;
  int pages, ps;
  int k_bits, v_bits, qjl;
  uint8_t* k_codes;
  uint8_t* k_signs;
  float* k_norm;
  float* k_rnorm;
  uint8_t* v_codes;
  float* v_norm;
  const float* Pi;
  const float* S;
  const float* kc;
  const float* kt;
  const float* vc;
  const float* vt;
};

constexpr int ROWS = 4;
// Rows per SM up to which the fp64 kernel is used.  Both sides in us, a call by itself with cold caches (the
// other routes' range is over 2, 3 and 4 bits):
//   rows per SM          2      4      8     12     16     20     32
//   fp64 kernel         15     17     26     35     45     54     82
//   bf16 pipeline    28-31  28-32  28-35  29-35  30-38  30-38  30-40
//   fp32 general     29-41  41-58  45-70  46-70  48-74  47-72  49-75
// (Quantize calls back to back, which overlap in the pipeline and find Pi and S in cache: fp64 kernel 10, 10,
// 18, 26, 34, 42, 66, pipeline 7 to 18 throughout, general 21 to 64.  A step has other kernels in between.)
constexpr int kRowsPerSmBf16 = 8, kRowsPerSmF32 = 16;
constexpr int QT = 256;    // eight warps of 16 matrix rows
constexpr int XS = D + 2;  // stride of a vector in shared memory (in doubles; no bank conflicts)

struct RowSmem {
  double x[2 * ROWS][XS];  // keys (0 .. ROWS-1), values
  double rho[2 * ROWS][XS];
  double n[2 * ROWS];
  double r2[ROWS];
  uint32_t kw[ROWS][16], vw[ROWS][16], sw[ROWS][4];  // packed rows
  float kc[16], kt[16], vc[16], vt[16];
};

__device__ __forceinline__ double warp_sumsq(const double* x) {
  const int lane = threadIdx.x & 31;
  double acc = 0.0;
#pragma unroll
  for (int k = 0; k < 4; ++k) acc = fma(x[lane + 32 * k], x[lane + 32 * k], acc);
#pragma unroll
  for (int o = 16; o; o >>= 1) acc += __shfl_xor_sync(FULL, acc, o);
  return acc;
}
__device__ __forceinline__ void put_code(uint32_t* w, int bit, int bits, uint32_t code) {
  atomicOr(w + (bit >> 5), code << (bit & 31));
  if ((bit & 31) + bits > 32) atomicOr(w + (bit >> 5) + 1, code >> (32 - (bit & 31)));
}

// A warp's 16 rows of a row-major fp32 matrix as m16n8k4 fp64 A fragments.  The order of the k-steps'
// columns is free: step 4m + i of lane t takes column 16m + 4t + i, so that a lane loads and reads four
// columns at a time.
struct Rows16 {
  float4 m[8][2];  // rows gq, gq + 8
  __device__ __forceinline__ void load(const float* M, int warp, int gq, int t) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
#pragma unroll
      for (int r = 0; r < 2; ++r) m[k][r] = __ldg(reinterpret_cast<const float4*>(M + (16 * warp + gq + 8 * r) * D + 16 * k + 4 * t));
  }
  // Products with eight vectors (column n: x[n]), in fp64: d[0], d[1]: row gq of columns 2t, 2t + 1;
  // d[2], d[3]: row gq + 8.
  __device__ __forceinline__ void times(const double (*x)[XS], int gq, int t, double (&d)[4]) const {
    double e[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i] = e[i] = 0.0;
    auto step = [](double (&s)[4], float a0, float a1, double b) {
      asm("mma.sync.aligned.m16n8k4.row.col.f64.f64.f64.f64 {%0,%1,%2,%3}, {%4,%5}, {%6}, {%0,%1,%2,%3};\n"
          : "+d"(s[0]), "+d"(s[1]), "+d"(s[2]), "+d"(s[3])
          : "d"((double)a0), "d"((double)a1), "d"(b));
    };
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const double2 b0 = *reinterpret_cast<const double2*>(&x[gq][16 * k + 4 * t]);
      const double2 b1 = *reinterpret_cast<const double2*>(&x[gq][16 * k + 4 * t + 2]);
      step(d, m[k][0].x, m[k][1].x, b0.x);
      step(e, m[k][0].y, m[k][1].y, b0.y);
      step(d, m[k][0].z, m[k][1].z, b1.x);
      step(e, m[k][0].w, m[k][1].w, b1.y);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i] += e[i];
  }
};

__global__ void __launch_bounds__(QT, 1) quantize_rows(const __grid_constant__ RowArgs a) {
  __shared__ RowSmem s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, gq = lane >> 2, t = lane & 3;
  const int64_t r0 = (int64_t)blockIdx.x * a.rows;
  const int nr = (int)min((int64_t)a.rows, (int64_t)a.N * a.Hkv - r0);
  Rows16 pi, sk;
  pi.load(a.Pi, warp, gq, t);
  if (a.qjl) sk.load(a.S, warp, gq, t);
  for (int i = tid; i < 2 * ROWS * D; i += QT) {  // (columns without a row: zeros)
    const int v = i / D, e = i % D, row = v % ROWS;
    double x = 0.0;
    if (row < nr) {
      const int64_t n = (r0 + row) / a.Hkv, h = (r0 + row) % a.Hkv;
      const int64_t at = n * a.sn + h * a.sh + e;
      const void* src = v < ROWS ? a.k : a.v;
      x = a.in_f32 ? (double)reinterpret_cast<const float*>(src)[at]
                   : (double)__bfloat162float(reinterpret_cast<const __nv_bfloat16*>(src)[at]);
    }
    s.x[v][e] = x;
  }
  if (tid < 16) s.kc[tid] = tid < (1 << a.k_bits) ? a.kc[tid] : 0.0f;
  else if (tid < 32) s.vc[tid - 16] = tid - 16 < (1 << a.v_bits) ? a.vc[tid - 16] : 0.0f;
  else if (tid < 48) s.kt[tid - 32] = tid - 32 < (1 << a.k_bits) - 1 ? a.kt[tid - 32] : INFINITY;
  else if (tid < 64) s.vt[tid - 48] = tid - 48 < (1 << a.v_bits) - 1 ? a.vt[tid - 48] : INFINITY;
  for (int i = tid; i < ROWS * 36; i += QT) (&s.kw[0][0])[i] = 0u;  // kw, vw and sw lie together
  static_assert(offsetof(RowSmem, sw) - offsetof(RowSmem, kw) == ROWS * 32 * 4, "packed rows");
  __syncthreads();
  {
    const double ss = warp_sumsq(s.x[warp]);  // eight warps, eight vectors
    if (lane == 0) s.n[warp] = sqrt(ss);
  }
  const double sqd = sqrt((double)D);
  double d[4];
  pi.times(s.x, gq, t, d);
  __syncthreads();  // the norms
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int v = 2 * t + (i & 1), j = 16 * warp + gq + 8 * (i >> 1), row = v % ROWS;
    const bool isv = v >= ROWS;
    const double n = s.n[v];
    // a zero row, or one with infinities or NaN, has the codes of u = 0
    const double u = n > 0.0 && n < INFINITY ? sqd * d[i] / n : 0.0;
    const float* th = isv ? s.vt : s.kt;
    uint32_t idx = 0;
#pragma unroll
    for (int c = 0; c < 15; ++c) idx += u >= (double)th[c] ? 1u : 0u;
    s.rho[v][j] = isv ? 0.0 : u - (double)s.kc[idx];
    const int bits = isv ? a.v_bits : a.k_bits;
    put_code(isv ? s.vw[row] : s.kw[row], bits * (isv ? v_slot_of_coord(j) : k_slot_of_coord(j)), bits, idx);
  }
  __syncthreads();
  if (a.qjl) {
    if (warp < ROWS) {
      const double ss = warp_sumsq(s.rho[warp]);
      if (lane == 0) s.r2[warp] = ss;
    }
    sk.times(s.rho, gq, t, d);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int v = 2 * t + (i & 1), l = 16 * warp + gq + 8 * (i >> 1);
      if (v < ROWS && d[i] >= 0.0) {
        const int bit = sign_bit_of_row(l);
        atomicOr(&s.sw[v][bit >> 5], 1u << (bit & 31));
      }
    }
    __syncthreads();
  }
  // one warp writes one row: key words, value words, signs and norms
  if (warp < nr) {
    const int64_t n = (r0 + warp) / a.Hkv;
    const int64_t to = slot_row(a.slots[n], (int)((r0 + warp) % a.Hkv), a.Hkv, a.pages, a.ps);
    if (to >= 0) {
      if (lane < 4 * a.k_bits) reinterpret_cast<uint32_t*>(a.k_codes)[to * 4 * a.k_bits + lane] = s.kw[warp][lane];
      if (lane < 4 * a.v_bits) reinterpret_cast<uint32_t*>(a.v_codes)[to * 4 * a.v_bits + lane] = s.vw[warp][lane];
      if (a.qjl && lane < 4) reinterpret_cast<uint32_t*>(a.k_signs)[to * 4 + lane] = s.sw[warp][lane];
      if (lane == 0) {
        a.k_norm[to] = (float)s.n[warp];
        a.v_norm[to] = (float)s.n[ROWS + warp];
        if (a.qjl) a.k_rnorm[to] = (float)(s.n[warp] * sqrt(s.r2[warp]) / sqd);
      }
    }
  }
}

// ------------------------------------------------------------------------------------- read
//
// Eight lanes per row, lane part p holding coordinates 16p .. 16p + 15: in the packed orders those
// are four runs of four key codes (slots 32t + 4p ..), eight runs of two value codes (slots
// 16g + 2p ..) and eight bits of each sign word, so a lane needs a few bytes of each array and writes
// 16 neighbouring values.  The lanes of a row fetch its codes in 16-byte pieces and pass them through
// shared memory (each lane its own bytes from global memory, 27 narrow loads that kept the L1 87% busy, took
// 53 us for 32K tokens in 3/3 bits where this takes 41 us, calls back to back).  Two or three sets of rows per
// warp, all loads first, took 46 and 53 us.  Bound by the values written and the latency of a row's chain slot -> codes -> values.

struct ReadArgs {
  int N, Hkv, pages, ps;
  const int32_t* slots;
  const uint8_t* k_codes;
  const uint8_t* k_signs;
  const float* k_norm;
  const float* k_rnorm;
  const uint8_t* v_codes;
  const float* v_norm;
  const float* kc;
  const float* vc;
  void* k_out;
  void* v_out;
  int8_t* signs;
  float* rnorm;
};

// 32 bytes at once: a whole sector per lane, where two 16-byte stores of 32-byte strides would write
// each sector in halves (54 -> 52 us for 32K tokens).
__device__ __forceinline__ void store32(void* dst, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
               "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
template <typename T>
__device__ __forceinline__ void store16(T* dst, const float (&v)[16]) {
  uint32_t w[8];
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(v[8 * h + i]);
      store32(dst + 8 * h, w);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    store32(dst, w);
  }
}

// Threads of a CTA: rows leave in small portions, so that others start (a call of 32K tokens, 3/3 bits, slots
// in random order: 43.2, 43.7 and 45.0 us with 64, 128 and 256 threads).
constexpr int RT = 64;

template <int KB, int VB, typename T>
__global__ void __launch_bounds__(RT) read_rows(const __grid_constant__ ReadArgs a) {
  constexpr int PITCH = 16 * (KB + VB) + 16;  // packed codes of a row (the fields of four rows in different banks)
  __shared__ __align__(16) unsigned char rows[RT / 8][PITCH];
  const int p = threadIdx.x & 7;
  const uint32_t r = blockIdx.x * (uint32_t)(RT / 8) + (threadIdx.x >> 3);
  const bool live = r < (uint32_t)a.N * (uint32_t)a.Hkv;  // (at most 2^30)
  // the codebooks, an entry per lane: a lookup is a shuffle (so whole warps stay to the end)
  const float kc = __ldg(a.kc + (threadIdx.x & ((1 << KB) - 1))), vc = __ldg(a.vc + (threadIdx.x & ((1 << VB) - 1)));
  unsigned char* mine = rows[threadIdx.x >> 3];
  int64_t row = -1;
  if (live) {
    const uint32_t n = r / (uint32_t)a.Hkv;
    row = slot_row(a.slots[n], (int)(r - n * a.Hkv), a.Hkv, a.pages, a.ps);
  }
  uint4 codes = make_uint4(0, 0, 0, 0), sg = codes;
  float kn = 0.0f, vn = 0.0f, rn = 0.0f;
  if (row >= 0) {
    if (p < KB + VB) {
      const uint8_t* src = p < KB ? a.k_codes + row * (16 * KB) + 16 * p : a.v_codes + row * (16 * VB) + 16 * (p - KB);
      codes = __ldg(reinterpret_cast<const uint4*>(src));
    }
    if (a.signs) sg = *reinterpret_cast<const uint4*>(a.k_signs + row * 16);
    kn = a.k_norm[row] * 0.08838834764831845f;  // 1 / sqrt(128)
    vn = a.v_norm[row] * 0.08838834764831845f;
    if (a.rnorm) rn = a.k_rnorm[row];
  }
  if (p < KB + VB) *reinterpret_cast<uint4*>(mine + 16 * p) = codes;
  __syncwarp();
  uint32_t kq[4], vq[8];
  // key codes: 4 KB bits at bit KB (32t + 4p); value codes: 2 VB bits at bit VB (16g + 2p)
  const unsigned char* kr = mine + (4 * KB * p) / 8;
  const unsigned char* vr = mine + 16 * KB + (2 * VB * p) / 8;
  const int ks = (4 * KB * p) & 7, vs = (2 * VB * p) & 7;
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    if constexpr (KB == 4) kq[t] = *reinterpret_cast<const uint16_t*>(kr + 16 * t);
    else if constexpr (KB == 2) kq[t] = kr[8 * t];
    else kq[t] = ((uint32_t)kr[12 * t] | (uint32_t)kr[12 * t + 1] << 8) >> ks;
  }
#pragma unroll
  for (int g = 0; g < 8; ++g) {
    if constexpr (VB == 3) vq[g] = ((uint32_t)vr[6 * g] | (uint32_t)vr[6 * g + 1] << 8) >> vs;  // (inside the pad at the end)
    else vq[g] = vr[2 * VB * g] >> vs;
  }
  float v[16];
#pragma unroll
  for (int t = 0; t < 4; ++t)
#pragma unroll
    for (int x = 0; x < 4; ++x)  // slot 32t + 4p + x is coordinate 16p + 8 (x / 2) + 2t + x % 2
      v[8 * (x >> 1) + 2 * t + (x & 1)] = __shfl_sync(FULL, kc, (int)(kq[t] >> (KB * x)), 1 << KB) * kn;
  if (live) store16(reinterpret_cast<T*>(a.k_out) + (int64_t)r * D + 16 * p, v);
#pragma unroll
  for (int g = 0; g < 8; ++g)
#pragma unroll
    for (int x = 0; x < 2; ++x)  // slot 16g + 2p + x is coordinate 16p + 8x + g
      v[8 * x + g] = __shfl_sync(FULL, vc, (int)(vq[g] >> (VB * x)), 1 << VB) * vn;
  if (!live) return;
  store16(reinterpret_cast<T*>(a.v_out) + (int64_t)r * D + 16 * p, v);
  if (a.signs) {
    // sketch row 16p + 8h + 2t + e is bit 2p + h + 16e of word t: byte 1 or -1 (0: no row)
    const uint32_t w[4] = {sg.x >> (2 * p), sg.y >> (2 * p), sg.z >> (2 * p), sg.w >> (2 * p)};
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {  // four rows: h = k / 2, words 2 (k % 2) and + 1, e = 0, 1
      const uint32_t x = (w[2 * (k & 1)] >> (k >> 1)) & 0x00010001u, y = (w[2 * (k & 1) + 1] >> (k >> 1)) & 0x00010001u;
      const uint32_t b = __byte_perm(x, y, 0x6420);
      o[k] = row >= 0 ? b | ((b ^ 0x01010101u) * 255u) : 0u;
    }
    reinterpret_cast<uint4*>(a.signs)[(int64_t)r * 8 + p] = make_uint4(o[0], o[1], o[2], o[3]);
  }
  if (a.rnorm && p == 0) a.rnorm[r] = rn;
}

template <int KB, int VB, typename T>
void launch_read(const ReadArgs& a, cudaStream_t s) {
  const int64_t rows = (int64_t)a.N * a.Hkv;
  read_rows<KB, VB, T><<<(unsigned)((rows * 8 + RT - 1) / RT), RT, 0, s>>>(a);
}
template <int KB, int VB>
void launch_read_t(const ReadArgs& a, int dtype, cudaStream_t s) {
  if (dtype == TQ_F32) launch_read<KB, VB, float>(a, s);
  else launch_read<KB, VB, __nv_bfloat16>(a, s);
}
template <int KB>
void launch_read_k(const ReadArgs& a, int vb, int dtype, cudaStream_t s) {
  if (vb == 2) launch_read_t<KB, 2>(a, dtype, s);
  else if (vb == 3) launch_read_t<KB, 3>(a, dtype, s);
  else launch_read_t<KB, 4>(a, dtype, s);
}

tq_status check_slots(const int32_t* slots, int N, const tq_cache* pool) {
  if (N < 0) return fail(TQ_ERR_INVALID_ARG, "N %d", N);
  if (N > 0 && (!slots || !aligned4(slots))) return fail(TQ_ERR_INVALID_ARG, "slots NULL or misaligned");
  if ((int64_t)N * pool->Hkv > (1LL << 30)) return fail(TQ_ERR_INVALID_ARG, "%d tokens of %d kv-heads: too many rows", N, pool->Hkv);
  return TQ_OK;
}

}  // namespace
}  // namespace tq

extern "C" tq_status tq_paged_quantize(const tq_params* params, const void* k, const void* v, int dtype,
                                       int64_t stride_n, int64_t stride_h, int N, const int32_t* slots,
                                       const tq_cache* pool, void* stream) {
  using namespace tq;
  const NvtxRange nvtx_range("tq_paged_quantize");
  clear_error();
  tq_status st = check_pool(pool);
  if (st == TQ_OK) st = check_params(params, pool);
  if (st == TQ_OK) st = check_slots(slots, N, pool);
  if (st != TQ_OK) return st;
  if (dtype != TQ_F32 && dtype != TQ_BF16) return fail(TQ_ERR_UNSUPPORTED, "dtype %d", dtype);
  if (N == 0) return TQ_OK;
  const int64_t es = dtype == TQ_F32 ? 4 : 2;
  if (!k || !v || !aligned16(k) || !aligned16(v)) return fail(TQ_ERR_INVALID_ARG, "k / v NULL or not 16-byte aligned");
  if (stride_n < 0 || stride_h < 0 || (stride_n * es) % 16 || (stride_h * es) % 16)
    return fail(TQ_ERR_INVALID_ARG, "strides (%lld, %lld) invalid", (long long)stride_n, (long long)stride_h);
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return fail(TQ_ERR_CUDA, "device query: %s", cudaGetErrorString(e));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int64_t rows = (int64_t)N * pool->Hkv;
  if (rows > (int64_t)(dtype == TQ_BF16 ? kRowsPerSmBf16 : kRowsPerSmF32) * sms) {
    if (dtype == TQ_BF16) {
      bool handled = false;
      st = quantize_bf16_pipeline(params, k, v, 0, stride_h, stride_n, N, 0, slots, pool, sms, s, &handled);
      if (handled || st != TQ_OK) return st;
    }
    return quantize_general_paged(params, k, v, dtype, stride_n, stride_h, N, slots, pool, sms, s);
  }
  RowArgs a;
  a.k = k;
  a.v = v;
  a.sn = stride_n;
  a.sh = stride_h;
  a.in_f32 = dtype == TQ_F32;
  a.N = N;
  a.Hkv = pool->Hkv;
  a.rows = (int)std::min<int64_t>(ROWS, (rows + sms - 1) / sms);
  a.slots = slots;
  a.pages = pool->B;
  a.ps = pool->T_cap;
  a.k_bits = pool->k_bits;
  a.v_bits = pool->v_bits;
  a.qjl = pool->qjl_m ? 1 : 0;
  a.k_codes = pool->k_codes;
  a.k_signs = pool->k_signs;
  a.k_norm = pool->k_norm;
  a.k_rnorm = pool->k_rnorm;
  a.v_codes = pool->v_codes;
  a.v_norm = pool->v_norm;
  a.Pi = params->Pi;
  a.S = params->S;
  a.kc = params->k_centroids;
  a.kt = params->k_thresholds;
  a.vc = params->v_centroids;
  a.vt = params->v_thresholds;
  quantize_rows<<<(unsigned)((rows + a.rows - 1) / a.rows), QT, 0, s>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return fail(TQ_ERR_CUDA, "paged quantize launch: %s", cudaGetErrorString(e));
  return TQ_OK;
}

extern "C" tq_status tq_paged_read(const tq_params* params, const tq_cache* pool, const int32_t* slots, int N, int dtype,
                                   void* k_out, void* v_out, int8_t* signs_out, float* rnorm_out, void* stream) {
  using namespace tq;
  const NvtxRange nvtx_range("tq_paged_read");
  clear_error();
  tq_status st = check_pool(pool);
  if (st == TQ_OK) st = check_params(params, pool);
  if (st == TQ_OK) st = check_slots(slots, N, pool);
  if (st != TQ_OK) return st;
  if (dtype != TQ_F32 && dtype != TQ_BF16) return fail(TQ_ERR_UNSUPPORTED, "dtype %d", dtype);
  if ((signs_out || rnorm_out) && !pool->qjl_m) return fail(TQ_ERR_INVALID_ARG, "signs / rnorm of a pool without a sketch");
  if (N == 0) return TQ_OK;
  if (!k_out || !v_out || ((reinterpret_cast<uintptr_t>(k_out) | reinterpret_cast<uintptr_t>(v_out)) & 31) || !aligned16(signs_out) ||
      !aligned4(rnorm_out))
    return fail(TQ_ERR_INVALID_ARG, "outputs NULL or misaligned (k_out, v_out: 32 bytes)");
  ReadArgs a;
  a.N = N;
  a.Hkv = pool->Hkv;
  a.pages = pool->B;
  a.ps = pool->T_cap;
  a.slots = slots;
  a.k_codes = pool->k_codes;
  a.k_signs = pool->k_signs;
  a.k_norm = pool->k_norm;
  a.k_rnorm = pool->k_rnorm;
  a.v_codes = pool->v_codes;
  a.v_norm = pool->v_norm;
  a.kc = params->k_centroids;
  a.vc = params->v_centroids;
  a.k_out = k_out;
  a.v_out = v_out;
  a.signs = signs_out;
  a.rnorm = rnorm_out;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (pool->k_bits == 2) launch_read_k<2>(a, pool->v_bits, dtype, s);
  else if (pool->k_bits == 3) launch_read_k<3>(a, pool->v_bits, dtype, s);
  else launch_read_k<4>(a, pool->v_bits, dtype, s);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(TQ_ERR_CUDA, "paged read launch: %s", cudaGetErrorString(e));
  return TQ_OK;
}
