// tq_paged_decode_attn: single-token attention of a ragged batch over a paged pool.
//
//   est_i = <q', khat'_i> + ||r_i|| sqrt(pi/2)/m <S q', 2 sign_i - 1>,  q' = Pi q,
//   out = Pi^T sum_i softmax(scale est)_i vhat'_i,  lse = log sum_i exp(scale est_i).
//
// Three launches, each a programmatic dependent of the one before:
//   prep    q' and S q' of every head and their tensor-core operands; the running sum of the lengths
//   split   the stream over the pages (tq_paged_split.cuh): one CTA per SM over an even share
//   merge   joins the partials of a head by log-sum-exp and turns o' back with Pi^T
// Prep and merge read Pi and S (64 KB each) once per CTA, not once per head: a CTA holds its share of
// the matrix in registers and takes the heads of a unit, or several units, past it.
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

// ------------------------------------------------------------------------------------------ prep

constexpr int PREP_THREADS = 512;  // four per matrix row

struct PrepArgs {
  int B, Hq, Hkv, g, hgroups, nb, qjl;
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

__device__ __forceinline__ void load_quarter(const float* M, int j, int q, float4 (&m)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) m[k] = __ldg(reinterpret_cast<const float4*>(M + j * D) + q + 4 * k);
}
__device__ __forceinline__ float dot_quarter(const float4 (&m)[8], const float* x, int q) {
  const float4* v = reinterpret_cast<const float4*>(x) + q;
  float a0 = 0.0f, a1 = 0.0f;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float4 w = v[4 * k];
    a0 = fmaf(m[k].x, w.x, a0);
    a1 = fmaf(m[k].y, w.y, a1);
    a0 = fmaf(m[k].z, w.z, a0);
    a1 = fmaf(m[k].w, w.w, a1);
  }
  float acc = a0 + a1;
  acc += __shfl_xor_sync(FULL, acc, 1);
  return acc + __shfl_xor_sync(FULL, acc, 2);
}

__global__ void __launch_bounds__(PREP_THREADS, 1) paged_prep(const __grid_constant__ PrepArgs a) {
  __shared__ float xs[HG][D], qs[HG][D], ss[HG][D];
  __shared__ float4 hc[HG];
  __shared__ int64_t wsum[PREP_THREADS / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  if (blockIdx.x == gridDim.x - 1) {
    // the last CTA: groups of the sequences before each one
    if (tid == 0) *a.err = 0u;
    int64_t base = 0;
    for (int b0 = 0; b0 < a.B; b0 += PREP_THREADS) {
      int first, len;
      int64_t x = b0 + tid < a.B ? seq_groups(a.lens[b0 + tid], a.max_tokens, a.window, first, len) : 0;
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
      for (int w = 0; w < PREP_THREADS / 32; ++w) {
        low += w < warp ? wsum[w] : 0;
        all += wsum[w];
      }
      if (b0 + tid < a.B) a.before[b0 + tid] = base + low + x - own;
      base += all;
    }
    if (tid == 0) a.before[a.B] = base;
    return;
  }
  const int j = tid >> 2, q = tid & 3, hgn = 4 * a.nb, ctas = gridDim.x - 1;
  const int seg_words = seg_bytes(a.nb) / 4;
  float4 pm[8], sm[8];
  load_quarter(a.Pi, j, q, pm);
  if (a.qjl) load_quarter(a.S, j, q, sm);
  for (int u = blockIdx.x; u < a.units; u += ctas) {
    const int hg = u % a.hgroups, kvh = (u / a.hgroups) % a.Hkv, b = u / (a.hgroups * a.Hkv);
    const int nh = min(HG, a.g - hg * HG);
    const int64_t q0 = ((int64_t)b * a.Hq + (int64_t)kvh * a.g + hg * HG) * D;
    for (int i = tid; i < nh * D; i += PREP_THREADS)
      (&xs[0][0])[i] = a.q_bf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(a.q)[q0 + i])
                                : reinterpret_cast<const float*>(a.q)[q0 + i];
    __syncthreads();
    for (int h = 0; h < nh; ++h) {
      const float y = dot_quarter(pm, xs[h], q);
      if (q == (h & 3)) qs[h][j] = y;
    }
    __syncthreads();
    if (a.qjl) {
      for (int h = 0; h < nh; ++h) {
        const float y = dot_quarter(sm, qs[h], q);
        if (q == (h & 3)) ss[h][j] = y;
      }
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
        for (int k = lane; k < D; k += 32) mx = fmaxf(mx, fmaxf(fabsf(qs[h][k]), a.qjl ? 16.0f * fabsf(ss[h][k]) : 0.0f));
#pragma unroll
        for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, o));
        const int ex = (mx < 16384.0f || !(mx < INFINITY)) ? 0 : ((__float_as_int(mx) >> 23) & 255) - 127 - 13;
        const float dn = __int_as_float((127 - ex) << 23);
        float ch = 0.0f, sh = 0.0f;
        if (a.qjl) {
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
    // Fragments: column gq of n-block nb is head 4 nb + gq / 2, part gq % 2 (0: fp16 hi, 1: lo); k-step
    // kk holds k = 16kk + 2t, +1 (register 0), +8, +9 (register 1) of lane (gq, t).  Word 2kk + r of a
    // lane is q', word 16 + 2kk + r is S q'; stored [n-block][word / 4][lane][word % 4].
    uint32_t* dst = a.ops + (int64_t)u * seg_words;
    for (int i = tid; i < a.nb * 1024; i += PREP_THREADS) {
      const int word = ((i >> 7) & 7) * 4 + (i & 3), ln = (i >> 2) & 31, nb = i >> 10;
      const int kk = (word >> 1) & 7, r = word & 1, sq = word >> 4;
      const int h = 4 * nb + (ln >> 3), t = ln & 3;
      const bool lo = (ln >> 2) & 1;
      uint32_t v = 0u;
      if (h < nh && (!sq || a.qjl)) {
        const float* src = (sq ? ss[h] : qs[h]) + 16 * kk + 8 * r + 2 * t;
        const float f = hc[h].w * (sq ? sgn_scale(2 * kk + r) : 1.0f);
        float h0, l0, h1, l1;
        split_half(src[0] * f, h0, l0);
        split_half(src[1] * f, h1, l1);
        v = lo ? pack_half2(l0, l1) : pack_half2(h0, h1);
      }
      dst[i] = v;
    }
    if (tid < hgn) reinterpret_cast<float4*>(dst + a.nb * 1024)[tid] = hc[tid];
    __syncthreads();  // the next unit reuses the vectors
  }
}

// ------------------------------------------------------------------------------------------ merge
//
// A CTA of 1024 threads (d = tid % 128, q = tid / 128) takes HPC heads of one unit: all of them, so
// that Pi is read once per unit, or one when there are too few units to fill the SMs.  With one head
// the eight thread groups share its partials; with several, group q joins head q's.  The turn back
// o_i = sum_j Pi[j][i] o'_j gives thread (i, q) rows 16q .. 16q + 15, loaded before the wait.

constexpr int MG = 8, MERGE_T = MG * D, MROWS = D / MG;

struct MergeArgs {
  int B, Hq, Hkv, g, hgroups, hgn, ctas;
  const float* part;
  const int64_t* before;
  const float* Pi;
  const unsigned int* err;
  void* out;
  int out_bf16;
  float* lse;
};

__device__ __forceinline__ void put_out(const MergeArgs& a, int64_t i, float v) {
  if (a.out_bf16) reinterpret_cast<__nv_bfloat16*>(a.out)[i] = __float2bfloat16_rn(v);
  else reinterpret_cast<float*>(a.out)[i] = v;
}

template <bool ONE>
__global__ void __launch_bounds__(MERGE_T) paged_merge(const __grid_constant__ MergeArgs a) {
  __shared__ float ob[HG][D];             // joined o' of each head
  __shared__ float red[MG][ONE ? 3 : HG][D];
  const int tid = threadIdx.x, d = tid % D, q = tid / D;
  float pj[MROWS];
#pragma unroll
  for (int r = 0; r < MROWS; ++r) pj[r] = __ldg(a.Pi + (MROWS * q + r) * D + d);
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  if (blockIdx.x == 0 && tid == 0 && *a.err) atomicOr(&g_paged_error, *a.err);
  const int u = ONE ? blockIdx.x / a.hgn : blockIdx.x;
  const int U = a.Hkv * a.hgroups, b = u / U, uu = u % U;
  const int hg = uu % a.hgroups, kvh = uu / a.hgroups;
  const int nh = min(HG, a.g - hg * HG);
  const int h0 = ONE ? blockIdx.x % a.hgn : 0;
  if (ONE && h0 >= nh) return;
  const int64_t orow = (int64_t)b * a.Hq + (int64_t)kvh * a.g + hg * HG;
  const int64_t lo = __ldcg(a.before + b), G = __ldcg(a.before + b + 1) - lo, N = __ldcg(a.before + a.B) * U;
  if (G == 0) {
    for (int h = ONE ? h0 : q; h < (ONE ? h0 + 1 : nh); h += MG) {
      if (ONE && q) break;
      put_out(a, (orow + h) * D + d, 0.0f);
      if (a.lse && d == 0) a.lse[orow + h] = -INFINITY;
    }
    return;
  }
  const int C = active_ctas(N, a.ctas);
  const int64_t f0 = lo * U + (int64_t)uu * G;
  const int c0 = range_of(N, C, f0), c1 = range_of(N, C, f0 + G - 1);
  // partials: the unit's own record, then those of the CTAs that go on with it
  const int S = 1 + c1 - c0;
  auto record = [&](int s, int h) {
    const int64_t slot = s == 0 ? u : (int64_t)a.B * U + c0 + s;
    return a.part + (slot * a.hgn + h) * PART;
  };
  float M = -1e30f, L = 0.0f, O = 0.0f;
  const int h = ONE ? h0 : q;
  if (ONE || q < nh) {
#pragma unroll 4
    for (int s = ONE ? q : 0; s < S; s += ONE ? MG : 1) {
      const float* p = record(s, h);
      const float2 ml = __ldcg(reinterpret_cast<const float2*>(p));
      const float o = __ldcg(p + 4 + d);
      const float Mn = fmaxf(M, ml.x);
      const float w0 = ex2(M - Mn), w1 = ex2(ml.x - Mn);
      L = fmaf(w1, ml.y, L * w0);
      O = fmaf(w1, o, O * w0);
      M = Mn;
    }
  }
  if constexpr (ONE) {
    red[q][0][d] = M;
    red[q][1][d] = L;
    red[q][2][d] = O;
    __syncthreads();
    if (q == 0) {
#pragma unroll
      for (int k = 0; k < MG; ++k) M = fmaxf(M, red[k][0][d]);
      L = 0.0f;
      O = 0.0f;
#pragma unroll
      for (int k = 0; k < MG; ++k) {
        const float w = ex2(red[k][0][d] - M);
        L = fmaf(w, red[k][1][d], L);
        O = fmaf(w, red[k][2][d], O);
      }
    }
    __syncthreads();
  }
  if (ONE ? q == 0 : q < nh) {
    ob[ONE ? 0 : q][d] = L != 0.0f ? O / L : 0.0f;
    if (a.lse && d == 0) a.lse[orow + h] = M * 0.69314718055994531f + logf(L);
  }
  __syncthreads();
#pragma unroll
  for (int x = 0; x < (ONE ? 1 : HG); ++x) {
    if (!ONE && x >= nh) break;
    float r = 0.0f;
#pragma unroll
    for (int k = 0; k < MROWS; ++k) r = fmaf(pj[k], ob[x][MROWS * q + k], r);
    red[q][x][d] = r;
  }
  __syncthreads();
  if (ONE ? q == 0 : q < nh) {
    float r = 0.0f;
#pragma unroll
    for (int k = 0; k < MG; ++k) r += red[k][ONE ? 0 : q][d];
    put_out(a, (orow + h) * D + d, r);
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
  w.before = w.part + up((size_t)(w.units + ctas) * 4 * w.nb * PART * 4);
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
  a.table_stride = table_stride;
  a.max_tokens = max_pages * pool->T_cap;
  a.window = window;
  a.ctas = sms;
  a.dyn_smem = attr_of(cudaDevAttrMaxSharedMemoryPerBlockOptin, 232448) / 256 * 256;
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
  p.qjl = pool->qjl_m ? 1 : 0;
  p.units = (int)w.units;
  p.max_tokens = a.max_tokens;
  p.window = window;
  p.sK = (float)(sc / sqrt((double)D));
  p.sQ = p.qjl ? (float)(sc * 2.0 * sqrt(M_PI / 2.0) / pool->qjl_m) : 0.0f;
  p.q = q;
  p.q_bf16 = q_dtype == TQ_BF16;
  p.Pi = params->Pi;
  p.S = params->S;
  p.lens = seq_lens;
  p.ops = a.ops;
  p.before = a.before;
  p.err = a.err;
  st = launch_dep(paged_prep, std::min<int64_t>(w.units, sms - 1) + 1, PREP_THREADS, s, false, "paged prep", p);
  if (st != TQ_OK) return st;
  const bool qjl = p.qjl != 0;
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
  m.part = a.part;
  m.before = a.before;
  m.Pi = params->Pi;
  m.err = a.err;
  m.out = out;
  m.out_bf16 = out_dtype == TQ_BF16;
  m.lse = lse;
  // one head per CTA while the units alone would leave SMs idle
  if (w.units < sms) return launch_dep(paged_merge<true>, w.units * m.hgn, MERGE_T, s, true, "paged merge", m);
  return launch_dep(paged_merge<false>, w.units, MERGE_T, s, true, "paged merge", m);
}
