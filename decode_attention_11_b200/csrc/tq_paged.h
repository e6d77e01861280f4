// What the kernels of tq_paged_decode_attn share: the arguments, the cut of a ragged batch into even
// ranges, and the layout of the workspace.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "tq_internal.h"

namespace tq {

constexpr int kGroup = kPageTokens;  // tokens of a group: the unit of work, inside one page

// Running maximum before any score.  Finite, so that differences of maxima are never inf - inf, and not above
// any finite score (at -1e30 a head whose scores were all below that came out as 0).
constexpr float kNoScore = -3.40282347e38f;

// Warps of a split CTA: multiples of four, so that its schedulers are loaded alike.  Up to four heads per
// unit (nb = 1): 12 warps of 168 registers (a call of 4 x 128K tokens in 4 bits: 184 us; 8 warps 194 us, 16 warps
// 196 us).  Up to eight: 8 warps of 237 (64 sequences to 16K, 3/2 bits: 125 us; 12 warps 134 us, 4 warps 160 us).
constexpr int paged_warps(int nb) { return nb == 1 ? 12 : 8; }

// Groups of 16 tokens that hold the tokens [first, len) a sequence of length n shows; a length outside
// [0, max_tokens] counts as 0.
__host__ __device__ inline int seq_groups(int n, int max_tokens, int window, int& first, int& len) {
  len = n < 0 || n > max_tokens ? 0 : n;
  first = window > 0 && len > window ? len - window : 0;
  return len ? (len + kGroup - 1) / kGroup - first / kGroup : 0;
}

// 64-bit division, on the 32-bit path when both operands fit.
__host__ __device__ inline int64_t div64(int64_t x, int64_t y) {
  return ((x | y) >> 31) == 0 ? (int64_t)((uint32_t)x / (uint32_t)y) : x / y;
}

// How N groups are cut: `warps` warps of each of `ctas` CTAs, warp W = cta * warps + w of them taking
// groups [range_start(W), range_start(W + 1)), at least one each.  Few groups go to many CTAs rather
// than to many warps of few.
struct Cut {
  int ctas, warps;
};
__host__ __device__ inline Cut cut_of(int64_t N, int ctas, int most_warps) {
  Cut c;
  const int64_t w = div64(N + ctas - 1, ctas);
  c.warps = w < 1 ? 1 : w > most_warps ? most_warps : (int)w;
  const int64_t n = div64(N, c.warps);
  c.ctas = n < 1 ? 1 : n > ctas ? ctas : (int)n;
  return c;
}
__host__ __device__ inline int64_t range_start(int64_t N, const Cut& c, int64_t W) {
  return div64(W * N, (int64_t)c.ctas * c.warps);
}
// the warp whose range holds group f
__host__ __device__ inline int range_of(int64_t N, const Cut& c, int64_t f) {
  return (int)div64((f + 1) * ((int64_t)c.ctas * c.warps) - 1, N);
}

// Query operands of one unit: the B fragments of q' and S q' (1024 words per block), then (fK, fQ, Kh,
// 2^-e) per head.  Up to four heads (nb = 1): one block, head h hi and lo in columns 2h, 2h + 1.  Up to
// eight (nb = 2): head h in column h, hi in block 0, lo in block 1.
__host__ __device__ constexpr int seg_bytes(int nb) { return nb * (4096 + 4 * 16); }

struct PagedArgs {
  int B, Hkv, g, hgroups;
  int pages, ps;          // of the pool
  uint64_t gpp_inv;       // ceil(2^64 / groups per page): group / groups per page by one product
  int64_t table_stride;
  int max_tokens, window;
  int ctas;
  const int32_t* table;
  const int32_t* lens;
  const uint8_t* k_codes;
  const uint8_t* k_signs;
  const float* k_norm;
  const float* k_rnorm;
  const uint8_t* v_codes;
  const float* v_norm;
  const float* kc;
  const float* vc;
  // workspace
  uint32_t* ops;          // [units] query operands
  float* part;            // [units + ctas x warps][heads] partials
  int64_t* before;        // [B + 1] groups of the sequences before b
  unsigned int* err;
};

tq_status paged_split_k2(const PagedArgs& a, int v_bits, bool qjl, cudaStream_t s);
tq_status paged_split_k3(const PagedArgs& a, int v_bits, bool qjl, cudaStream_t s);
tq_status paged_split_k4(const PagedArgs& a, int v_bits, bool qjl, cudaStream_t s);

// Error bits of paged decode calls so far (tq_decode_device_errors adds them to its own).
unsigned int paged_decode_errors(bool* ok);
int paged_reset_errors();

}  // namespace tq
