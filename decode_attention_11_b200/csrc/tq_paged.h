// What the kernels of tq_paged_decode_attn share: the arguments, the cut of a ragged batch into even
// ranges, and the layout of the workspace.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "tq_internal.h"

namespace tq {

constexpr int kGroup = kPageTokens;  // tokens of a group: the unit of work, inside one page
constexpr int kMinGroups = 11;       // groups a CTA gets at least: one per consumer warp

// Groups of 16 tokens that hold the tokens [first, len) a sequence of length n shows; a length outside
// [0, max_tokens] counts as 0.
__host__ __device__ inline int seq_groups(int n, int max_tokens, int window, int& first, int& len) {
  len = n < 0 || n > max_tokens ? 0 : n;
  first = window > 0 && len > window ? len - window : 0;
  return len ? (len + kGroup - 1) / kGroup - first / kGroup : 0;
}

// N groups over at most `ctas` CTAs: CTA c of active_ctas takes [range_start(c), range_start(c + 1)).
__host__ __device__ inline int active_ctas(int64_t N, int ctas) {
  const int64_t c = N / kMinGroups;
  return c < 1 ? 1 : c > ctas ? ctas : (int)c;
}
__host__ __device__ inline int64_t range_start(int64_t N, int C, int c) { return (int64_t)c * N / C; }
__host__ __device__ inline int range_of(int64_t N, int C, int64_t f) { return (int)(((f + 1) * C - 1) / N); }

// Query operands of one unit: the B fragments of q' and S q' (1024 words per n-block of four heads),
// then (fK, fQ, Kh, 2^-e) per head.
__host__ __device__ constexpr int seg_bytes(int nb) { return nb * (4096 + 4 * 16); }

struct PagedArgs {
  int B, Hq, Hkv, g, hgroups;
  int pages, ps;          // of the pool
  int64_t table_stride;
  int max_tokens, window;
  int ctas, dyn_smem;
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
  float* part;            // [units + ctas][heads] partials
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
