// Paged split kernels of 2-bit keys.
#include "tq_paged_split.cuh"

namespace tq {
tq_status paged_split_k2(const PagedArgs& a, int v_bits, bool qjl, cudaStream_t s) {
  return launch_paged_k<2>(a, v_bits, qjl, s);
}
}  // namespace tq
