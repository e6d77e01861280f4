// Paged split kernels of 4-bit keys.
#include "tq_paged_split.cuh"

namespace tq {
tq_status paged_split_k4(const PagedArgs& a, int v_bits, bool qjl, cudaStream_t s) {
  return launch_paged_k<4>(a, v_bits, qjl, s);
}
}  // namespace tq
