// Attention over listed records at head dim 256 (kernel: prefill_umma_wide.cuh).
#include "prefill_umma_wide.cuh"

namespace tq {

cudaError_t launch_prefill_listed_d256(const PrefillParams& pp, cudaStream_t s) {
  return prefill_wide_launch<256, true>(pp, s);
}

}  // namespace tq
