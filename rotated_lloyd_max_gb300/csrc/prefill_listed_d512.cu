// Attention over listed records at head dim 512 (kernel: prefill_umma_wide.cuh).
#include "prefill_umma_wide.cuh"

namespace tq {

cudaError_t launch_prefill_listed_d512(const PrefillParams& pp, cudaStream_t s) {
  return prefill_wide_launch<512, true>(pp, s);
}

}  // namespace tq
