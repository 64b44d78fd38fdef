// Attention over listed records at head dim 128 (kernel: prefill_umma.cuh).
#include "prefill_umma.cuh"

namespace tq {

cudaError_t launch_prefill_listed_d128(const PrefillParams& pp, cudaStream_t s) {
  return prefill_umma_launch<128, true>(pp, s);
}

}  // namespace tq
