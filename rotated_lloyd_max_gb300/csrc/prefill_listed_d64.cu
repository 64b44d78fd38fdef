// Attention over listed records at head dim 64 (kernel: prefill_umma.cuh).
#include "prefill_umma.cuh"

namespace tq {

cudaError_t launch_prefill_listed_d64(const PrefillParams& pp, cudaStream_t s) {
  return prefill_umma_launch<64, true>(pp, s);
}

}  // namespace tq
