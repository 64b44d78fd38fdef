// Attention of several query tokens at head dim 64 (kernel: prefill_umma.cuh).
#include "prefill_umma.cuh"

namespace tq {

int prefill_rows_d64() { return kPfRows; }
cudaError_t launch_prefill_d64(const PrefillParams& pp, cudaStream_t s) { return prefill_umma_launch<64, false>(pp, s); }

}  // namespace tq
