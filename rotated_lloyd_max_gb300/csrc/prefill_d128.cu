// Attention of several query tokens at head dim 128 (kernel: prefill_umma.cuh).
#include "prefill_umma.cuh"

namespace tq {

int prefill_rows_d128() { return kPfRows; }
cudaError_t launch_prefill_d128(const PrefillParams& pp, cudaStream_t s) { return prefill_umma_launch<128, false>(pp, s); }

}  // namespace tq
