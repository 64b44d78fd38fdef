// Attention of several query tokens at head dim 256 (kernel: prefill_umma_wide.cuh).
#include "prefill_umma_wide.cuh"

namespace tq {

int prefill_rows_d256() { return kPwRows; }
cudaError_t launch_prefill_d256(const PrefillParams& pp, cudaStream_t s) { return prefill_wide_launch<256, false>(pp, s); }

}  // namespace tq
