// Attention of several query tokens at head dim 512 (kernel: prefill_umma_wide.cuh).
#include "prefill_umma_wide.cuh"

namespace tq {

int prefill_rows_d512() { return kPwRows; }
cudaError_t launch_prefill_d512(const PrefillParams& pp, cudaStream_t s) { return prefill_wide_launch<512, false>(pp, s); }

}  // namespace tq
