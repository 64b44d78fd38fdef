// Attention of several query tokens at head dim 256 (kernel: prefill.cuh).
#include "prefill.cuh"

namespace tq {

int prefill_rows_d256() { return PCfg<256>::BM; }
cudaError_t launch_prefill_d256(const PrefillParams& pp, cudaStream_t s) { return prefill_launch_d<256>(pp, s); }

}  // namespace tq
