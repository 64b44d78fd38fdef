// Attention of several query tokens at head dim 512 (kernel: prefill.cuh).
#include "prefill.cuh"

namespace tq {

int prefill_rows_d512() { return PCfg<512>::BM; }
cudaError_t launch_prefill_d512(const PrefillParams& pp, cudaStream_t s) { return prefill_launch_d<512>(pp, s); }

}  // namespace tq
