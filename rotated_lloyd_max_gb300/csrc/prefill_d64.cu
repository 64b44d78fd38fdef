// Attention of several query tokens at head dim 64 (kernel: prefill.cuh).
#include "prefill.cuh"

namespace tq {

int prefill_rows_d64() { return PCfg<64>::BM; }
cudaError_t launch_prefill_d64(const PrefillParams& pp, cudaStream_t s) { return prefill_launch_d<64>(pp, s); }

}  // namespace tq
