// Attention of several query tokens at head dim 128 (kernel: prefill.cuh).
#include "prefill.cuh"

namespace tq {

int prefill_rows_d128() { return PCfg<128>::BM; }
cudaError_t launch_prefill_d128(const PrefillParams& pp, cudaStream_t s) { return prefill_launch_d<128>(pp, s); }

}  // namespace tq
