// Attention of few rows over listed records, head dim 64, 2-bit keys (kernel: sparse_few.cuh).
#include "sparse_few.cuh"

namespace tq {

cudaError_t launch_sparse_few_d64_k2(const PrefillParams& pp, cudaStream_t s) { return sparse_few_launch<64, 2>(pp, s); }

}  // namespace tq
