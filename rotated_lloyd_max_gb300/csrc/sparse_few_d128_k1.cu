// Attention of few rows over listed records, head dim 128, 1-bit keys (kernel: sparse_few.cuh).
#include "sparse_few.cuh"

namespace tq {

cudaError_t launch_sparse_few_d128_k1(const PrefillParams& pp, cudaStream_t s) { return sparse_few_launch<128, 1>(pp, s); }

}  // namespace tq
