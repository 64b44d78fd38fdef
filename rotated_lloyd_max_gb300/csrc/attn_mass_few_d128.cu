// Accumulated attention weight of few query rows at head dim 128 (kernel: attn_mass_few.cuh).
#include "attn_mass_few.cuh"

namespace tq {

cudaError_t launch_attn_mass_few_d128(const MassParams& mp, cudaStream_t s) { return attn_mass_few_launch_d<128>(mp, s); }

}  // namespace tq
