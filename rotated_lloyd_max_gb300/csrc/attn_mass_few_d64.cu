// Accumulated attention weight of few query rows at head dim 64 (kernel: attn_mass_few.cuh).
#include "attn_mass_few.cuh"

namespace tq {

cudaError_t launch_attn_mass_few_d64(const MassParams& mp, cudaStream_t s) { return attn_mass_few_launch_d<64>(mp, s); }

}  // namespace tq
