// Accumulated attention weight of few query rows at head dim 256 (kernel: attn_mass_few.cuh).
#include "attn_mass_few.cuh"

namespace tq {

cudaError_t launch_attn_mass_few_d256(const MassParams& mp, cudaStream_t s) { return attn_mass_few_launch_d<256>(mp, s); }

}  // namespace tq
