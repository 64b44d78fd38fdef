// Accumulated attention weight of many query rows at head dim 64 (kernel: attn_mass_umma.cuh).
#include "attn_mass_umma.cuh"

namespace tq {

cudaError_t launch_attn_mass_umma_d64(const MassParams& mp, cudaStream_t s) { return mass_umma_launch<64>(mp, s); }

}  // namespace tq
