// Accumulated attention weight of many query rows at head dim 128 (kernel: attn_mass_umma.cuh).
#include "attn_mass_umma.cuh"

namespace tq {

cudaError_t launch_attn_mass_umma_d128(const MassParams& mp, cudaStream_t s) { return mass_umma_launch<128>(mp, s); }

}  // namespace tq
