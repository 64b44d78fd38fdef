// Accumulated attention weight at head dim 128 (kernel: attn_mass.cuh).
#include "attn_mass.cuh"

namespace tq {

cudaError_t launch_attn_mass_d128(const MassParams& mp, int NT, cudaStream_t s) {
  return attn_mass_launch_d<128>(mp, NT, s);
}

}  // namespace tq
