// A run of packed codes whose words are loaded ahead of their use.
#pragma once

#include <stdint.h>

namespace tq {

// NB bits of a packed row from bit `off` on, a multiple of NB, loaded now and aligned when used
template <int NB>
struct Run {
  static constexpr bool AL = NB % 32 == 0;
  static constexpr int STEP = NB % 16 ? 8 : 16;  // what an unaligned run's offset is a multiple of
  static constexpr int NW = (NB + 31) / 32, RAW = AL ? NW : (32 - STEP + NB + 31) / 32;
  uint32_t r[RAW];
  __device__ __forceinline__ void load(const uint8_t* row, int off) {
    const uint32_t* p = reinterpret_cast<const uint32_t*>(row) + (off >> 5);
    if constexpr (RAW == 4 && AL) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
      r[0] = v.x; r[1] = v.y; r[2] = v.z; r[3] = v.w;
    } else if constexpr (RAW == 2 && AL) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
      r[0] = v.x; r[1] = v.y;
    } else {
#pragma unroll
      for (int i = 0; i < RAW; ++i) r[i] = __ldg(p + i);
    }
  }
  // from shared memory
  __device__ __forceinline__ void fetch(const unsigned char* row, int off) {
    const uint32_t* p = reinterpret_cast<const uint32_t*>(row) + (off >> 5);
    if constexpr (RAW == 4 && AL) {
      const uint4 v = *reinterpret_cast<const uint4*>(p);
      r[0] = v.x; r[1] = v.y; r[2] = v.z; r[3] = v.w;
    } else if constexpr (RAW == 2 && AL) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      r[0] = v.x; r[1] = v.y;
    } else {
#pragma unroll
      for (int i = 0; i < RAW; ++i) r[i] = p[i];
    }
  }
  __device__ __forceinline__ void get(int off, uint32_t (&w)[NW]) const {
#pragma unroll
    for (int i = 0; i < NW; ++i) w[i] = AL ? r[i] : __funnelshift_r(r[i], i + 1 < RAW ? r[i + 1 < RAW ? i + 1 : i] : 0u, off & 31);
  }
};

}  // namespace tq
