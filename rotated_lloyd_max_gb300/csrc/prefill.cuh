// Attention of several query tokens per sequence over records and ring: what
// its kernels (prefill_umma.cuh, prefill_umma_wide.cuh) and the merge of
// their context splits (prefill_merge.cu) share.
//
// The query rows of a kv head are its query heads x new tokens, row = token *
// G + head, so that a tile of rows shares the keys it reads whatever the group
// size.  Packed codes become f16 operands in shared memory (centroids x 2^15,
// so that side-list values up to 1 fit and no centroid is subnormal).  Rounding
// to f16 (11 bits) of rotated queries, centroids, scales and weights is finer
// than the bf16 output's 8; softmax statistics and outputs accumulate in f32.
// O stays in the rotated basis; the merge of the splits turns it back once.
#pragma once

#include "attn_mass.cuh"

namespace tq {

struct PrefillParams {
  QueryParams q;
  int Sc, St, cps, tps;  // splits over records / ring tokens; records, ring tokens per split
  int rows, tiles;       // query rows of a unit, row tiles
  float* ws_acc;         // partial outputs and statistics (layouts: the kernels)
  float2* ws_ml;
  uint16_t* out;
  int64_t o_ls, o_bs, o_ts;
  float inv_sqrt_d;
};

// byte planes of a 16-entry f16 table: low and high bytes of entries 4 w .. 4 w + 3
struct Planes {
  uint32_t lo[4], hi[4];
};
__device__ __forceinline__ Planes make_planes(const CodecDev& c, float scale) {
  Planes pl;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    pl.lo[w] = pl.hi[w] = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t v = __half_as_ushort(__float2half_rn(c.centroids[4 * w + j] * scale));
      pl.lo[w] |= (v & 0xFFu) << (8 * j);
      pl.hi[w] |= (v >> 8) << (8 * j);
    }
  }
  return pl;
}
// eight nibble codes -> eight f16
__device__ __forceinline__ uint4 decode8(uint32_t w, const Planes& pl) {
  uint32_t o[4];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t sel = k ? w >> 16 : w;
    const uint32_t s7 = sel & 0x7777u, pick = 0x3210u + ((sel >> 3) & 0x1111u) * 4u;
    const uint32_t a = __byte_perm(__byte_perm(pl.lo[0], pl.lo[1], s7), __byte_perm(pl.lo[2], pl.lo[3], s7), pick);
    const uint32_t b = __byte_perm(__byte_perm(pl.hi[0], pl.hi[1], s7), __byte_perm(pl.hi[2], pl.hi[3], s7), pick);
    o[2 * k] = __byte_perm(a, b, 0x5140);
    o[2 * k + 1] = __byte_perm(a, b, 0x7362);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

constexpr float kTableScale = 32768.f;  // 2^15

__device__ __forceinline__ uint32_t pack2_f16(float a, float b) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack2_bf16(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

}  // namespace tq
