// Bounds of a record's keys: per coordinate the smallest and the largest of the
// 128 decoded keys, rounded outward to bf16.
//
// A CTA per record; a vector is spread over d / 32 lanes as in the decoder, whose
// f32 transform a single pass of butterflies replaces here (its split into a part
// on a grid and a rest serves a tolerance of 1e-5 that a bf16 result does not have).
#include "cache_params.h"
#include "tq_common.cuh"

namespace tq {

// f32 to the next bf16 below (DOWN) or above; NaN and infinities as they are
template <bool DOWN>
__device__ __forceinline__ uint32_t bf16_outward(float x) {
  const uint32_t u = __float_as_uint(x), cut = u >> 16;
  if (x != x) return 0x7FC0u;
  return cut + ((u & 0xFFFFu) != 0 && (u >> 31) == (DOWN ? 1u : 0u) ? 1u : 0u);
}
// minimum and maximum that keep a NaN
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

template <int D, int B, bool OUTL>
__global__ void __launch_bounds__(kThreads) key_bounds_kernel(const __grid_constant__ BoundsParams p) {
  constexpr int L = D / 32, VPW = 32 / L, VPC = 4 * VPW, RB = D * B / 8;
  __shared__ float lut[16];
  __shared__ int pre[kChunk];
  __shared__ float part[2][4][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, lg = lane % L, vi = lane / L;
  const int64_t unit = blockIdx.x / p.max_new;
  const int h = (int)(unit % p.Hkv), lb = (int)(unit / p.Hkv), b = lb % p.B, l = lb / p.B;
  const int n = min(max(p.n_chunks[lb], 0), min(p.max_chunks, p.rec_limit));
  const int64_t r = (int64_t)(p.first ? max(p.first[lb], 0) : 0) + blockIdx.x % p.max_new;
  if (r >= n) return;
  const uint8_t* rec = p.rec + l * p.rec_ls +
                       rec_offset(p.table, p.table_stride, p.rec_cap, p.Hkv, b, h, (int)r, p.c.rec_bytes);
  if (threadIdx.x < 16) lut[threadIdx.x] = p.c.centroids[threadIdx.x & ((1 << B) - 1)];
  if (OUTL && warp == 0) {  // where a slot's entries begin
    int run = 0;
    for (int k = 0; k < kChunk; k += 32) {
      const int v = rec[p.c.off_count + k + lane];
      int inc = v;
#pragma unroll
      for (int m = 1; m < 32; m <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, inc, m);
        if (lane >= m) inc += o;
      }
      pre[k + lane] = run + inc - v;
      run += __shfl_sync(0xffffffffu, inc, 31);
    }
  }
  __syncthreads();
  float lo[32], hi[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    lo[i] = INFINITY;
    hi[i] = -INFINITY;
  }
#pragma unroll 1
  for (int slot = warp * VPW + vi; slot < kChunk; slot += VPC) {
    const uint32_t* src = reinterpret_cast<const uint32_t*>(rec + slot * RB + lg * 4 * B);
    uint32_t w[B];
#pragma unroll
    for (int q = 0; q < B; ++q) w[q] = __ldg(src + q);
    float f = __ldg(reinterpret_cast<const float*>(rec + p.c.off_norm) + slot) * p.c.inv_sqrt_d;
    f = fmaf(f, 0.f, f);  // NaN where it is not finite
    float x[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const int bit = i * B;
      uint32_t code = w[bit >> 5] >> (bit & 31);
      if ((bit & 31) + B > 32) code |= w[(bit >> 5) + 1] << (32 - (bit & 31));
      x[i] = lut[code & ((1u << B) - 1u)];
    }
    if (OUTL) {
      const int e0 = pre[slot], e1 = min(e0 + rec[p.c.off_count + slot], p.c.cap);
      const uint32_t* ent = reinterpret_cast<const uint32_t*>(rec + p.c.off_entries);
      for (int e = e0; e < e1; ++e) {
        const uint32_t v = __ldg(ent + e);
        const int idx = (int)(v & (D - 1));
        if ((idx >> 5) == lg) {
          const float val = bf16_hi(v);
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] = i == (idx & 31) ? val : x[i];
        }
      }
      __syncwarp();
    }
    fwht_regs<32>(x);
    fwht_lanes<32>(x, lane, L);
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const float y = x[i] * f;
      lo[i] = min_nan(lo[i], y);
      hi[i] = max_nan(hi[i], y);
    }
  }
  // over the warp's vectors, then the four warps
#pragma unroll
  for (int m = L; m < 32; m <<= 1)
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      lo[i] = min_nan(lo[i], __shfl_xor_sync(0xffffffffu, lo[i], m));
      hi[i] = max_nan(hi[i], __shfl_xor_sync(0xffffffffu, hi[i], m));
    }
  if (vi == 0) {
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      part[0][warp][32 * lg + i] = lo[i];
      part[1][warp][32 * lg + i] = hi[i];
    }
  }
  __syncthreads();
  uint16_t* out = p.bounds + l * p.bounds_ls + rec_offset(p.table, p.table_stride, p.rec_cap, p.Hkv, b, h, (int)r, 2 * D);
  for (int j = threadIdx.x; j < D; j += kThreads) {
    float a = min_nan(min_nan(part[0][0][j], part[0][1][j]), min_nan(part[0][2][j], part[0][3][j]));
    float z = max_nan(max_nan(part[1][0][j], part[1][1][j]), max_nan(part[1][2][j], part[1][3][j]));
    if ((p.c.signs[j >> 5] >> (j & 31)) & 1u) {  // the coordinate's sign turns them around
      const float o = a;
      a = -z;
      z = -o;
    }
    out[j] = (uint16_t)bf16_outward<true>(a);
    out[D + j] = (uint16_t)bf16_outward<false>(z);
  }
}

template <int D, int B>
static cudaError_t bounds_launch(const BoundsParams& p, cudaStream_t s) {
  const unsigned grid = (unsigned)((int64_t)p.L * p.B * p.Hkv * p.max_new);
  if (p.c.has_outl) key_bounds_kernel<D, B, true><<<grid, kThreads, 0, s>>>(p);
  else key_bounds_kernel<D, B, false><<<grid, kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_key_bounds(const BoundsParams& p, cudaStream_t s) {
  switch (p.c.d * 10 + p.c.bits) {
#define TQ_CASE(D_) \
  case D_ * 10 + 1: return bounds_launch<D_, 1>(p, s); \
  case D_ * 10 + 2: return bounds_launch<D_, 2>(p, s); \
  case D_ * 10 + 3: return bounds_launch<D_, 3>(p, s); \
  case D_ * 10 + 4: return bounds_launch<D_, 4>(p, s);
    TQ_CASE(64) TQ_CASE(128) TQ_CASE(256) TQ_CASE(512)
#undef TQ_CASE
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace tq
