// Second pass of the accumulated weights for few query rows: weights from the
// kept logits, a thread per token (kernel of the first pass: attn_mass_few.cuh).
#include "attn_mass_few.cuh"

namespace tq {

constexpr int kAddThreads = 256, kAddTokens = 4;  // tokens per thread

// P logits a token (the rows padded to a power of two)
template <int P>
__global__ void __launch_bounds__(kAddThreads) attn_mass_add_kernel(const __grid_constant__ MassParams mp) {
  __shared__ float lse[8];
  pdl_wait();
  const QueryParams& p = mp.q;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.y % p.Hkv, b = blockIdx.y / p.Hkv, l = blockIdx.z;
  const int lb = l * p.B + b;
  const int64_t unit = (int64_t)lb * p.Hkv + h;
  const CacheLen cl = cache_len(p, lb);
  const int S = mp.Sc + mp.St;
  const int first = blockIdx.x * kAddThreads * kAddTokens;
  if (first >= cl.total) return;
  const float* lg = mp.logits + unit * few_columns(mp) * P;
  float* m = mp.mass + l * mp.mass_ls + ((int64_t)b * p.Hkv + h) * mp.mass_cap;
  float x[kAddTokens][P], old[kAddTokens];
#pragma unroll
  for (int k = 0; k < kAddTokens; ++k) {
    const int i = first + k * kAddThreads + tid;
    // the ring's logits lie behind max_chunks records
    const int64_t col = i < cl.n * kChunk ? i : (int64_t)p.max_chunks * kChunk + (i - cl.n * kChunk);
    if (i < cl.total) {
      if constexpr (P >= 4) {
#pragma unroll
        for (int q = 0; q < P; q += 4) *reinterpret_cast<float4*>(&x[k][q]) = __ldcs(reinterpret_cast<const float4*>(lg + col * P + q));
      } else if constexpr (P == 2) {
        *reinterpret_cast<float2*>(&x[k][0]) = __ldcs(reinterpret_cast<const float2*>(lg + col * P));
      } else {
        x[k][0] = __ldcs(lg + col);
      }
      old[k] = m[i];
    }
  }
  if (warp < mp.rows) {  // a warp per row: its log-sum over the splits (rows <= 8 warps)
    const float2* ml = mp.ml + unit * S * 8 + warp;
    float M = -INFINITY, W = 0.f;
    for (int s = lane; s < S; s += 32) M = fmaxf(M, ml[s * 8].x);
    M = warp_max(M);
    for (int s = lane; s < S; s += 32) {
      const float2 v = ml[s * 8];
      if (v.y > 0.f) W += v.y * exp2f(v.x - M);
      else if (v.y != v.y) W = v.y;
    }
    W = warp_sum(W);
    if (lane == 0) lse[warp] = log_sum(M, W, row_limit(p, cl, query_len(p, b), warp));
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kAddTokens; ++k) {
    const int i = first + k * kAddThreads + tid;
    if (i >= cl.total) continue;
    float s = 0.f;
#pragma unroll
    for (int q = 0; q < P; ++q)
      if (q < mp.rows && lse[q] != INFINITY) s += ex2(x[k][q] - lse[q]);
    m[i] = fmaf(mp.decay, old[k], s);
  }
}

cudaError_t launch_attn_mass_add(const MassParams& mp, cudaStream_t s) {
  const int most = mp.q.max_chunks * kChunk + mp.q.max_tail;
  const dim3 grid((most + kAddThreads * kAddTokens - 1) / (kAddThreads * kAddTokens), mp.q.B * mp.q.Hkv, mp.q.L);
  switch (mp.pitch) {
    case 1: return launch_after(attn_mass_add_kernel<1>, grid, kAddThreads, 0, s, 1, mp);
    case 2: return launch_after(attn_mass_add_kernel<2>, grid, kAddThreads, 0, s, 1, mp);
    case 4: return launch_after(attn_mass_add_kernel<4>, grid, kAddThreads, 0, s, 1, mp);
    case 8: return launch_after(attn_mass_add_kernel<8>, grid, kAddThreads, 0, s, 1, mp);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace tq
