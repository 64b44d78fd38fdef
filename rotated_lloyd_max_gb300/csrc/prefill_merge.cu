// Merge of the context splits of the several-query attention: a warp per
// query row, weights from the splits' (m, l), one inverse transform for the
// records' part (as the decode merge does), one rounding to bf16.  Rows
// behind a sequence's last query token are left as they are.
#include "prefill.cuh"

namespace tq {

// 1 / W; NaN where it is or where a row sees tokens of no finite logit, 0 where it sees no token
__device__ __forceinline__ float inverse_weight(const QueryParams& p, int lb, int tb, int row, float W) {
  if (W > 0.f || W != W) return 1.f / W;
  return row_limit(p, cache_len(p, lb), tb, row) > 0 ? __int_as_float(0x7fc00000) : 0.f;
}

template <int D>
__global__ void __launch_bounds__(kThreads) prefill_merge_kernel(const __grid_constant__ PrefillParams pp) {
  constexpr int E = D / 32;
  pdl_wait();
  const QueryParams& p = pp.q;
  const int lane = threadIdx.x & 31;
  const int64_t wrow = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int64_t units = (int64_t)p.L * p.B * p.Hkv;
  if (wrow >= units * pp.rows) return;
  const int64_t unit = wrow / pp.rows;
  const int row = (int)(wrow % pp.rows), tok = row / p.G;
  const int h = (int)(unit % p.Hkv), lb = (int)(unit / p.Hkv), b = lb % p.B, l = lb / p.B;
  const int tb = query_len(p, b);
  if (tok >= tb) return;
  const int S = pp.Sc + pp.St;
  const float2* ml = pp.ws_ml + wrow * S;
  const float* acc = pp.ws_acc + wrow * S * D + lane * E;
  float M = -INFINITY;
  for (int s = lane; s < S; s += 32) M = fmaxf(M, ml[s].y > 0.f ? ml[s].x : -INFINITY);
  M = warp_max(M);
  float c[E], d[E], W = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) c[e] = d[e] = 0.f;
#pragma unroll 2
  for (int s = 0; s < S; ++s) {
    const float2 v = ml[s];
    if (v.y != v.y) W = v.y;  // a split that gave up: the row comes out NaN
    if (!(v.y > 0.f)) continue;
    const float w = exp2f(v.x - M);
    W = fmaf(w, v.y, W);
    const float* a = acc + (int64_t)s * D;
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      const float2 x = *reinterpret_cast<const float2*>(a + e);
      if (s < pp.Sc) {
        c[e] = fmaf(w, x.x, c[e]);
        c[e + 1] = fmaf(w, x.y, c[e + 1]);
      } else {
        d[e] = fmaf(w, x.x, d[e]);
        d[e + 1] = fmaf(w, x.y, d[e + 1]);
      }
    }
  }
  if (pp.Sc > 0) {
    fwht_regs<E>(c);
    fwht_lanes<E>(c, lane, 32);
  }
  const float iw = inverse_weight(p, lb, tb, row, W);
  uint16_t* out = pp.out + l * pp.o_ls + b * pp.o_bs + (int64_t)tok * pp.o_ts + (int64_t)(h * p.G + row % p.G) * D +
                  lane * E;
#pragma unroll
  for (int e = 0; e < E; e += 2) {
    const int j = lane * E + e;
    const uint32_t sg = p.vc.signs[j >> 5] >> (j & 31);
    const float x = c[e] * ((sg & 1u) ? -pp.inv_sqrt_d : pp.inv_sqrt_d) + d[e];
    const float y = c[e + 1] * ((sg & 2u) ? -pp.inv_sqrt_d : pp.inv_sqrt_d) + d[e + 1];
    const __nv_bfloat162 w = __floats2bfloat162_rn(x * iw, y * iw);
    *reinterpret_cast<uint32_t*>(out + e) = *reinterpret_cast<const uint32_t*>(&w);
  }
}

// Merge of the narrow kernel's partials, [tile][split][D / 4][128 rows][4]: four
// threads per row with D / 4 coordinates each (the transform's last two stages
// cross them), so that a warp reads eight rows' 16-byte pieces side by side.
// A CTA takes 256 / (4 SL) rows; with SL > 1 the splits of a row are shared by SL
// groups of threads, whose sums meet in shared memory (a few rows with many
// splits would otherwise wait for one load after another: the call for 30 rows of
// 2 kv heads takes 33 us with SL = 1 and 23 with 8 over 18 splits, 25 and 21 over 7).
template <int D, int SL>
__global__ void __launch_bounds__(256) prefill_merge_tiles_kernel(const __grid_constant__ PrefillParams pp) {
  constexpr int E = D / 4, ROWS = 256 / (4 * SL);
  __shared__ float part[SL > 1 ? (SL - 1) * 4 * ROWS : 1][E + 1];
  __shared__ float wsum[SL > 1 ? SL * 4 * ROWS : 1];
  pdl_wait();
  const QueryParams& p = pp.q;
  const int tid = threadIdx.x, qd = tid & 3, sl = SL > 1 ? tid / (4 * ROWS) : 0, lr = (tid >> 2) % ROWS;
  const int ntile = (pp.rows + 127) / 128, per = 128 / ROWS;  // CTAs of a tile
  const int64_t blk = blockIdx.x / per;
  const int r = (int)(blockIdx.x % per) * ROWS + lr;
  const int tile = (int)(blk % ntile);
  const int64_t unit = blk / ntile;
  const int row = tile * 128 + r, tok = row / p.G;
  const int h = (int)(unit % p.Hkv), lb = (int)(unit / p.Hkv), b = lb % p.B, l = lb / p.B;
  const int tb = query_len(p, b);
  if (tile * 128 + (int)(blockIdx.x % per) * ROWS >= tb * p.G) return;
  const bool live = row < tb * p.G;
  const int S = pp.Sc + pp.St;
  const float2* ml = pp.ws_ml + blk * S * 128 + r;
  const float4* acc = reinterpret_cast<const float4*>(pp.ws_acc) + (blk * S * (D / 4) + qd * (E / 4)) * 128 + r;
  float M = -INFINITY, W = 0.f;
  if (live) {
#pragma unroll 4
    for (int s = 0; s < S; ++s) {
      const float2 v = ml[s * 128];
      M = fmaxf(M, v.y > 0.f ? v.x : -INFINITY);
    }
  }
  // the records' splits, then (in a second round) the ring's: sum of w x over this thread's share
  float c[E];
  auto round = [&](int s0, int s1) {
#pragma unroll 2
    for (int s = s0 + sl; s < s1; s += SL) {
      const float2 v = live ? ml[s * 128] : make_float2(0.f, 0.f);
      if (v.y != v.y) W = v.y;  // a split that gave up: the row comes out NaN
      const bool on = v.y > 0.f;
      const float w = on ? exp2f(v.x - M) : 0.f;
      W = on ? fmaf(w, v.y, W) : W;
      const float4* a = acc + (int64_t)s * (D / 4) * 128;
#pragma unroll
      for (int k = 0; k < E / 4; ++k) {
        const float4 x = on ? a[k * 128] : make_float4(0.f, 0.f, 0.f, 0.f);  // an empty split wrote nothing
        c[4 * k] = fmaf(w, x.x, c[4 * k]);
        c[4 * k + 1] = fmaf(w, x.y, c[4 * k + 1]);
        c[4 * k + 2] = fmaf(w, x.z, c[4 * k + 2]);
        c[4 * k + 3] = fmaf(w, x.w, c[4 * k + 3]);
      }
    }
  };
  auto join = [&] {  // group 0 gathers the other groups' sums
    if constexpr (SL > 1) {
      const int at = 4 * lr + qd;
      __syncthreads();
      if (sl > 0) {
#pragma unroll
        for (int e = 0; e < E; ++e) part[(sl - 1) * 4 * ROWS + at][e] = c[e];
      }
      __syncthreads();
      if (sl == 0) {
        for (int g = 0; g < SL - 1; ++g)
#pragma unroll
          for (int e = 0; e < E; ++e) c[e] += part[g * 4 * ROWS + at][e];
      }
    }
  };
#pragma unroll
  for (int e = 0; e < E; ++e) c[e] = 0.f;
  if (pp.Sc > 0) {
    round(0, pp.Sc);
    join();
    __syncwarp();
    fwht_regs<E>(c);
    fwht_lanes<E>(c, tid & 31, 4);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int j = qd * E + e;
      c[e] *= ((p.vc.signs[j >> 5] >> (j & 31)) & 1u) ? -pp.inv_sqrt_d : pp.inv_sqrt_d;
      if (sl > 0) c[e] = 0.f;
    }
  }
  round(pp.Sc, S);
  join();
  if constexpr (SL > 1) {
    wsum[tid] = W;
    __syncthreads();
    if (sl > 0) return;
    for (int g = 1; g < SL; ++g) W += wsum[g * 4 * ROWS + 4 * lr + qd];
  }
  if (!live) return;
  const float iw = inverse_weight(p, lb, tb, row, W);
  uint16_t* out = pp.out + l * pp.o_ls + b * pp.o_bs + (int64_t)tok * pp.o_ts + (int64_t)(h * p.G + row % p.G) * D + qd * E;
#pragma unroll
  for (int e = 0; e < E; e += 8)
    *reinterpret_cast<uint4*>(out + e) =
        make_uint4(pack2_bf16(c[e] * iw, c[e + 1] * iw), pack2_bf16(c[e + 2] * iw, c[e + 3] * iw),
                   pack2_bf16(c[e + 4] * iw, c[e + 5] * iw), pack2_bf16(c[e + 6] * iw, c[e + 7] * iw));
}

template <int D>
static cudaError_t merge_tiles_launch(const PrefillParams& pp, int64_t tiles, cudaStream_t s) {
  if (pp.Sc + pp.St > 6) return launch_after(prefill_merge_tiles_kernel<D, 8>, dim3((unsigned)(tiles * 16)), 256, 0, s, 1, pp);
  return launch_after(prefill_merge_tiles_kernel<D, 1>, dim3((unsigned)(tiles * 2)), 256, 0, s, 1, pp);
}

cudaError_t launch_prefill_merge(const PrefillParams& pp, cudaStream_t s) {
  const int64_t rows = (int64_t)pp.q.L * pp.q.B * pp.q.Hkv * pp.rows;
  const unsigned grid = (unsigned)((rows + 3) / 4);
  const int64_t tiles = (int64_t)pp.q.L * pp.q.B * pp.q.Hkv * ((pp.rows + 127) / 128);
  switch (pp.q.D) {
    case 64: return merge_tiles_launch<64>(pp, tiles, s);
    case 128: return merge_tiles_launch<128>(pp, tiles, s);
    case 256: return launch_after(prefill_merge_kernel<256>, dim3(grid), kThreads, 0, s, 1, pp);
    case 512: return launch_after(prefill_merge_kernel<512>, dim3(grid), kThreads, 0, s, 1, pp);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace tq
