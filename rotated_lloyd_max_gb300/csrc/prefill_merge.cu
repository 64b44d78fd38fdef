// Merge of the context splits of the several-query attention: a warp per
// query row, weights from the splits' (m, l), one inverse transform for the
// records' part (as the decode merge does), one rounding to bf16.  Rows
// behind a sequence's last query token are left as they are.
#include "prefill.cuh"

namespace tq {

template <int D>
__global__ void __launch_bounds__(kThreads) prefill_merge_kernel(const __grid_constant__ PrefillParams pp) {
  constexpr int E = D / 32;
  const QueryParams& p = pp.q;
  const int lane = threadIdx.x & 31;
  const int64_t wrow = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int64_t units = (int64_t)p.L * p.B * p.Hkv;
  if (wrow >= units * pp.rows) return;
  const int64_t unit = wrow / pp.rows;
  const int row = (int)(wrow % pp.rows), tok = row / p.G;
  const int h = (int)(unit % p.Hkv), lb = (int)(unit / p.Hkv), b = lb % p.B, l = lb / p.B;
  if (tok >= query_len(p, b)) return;
  const int S = pp.Sc + pp.St;
  const float2* ml = pp.ws_ml + wrow * S;
  const float* acc = pp.ws_acc + wrow * S * D + lane * E;
  float M = -INFINITY;
  for (int s = lane; s < S; s += 32) M = fmaxf(M, ml[s].y > 0.f ? ml[s].x : -INFINITY);
  M = warp_max(M);
  float c[E], d[E], W = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) c[e] = d[e] = 0.f;
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
  const float iw = W > 0.f || W != W ? 1.f / W : 0.f;  // a row that sees no token is zero
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

// Merge of the tcgen05 kernel's partials, [tile][split][D / 4][128 rows][4]: a
// CTA per 128-row tile, four threads per row with D / 4 coordinates each (the
// transform's last two stages cross them), so that a warp reads eight rows'
// 16-byte pieces side by side.
template <int D>
__global__ void __launch_bounds__(512) prefill_merge_tiles_kernel(const __grid_constant__ PrefillParams pp) {
  constexpr int E = D / 4;
  const QueryParams& p = pp.q;
  const int tid = threadIdx.x, r = tid >> 2, qd = tid & 3;
  const int ntile = (pp.rows + 127) / 128, tile = blockIdx.x % ntile;
  const int64_t unit = blockIdx.x / ntile;
  const int row = tile * 128 + r, tok = row / p.G;
  const int h = (int)(unit % p.Hkv), lb = (int)(unit / p.Hkv), b = lb % p.B, l = lb / p.B;
  const int tb = query_len(p, b);
  if (tile * 128 >= tb * p.G) return;
  const bool live = row < pp.rows && tok < tb;
  const int S = pp.Sc + pp.St;
  const float2* ml = pp.ws_ml + (int64_t)blockIdx.x * S * 128 + r;
  const float4* acc = reinterpret_cast<const float4*>(pp.ws_acc) + ((int64_t)blockIdx.x * S * (D / 4) + qd * (E / 4)) * 128 + r;
  float M = -INFINITY, W = 0.f;
  if (live)
    for (int s = 0; s < S; ++s) {
      const float2 v = ml[s * 128];
      if (v.y > 0.f) M = fmaxf(M, v.x);
    }
  float c[E];
#pragma unroll
  for (int e = 0; e < E; ++e) c[e] = 0.f;
  auto add = [&](int s) {
    const float2 v = live ? ml[s * 128] : make_float2(0.f, 0.f);
    if (v.y != v.y) W = v.y;  // a split that gave up: the row comes out NaN
    if (!(v.y > 0.f)) return;
    const float w = exp2f(v.x - M);
    W = fmaf(w, v.y, W);
    const float4* a = acc + (int64_t)s * (D / 4) * 128;
#pragma unroll
    for (int k = 0; k < E / 4; ++k) {
      const float4 x = a[k * 128];
      c[4 * k] = fmaf(w, x.x, c[4 * k]);
      c[4 * k + 1] = fmaf(w, x.y, c[4 * k + 1]);
      c[4 * k + 2] = fmaf(w, x.z, c[4 * k + 2]);
      c[4 * k + 3] = fmaf(w, x.w, c[4 * k + 3]);
    }
  };
  if (pp.Sc > 0) {
    for (int s = 0; s < pp.Sc; ++s) add(s);
    __syncwarp();
    fwht_regs<E>(c);
    fwht_lanes<E>(c, tid & 31, 4);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int j = qd * E + e;
      c[e] *= ((p.vc.signs[j >> 5] >> (j & 31)) & 1u) ? -pp.inv_sqrt_d : pp.inv_sqrt_d;
    }
  }
  for (int s = pp.Sc; s < S; ++s) add(s);
  if (!live) return;
  const float iw = W > 0.f || W != W ? 1.f / W : 0.f;  // a row that sees no token is zero
  uint16_t* out = pp.out + l * pp.o_ls + b * pp.o_bs + (int64_t)tok * pp.o_ts + (int64_t)(h * p.G + row % p.G) * D + qd * E;
#pragma unroll
  for (int e = 0; e < E; e += 8)
    *reinterpret_cast<uint4*>(out + e) =
        make_uint4(pack2_bf16(c[e] * iw, c[e + 1] * iw), pack2_bf16(c[e + 2] * iw, c[e + 3] * iw),
                   pack2_bf16(c[e + 4] * iw, c[e + 5] * iw), pack2_bf16(c[e + 6] * iw, c[e + 7] * iw));
}

cudaError_t launch_prefill_merge(const PrefillParams& pp, cudaStream_t s) {
  const int64_t rows = (int64_t)pp.q.L * pp.q.B * pp.q.Hkv * pp.rows;
  const unsigned grid = (unsigned)((rows + 3) / 4);
  const unsigned tiles = (unsigned)((int64_t)pp.q.L * pp.q.B * pp.q.Hkv * ((pp.rows + 127) / 128));
  switch (pp.q.D) {
    case 64: prefill_merge_tiles_kernel<64><<<tiles, 512, 0, s>>>(pp); break;
    case 128: prefill_merge_tiles_kernel<128><<<tiles, 512, 0, s>>>(pp); break;
    case 256: prefill_merge_kernel<256><<<grid, kThreads, 0, s>>>(pp); break;
    case 512: prefill_merge_kernel<512><<<grid, kThreads, 0, s>>>(pp); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

}  // namespace tq
