// Attention of several query tokens per sequence over records and ring
// (mma.sync; every head dim, any group size, side lists, soft cap).
//
// The query rows of a kv head are its query heads x new tokens, row = token *
// G + head, so that a tile of rows shares the keys it reads whatever the
// group size.  A CTA keeps one tile of rows and walks a run of 64-token tiles
// (a split of the context): packed codes become f16 keys and values in shared
// memory (centroids x 2^15, so that outlier values up to 1 fit and no centroid
// is subnormal), scores and weighted values are m16n8k16 MMAs with f32
// accumulation, the softmax runs in registers with an exact running maximum.
//   score    t_ij = (2^15 2^s_i q~_i . c_j) * n_j * scale / 2^(15 + s_i),
//   weight   p_ij = 2^(t_ij - m_i), sum l_i in f32;
//   values   O_i += (p_ij n_j 2^kx) c_j with the V scale n_j folded into the
//            weight before it is rounded to f16, kx the exponent that keeps
//            the largest below 2^11 (it falls when a larger scale comes).
// Rounding to f16 (11 bits) of q~, c and p n is finer than the bf16 output's 8.
// O stays in the rotated basis; the merge of the splits turns it back once.
// The ring's tokens are splits of their own with bf16 operands.
#pragma once

#include "attn_mass.cuh"

namespace tq {

struct PrefillParams {
  QueryParams q;
  int Sc, St, cps, tps;  // splits over records / ring tokens; records, ring tokens per split
  int rows, tiles;       // query rows of a unit, row tiles
  float* ws_acc;         // [units * rows][Sc + St][D]
  float2* ws_ml;         // [units * rows][Sc + St]
  uint16_t* out;
  int64_t o_ls, o_bs, o_ts;
  float inv_sqrt_d;
};

// Tile shapes: BM rows (16 per row warp), CW warps side by side over the output columns
template <int D>
struct PCfg {
  static constexpr int BN = 64;
  static constexpr int CW = D == 512 ? 2 : 1;
  static constexpr int WARPS = 8;
  static constexpr int BM = 16 * WARPS / CW;
  static constexpr int P = D + 8;           // row pitch: 16 bytes of padding, no ldmatrix conflicts
  static constexpr int OC = D / CW;         // output columns of a warp
  static constexpr int SMEM = (BM + 2 * BN) * P * 2;
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a));
}
__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

// codes 8 u .. 8 u + 7 of a packed row, one per nibble
__device__ __forceinline__ uint32_t nibbles(const uint8_t* row, int u, int bits) {
  if (bits == 4) return __ldg(reinterpret_cast<const uint32_t*>(row) + u);
  if (bits == 2) {
    uint32_t x = __ldg(reinterpret_cast<const uint16_t*>(row) + u);
    x = (x | (x << 8)) & 0x00FF00FFu;
    x = (x | (x << 4)) & 0x0F0F0F0Fu;
    return (x | (x << 2)) & 0x33333333u;
  }
  if (bits == 1) {
    uint32_t x = __ldg(row + u);
    x = (x | (x << 12)) & 0x000F000Fu;
    x = (x | (x << 6)) & 0x03030303u;
    return (x | (x << 3)) & 0x11111111u;
  }
  // 3 bytes at 3 u: the two words around them (the second may lie past the row, inside the record)
  const uint32_t* w = reinterpret_cast<const uint32_t*>(row) + ((3 * u) >> 2);
  return spread3(__funnelshift_r(__ldg(w), __ldg(w + 1), 8 * ((3 * u) & 3)));
}

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

template <int D, bool DENSE>
__global__ void __launch_bounds__(256) prefill_kernel(const __grid_constant__ PrefillParams pp) {
  using C = PCfg<D>;
  constexpr int BM = C::BM, BN = C::BN, P = C::P, CW = C::CW, OC = C::OC;
  constexpr int E = D / 32;
  const QueryParams& p = pp.q;
  extern __shared__ __align__(128) unsigned char sm[];
  uint16_t* qs = reinterpret_cast<uint16_t*>(sm);
  uint16_t* ks = qs + BM * P;
  uint16_t* vs = ks + BN * P;
  __shared__ float s_nk[BN], s_nv[BN], s_qsc[BM];
  __shared__ int s_lim[BM], s_pre[kChunk];

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int h = blockIdx.y % p.Hkv, b = blockIdx.y / p.Hkv, l = blockIdx.z;
  const int S = pp.Sc + pp.St, nsp = DENSE ? pp.St : pp.Sc;
  const int tile = blockIdx.x / nsp, split = blockIdx.x % nsp;
  const int lb = l * p.B + b;
  const int64_t unit = (int64_t)lb * p.Hkv + h;
  const CacheLen cl = cache_len(p, lb);
  const int tb = query_len(p, b);
  const int r0 = tile * BM, rn = min(BM, tb * p.G - r0);  // the tile's rows that are queries
  if (rn <= 0) return;
  // tokens [k0, k1) of the records or of the ring; nothing past the last row's limit
  const int base = DENSE ? cl.n * kChunk : 0;
  const int top = row_limit(p, cl, tb, r0 + rn - 1) - base;
  const int per = DENSE ? pp.tps : pp.cps * kChunk;
  const int k0 = split * per, k1 = min(min(k0 + per, DENSE ? cl.len : cl.n * kChunk), top);
  const int sidx = DENSE ? pp.Sc + split : split;
  const int64_t wrow = unit * pp.rows + r0;
  if (k0 >= k1) {
    for (int r = tid; r < rn; r += 256) pp.ws_ml[(wrow + r) * S + sidx] = make_float2(-INFINITY, 0.f);
    return;
  }
  // ---------------------------------------------------------------- queries
  for (int r = warp; r < BM; r += 8) {
    float x[E];
    const int row = r0 + r;
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = 0.f;
    if (r < rn) {
      const uint16_t* qp = p.q + l * p.q_ls + b * p.q_bs + (int64_t)(row / p.G) * p.q_ts +
                           (int64_t)(h * p.G + row % p.G) * D + lane * E;
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(qp + e);
        x[e] = bf16_lo(w);
        x[e + 1] = bf16_hi(w);
      }
    }
    float f = p.sscale;
    uint16_t* dst = qs + r * P + lane * E;
    if constexpr (!DENSE) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int j = lane * E + e;
        if ((p.kc.signs[j >> 5] >> (j & 31)) & 1u) x[e] = -x[e];
      }
      fwht_regs<E>(x);
      fwht_lanes<E>(x, lane, 32);
      float mx = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        x[e] *= inv_sqrt_dim<D>();
        mx = fmaxf(mx, fabsf(x[e]));
      }
      mx = warp_max(mx);
      const int s = mx > 0.f ? 13 - exp_of(mx) : 0;
      const float sc = pow2i(s);
      f = p.sscale * pow2i(-15 - s);
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const __half2 v = __floats2half2_rn(x[e] * sc, x[e + 1] * sc);
        *reinterpret_cast<uint32_t*>(dst + e) = *reinterpret_cast<const uint32_t*>(&v);
      }
    } else {
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(x[e], x[e + 1]);
        *reinterpret_cast<uint32_t*>(dst + e) = *reinterpret_cast<const uint32_t*>(&v);
      }
    }
    if (lane == 0) {
      s_qsc[r] = f;
      s_lim[r] = r < rn ? row_limit(p, cl, tb, row) - base : 0;
    }
  }
  Planes kpl, vpl;
  if constexpr (!DENSE) {
    kpl = make_planes(p.kc, kTableScale);
    vpl = make_planes(p.vc, kTableScale);
  }
  const int rw = warp / CW, cw = warp % CW;  // row warp, column warp
  const bool busy = 16 * rw < rn;
  const bool one = DENSE ? p.ktail == p.vtail : p.shared_kv != 0;  // keys are the values
  const uint16_t* vt = one ? ks : vs;
  __syncthreads();
  const float f0 = s_qsc[16 * rw + g], f1 = s_qsc[16 * rw + g + 8];
  const int lim0 = s_lim[16 * rw + g], lim1 = s_lim[16 * rw + g + 8];
  const int cap = p.tail_cap;
  const int rstart = DENSE && p.tail_start ? ((p.tail_start[lb] % cap) + cap) % cap : 0;
  const int64_t ring = l * p.tail_ls + (int64_t)(b * p.Hkv + h) * cap * D;

  float o[OC / 8][4];
#pragma unroll
  for (int n = 0; n < OC / 8; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
  int kx = DENSE ? 0 : 127;  // exponent of the weights' V scale

#pragma unroll 1
  for (int k = k0; k < k1; k += BN) {
    // -------------------------------------------------------------- keys and values of 64 tokens
    if constexpr (DENSE) {
      for (int i = tid; i < BN * (D / 8); i += 256) {
        const int tok = i / (D / 8), c = i % (D / 8);
        const int at = min(k + tok, cl.len - 1);
        const int64_t src = ring + (int64_t)((rstart + (int64_t)at) % cap) * D + 8 * c;
        *reinterpret_cast<uint4*>(ks + tok * P + 8 * c) = *reinterpret_cast<const uint4*>(p.ktail + src);
        if (!one) *reinterpret_cast<uint4*>(vs + tok * P + 8 * c) = *reinterpret_cast<const uint4*>(p.vtail + src);
      }
    } else {
      const int c = k / kChunk, s0 = k % kChunk;
      for (int kv = 0; kv < (one ? 1 : 2); ++kv) {
        const CodecDev& cd = kv ? p.vc : p.kc;
        const uint8_t* rec = (kv ? p.vrec + l * p.vrec_ls : p.krec + l * p.krec_ls) +
                             rec_offset(p.table, p.table_stride, p.rec_cap, p.Hkv, b, h, c, cd.rec_bytes);
        const int bits = cd.bits, rb = D * bits / 8;
        uint16_t* dst = kv ? vs : ks;
        for (int i = tid; i < BN * (D / 8); i += 256) {
          const int tok = i / (D / 8), u = i % (D / 8);
          *reinterpret_cast<uint4*>(dst + tok * P + 8 * u) = decode8(nibbles(rec + (s0 + tok) * rb, u, bits), kv ? vpl : kpl);
        }
        if (tid < BN) {
          const float n = __ldg(reinterpret_cast<const float*>(rec + cd.off_norm) + s0 + tid);
          (kv ? s_nv : s_nk)[tid] = n;
          if (one) s_nv[tid] = n;
        }
        if (cd.has_outl) {
          __syncthreads();
          if (warp < 4) s_pre[32 * warp + lane] = slot_entries(rec + cd.off_count, warp, lane);
          __syncthreads();
          const uint32_t* ent = reinterpret_cast<const uint32_t*>(rec + cd.off_entries);
          for (int tok = warp; tok < BN; tok += 8) {
            const int e = s_pre[s0 + tok], from = e >> 8, cnt = min(e & 255, max(cd.cap - from, 0));
            for (int i = lane; i < cnt; i += 32) {
              const uint32_t en = __ldg(ent + from + i);
              dst[tok * P + (en & (D - 1))] = __half_as_ushort(__float2half_rn(bf16_hi(en) * kTableScale));
            }
          }
          __syncthreads();
        }
      }
    }
    __syncthreads();
    if (busy) {
      // ------------------------------------------------------------ scores
      float s[BN / 8][4];
#pragma unroll
      for (int n = 0; n < BN / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
      const uint32_t qa = smem_addr(qs + (16 * rw + (lane & 15)) * P + 8 * (lane >> 4));
      const uint32_t ka = smem_addr(ks + ((lane & 7) + 8 * (lane >> 4)) * P + 8 * ((lane >> 3) & 1));
#pragma unroll 4
      for (int kk = 0; kk < D / 16; ++kk) {
        uint32_t a[4];
        ldsm4(a, qa + 32 * kk);
#pragma unroll
        for (int n = 0; n < BN / 16; ++n) {
          uint32_t bk[4];
          ldsm4(bk, ka + 2 * (16 * n * P + 16 * kk));
          if constexpr (DENSE) {
            mma_bf16(s[2 * n], a, bk[0], bk[1]);
            mma_bf16(s[2 * n + 1], a, bk[2], bk[3]);
          } else {
            mma_f16(s[2 * n], a, bk[0], bk[1]);
            mma_f16(s[2 * n + 1], a, bk[2], bk[3]);
          }
        }
      }
      // ------------------------------------------------------------ softmax
      float x0 = m0, x1 = m1;
#pragma unroll
      for (int n = 0; n < BN / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int tok = 8 * n + 2 * t + (e & 1);
          const float f = (e < 2 ? f0 : f1) * (DENSE ? 1.f : s_nk[tok]);
          s[n][e] = mass_logit(p, s[n][e], f, k + tok < min(e < 2 ? lim0 : lim1, k1));
          if (e < 2) x0 = fmaxf(x0, s[n][e]);
          else x1 = fmaxf(x1, s[n][e]);
        }
#pragma unroll
      for (int x = 1; x < 4; x <<= 1) {
        x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, x));
        x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, x));
      }
      int kn = kx;
      if constexpr (!DENSE) {
        const float nm = warp_max(fmaxf(s_nv[lane], s_nv[lane + 32]));
        if (nm > 0.f) kn = min(kx, 10 - exp_of(nm));
      }
      const float gam = DENSE ? 1.f : pow2i(kn - kx);
      const float z0 = x0 == -INFINITY ? 0.f : x0, z1 = x1 == -INFINITY ? 0.f : x1;  // all masked so far
      const float a0 = ex2(m0 - z0), a1 = ex2(m1 - z1);
      m0 = x0;
      m1 = x1;
      l0 *= a0;
      l1 *= a1;
      kx = kn;
      const float vsc = DENSE ? 1.f : pow2i(kx);
      uint32_t pa[BN / 16][4];
#pragma unroll
      for (int n = 0; n < BN / 8; ++n) {
        const float w0 = ex2(s[n][0] - z0), w1 = ex2(s[n][1] - z0), w2 = ex2(s[n][2] - z1), w3 = ex2(s[n][3] - z1);
        l0 += w0 + w1;
        l1 += w2 + w3;
        if constexpr (DENSE) {
          const __nv_bfloat162 u = __floats2bfloat162_rn(w0, w1), v = __floats2bfloat162_rn(w2, w3);
          pa[n >> 1][2 * (n & 1)] = *reinterpret_cast<const uint32_t*>(&u);
          pa[n >> 1][2 * (n & 1) + 1] = *reinterpret_cast<const uint32_t*>(&v);
        } else {
          const float n0 = s_nv[8 * n + 2 * t] * vsc, n1 = s_nv[8 * n + 2 * t + 1] * vsc;
          const __half2 u = __floats2half2_rn(w0 * n0, w1 * n1), v = __floats2half2_rn(w2 * n0, w3 * n1);
          pa[n >> 1][2 * (n & 1)] = *reinterpret_cast<const uint32_t*>(&u);
          pa[n >> 1][2 * (n & 1) + 1] = *reinterpret_cast<const uint32_t*>(&v);
        }
      }
#pragma unroll
      for (int n = 0; n < OC / 8; ++n) {
        o[n][0] *= a0 * gam;
        o[n][1] *= a0 * gam;
        o[n][2] *= a1 * gam;
        o[n][3] *= a1 * gam;
      }
      // ------------------------------------------------------------ values
      const uint32_t va = smem_addr(vt + (lane & 15) * P + cw * OC + 8 * (lane >> 4));
#pragma unroll
      for (int kk = 0; kk < BN / 16; ++kk)
#pragma unroll
        for (int n = 0; n < OC / 16; ++n) {
          uint32_t bv[4];
          ldsm4t(bv, va + 2 * (16 * kk * P + 16 * n));
          if constexpr (DENSE) {
            mma_bf16(o[2 * n], pa[kk], bv[0], bv[1]);
            mma_bf16(o[2 * n + 1], pa[kk], bv[2], bv[3]);
          } else {
            mma_f16(o[2 * n], pa[kk], bv[0], bv[1]);
            mma_f16(o[2 * n + 1], pa[kk], bv[2], bv[3]);
          }
        }
    }
    __syncthreads();
  }
  if (!busy) return;
#pragma unroll
  for (int x = 1; x < 4; x <<= 1) {
    l0 += __shfl_xor_sync(0xffffffffu, l0, x);
    l1 += __shfl_xor_sync(0xffffffffu, l1, x);
  }
  const float un = DENSE ? 1.f : pow2i(-15) * pow2i(-kx);
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int r = 16 * rw + g + 8 * half;
    if (r >= rn) continue;
    float* dst = pp.ws_acc + ((wrow + r) * S + sidx) * D + cw * OC + 2 * t;
#pragma unroll
    for (int n = 0; n < OC / 8; ++n)
      *reinterpret_cast<float2*>(dst + 8 * n) = f2(o[n][2 * half] * un, o[n][2 * half + 1] * un);
    if (t == 0 && cw == 0) pp.ws_ml[(wrow + r) * S + sidx] = half ? make_float2(m1, l1) : make_float2(m0, l0);
  }
}

template <int D>
cudaError_t prefill_launch_d(const PrefillParams& pp, cudaStream_t s) {
  using C = PCfg<D>;
  const dim3 grid(pp.tiles, pp.q.B * pp.q.Hkv, pp.q.L);
  cudaError_t e = cudaFuncSetAttribute(prefill_kernel<D, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(prefill_kernel<D, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  if (pp.Sc > 0) prefill_kernel<D, false><<<dim3(grid.x * pp.Sc, grid.y, grid.z), 256, C::SMEM, s>>>(pp);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if (pp.St > 0) prefill_kernel<D, true><<<dim3(grid.x * pp.St, grid.y, grid.z), 256, C::SMEM, s>>>(pp);
  return cudaGetLastError();
}

}  // namespace tq
