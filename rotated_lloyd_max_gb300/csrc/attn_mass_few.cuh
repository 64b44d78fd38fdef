// Accumulated attention weight for at most eight query rows per kv head (a
// decode step): one pass over the keys that keeps the logits, then one over
// the logits.
//
// First pass (attn_mass_few_kernel): the arithmetic of attn_mass_kernel with
// the rows as a single n-tile of 8; the logits of a token (4 bytes a row, 16
// to 32 bytes against 68 of a 4-bit key record at head dim 128) go to the
// workspace, the rows' (max, sum) per split beside them.  Bound by the table
// lookups (8 bytes of shared memory a pair of codes) and the packed keys'
// bytes; the words of the next 32 codes are loaded while this run's are
// multiplied.  At most four rows share one MMA between their hi and lo parts
// (columns r and r + 4), two MMAs a k-step instead of three.
// Five CTAs per SM (a few spilled words; 32 sequences of 32768 tokens, 8 kv heads
// of 4 query heads: both passes 289 us; at an earlier stage 294, four CTAs 305, six 312).
// Second pass (attn_mass_add_kernel): a thread per token turns its logits into
// weights with the rows' log-sums and adds them to the mass.
#pragma once

#include "attn_mass.cuh"

namespace tq {

struct FewMisc {
  float qsc[8];
  int lim[8];
  float2 part[4][8];
  uint2 cent[16];
};

// where the logits of a unit's tokens lie: records first, the ring behind max_chunks records
__device__ __forceinline__ int64_t few_columns(const MassParams& mp) {
  return (int64_t)mp.q.max_chunks * kChunk + (int64_t)mp.St * mp.tps;
}

template <int D, int KB, bool OUTL>
__global__ void __launch_bounds__(kThreads, 5) attn_mass_few_kernel(const __grid_constant__ MassParams mp) {
  constexpr int KS = D / 16, RUN = D / 4;
  constexpr int STEP = RUN < 32 ? RUN : 32, NS = RUN / STEP;  // codes of a run taken at a time, such pieces
  constexpr int NB = STEP * KB, NW = (NB + 31) / 32;
  constexpr bool AL = NB % 32 == 0;
  const QueryParams& p = mp.q;
  pdl_start();
  extern __shared__ __align__(128) unsigned char sm[];
  uint4* qfrag = reinterpret_cast<uint4*>(sm + mp.sm_frag);
  uint2* qfragd = reinterpret_cast<uint2*>(sm + mp.sm_frag);
  FewMisc& ms = *reinterpret_cast<FewMisc*>(sm + mp.sm_misc);
  float* qrot = reinterpret_cast<float*>(sm + mp.sm_qrot);  // side lists: rotated queries [D][8]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int S = mp.Sc + mp.St;
  const int h = blockIdx.y % p.Hkv, b = blockIdx.y / p.Hkv, l = blockIdx.z, split = blockIdx.x;
  const int lb = l * p.B + b;
  const int64_t unit = (int64_t)lb * p.Hkv + h;
  const bool dense = split >= mp.Sc;
  const CacheLen cl = cache_len(p, lb);
  const int tb = query_len(p, b);
  const int per = dense ? mp.tps / kChunk : mp.cps;
  const int c0 = (dense ? split - mp.Sc : split) * per;
  const int c1 = min(c0 + per, dense ? (cl.len + kChunk - 1) / kChunk : cl.n);
  float2* ml = mp.ml + (unit * S + split) * 8;
  if (c0 >= c1 || tb == 0) {  // no token here, or no query (no logit of theirs is read then)
    if (tid < 8) ml[tid] = make_float2(-INFINITY, 0.f);
    return;
  }
  const bool packed = mp.rows <= 4 && !dense;
  const int base = dense ? cl.n * kChunk : 0;
  const int row_bytes = D * KB / 8;
  const uint8_t* kl = p.krec + l * p.krec_ls;
  const int cap = p.tail_cap;
  const uint16_t* ring = p.ktail + l * p.tail_ls + (int64_t)(b * p.Hkv + h) * cap * D;
  const int rstart = dense && p.tail_start ? ((p.tail_start[lb] % cap) + cap) % cap : 0;
  const uint32_t loff = (lane & 15) * 8;
  const ByteTable tab = byte_table(sm, loff, 128);
  // the lane's token rows of a record, and the words of one run piece
  const int off0 = (32 * warp + g) * row_bytes;
  auto rec_at = [&](int c) {
    return kl + rec_offset(p.table, p.table_stride, p.rec_cap, p.Hkv, b, h, c, p.kc.rec_bytes);
  };
  uint32_t w[4][NW], wn[4][NW];
  float nk[4], nkn[4];
  auto load_words = [&](const uint8_t* rec, int s, uint32_t (&x)[4][NW]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) load_run<NB, AL>(rec + off0 + 8 * i * row_bytes, (t * RUN + s * STEP) * KB, x[i]);
  };
  auto load_norms = [&](const uint8_t* rec, float (&x)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = __ldg(reinterpret_cast<const float*>(rec + p.kc.off_norm) + 32 * warp + 8 * i + g);
  };
  const uint8_t* rec = nullptr;
  if (!dense) {
    rec = rec_at(c0);
    load_words(rec, 0, w);
    load_norms(rec, nk);
    if (tid < 16) {
      const float v = p.kc.centroids[tid] * 65536.f;
      const __half hi = __float2half_rn(v);
      ms.cent[tid] = make_uint2(__half_as_ushort(hi), __half_as_ushort(__float2half_rn(v - __half2float(hi))));
    }
  }
  // ---------------------------------------------------------------- query fragments: a warp for two rows
  if (packed)
    for (int i = tid; i < KS * 32; i += kThreads) qfrag[i] = make_uint4(0, 0, 0, 0);
  __syncthreads();
  for (int r = warp; r < 8; r += 4) {
    const bool live = r < mp.rows && r / p.G < tb;
    if (packed && r >= 4) break;
    constexpr int E = D / 32;
    float x[E];
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = 0.f;
    if (live) {
      const uint16_t* qp = p.q + l * p.q_ls + b * p.q_bs + (int64_t)(r / p.G) * p.q_ts + (int64_t)(h * p.G + r % p.G) * D +
                           lane * E;
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const uint32_t v = *reinterpret_cast<const uint32_t*>(qp + e);
        x[e] = bf16_lo(v);
        x[e + 1] = bf16_hi(v);
      }
    }
    float sc = 1.f, f = p.sscale;
    if (!dense) {
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
      sc = pow2i(s);
      f *= pow2i(-16 - s);
      if constexpr (OUTL) {
#pragma unroll
        for (int e = 0; e < E; ++e) qrot[(lane * E + e) * 8 + r] = x[e];
      }
    }
    if (lane == 0) {
      ms.qsc[r] = f;
      ms.lim[r] = live ? row_limit(p, cl, tb, r) : 0;
    }
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      const int j = lane * E + e, tt = j / RUN, kk = (j % RUN) / 4, half = (j % 4) / 2;
      const int at = kk * 32 + r * 4 + tt;
      if (dense) {
        reinterpret_cast<uint32_t*>(qfragd + at)[half] = pack_bf16x2(x[e], x[e + 1]);
      } else {
        uint32_t hi, lo;
        split_f16x2(x[e] * sc, x[e + 1] * sc, hi, lo);
        reinterpret_cast<uint32_t*>(qfrag + at)[half] = hi;
        reinterpret_cast<uint32_t*>(qfrag + at + (packed ? 16 : 0))[packed ? half : 2 + half] = lo;
      }
    }
  }
  if (packed && tid >= 4 && tid < 8) {
    ms.qsc[tid] = 0.f;
    ms.lim[tid] = 0;
  }
  if (!dense)  // pair table, as in attn_mass_kernel
    for (int i = tid; i < (1 << (2 * KB)) * 16; i += kThreads) {
      const uint2 a = ms.cent[(i >> 4) & ((1 << KB) - 1)], c = ms.cent[i >> (4 + KB)];
      *reinterpret_cast<uint2*>(sm + i * 8) = make_uint2(__byte_perm(a.x, c.x, 0x5410), __byte_perm(a.y, c.y, 0x5410));
    }
  __syncthreads();
  // ---------------------------------------------------------------- scores
  const int r0 = packed ? 2 * (t & 1) : 2 * t;  // the lane's rows r0, r0 + 1
  const float q0 = ms.qsc[r0], q1 = ms.qsc[r0 + 1];
  const int lim0 = ms.lim[r0], lim1 = ms.lim[r0 + 1];
  const int pitch = mp.pitch;
  float* keep = mp.logits + (unit * few_columns(mp) + (dense ? (int64_t)p.max_chunks * kChunk : 0)) * pitch + r0;
  const bool writes = r0 < pitch && (!packed || t < 2);
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
#pragma unroll 1
  for (int c = c0; c < c1; ++c) {
    float acc[2][4], ac2[2][4];
#pragma unroll
    for (int mi = 0; mi < 2; ++mi)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[mi][e] = ac2[mi][e] = 0.f;
    if (!dense) {
      const uint8_t* next = c + 1 < c1 ? rec_at(c + 1) : rec;
      load_norms(next, nkn);
#pragma unroll 1
      for (int s = 0; s < NS; ++s) {
        load_words(s + 1 < NS ? rec : next, s + 1 < NS ? s + 1 : 0, wn);
        const uint4* bq = qfrag + s * (STEP / 4) * 32 + lane;
#pragma unroll
        for (int k = 0; k < STEP / 4; ++k) {
          uint32_t ah[2][4], al[2][4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint2 v = pair_at<KB>(tab, sm, w[i], 4 * k + 2 * e, loff);
              ah[i >> 1][(i & 1) + 2 * e] = v.x;
              al[i >> 1][(i & 1) + 2 * e] = v.y;
            }
          const uint4 q4 = bq[k * 32];
#pragma unroll
          for (int mi = 0; mi < 2; ++mi) {
            mma_f16(acc[mi], ah[mi], q4.x, q4.y);
            mma_f16(ac2[mi], al[mi], q4.x, q4.y);
            if (!packed) mma_f16(ac2[mi], ah[mi], q4.z, q4.w);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int k = 0; k < NW; ++k) w[i][k] = wn[i][k];
      }
#pragma unroll
      for (int mi = 0; mi < 2; ++mi)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          acc[mi][e] += ac2[mi][e];
          if (packed) acc[mi][e] += __shfl_xor_sync(0xffffffffu, acc[mi][e], 2);
        }
      if constexpr (OUTL) {  // lane tk's side list, entry by entry, for every row; then to the token's lanes
        const int oc = slot_entries(rec + p.kc.off_count, warp, lane);
        const int from = oc >> 8, cnt = min(oc & 255, max(p.kc.cap - from, 0));
        const uint32_t* ent = reinterpret_cast<const uint32_t*>(rec + p.kc.off_entries) + from;
        const unsigned char* row = rec + (32 * warp + lane) * row_bytes;
        float d[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) d[r] = 0.f;
        for (int e = 0; e < cnt; ++e) {
          const uint32_t en = __ldg(ent + e);
          const int j = en & (D - 1);
          const float delta = bf16_hi(en) - p.kc.centroids[row_code<KB>(row, j)];
          const float4 a = *reinterpret_cast<const float4*>(qrot + j * 8), c4 = *reinterpret_cast<const float4*>(qrot + j * 8 + 4);
          d[0] = fmaf(delta, a.x, d[0]);
          d[1] = fmaf(delta, a.y, d[1]);
          d[2] = fmaf(delta, a.z, d[2]);
          d[3] = fmaf(delta, a.w, d[3]);
          d[4] = fmaf(delta, c4.x, d[4]);
          d[5] = fmaf(delta, c4.y, d[5]);
          d[6] = fmaf(delta, c4.z, d[6]);
          d[7] = fmaf(delta, c4.w, d[7]);
        }
        float* corr = reinterpret_cast<float*>(sm + mp.sm_corr) + warp * 32 * 9;
#pragma unroll
        for (int r = 0; r < 8; ++r) corr[lane * 9 + r] = d[r];
        __syncwarp();
      }
      rec = next;
    } else {
      const uint16_t* rows[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int tok = min(c * kChunk + 32 * warp + 8 * i + g, cl.len - 1);
        rows[i] = ring + (int64_t)((rstart + (int64_t)tok) % cap) * D + t * RUN;
        nk[i] = 1.f;
      }
#pragma unroll 4
      for (int kk = 0; kk < KS; kk += 2) {
        uint4 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const uint4*>(rows[i] + 4 * kk);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t a[2][4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            a[i >> 1][i & 1] = k ? x[i].z : x[i].x;
            a[i >> 1][(i & 1) + 2] = k ? x[i].w : x[i].y;
          }
          const uint2 q2 = qfragd[(kk + k) * 32 + lane];
          mma_bf16(acc[0], a[0], q2.x, q2.y);
          mma_bf16(acc[1], a[1], q2.x, q2.y);
        }
      }
    }
    float x[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int tok = c * kChunk + 32 * warp + 8 * i + g;
      const float n = finite_or_nan(nk[i]);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float v = acc[i >> 1][2 * (i & 1) + e] * (e ? q1 : q0);
        if constexpr (OUTL) {
          if (!dense) v = fmaf(reinterpret_cast<const float*>(sm + mp.sm_corr)[(warp * 32 + 8 * i + g) * 9 + r0 + e], p.sscale, v);
        }
        x[i][e] = mass_logit(p, v, n, base + tok < (e ? lim1 : lim0));
      }
      if (writes) {
        float* dst = keep + (int64_t)tok * pitch;
        if (pitch > 1) *reinterpret_cast<float2*>(dst) = f2(x[i][0], x[i][1]);
        else *dst = x[i][0];
      }
    }
    const float a0 = fmaxf(fmaxf(fmaxf(x[0][0], x[1][0]), fmaxf(x[2][0], x[3][0])), m0);
    const float a1 = fmaxf(fmaxf(fmaxf(x[0][1], x[1][1]), fmaxf(x[2][1], x[3][1])), m1);
    // a NaN reaches the sums, whatever the maxima are
    if (a0 > -INFINITY) {
      l0 = l0 * ex2(m0 - a0) + ((ex2(x[0][0] - a0) + ex2(x[1][0] - a0)) + (ex2(x[2][0] - a0) + ex2(x[3][0] - a0)));
      m0 = a0;
    } else {
      const float y = (x[0][0] + x[1][0]) + (x[2][0] + x[3][0]);
      if (y != y) l0 = y;
    }
    if (a1 > -INFINITY) {
      l1 = l1 * ex2(m1 - a1) + ((ex2(x[0][1] - a1) + ex2(x[1][1] - a1)) + (ex2(x[2][1] - a1) + ex2(x[3][1] - a1)));
      m1 = a1;
    } else {
      const float y = (x[0][1] + x[1][1]) + (x[2][1] + x[3][1]);
      if (y != y) l1 = y;
    }
    if (!dense) {
#pragma unroll
      for (int i = 0; i < 4; ++i) nk[i] = nkn[i];
    }
    if constexpr (OUTL) __syncwarp();  // the corrections are read before the next record's are written
  }
  // statistics over the eight token lanes, then the four warps
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    float m = e ? m1 : m0, s = e ? l1 : l0;
#pragma unroll
    for (int k = 4; k < 32; k <<= 1) {
      const float mo = __shfl_xor_sync(0xffffffffu, m, k), so = __shfl_xor_sync(0xffffffffu, s, k);
      const float mx = fmaxf(m, mo);
      s = mx > -INFINITY ? s * ex2(m - mx) + so * ex2(mo - mx) : s + so;
      m = mx;
    }
    if (g == 0 && (!packed || t < 2)) ms.part[warp][r0 + e] = make_float2(m, s);
  }
  __syncthreads();
  if (tid < 8) {
    float m = -INFINITY, s = 0.f;
    if (!packed || tid < 4) {
      for (int k = 0; k < 4; ++k) m = fmaxf(m, ms.part[k][tid].x);
      for (int k = 0; k < 4; ++k) s += ms.part[k][tid].y * (m > -INFINITY ? ex2(ms.part[k][tid].x - m) : 1.f);
    }
    ml[tid] = make_float2(m, s);
  }
}

// shared memory of one instantiation
inline void attn_mass_few_layout(MassParams& mp, int D, int KB, bool outl) {
  auto al = [](int x) { return (x + 127) / 128 * 128; };
  int off = (1 << (2 * KB)) * 128;  // the pair table comes first
  mp.sm_frag = off;
  off = al(off + D / 16 * 32 * 16);
  mp.sm_misc = off;
  off = al(off + (int)sizeof(FewMisc));
  mp.sm_qrot = off;
  off = al(off + (outl ? D * 8 * 4 : 0));
  mp.sm_corr = off;
  off = al(off + (outl ? kChunk * 9 * 4 : 0));
  mp.sm_total = off;
}

template <int D, int KB, bool OUTL>
cudaError_t attn_mass_few_launch_t(const MassParams& mp, cudaStream_t s) {
  auto kern = attn_mass_few_kernel<D, KB, OUTL>;
  if (mp.sm_total > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, mp.sm_total);
    if (e != cudaSuccess) return e;
  }
  kern<<<dim3(mp.Sc + mp.St, mp.q.B * mp.q.Hkv, mp.q.L), kThreads, mp.sm_total, s>>>(mp);
  return cudaGetLastError();
}

template <int D>
cudaError_t attn_mass_few_launch_d(const MassParams& mp, cudaStream_t s) {
  const bool outl = mp.q.krec && mp.q.kc.has_outl;
  switch (mp.q.krec ? mp.q.kc.bits : 1) {
    case 1: return outl ? attn_mass_few_launch_t<D, 1, true>(mp, s) : attn_mass_few_launch_t<D, 1, false>(mp, s);
    case 2: return outl ? attn_mass_few_launch_t<D, 2, true>(mp, s) : attn_mass_few_launch_t<D, 2, false>(mp, s);
    case 3: return outl ? attn_mass_few_launch_t<D, 3, true>(mp, s) : attn_mass_few_launch_t<D, 3, false>(mp, s);
    case 4: return outl ? attn_mass_few_launch_t<D, 4, true>(mp, s) : attn_mass_few_launch_t<D, 4, false>(mp, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace tq
