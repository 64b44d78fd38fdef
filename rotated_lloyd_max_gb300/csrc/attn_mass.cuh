// Accumulated attention weight: mass_j = decay mass_j + sum over the query
// rows of a kv head (query heads x new tokens) of softmax_ij.
//
// Two passes over the keys.  The first leaves each row's (max, sum) per split
// of the context; the second forms the scores again, subtracts the row's
// log-sum and adds the weights up over the rows.  Forming the scores twice
// costs a second read of the packed keys (half a byte per coordinate at 4
// bits), where keeping them would cost 8 bytes written and read per row and
// token.
//
// Tokens are the M dimension of the MMA, query rows its N: a warp holds 32
// tokens of a record (two m-tiles), dequantises their packed codes straight
// from memory into A fragments, a k-step at a time, and runs up to 64 rows
// (8 NT) against them, so that a code is decoded once per 64 rows and never
// stored.  The weights are f32 results, and a logit's absolute error is a
// weight's relative one: centroids and rotated queries enter as f16 hi + lo
// pairs (22 bits) and a product takes three MMAs.  The ring's bf16 keys and
// queries are exact operands of one bf16 MMA.
//
// A lane's coordinates are the contiguous run (d/4) (lane % 4) .. of a packed
// row: fragment columns 2t, 2t + 1, 2t + 8, 2t + 9 of k-step kk hold the
// run's codes 4 kk .. 4 kk + 3.  Queries are laid out to match, per k-step and
// lane one 16-byte word (hi, hi, lo, lo).  Pairs of codes become f16 pairs by
// one 64-bit lookup in a table that is replicated so that no two lanes of a
// half-warp share a bank.
#pragma once

#include "attn_mma.cuh"
#include "cache_params.h"

namespace tq {

// 128-token tiles of a split on tcgen05 at most: their sums lie in shared memory (24 KB)
constexpr int kMassUmmaPer = 48;

struct MassParams {
  QueryParams q;
  int Sc, St;         // context splits over records and over ring tokens
  int cps, tps;       // records and ring tokens (a multiple of 128) per split
  int rows, nrb;      // query rows T * G, row blocks of 8 NT
  int pass;           // 0: row statistics, 1: weights
  float2* ml;         // [units][Sc + St][rows padded to nrb * 8 NT]
  uint4* frag;        // [units][nrb][D / 16][NT][32] query fragments hi, lo
  uint2* fragd;       // the same for the ring: bf16 queries as they are
  float* qsc;         // [units][nrb * 8 NT] score scales
  float* qrot;        // [units][nrb][D][8 NT] rotated queries (side lists only)
  int pitch;          // few rows: logits kept per token (rows padded to a power of two)
  float* logits;      // [units][records' then the ring's tokens][pitch]
  float* mass;
  int64_t mass_ls;
  int mass_cap;
  float decay;
  // dynamic shared memory (bytes)
  int sm_frag, sm_misc, sm_cent, sm_sum, sm_qrot, sm_corr, sm_total;
};

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// x, or NaN in the place of an infinity: an infinite scale makes coordinates of both signs infinite,
// and a product with them no number
__device__ __forceinline__ float finite_or_nan(float x) { return fmaf(x, 0.f, x); }

// new tokens of sequence b
__device__ __forceinline__ int query_len(const QueryParams& p, int b) {
  return p.q_lens ? min(max(p.q_lens[b], 0), p.T) : p.T;
}
struct CacheLen {
  int n, len, total;
};
__device__ __forceinline__ CacheLen cache_len(const QueryParams& p, int lb) {
  CacheLen c;
  c.n = p.n_chunks ? min(max(p.n_chunks[lb], 0), min(p.max_chunks, p.rec_limit)) : 0;
  c.len = p.tail_len ? min(max(p.tail_len[lb], 0), min(p.max_tail, p.tail_cap)) : 0;
  c.total = c.n * kChunk + c.len;
  return c;
}
// tokens that query row r (token r / G) sees: those of index below the result
__device__ __forceinline__ int row_limit(const QueryParams& p, const CacheLen& c, int tb, int r) {
  const int t = r / p.G;
  return t >= tb ? 0 : p.causal ? min(c.total, c.total - tb + t + 1) : c.total;
}

// the table's entry (f16 pairs hi, lo) for codes at and at + 1 of a run's words
template <int KB, int NW>
__device__ __forceinline__ uint2 pair_at(const ByteTable& tab, const unsigned char* table, const uint32_t (&w)[NW], int at,
                                         uint32_t loff) {
  if constexpr (KB == 4) return byte_lookup2(tab, w[at / 8], at % 8 / 2);
  else return *reinterpret_cast<const uint2*>(table + pair_off(w, at * KB, 2 * KB, loff));
}

template <int NT>
struct MassMisc {
  float qsc[8 * NT];      // score scale of a row
  int lim[8 * NT];        // tokens it sees
  float lse[8 * NT];      // log2 of its sum (pass 1)
  float2 part[4][8 * NT]; // the warps' statistics (pass 0)
};

__device__ __forceinline__ uint32_t pack_bf16x2(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// log2 of a row's sum W 2^M: INFINITY for a row that sees no token and weighs nothing, NaN for one of
// no finite softmax, which leaves NaN in every entry
__device__ __forceinline__ float log_sum(float M, float W, int limit) {
  if (W > 0.f) return M + log2f(W);
  return W != W || limit > 0 ? __int_as_float(0x7fc00000) : INFINITY;
}
// a logit in log2 units, -inf past the row's limit
__device__ __forceinline__ float mass_logit(const QueryParams& p, float acc, float f, bool seen) {
  float t = acc * f;
  if (p.scap > 0.f) t = soft_cap(t, p.scap, p.iscap);
  return seen ? t : -INFINITY;
}

template <int D, int KB, int NT, bool OUTL>
__global__ void __launch_bounds__(kThreads) attn_mass_kernel(const __grid_constant__ MassParams mp) {
  constexpr int KS = D / 16, RUN = D / 4;
  constexpr int STEP = RUN < 32 ? RUN : 32;   // codes of a run taken at a time
  constexpr int NB = STEP * KB, NW = (NB + 31) / 32;
  constexpr bool AL = NB % 32 == 0;
  constexpr int R = 8 * NT;
  const QueryParams& p = mp.q;
  extern __shared__ __align__(128) unsigned char sm[];
  uint4* qfrag = reinterpret_cast<uint4*>(sm + mp.sm_frag);
  uint2* qfragd = reinterpret_cast<uint2*>(sm + mp.sm_frag);
  MassMisc<NT>& ms = *reinterpret_cast<MassMisc<NT>*>(sm + mp.sm_misc);
  uint2* cent = reinterpret_cast<uint2*>(sm + mp.sm_cent);
  float* sums = reinterpret_cast<float*>(sm + mp.sm_sum);

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int S = mp.Sc + mp.St;
  const int h = blockIdx.y % p.Hkv, b = blockIdx.y / p.Hkv, l = blockIdx.z;
  const int split = mp.pass == 0 ? blockIdx.x / mp.nrb : blockIdx.x;
  const int rb0 = mp.pass == 0 ? blockIdx.x % mp.nrb : 0, rb1 = mp.pass == 0 ? rb0 + 1 : mp.nrb;
  const int lb = l * p.B + b;
  const int64_t unit = (int64_t)lb * p.Hkv + h;
  const bool dense = split >= mp.Sc;
  const CacheLen cl = cache_len(p, lb);
  const int tb = query_len(p, b);
  // the split's tokens: records [c0, c1), or 128-token tiles of the ring
  const int per = dense ? mp.tps / kChunk : mp.cps;
  const int c0 = (dense ? split - mp.Sc : split) * per;
  const int c1 = min(c0 + per, dense ? (cl.len + kChunk - 1) / kChunk : cl.n);
  const int rows_pad = mp.nrb * R;
  const int base = dense ? cl.n * kChunk : 0;  // index of the first record's / the ring's first token
  if (mp.pass == 0) {
    if (c0 >= c1 || tb == 0) {
      float2* ml = mp.ml + (unit * S + split) * rows_pad + rb0 * R;
      if (tid < R) ml[tid] = make_float2(-INFINITY, 0.f);
      return;
    }
  } else if (c0 >= c1) {
    return;
  }

  const uint8_t* kl = p.krec + l * p.krec_ls;
  const int row_bytes = D * KB / 8;
  const int cap = p.tail_cap;
  const uint16_t* ring = p.ktail + l * p.tail_ls + (int64_t)(b * p.Hkv + h) * cap * D;
  const int rstart = dense && p.tail_start ? ((p.tail_start[lb] % cap) + cap) % cap : 0;
  const uint32_t loff = (lane & 15) * 8;
  const ByteTable tab = byte_table(sm, loff, 128);

  if (!dense) {  // pair table: entry e at byte 128 e + 8 (lane % 16): f16 pairs hi, lo of centroids x 2^16
    if (tid < 16) {
      const float v = p.kc.centroids[tid] * 65536.f;
      const __half hi = __float2half_rn(v);
      cent[tid] = make_uint2(__half_as_ushort(hi), __half_as_ushort(__float2half_rn(v - __half2float(hi))));
    }
    __syncthreads();
    for (int i = tid; i < (1 << (2 * KB)) * 16; i += kThreads) {
      const uint2 a = cent[(i >> 4) & ((1 << KB) - 1)], c = cent[i >> (4 + KB)];
      *reinterpret_cast<uint2*>(sm + i * 8) = make_uint2(__byte_perm(a.x, c.x, 0x5410), __byte_perm(a.y, c.y, 0x5410));
    }
  }
  if (mp.pass == 1)
    for (int i = tid; i < (c1 - c0) * kChunk; i += kThreads) sums[i] = 0.f;

#pragma unroll 1
  for (int rb = rb0; rb < rb1; ++rb) {
    const int64_t ub = unit * mp.nrb + rb;
    __syncthreads();  // the previous block's fragments and sums are done with
    // ------------------------------------------------------------ query fragments
    if (mp.pass == 0) {
      const bool keep = dense ? split == mp.Sc : split == 0;  // the first split leaves them for pass 1
      for (int r = warp; r < R; r += 4) {  // a warp per row, a lane per D / 32 coordinates
        const int row = rb * R + r;
        const bool live = row < mp.rows && row / p.G < tb;
        constexpr int E = D / 32;
        float x[E];
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = 0.f;
        if (live) {
          const uint16_t* qp = p.q + l * p.q_ls + b * p.q_bs + (int64_t)(row / p.G) * p.q_ts +
                               (int64_t)(h * p.G + row % p.G) * D + lane * E;
#pragma unroll
          for (int e = 0; e < E; e += 2) {
            const uint32_t w = *reinterpret_cast<const uint32_t*>(qp + e);
            x[e] = bf16_lo(w);
            x[e + 1] = bf16_hi(w);
          }
        }
        float sc = 1.f;
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
          const int s = mx > 0.f ? 13 - exp_of(mx) : 0;  // largest |q~| in [2^13, 2^14)
          if constexpr (OUTL) {
            float* qr = mp.qrot + (ub * D + lane * E) * R + r;
#pragma unroll
            for (int e = 0; e < E; ++e) {
              reinterpret_cast<float*>(sm + mp.sm_qrot)[(lane * E + e) * R + r] = x[e];
              if (keep) qr[e * R] = x[e];
            }
          }
          sc = pow2i(s);
          if (lane == 0) ms.qsc[r] = p.sscale * pow2i(-16 - s);
        } else if (lane == 0) {
          ms.qsc[r] = p.sscale;
        }
        if (lane == 0) ms.lim[r] = live ? row_limit(p, cl, tb, row) : 0;
        // coordinate j sits in lane j / RUN's word of k-step (j % RUN) / 4
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          const int j = lane * E + e, tt = j / RUN, kk = (j % RUN) / 4, half = (j % 4) / 2;
          const int at = (kk * NT + (r >> 3)) * 32 + (r & 7) * 4 + tt;
          if (dense) {
            const __nv_bfloat162 w = __floats2bfloat162_rn(x[e], x[e + 1]);
            reinterpret_cast<uint32_t*>(qfragd + at)[half] = *reinterpret_cast<const uint32_t*>(&w);
          } else {
            uint32_t hi, lo;
            split_f16x2(x[e] * sc, x[e + 1] * sc, hi, lo);
            reinterpret_cast<uint32_t*>(qfrag + at)[half] = hi;
            reinterpret_cast<uint32_t*>(qfrag + at)[2 + half] = lo;
          }
        }
      }
      __syncthreads();
      if (keep) {
        if (dense) {
          for (int i = tid; i < KS * NT * 32; i += kThreads) mp.fragd[ub * (KS * NT * 32) + i] = qfragd[i];
        } else {
          for (int i = tid; i < KS * NT * 32; i += kThreads) mp.frag[ub * (KS * NT * 32) + i] = qfrag[i];
          if (tid < R) mp.qsc[ub * R + tid] = ms.qsc[tid];
        }
      }
    } else {
      if (dense) {
        for (int i = tid; i < KS * NT * 32; i += kThreads) qfragd[i] = mp.fragd[ub * (KS * NT * 32) + i];
      } else {
        for (int i = tid; i < KS * NT * 32; i += kThreads) qfrag[i] = mp.frag[ub * (KS * NT * 32) + i];
        if constexpr (OUTL)
          for (int i = tid; i < D * R; i += kThreads)
            reinterpret_cast<float*>(sm + mp.sm_qrot)[i] = mp.qrot[ub * D * R + i];
      }
      if (tid < R) {
        const int row = rb * R + tid;
        const bool live = row < mp.rows && row / p.G < tb;
        ms.qsc[tid] = dense ? p.sscale : mp.qsc[ub * R + tid];
        ms.lim[tid] = live ? row_limit(p, cl, tb, row) : 0;
        float M = -INFINITY, W = 0.f;
        const float2* ml = mp.ml + unit * S * rows_pad + row;
        for (int s = 0; s < S; ++s) M = fmaxf(M, ml[(int64_t)s * rows_pad].x);
        for (int s = 0; s < S; ++s) {
          const float2 v = ml[(int64_t)s * rows_pad];
          if (v.y > 0.f) W += v.y * exp2f(v.x - M);
          else if (v.y != v.y) W = v.y;
        }
        ms.lse[tid] = log_sum(M, W, ms.lim[tid]);
      }
      __syncthreads();
    }
    // ------------------------------------------------------------ scores
    float m_[NT][2], l_[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m_[nt][0] = m_[nt][1] = -INFINITY;
      l_[nt][0] = l_[nt][1] = 0.f;
    }
#pragma unroll 1
    for (int c = c0; c < c1; ++c) {
      float acc[2][NT][4];
#pragma unroll
      for (int mi = 0; mi < 2; ++mi)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[mi][nt][e] = 0.f;
      float nk[4];  // score scales of tokens 32 warp + 16 mi + 8 k + g
      if (!dense) {
        const uint8_t* rec = kl + rec_offset(p.table, p.table_stride, p.rec_cap, p.Hkv, b, h, c, p.kc.rec_bytes);
        const unsigned char* rows[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int tok = 32 * warp + 8 * i + g;
          rows[i] = rec + tok * row_bytes;
          nk[i] = __ldg(reinterpret_cast<const float*>(rec + p.kc.off_norm) + tok);
        }
#pragma unroll 1
        for (int s = 0; s < RUN / STEP; ++s) {
          uint32_t w[4][NW];
#pragma unroll
          for (int i = 0; i < 4; ++i) load_run<NB, AL>(rows[i], (t * RUN + s * STEP) * KB, w[i]);
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
            const uint4* bq = qfrag + (s * (STEP / 4) + k) * NT * 32 + lane;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const uint4 q4 = bq[nt * 32];
#pragma unroll
              for (int mi = 0; mi < 2; ++mi) {
                mma_f16(acc[mi][nt], ah[mi], q4.x, q4.y);
                mma_f16(acc[mi][nt], al[mi], q4.x, q4.y);
                mma_f16(acc[mi][nt], ah[mi], q4.z, q4.w);
              }
            }
          }
        }
        if constexpr (OUTL) {
          // side list: token by token, a lane per query row, (value - centroid) q~_j;
          // entries past the capacity or past a row's coordinates are not read
          const float* qr = reinterpret_cast<const float*>(sm + mp.sm_qrot);
          float* corr = reinterpret_cast<float*>(sm + mp.sm_corr) + warp * 32 * R;
          const int oc = slot_entries(rec + p.kc.off_count, warp, lane);
          const uint32_t* ent = reinterpret_cast<const uint32_t*>(rec + p.kc.off_entries);
          for (int tk = 0; tk < 32; ++tk) {
            const int o = __shfl_sync(0xffffffffu, oc, tk), from = o >> 8;
            const int cnt = min(o & 255, max(p.kc.cap - from, 0));
            float a[(R + 31) / 32];
#pragma unroll
            for (int i = 0; i < (R + 31) / 32; ++i) a[i] = 0.f;
            for (int e = 0; e < cnt; ++e) {
              const uint32_t en = __ldg(ent + from + e);
              const int j = en & (D - 1);
              const float delta = bf16_hi(en) - p.kc.centroids[row_code<KB>(rec + (32 * warp + tk) * row_bytes, j)];
#pragma unroll
              for (int i = 0; i < (R + 31) / 32; ++i)
                if (lane + 32 * i < R) a[i] = fmaf(delta, qr[j * R + lane + 32 * i], a[i]);
            }
#pragma unroll
            for (int i = 0; i < (R + 31) / 32; ++i)
              if (lane + 32 * i < R) corr[tk * R + lane + 32 * i] = a[i] * p.sscale;
          }
          __syncwarp();
        }
      } else {
        const uint16_t* rows[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int tok = min(c * kChunk + 32 * warp + 8 * i + g, cl.len - 1);
          rows[i] = ring + (int64_t)((rstart + (int64_t)tok) % cap) * D + t * RUN;
          nk[i] = 1.f;
        }
#pragma unroll 2
        for (int kk = 0; kk < KS; kk += 2) {
          uint4 w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const uint4*>(rows[i] + 4 * kk);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint32_t a[2][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              a[i >> 1][i & 1] = k ? w[i].z : w[i].x;
              a[i >> 1][(i & 1) + 2] = k ? w[i].w : w[i].y;
            }
            const uint2* bq = qfragd + (kk + k) * NT * 32 + lane;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const uint2 q2 = bq[nt * 32];
              mma_bf16(acc[0][nt], a[0], q2.x, q2.y);
              mma_bf16(acc[1][nt], a[1], q2.x, q2.y);
            }
          }
        }
      }
      // element e of tile mi: token 32 warp + 16 mi + 8 (e / 2) + g, row 8 nt + 2 t + e % 2
#pragma unroll
      for (int i = 0; i < 4; ++i) nk[i] = finite_or_nan(nk[i]);
      const int tok0 = base + c * kChunk + 32 * warp + g;
      float w4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e1 = 0; e1 < 2; ++e1) {
          const int r = 8 * nt + 2 * t + e1;
          const float qs = ms.qsc[r];
          const int lim = ms.lim[r];
          float x[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float v = acc[i >> 1][nt][2 * (i & 1) + e1] * qs;
            if constexpr (OUTL) {
              if (!dense) v += reinterpret_cast<const float*>(sm + mp.sm_corr)[(warp * 32 + 8 * i + g) * R + r];
            }
            x[i] = mass_logit(p, v, nk[i], tok0 + 8 * i < lim);
          }
          if (mp.pass == 0) {
            const float mx = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), m_[nt][e1]);
            const float rf = mx > -INFINITY ? mx : 0.f;  // a NaN reaches the sum, whatever the maximum is
            l_[nt][e1] = l_[nt][e1] * ex2(m_[nt][e1] - rf) + ((ex2(x[0] - rf) + ex2(x[1] - rf)) +
                                                             (ex2(x[2] - rf) + ex2(x[3] - rf)));
            m_[nt][e1] = mx;
          } else {
            const float lse = ms.lse[r];
#pragma unroll
            for (int i = 0; i < 4; ++i) w4[i] += ex2(x[i] - lse);
          }
        }
      if (mp.pass == 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          w4[i] += __shfl_xor_sync(0xffffffffu, w4[i], 1);
          w4[i] += __shfl_xor_sync(0xffffffffu, w4[i], 2);
          if (t == i) sums[(c - c0) * kChunk + 32 * warp + 8 * i + g] += w4[i];
        }
      }
      if constexpr (OUTL) __syncwarp();  // the corrections are read before the next record's are written
    }
    if (mp.pass == 0) {  // statistics over the eight token lanes, then the four warps
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e1 = 0; e1 < 2; ++e1) {
          float m = m_[nt][e1], s = l_[nt][e1];
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) {
            const float mo = __shfl_xor_sync(0xffffffffu, m, x), so = __shfl_xor_sync(0xffffffffu, s, x);
            const float mx = fmaxf(m, mo);
            s = mx > -INFINITY ? s * ex2(m - mx) + so * ex2(mo - mx) : s + so;
            m = mx;
          }
          if (g == 0) ms.part[warp][8 * nt + 2 * t + e1] = make_float2(m, s);
        }
      __syncthreads();
      if (tid < R) {
        float m = -INFINITY, s = 0.f;
        for (int w = 0; w < 4; ++w) m = fmaxf(m, ms.part[w][tid].x);
        for (int w = 0; w < 4; ++w) s += ms.part[w][tid].y * (m > -INFINITY ? ex2(ms.part[w][tid].x - m) : 1.f);
        mp.ml[(unit * S + split) * rows_pad + rb * R + tid] = make_float2(m, s);
      }
    }
  }
  if (mp.pass == 1) {
    __syncthreads();
    float* m = mp.mass + l * mp.mass_ls + ((int64_t)b * p.Hkv + h) * mp.mass_cap;
    const int first = base + c0 * kChunk, end = min((c1 - c0) * kChunk, (dense ? cl.total : cl.n * kChunk) - first);
    for (int i = tid; i < end; i += kThreads) m[first + i] = fmaf(mp.decay, m[first + i], sums[i]);
  }
}

// shared memory of one instantiation
inline void attn_mass_layout(MassParams& mp, int D, int KB, int NT, bool outl) {
  auto al = [](int x) { return (x + 127) / 128 * 128; };
  int off = (1 << (2 * KB)) * 128;  // the pair table comes first
  mp.sm_frag = off;
  off = al(off + D / 16 * NT * 32 * 16);
  mp.sm_misc = off;
  off = al(off + 8 * NT * (4 + 4 + 4 + 32));
  mp.sm_cent = off;
  off += 128;
  mp.sm_sum = off;
  off = al(off + 4 * std::max(mp.cps * kChunk, mp.tps));
  mp.sm_qrot = off;
  off = al(off + (outl ? D * 8 * NT * 4 : 0));
  mp.sm_corr = off;
  off = al(off + (outl ? kChunk * 8 * NT * 4 : 0));
  mp.sm_total = off;
}

template <int D, int KB, int NT, bool OUTL>
cudaError_t attn_mass_launch_t(const MassParams& mp, cudaStream_t s) {
  auto kern = attn_mass_kernel<D, KB, NT, OUTL>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, mp.sm_total);
  if (e != cudaSuccess) return e;
  const int S = mp.Sc + mp.St;
  const dim3 grid(mp.pass == 0 ? S * mp.nrb : S, mp.q.B * mp.q.Hkv, mp.q.L);
  kern<<<grid, kThreads, mp.sm_total, s>>>(mp);
  return cudaGetLastError();
}

// row blocks of 32 for up to 32 rows, else of 64; of 16 with side lists, whose
// corrections keep the rotated queries in shared memory as f32
template <int D, int KB>
cudaError_t attn_mass_launch_kb(const MassParams& mp, int NT, cudaStream_t s) {
  if (mp.q.kc.has_outl) return attn_mass_launch_t<D, KB, 2, true>(mp, s);
  return NT == 4 ? attn_mass_launch_t<D, KB, 4, false>(mp, s) : attn_mass_launch_t<D, KB, 8, false>(mp, s);
}

template <int D>
cudaError_t attn_mass_launch_d(const MassParams& mp, int NT, cudaStream_t s) {
  switch (mp.q.krec ? mp.q.kc.bits : 1) {
    case 1: return attn_mass_launch_kb<D, 1>(mp, NT, s);
    case 2: return attn_mass_launch_kb<D, 2>(mp, NT, s);
    case 3: return attn_mass_launch_kb<D, 3>(mp, NT, s);
    case 4: return attn_mass_launch_kb<D, 4>(mp, NT, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace tq
