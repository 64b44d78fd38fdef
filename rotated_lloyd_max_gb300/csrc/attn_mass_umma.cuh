// Accumulated attention weight for many query rows on the fifth-generation
// tensor cores (head dims 64 and 128): the two passes of attn_mass_kernel with
// 128 rows per CTA.
//
// Scores S = Q~ K^T of a record (128 rows x 128 tokens, f32 in tensor memory)
// are three f16 products, hi hi + lo hi + hi lo, of operands that hold 22
// bits: the rotated queries stay in tensor memory for the whole run as the A
// operand, hi and lo, so that only the decoded keys are read from shared
// memory (an MMA with both operands there would need all of its bandwidth).
// Three score buffers; two warpgroups take records in turn, a thread a row.
//   pass 0: running sum of 2^(t - ref), the reference moving only when it is
//           passed by 2^40 (f32 holds the terms exactly enough either way);
//   pass 1: 2^(t - log-sum), summed over a warp's 32 rows by a transposing
//           butterfly (lane j ends with column j), then over the four warps.
// Sixteen warps decode keys into two stages (hi and lo tiles) by one 64-bit
// lookup a pair of codes; the ring's bf16 keys are copied as they are (one
// exact product).  32 tokens of 32 heads over 131072 + 1024 (3 bits, head dim 128):
// 217 us, 41% of the tensor cores' time (107 us for the six products); the rest is
// instruction issue, the column sums and the decoding of hi and lo above all.
// Every wait is bounded; a CTA whose wait expired leaves NaN.
#pragma once

#include <cstddef>

#include "attn_mass.cuh"
#include "prefill_umma.cuh"

namespace tq {

constexpr int kMuThreads = 800, kMuLoad = 16, kMuIssue = 24;
constexpr float kMuMargin = 40.f;

template <int D>
struct MuCfg {
  static constexpr int TILE = 128 * D * 2;  // one operand tile
  static constexpr int K = 0, LUT = 4 * TILE, MISC = LUT + 32768, SUMS = MISC + 11264;
  static constexpr int SMEM = SUMS + kMassUmmaPer * 512 + 1024;
};

struct MuMisc {
  uint64_t k_full[2], k_empty[2], s_full[3], s_empty[3], rot, fin;
  uint32_t tbase;
  int abort_;
  alignas(16) float nk[8][128];  // a consumer warp's copy of a record's scales
  float part[2][4][128]; // pass 1: column sums of a warpgroup's warps
  float2 st[2][128];     // pass 0: the warpgroups' statistics; pass 1: [0][r].x = log-sum of row r
};
static_assert(sizeof(MuMisc) <= 11264 && offsetof(MuMisc, nk) % 16 == 0 && offsetof(MuMisc, st) % 8 == 0, "bookkeeping block");

// eight codes -> f16 pairs hi (one uint4) and lo through the pair table
template <int B>
__device__ __forceinline__ void lookup8(const unsigned char* lut, uint32_t x, uint32_t lo, uint4& vh, uint4& vl) {
  constexpr uint32_t M = ((1u << (2 * B)) - 1u) << 7;
  const ByteTable tab = byte_table(lut, lo, 128);
  uint2 e[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (B == 4) {
      e[k] = byte_lookup2(tab, x, k);
    } else {
      const int sh = 2 * B * k;
      const uint32_t o = ((sh >= 7 ? x >> (sh - 7) : x << (7 - sh)) & M) | lo;
      e[k] = *reinterpret_cast<const uint2*>(lut + o);
    }
  }
  vh = make_uint4(e[0].x, e[1].x, e[2].x, e[3].x);
  vl = make_uint4(e[0].y, e[1].y, e[2].y, e[3].y);
}

template <int D, int B>
__device__ __forceinline__ void store_hi_lo(const Packed<D>& k, const unsigned char* lut, unsigned char* st, int w,
                                            int lane) {
  using P = Packed<D>;
  const uint32_t lo = (lane & 15) * 8;
  st += w * kPfTok * 128;
#pragma unroll
  for (int i = 0; i < P::PER; ++i) {
    const int row = (lane + 32 * i) / P::CH, ch = (lane + 32 * i) % P::CH;
    uint4 vh, vl;
    lookup8<B>(lut, k.x[i], lo, vh, vl);
    unsigned char* d = st + (ch >> 3) * 16384 + row * 128 + (((ch ^ row) & 7) << 4);
    *reinterpret_cast<uint4*>(d) = vh;
    *reinterpret_cast<uint4*>(d + MuCfg<D>::TILE) = vl;
  }
}

__device__ __forceinline__ void bar_wg(int wg) {
  if (wg == 0) asm volatile("bar.sync 1, 128;" ::: "memory");
  else asm volatile("bar.sync 2, 128;" ::: "memory");
}

// sums of 32 values over a warp: lane j returns the sum of v[j]
__device__ __forceinline__ float column_sum(float (&v)[32], int lane) {
#pragma unroll
  for (int half = 16; half >= 1; half >>= 1) {
    const bool up = (lane & half) != 0;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float keep = up ? v[half + i] : v[i];
      const float give = up ? v[i] : v[half + i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, half);
    }
  }
  return v[0];
}

template <int D, bool DENSE>
__device__ __forceinline__ void mass_umma_body(const MassParams& mp, unsigned char* sm, int64_t unit, int split,
                                               int tile0, int tile1) {
  using C = MuCfg<D>;
  const QueryParams& p = mp.q;
  MuMisc& ms = *reinterpret_cast<MuMisc*>(sm + C::MISC);
  float* sums = reinterpret_cast<float*>(sm + C::SUMS);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = (int)(unit % p.Hkv), lb = (int)(unit / p.Hkv), b = lb % p.B, l = lb / p.B;
  const int S = mp.Sc + mp.St;
  const CacheLen cl = cache_len(p, lb);
  const int tb = query_len(p, b);
  const int per = DENSE ? mp.tps / kChunk : mp.cps;
  const int c0 = split * per, c1 = min(c0 + per, DENSE ? (cl.len + kChunk - 1) / kChunk : cl.n);
  const int sidx = DENSE ? mp.Sc + split : split;
  const int base = DENSE ? cl.n * kChunk : 0;
  if (mp.pass == 0) {
    const int64_t at = ((unit * mp.nrb + tile0) * S + sidx) * 128;
    if (c0 >= c1 || tile0 * 128 >= tb * p.G) {
      if (tid < 128) mp.ml[at + tid] = make_float2(-INFINITY, 0.f);
      return;
    }
  } else if (c0 >= c1) {
    return;
  }
  const int n = c1 - c0;
  // ---------------------------------------------------------------- set-up
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ms.k_full[i], kMuLoad);
      mbar_init(&ms.k_empty[i], 1);
    }
    for (int i = 0; i < 3; ++i) {
      mbar_init(&ms.s_full[i], 1);
      mbar_init(&ms.s_empty[i], 4);
    }
    mbar_init(&ms.rot, 1);
    mbar_init(&ms.fin, 1);
    ms.abort_ = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMuIssue) tmem_alloc(&ms.tbase, 512);
  if constexpr (!DENSE)
    for (int i = tid; i < (1 << (2 * p.kc.bits)) * 16; i += kMuThreads) {
      const int e = i >> 4, m = (1 << p.kc.bits) - 1;
      uint32_t hi, lo;
      split_f16x2(p.kc.centroids[e & m] * kTableScale, p.kc.centroids[e >> p.kc.bits] * kTableScale, hi, lo);
      *reinterpret_cast<uint2*>(sm + C::LUT + i * 8) = make_uint2(hi, lo);
    }
  if (mp.pass == 1)
    for (int i = tid; i < n * kChunk; i += kMuThreads) sums[i] = 0.f;
  volatile int* abort_f = &ms.abort_;
  uint32_t done = 0;  // records whose pipeline phases lie behind
#pragma unroll 1
  for (int tile = tile0; tile < tile1; ++tile) {
    const int r0 = tile * 128, rn = min(128, tb * p.G - r0);
    if (rn <= 0) break;
    // ---------------------------------------------------------------- queries into tensor memory
    constexpr int CH = D / 8;
    const uint32_t flip = p.sscale < 0.f ? 0x80008000u : 0u;  // the softmax scale's sign
    for (int i = tid; i < 128 * CH; i += kMuThreads) {
      const int r = i / CH, ch = i % CH, row = r0 + r;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (r < rn)
        v = __ldg(reinterpret_cast<const uint4*>(p.q + l * p.q_ls + b * p.q_bs + (int64_t)(row / p.G) * p.q_ts +
                                                 (int64_t)(h * p.G + row % p.G) * D) + ch);
      v = make_uint4(v.x ^ flip, v.y ^ flip, v.z ^ flip, v.w ^ flip);
      *reinterpret_cast<uint4*>(sm + C::K + (ch >> 3) * 16384 + sw128_off(r, ch & 7)) = v;
    }
    if constexpr (!DENSE) {  // signed Hadamard matrix, as in the prefill kernel
      for (int i = tid; i < D * CH; i += kMuThreads) {
        const int n_ = i / CH, ch = i % CH;
        const uint32_t sg = (p.kc.signs[ch >> 2] >> (8 * (ch & 3))) ^ (__popc((n_ >> 3) & ch) & 1 ? 0xFFu : 0u);
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t s0 = (sg >> (2 * j)) ^ __popc(n_ & (2 * j)), s1 = (sg >> (2 * j + 1)) ^ __popc(n_ & (2 * j + 1));
          w[j] = 0x3F803F80u | ((s0 & 1u) << 15) | ((s1 & 1u) << 31);
        }
        *reinterpret_cast<uint4*>(sm + C::K + C::TILE + (ch >> 3) * 16384 + sw128_off(n_, ch & 7)) =
            make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    if (mp.pass == 1 && tid < 512) {  // log-sums of the rows, four threads each
      const int r = tid >> 2, row = r0 + r;
      const float2* ml = mp.ml + (unit * mp.nrb + tile) * S * 128 + r;
      float M = -INFINITY, W = 0.f;
      for (int s = tid & 3; s < S; s += 4) M = fmaxf(M, ml[(int64_t)s * 128].x);
      M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 1));
      M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 2));
      for (int s = tid & 3; s < S; s += 4) {
        const float2 v = ml[(int64_t)s * 128];
        if (v.y != v.y) W = v.y;  // a split that gave up
        if (v.y > 0.f) W += v.y * exp2f(v.x - M);
      }
      W += __shfl_xor_sync(0xffffffffu, W, 1);
      W += __shfl_xor_sync(0xffffffffu, W, 2);
      if ((tid & 3) == 0) ms.st[0][r].x = log_sum(M, W, row < tb * p.G ? row_limit(p, cl, tb, row) : 0);
    }
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tQ = ms.tbase, tS = ms.tbase + 128;
    const uint32_t ph = (uint32_t)(tile - tile0) & 1;
    float f = fabsf(p.sscale);  // logit factor of the thread's row
    if (warp == kMuIssue) {
      if constexpr (!DENSE) {
        if (elect_one()) {
          const uint64_t dQ = sdesc_sw128(smem_u32(sm + C::K), 16, 1024), dH = dQ + C::TILE / 16;
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint64_t o = (ks >> 2) * 1024 + 2 * (ks & 3);
            umma_f16(tS, dQ + o, dH + o, idesc_f16(128, D, false, false) | kIdescBf16, ks != 0);
          }
          umma_commit(&ms.rot);
        }
        __syncwarp();
      }
    } else if (warp < 8) {  // both warpgroups learn their rows' factors; the first writes the operand
      const uint32_t lrow = (uint32_t)(32 * (warp & 3)) << 16;
      const int r = 32 * (warp & 3) + lane;
      if constexpr (DENSE) {
        if (warp < 4) {
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t w[16];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint4 v = *reinterpret_cast<const uint4*>(sm + C::K + (c >> 1) * 16384 + sw128_off(r, 4 * (c & 1) + k));
              w[4 * k] = v.x; w[4 * k + 1] = v.y; w[4 * k + 2] = v.z; w[4 * k + 3] = v.w;
            }
            tmem_st16(tQ + lrow + 16 * c, w);
          }
        }
      } else {
        mbar_wait_idle(&ms.rot, ph, abort_f);
        tc_fence_after();
        float mx = 0.f;
#pragma unroll 1
        for (int c = 0; c < D / 16; ++c) {
          uint32_t a[16];
          tmem_ld16(tS + lrow + 16 * c, a);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j) mx = fmaxf(mx, fabsf(__uint_as_float(a[j])));
        }
        mx *= inv_sqrt_dim<D>();
        const int s = mx > 0.f ? 13 - exp_of(mx) : 0;
        const float sc = pow2i(s);
        f *= pow2i(-15 - s);
        if (warp < 4) {
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t wh[16], wl[16];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              uint32_t a[16];
              tmem_ld16(tS + lrow + 32 * c + 16 * e, a);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 8; ++j)
                split_f16x2(__uint_as_float(a[2 * j]) * inv_sqrt_dim<D>() * sc,
                            __uint_as_float(a[2 * j + 1]) * inv_sqrt_dim<D>() * sc, wh[8 * e + j], wl[8 * e + j]);
            }
            tmem_st16(tQ + lrow + 16 * c, wh);
            tmem_st16(tQ + lrow + D / 2 + 16 * c, wl);
          }
        }
      }
      tmem_st_wait();
      tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    // ---------------------------------------------------------------- the run
    if (warp == kMuIssue) {
      if (elect_one()) {
        constexpr uint32_t IS = idesc_f16(128, 128, false, false) | (DENSE ? kIdescBf16 : 0u);
        const uint64_t dK = sdesc_sw128(smem_u32(sm + C::K), 16, 1024);
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
          const uint32_t g = done + i, sb = g % 3;
          mbar_wait_idle(&ms.k_full[g & 1], (g >> 1) & 1, abort_f);
          mbar_wait_idle(&ms.s_empty[sb], ((g / 3) & 1) ^ 1, abort_f);
          tc_fence_after();
          const uint64_t kh = dK + (g & 1) * (2 * C::TILE / 16), kL = kh + C::TILE / 16;
          const uint32_t d = tS + 128 * sb;
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint64_t o = (ks >> 2) * 1024 + 2 * (ks & 3);
            umma_f16_ts(d, tQ + 8 * ks, kh + o, IS, ks != 0);
            if constexpr (!DENSE) {
              umma_f16_ts(d, tQ + 8 * ks, kL + o, IS, 1);
              umma_f16_ts(d, tQ + D / 2 + 8 * ks, kh + o, IS, 1);
            }
          }
          umma_commit(&ms.k_empty[g & 1]);
          umma_commit(&ms.s_full[sb]);
        }
      }
      __syncwarp();
    } else if (warp >= 8) {
      const int w = warp - 8;
      if constexpr (DENSE) {
        constexpr int PER = kPfTok * CH / 32;
        const int cap = p.tail_cap;
        const int start = p.tail_start ? ((p.tail_start[lb] % cap) + cap) % cap : 0;
        const uint16_t* src = p.ktail + l * p.tail_ls + (int64_t)(b * p.Hkv + h) * cap * D;
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
          const uint32_t g = done + i;
          mbar_wait_idle(&ms.k_empty[g & 1], ((g >> 1) & 1) ^ 1, abort_f);
          unsigned char* st = sm + C::K + (g & 1) * 2 * C::TILE;
#pragma unroll
          for (int k = 0; k < PER; ++k) {
            const int x = lane + 32 * k, row = kPfTok * w + x / CH, ch = x % CH;
            const int tok = min((c0 + i) * kChunk + row, cl.len - 1);
            cp_async16(st + (ch >> 3) * 16384 + sw128_off(row, ch & 7),
                       src + (int64_t)((start + (int64_t)tok) % cap) * D + 8 * ch);
          }
          cp_async_commit();
          cp_async_wait<0>();
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ms.k_full[g & 1]);
        }
      } else {
        RecSource ks = rec_source<D>(p.kc, p.krec + l * p.krec_ls, w, lane);
        auto seek = [&](int c) {
          if (p.table || c == c0) ks.next = ks.layer + rec_offset(p.table, p.table_stride, p.rec_cap, p.Hkv, b, h, c, ks.bytes);
          else ks.next += ks.bytes;
        };
        Packed<D> xk;
        seek(c0);
        load_tile<D>(ks, xk);
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
          const uint32_t g = done + i;
          mbar_wait_idle(&ms.k_empty[g & 1], ((g >> 1) & 1) ^ 1, abort_f);
          unsigned char* st = sm + C::K + (g & 1) * 2 * C::TILE;
          switch (ks.bits) {
            case 1: store_hi_lo<D, 1>(xk, sm + C::LUT, st, w, lane); break;
            case 2: store_hi_lo<D, 2>(xk, sm + C::LUT, st, w, lane); break;
            case 3: store_hi_lo<D, 3>(xk, sm + C::LUT, st, w, lane); break;
            default: store_hi_lo<D, 4>(xk, sm + C::LUT, st, w, lane); break;
          }
          if (p.kc.has_outl) {  // values are bf16: exact in the hi tile
            side_list<D>(p.kc, ks.next, w, lane, 1.f, [&](int row, int j, float y, float) {
              unsigned char* d = st + (j >> 6) * 16384 + sw128_off(kPfTok * w + row, (j >> 3) & 7) + 2 * (j & 7);
              *reinterpret_cast<__half*>(d) = __float2half_rn(y * kTableScale);
              *reinterpret_cast<uint16_t*>(d + C::TILE) = 0;
            });
          }
          fence_async_smem();  // before the next loads, which it would wait for
          __syncwarp();
          if (lane == 0) mbar_arrive(&ms.k_full[g & 1]);
          if (i + 1 < n) {
            seek(c0 + i + 1);
            load_tile<D>(ks, xk);
          }
        }
      }
    } else {
      // a warpgroup takes every other record, a thread a row
      const int wg = warp >> 2, r = 32 * (warp & 3) + lane;
      const uint32_t lrow = (uint32_t)(32 * (warp & 3)) << 16;
      const int lim = r < rn ? row_limit(p, cl, tb, r0 + r) - base - c0 * kChunk : 0x7FFFFFFF;
      const float lse = mp.pass == 1 ? ms.st[0][r].x : 0.f;
      float ref = mp.pass == 1 ? lse : -INFINITY, lsum = 0.f;
      auto norms = [&](int i) {
        if constexpr (DENSE) return make_float4(1.f, 1.f, 1.f, 1.f);
        const uint8_t* rec = p.krec + l * p.krec_ls +
                             rec_offset(p.table, p.table_stride, p.rec_cap, p.Hkv, b, h, c0 + i, p.kc.rec_bytes);
        return __ldg(reinterpret_cast<const float4*>(rec + p.kc.off_norm) + lane);
      };
      float4 nk = wg < n ? norms(wg) : make_float4(0, 0, 0, 0);
#pragma unroll 1
      for (int i = wg; i < n; i += 2) {
        const uint32_t g = done + i, sb = g % 3;
        const uint32_t tB = tS + 128 * sb + lrow;
        __syncwarp();
        *reinterpret_cast<float4*>(&ms.nk[warp][4 * lane]) =
            make_float4(finite_or_nan(nk.x), finite_or_nan(nk.y), finite_or_nan(nk.z), finite_or_nan(nk.w));
        __syncwarp();
        if (i + 2 < n) nk = norms(i + 2);
        mbar_wait_idle(&ms.s_full[sb], (g / 3) & 1, abort_f);
        tc_fence_after();
        const int seen = lim - i * kChunk;
        const bool edge = __any_sync(0xffffffffu, seen < kChunk), plain = !edge && !(p.scap > 0.f);
        // logits of 32 columns
        auto logits = [&](int c, float (&v)[32]) {
          uint32_t a[2][16];
          tmem_ld16(tB + 32 * c, a[0]);
          tmem_ld16(tB + 32 * c + 16, a[1]);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            const float4 s = *reinterpret_cast<const float4*>(&ms.nk[warp][32 * c + j]);
            const float2 x = mul2(f2(__uint_as_float(a[j >> 4][j & 15]), __uint_as_float(a[j >> 4][(j & 15) + 1])), f2(s.x, s.y));
            const float2 y = mul2(f2(__uint_as_float(a[j >> 4][(j & 15) + 2]), __uint_as_float(a[j >> 4][(j & 15) + 3])), f2(s.z, s.w));
            v[j] = x.x;
            v[j + 1] = x.y;
            v[j + 2] = y.x;
            v[j + 3] = y.y;
          }
          if (plain) return;
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            float t = v[j] * f;
            if (p.scap > 0.f) t = soft_cap(t, p.scap, p.iscap);
            v[j] = 32 * c + j < seen ? t : -INFINITY;
          }
        };
        const float ff = plain ? f : 1.f;
        if (mp.pass == 0) {
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            float v[32];
            logits(c, v);
            float m = v[0];
#pragma unroll
            for (int j = 1; j < 31; j += 2) m = max3(m, v[j], v[j + 1]);
            m = fmaxf(m, v[31]);
            m = m > -INFINITY ? m * ff : -INFINITY;
            if (m > ref + kMuMargin) {
              if (ref > -INFINITY) lsum *= ex2(ref - m);  // else it is zero or NaN
              ref = m;
            }
            const float rr = ref > -INFINITY ? ref : 0.f;
            const float2 F = f2(ff, ff), M2 = f2(-rr, -rr);
            float2 s = f2(0.f, 0.f);
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
              const float2 x = fma2(f2(v[j], v[j + 1]), F, M2);
              s = add2(s, f2(ex2(x.x), ex2(x.y)));
            }
            lsum += s.x + s.y;
          }
        } else {
          const float2 F = f2(ff, ff), M2 = f2(-ref, -ref);
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            float v[32];
            logits(c, v);
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
              const float2 x = fma2(f2(v[j], v[j + 1]), F, M2);
              v[j] = ex2(x.x);
              v[j + 1] = ex2(x.y);
            }
            ms.part[wg][warp & 3][32 * c + lane] = column_sum(v, lane);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ms.s_empty[sb]);
        if (mp.pass == 1) {
          bar_wg(wg);
          sums[i * kChunk + r] += (ms.part[wg][0][r] + ms.part[wg][1][r]) + (ms.part[wg][2][r] + ms.part[wg][3][r]);
          bar_wg(wg);
        }
      }
      if (mp.pass == 0) ms.st[wg][r] = make_float2(ref, lsum);
    }
    done += n;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (mp.pass == 0 && tid < 128) {
      const float2 x = ms.st[0][tid], y = ms.st[1][tid];
      const float m = fmaxf(x.x, y.x);
      float w = m > -INFINITY ? x.y * ex2(x.x - m) + y.y * ex2(y.x - m) : x.y + y.y;
      if (*abort_f) w = __int_as_float(0x7fc00000);
      mp.ml[((unit * mp.nrb + tile) * S + sidx) * 128 + tid] = make_float2(m, tid < rn ? w : 0.f);
    }
  }
  if (mp.pass == 1) {
    float* m = mp.mass + l * mp.mass_ls + ((int64_t)b * p.Hkv + h) * mp.mass_cap;
    const int first = base + c0 * kChunk, end = min(n * kChunk, (DENSE ? cl.total : cl.n * kChunk) - first);
    const float bad = *abort_f ? __int_as_float(0x7fc00000) : 0.f;
    for (int i = tid; i < end; i += kMuThreads) m[first + i] = fmaf(mp.decay, m[first + i], sums[i]) + bad;
  }
  if (warp == kMuIssue) {
    if (elect_one()) umma_commit(&ms.fin);
    __syncwarp();
    volatile int drain = 0;  // every MMA has completed, whatever the abort flag says
    mbar_wait_idle(&ms.fin, 0, &drain);
    tc_fence_after();
    tmem_dealloc(ms.tbase, 512);
  }
}

template <int D>
__global__ void __launch_bounds__(kMuThreads, 1) mass_umma_kernel(const __grid_constant__ MassParams mp) {
  extern __shared__ __align__(1024) unsigned char smraw[];
  unsigned char* sm = smraw + ((1024u - (smem_u32(smraw) & 1023u)) & 1023u);
  // pass 0: a row tile per CTA; pass 1: a CTA keeps its tokens and walks the row tiles
  const int64_t U = (int64_t)mp.q.L * mp.q.B * mp.q.Hkv * (mp.pass == 0 ? mp.nrb : 1);
  const int split = (int)(blockIdx.x / U);
  const int64_t u = blockIdx.x % U;
  const int64_t unit = mp.pass == 0 ? u / mp.nrb : u;
  const int t0 = mp.pass == 0 ? (int)(u % mp.nrb) : 0, t1 = mp.pass == 0 ? t0 + 1 : mp.nrb;
  if (split < mp.Sc) mass_umma_body<D, false>(mp, sm, unit, split, t0, t1);
  else mass_umma_body<D, true>(mp, sm, unit, split - mp.Sc, t0, t1);
}

template <int D>
cudaError_t mass_umma_launch(const MassParams& mp, cudaStream_t s) {
  const cudaError_t e = cudaFuncSetAttribute(mass_umma_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, MuCfg<D>::SMEM);
  if (e != cudaSuccess) return e;
  const int64_t grid = (int64_t)mp.q.L * mp.q.B * mp.q.Hkv * (mp.pass == 0 ? mp.nrb : 1) * (mp.Sc + mp.St);
  mass_umma_kernel<D><<<(unsigned)grid, kMuThreads, MuCfg<D>::SMEM, s>>>(mp);
  return cudaGetLastError();
}

}  // namespace tq
