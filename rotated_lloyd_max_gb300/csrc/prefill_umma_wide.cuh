// Attention of several query tokens per sequence on the fifth-generation
// tensor cores at head dims 256 and 512, where the outputs of 128 rows would
// fill tensor memory: scores and outputs are transposed, 64 query rows a CTA.
//
//   S^T[token][row]  = K Q~^T   (A: 128 decoded tokens, B: 64 rows; N = 64)
//   O^T[coord][row] += V^T P    (A: 128 coordinates of the decoded tokens,
//                                MN-major; B: P [token][row], MN-major)
// A thread owns a token (its lane) for the softmax and a coordinate for the
// outputs, so that a token's scales are one factor of its thread's logits and one
// of its weights, and decoding is a table lookup and nothing else.  References
// of the softmax as in the narrower kernel (prefill_umma.cuh), but that a row whose
// weights have become small is found by their sums, two records late and off the
// chain of the products; the ring's tokens are bf16 operands.
//
// Tokens are decoded in chunks of 64 coordinates (16 KB) into a ring of eight,
// sixteen warps in groups of four, a group a chunk.  Where keys and values share
// a record (or ring), a chunk serves the scores and, kept, the outputs, so that
// it is decoded once; otherwise the keys' chunks and the values' follow one another.
// A chunk is decoded into registers before its slot is waited for (5% more when it
// decodes into the slot).  64 tokens of 64 heads over 16384, head dim 512: 376 us.
//
// 128 tokens at head dim 512 take 640 KB of shared memory's traffic (two
// products of 192 KB, since an MMA of N = 64 reads 6 KB; 128 KB of tiles
// written; 128 KB of lookups), 5000 of the 9600 cycles measured.  The rest is
// waiting: the ring holds one such tile, so that the decoding of the next runs
// behind the products of this one, and scores, softmax and outputs follow one another.
#pragma once

#include "prefill_umma.cuh"

namespace tq {

constexpr int kPwThreads = 672, kPwRows = 64, kPwSlots = 8;
constexpr int kPwIssue = 20;

template <int D>
struct PwCfg {
  static constexpr int Q = 0, P = 64 * D * 2, RING = P + 16384, LUT = RING + kPwSlots * 16384, MISC = LUT + 16384;
  static constexpr int SMEM = MISC + 2048 + 1024;
};

struct PwMisc {
  uint64_t full[kPwSlots], empty[kPwSlots], s_full, p_full, o_done, fin;
  uint32_t tbase;
  int abort_;
  alignas(16) float qf[64];    // logit factor of a row
  alignas(16) float ref[64];   // its softmax reference (log2 units)
  int lim[64];                 // tokens it sees, counted from the run's first
  alignas(16) float red[4][64];
  uint4 small[2][2];           // by record parity, halves of the rows: those whose weights sum to less than
                               // 2^kPfLow, a word a warp
  uint32_t bound[2];           // rows whose reference may not move down
};
static_assert(sizeof(PwMisc) <= 2048, "bookkeeping block");

__device__ __forceinline__ void bar_soft() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ bool bar_soft_or(bool pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.red.or.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)pred)
      : "memory");
  return r != 0;
}

// 32 values per lane -> lane j holds the maximum / sum over the warp of value j
template <bool MAX>
__device__ __forceinline__ float transpose_reduce32(float (&v)[32], int lane) {
#pragma unroll
  for (int half = 16; half >= 1; half >>= 1) {
    const bool up = (lane & half) != 0;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float keep = up ? v[half + i] : v[i];
      const float give = up ? v[i] : v[half + i];
      const float got = __shfl_xor_sync(0xffffffffu, give, half);
      v[i] = MAX ? fmaxf(keep, got) : keep + got;
    }
  }
  return v[0];
}

// One chunk (coordinates 64 c ..) of a record: warp w of a group takes tokens
// 32 w .. 32 w + 31, a lane eight codes of every fourth token.
struct Chunk {
  uint32_t x[8];
};
// at: the lane's first token, codes of chunk c
template <int D, int B>
__device__ __forceinline__ void load_chunk(const uint8_t* at, Chunk& k) {
  constexpr int STEP = 4 * (D * B / 8);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (B == 4) k.x[i] = __ldg(reinterpret_cast<const uint32_t*>(at + i * STEP));
    else if constexpr (B == 2) k.x[i] = __ldg(reinterpret_cast<const uint16_t*>(at + i * STEP));
    else if constexpr (B == 1) k.x[i] = __ldg(at + i * STEP);
    else {
      const uint32_t o = (uint32_t)reinterpret_cast<uintptr_t>(at) & 3u;
      const uint32_t* q = reinterpret_cast<const uint32_t*>(at - o + i * STEP);
      k.x[i] = __funnelshift_r(__ldg(q), __ldg(q + 1), 8 * o);
    }
  }
}
template <int D>
__device__ __forceinline__ void load_chunk_b(int bits, const uint8_t* at, Chunk& k) {
  switch (bits) {
    case 1: load_chunk<D, 1>(at, k); break;
    case 2: load_chunk<D, 2>(at, k); break;
    case 3: load_chunk<D, 3>(at, k); break;
    default: load_chunk<D, 4>(at, k); break;
  }
}
// four 4-bit codes (16 bits) -> f16 pairs through the byte planes
__device__ __forceinline__ void half_planes(uint32_t sel, const Planes& pl, uint32_t& x, uint32_t& y) {
  const uint32_t s7 = sel & 0x7777u, pick = 0x3210u + ((sel >> 3) & 0x1111u) * 4u;
  const uint32_t a = __byte_perm(__byte_perm(pl.lo[0], pl.lo[1], s7), __byte_perm(pl.lo[2], pl.lo[3], s7), pick);
  const uint32_t b = __byte_perm(__byte_perm(pl.hi[0], pl.hi[1], s7), __byte_perm(pl.hi[2], pl.hi[3], s7), pick);
  x = __byte_perm(a, b, 0x5140);
  y = __byte_perm(a, b, 0x7362);
}
// LUT: half of the 4-bit codes through a table of 16 copies (a pair's entry e at
// 64 e + 4 (lane % 16)), half through the planes: the lookups alone queue for
// shared memory (two lanes meet in a bank), the planes alone for the ALUs.
template <int B, bool LUT>
__device__ __forceinline__ void decode_chunk(const Chunk& k, const Planes& pl, const unsigned char* lut, uint4 (&v)[8],
                                             int lane) {
  const ByteTable tab = byte_table(lut, 4 * (lane & 15), 64);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (LUT) {
      const uint32_t x = k.x[i];
      v[i].x = byte_lookup(tab, x, 0);
      v[i].y = byte_lookup(tab, x, 1);
      half_planes(x >> 16, pl, v[i].z, v[i].w);
    } else {
      v[i] = decode_codes<B>(k.x[i], pl);
    }
  }
}
__device__ __forceinline__ void decode_chunk_b(int bits, const Chunk& k, const Planes& pl, const unsigned char* lut,
                                               uint4 (&v)[8], int lane) {
  switch (bits) {
    case 1: decode_chunk<1, false>(k, pl, lut, v, lane); break;
    case 2: decode_chunk<2, false>(k, pl, lut, v, lane); break;
    case 3: decode_chunk<3, false>(k, pl, lut, v, lane); break;
    default:
      if (lut) decode_chunk<4, true>(k, pl, lut, v, lane);
      else decode_chunk<4, false>(k, pl, lut, v, lane);
  }
}
// side list entries of chunk c's coordinates, a lane a token
template <int D>
__device__ __forceinline__ void patch_chunk(const CodecDev& cd, const uint8_t* rec, int c, unsigned char* st, int w,
                                            int lane) {
  const int e = slot_entries(rec + cd.off_count, w, lane), from = e >> 8, cnt = min(e & 255, max(cd.cap - from, 0));
  const uint32_t* ent = reinterpret_cast<const uint32_t*>(rec + cd.off_entries) + from;
  __syncwarp();
  for (int i = 0; i < cnt; ++i) {
    const uint32_t en = __ldg(ent + i);
    const int j = en & (D - 1);
    if ((j >> 6) == c)
      *reinterpret_cast<__half*>(st + sw128_off(32 * w + lane, (j >> 3) & 7) + 2 * (j & 7)) =
          __float2half_rn(bf16_hi(en) * kTableScale);
  }
}

template <int D, bool DENSE>
__device__ __forceinline__ void prefill_wide_body(const PrefillParams& pp, unsigned char* sm, int64_t unit, int tile,
                                                  int split) {
  using C = PwCfg<D>;
  constexpr int NCH = D / 64, NBL = D / 128, E = D / 32;
  const QueryParams& p = pp.q;
  PwMisc& ms = *reinterpret_cast<PwMisc*>(sm + C::MISC);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = (int)(unit % p.Hkv), lb = (int)(unit / p.Hkv), b = lb % p.B, l = lb / p.B;
  const int S = pp.Sc + pp.St;
  const CacheLen cl = cache_len(p, lb);
  const int tb = query_len(p, b);
  const int r0 = tile * kPwRows, rn = min(kPwRows, tb * p.G - r0);
  if (rn <= 0) return;
  const int base = DENSE ? cl.n * kChunk : 0;
  const int top = row_limit(p, cl, tb, r0 + rn - 1) - base;
  const int k0 = split * (DENSE ? pp.tps : pp.cps * kChunk);
  const int k1 = min(min(k0 + (DENSE ? pp.tps : pp.cps * kChunk), DENSE ? cl.len : cl.n * kChunk), top);
  const int sidx = DENSE ? pp.Sc + split : split;
  const int64_t wrow = unit * pp.rows + r0;
  if (k0 >= k1) {
    for (int r = tid; r < rn; r += kPwThreads) pp.ws_ml[(wrow + r) * S + sidx] = make_float2(-INFINITY, 0.f);
    return;
  }
  const int n = (k1 - k0 + kChunk - 1) / kChunk, c0 = k0 / kChunk;
  const bool one = DENSE ? p.ktail == p.vtail : p.shared_kv != 0;  // keys are the values
  const uint8_t* kl = p.krec + l * p.krec_ls;
  const uint8_t* vl = p.vrec + l * p.vrec_ls;
  auto rec_at = [&](bool key, int c) {
    return (key ? kl : vl) + rec_offset(p.table, p.table_stride, p.rec_cap, p.Hkv, b, h, c,
                                        key ? p.kc.rec_bytes : p.vc.rec_bytes);
  };
  // ---------------------------------------------------------------- set-up
  if (tid == 0) {
    for (int i = 0; i < kPwSlots; ++i) {
      mbar_init(&ms.full[i], 4);
      mbar_init(&ms.empty[i], 1);
    }
    mbar_init(&ms.s_full, 1);
    mbar_init(&ms.p_full, 4);
    mbar_init(&ms.o_done, 1);
    mbar_init(&ms.fin, 1);
    ms.abort_ = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kPwIssue) tmem_alloc(&ms.tbase, 512);
  bool vtable = false;  // the values are decoded through the lookup table
  if constexpr (!DENSE) {
    vtable = p.vc.bits == 4;
    if (p.kc.bits == 4)
      for (int k = 8; k < 16; ++k) vtable = vtable && p.kc.centroids[k] == p.vc.centroids[k];
    float mv = 0.f;  // the run's largest value scale
    for (int i = tid; i < n * (kChunk / 4); i += kPwThreads) {
      const float4 y = __ldg(reinterpret_cast<const float4*>(rec_at(false, c0 + i / (kChunk / 4)) + p.vc.off_norm) + i % (kChunk / 4));
      mv = fmaxf(mv, fmaxf(fmaxf(fabsf(y.x), fabsf(y.y)), fmaxf(fabsf(y.z), fabsf(y.w))));
    }
    mv = warp_max(mv);
    if (lane == 0) ms.red[0][warp] = mv;
    const CodecDev& c4 = p.kc.bits == 4 ? p.kc : p.vc;
    if (c4.bits == 4)
      for (int i = tid; i < 256 * 16; i += kPwThreads)
        reinterpret_cast<uint32_t*>(sm + C::LUT)[i] =
            pack2_f16(c4.centroids[(i >> 4) & 15] * kTableScale, c4.centroids[i >> 8] * kTableScale);
    __syncthreads();
  }
  float ev = 1.f;  // 2^-(E+1) of the values' scales: weights times scales stay in f16's range
  if constexpr (!DENSE) ev = pow2i(-1 - exp_of(warp_max(ms.red[0][lane < 21 ? lane : 0])));
  {  // query rows, a warp each; lane holds E coordinates
    const float sgn = p.sscale < 0.f ? -1.f : 1.f;
    for (int r = warp; r < kPwRows; r += kPwThreads / 32) {
      const int row = r0 + r;
      float x[E];
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] = 0.f;
      if (r < rn) {
        const uint16_t* qp = p.q + l * p.q_ls + b * p.q_bs + (int64_t)(row / p.G) * p.q_ts +
                             (int64_t)(h * p.G + row % p.G) * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; e += 8) {
          const uint4 v = *reinterpret_cast<const uint4*>(qp + e);
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            x[e + 2 * k] = bf16_lo(w[k]) * sgn;
            x[e + 2 * k + 1] = bf16_hi(w[k]) * sgn;
          }
        }
      }
      float f = fabsf(p.sscale);
      uint32_t w[E / 2];
      if constexpr (DENSE) {
#pragma unroll
        for (int e = 0; e < E; e += 2) w[e / 2] = pack2_bf16(x[e], x[e + 1]);
      } else {
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
        f *= pow2i(-15 - s);
#pragma unroll
        for (int e = 0; e < E; e += 2) w[e / 2] = pack2_f16(x[e] * sc, x[e + 1] * sc);
      }
#pragma unroll
      for (int e = 0; e < E; e += 8) {
        const int j = lane * E + e;
        *reinterpret_cast<uint4*>(sm + C::Q + (j >> 6) * 8192 + sw128_off(r, (j >> 3) & 7)) =
            make_uint4(w[e / 2], w[e / 2 + 1], w[e / 2 + 2], w[e / 2 + 3]);
      }
      if (lane == 0) {
        ms.qf[r] = f;
        ms.ref[r] = -INFINITY;
        ms.lim[r] = r < rn ? row_limit(p, cl, tb, row) - base - k0 : 0x7FFFFFFF;
      }
    }
  }
  fence_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tS = ms.tbase, tO = ms.tbase + 64;  // S^T: 64 columns; O^T: NBL blocks of 64
  volatile int* abort_f = &ms.abort_;
  // chunk g of the run: record i's NCH chunks, once or (keys, then values) twice
  const int perrec = one ? NCH : 2 * NCH;

  if (warp == kPwIssue) {
    // ---------------------------------------------------------------- MMA issue
    if (elect_one()) {
      constexpr uint32_t T = DENSE ? kIdescBf16 : 0u;
      constexpr uint32_t IS = idesc_f16(128, 64, false, false) | T, IV = idesc_f16(128, 64, true, true) | T;
      const uint64_t dQ = sdesc_sw128(smem_u32(sm + C::Q), 16, 1024);
      const uint64_t dK = sdesc_sw128(smem_u32(sm + C::RING), 16, 1024);
      const uint64_t dP = sdesc_sw128(smem_u32(sm + C::P), 1024, 1024);
      const uint64_t dV = sdesc_sw128(smem_u32(sm + C::RING), 16384, 1024);
      // slots and parities of a record's chunks: one record in turn takes NCH slots
      // where keys are the values, else 2 NCH (all of them, twice at head dim 512)
#pragma unroll 1
      for (int i = 0; i < n; ++i) {
        const uint32_t q0 = i * perrec, s0 = q0 % kPwSlots, p0 = (q0 / kPwSlots) & 1;
        const uint32_t q1 = one ? q0 : q0 + NCH, s1 = q1 % kPwSlots, p1 = (q1 / kPwSlots) & 1;
        const uint64_t a0 = dK + s0 * 1024, v0 = dV + s1 * 1024;
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
          mbar_wait_idle(&ms.full[s0 + c], p0, abort_f);
          tc_fence_after();
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) umma_f16(tS, a0 + c * 1024 + 2 * ks, dQ + c * 512 + 2 * ks, IS, (c | ks) != 0);
          if (!one) umma_commit(&ms.empty[s0 + c]);
        }
        umma_commit(&ms.s_full);
        mbar_wait_idle(&ms.p_full, i & 1, abort_f);
        tc_fence_after();
#pragma unroll
        for (int j = 0; j < NBL; ++j) {
          // a block of 128 coordinates: two chunks, 64 coordinates (M rows) apart in the ring
          if (!one) {
            mbar_wait_idle(&ms.full[s1 + 2 * j], p1, abort_f);
            mbar_wait_idle(&ms.full[s1 + 2 * j + 1], p1, abort_f);
            tc_fence_after();
          }
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)
            umma_f16(tO + 64 * j, v0 + j * 2048 + 128 * ks, dP + 128 * ks, IV, i > 0 || ks > 0);
          umma_commit(&ms.empty[s1 + 2 * j]);
          umma_commit(&ms.empty[s1 + 2 * j + 1]);
        }
        umma_commit(&ms.o_done);
      }
      umma_commit(&ms.fin);
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ---------------------------------------------------------------- chunks: group grp takes every fourth
    const int grp = (warp - 4) >> 2, w = (warp - 4) & 3;
    const int total = n * perrec;
    if constexpr (DENSE) {
      const int cap = p.tail_cap;
      const int start = p.tail_start ? ((p.tail_start[lb] % cap) + cap) % cap : 0;
      const int64_t ring = l * p.tail_ls + (int64_t)(b * p.Hkv + h) * cap * D;
#pragma unroll 1
      for (int q = grp; q < total; q += 4) {
        const int i = q / perrec, x = q % perrec, c = x % NCH, s = q % kPwSlots;
        const uint16_t* src = (x >= NCH ? p.vtail : p.ktail) + ring + 64 * c;
        mbar_wait_idle(&ms.empty[s], ((q / kPwSlots) & 1) ^ 1, abort_f);
        unsigned char* st = sm + C::RING + s * 16384;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int row = 32 * w + 4 * k + (lane >> 3), tok = min(k0 + i * kChunk + row, cl.len - 1);
          cp_async16(st + sw128_off(row, lane & 7), src + (int64_t)((start + (int64_t)tok) % cap) * D + 8 * (lane & 7));
        }
        cp_async_commit();
        cp_async_wait<0>();
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ms.full[s]);
      }
    } else {
      // a group's chunks of a record: c = grp, grp + 4, .. of the keys, then of the
      // values where those are apart; the same chunk of the next record is loaded
      // as soon as one is stored
      constexpr int PER = NCH / 4;
      const Planes kpl = make_planes(p.kc, kTableScale), vpl = make_planes(p.vc, kTableScale);
      const unsigned char* klut = p.kc.bits == 4 ? sm + C::LUT : nullptr;
      const unsigned char* vlut = vtable ? sm + C::LUT : nullptr;
      const int kbits = p.kc.bits, vbits = p.vc.bits;
      const int kat = (32 * w + (lane >> 3)) * (D * kbits / 8) + (8 * grp + (lane & 7)) * kbits;
      const int vat = (32 * w + (lane >> 3)) * (D * vbits / 8) + (8 * grp + (lane & 7)) * vbits;
      Chunk kx[PER], vx[PER];
      const uint8_t *krec = rec_at(true, c0), *vrec = rec_at(false, c0);
#pragma unroll
      for (int x = 0; x < PER; ++x) {
        load_chunk_b<D>(kbits, krec + kat + 32 * x * kbits, kx[x]);
        if (!one) load_chunk_b<D>(vbits, vrec + vat + 32 * x * vbits, vx[x]);
      }
      // a chunk is decoded before its slot is waited for
      uint32_t q = grp;
      uint4 v[8];
      auto put = [&](const CodecDev& cd, const uint8_t* rec, int x) {
        const uint32_t s = q % kPwSlots;
        mbar_wait_idle(&ms.empty[s], ((q / kPwSlots) & 1) ^ 1, abort_f);
        unsigned char* st = sm + C::RING + s * 16384;
#pragma unroll
        for (int k = 0; k < 8; ++k) *reinterpret_cast<uint4*>(st + sw128_off(32 * w + 4 * k + (lane >> 3), lane & 7)) = v[k];
        if (cd.has_outl) patch_chunk<D>(cd, rec, grp + 4 * x, st, w, lane);
        fence_async_smem();  // before the next loads, which it would wait for
        __syncwarp();
        if (lane == 0) mbar_arrive(&ms.full[s]);
        q += 4;
      };
      decode_chunk_b(kbits, kx[0], kpl, klut, v, lane);
#pragma unroll 1
      for (int i = 0; i < n; ++i) {
        const bool more = i + 1 < n;
        const uint8_t* knext = more ? rec_at(true, c0 + i + 1) : krec;
        const uint8_t* vnext = one || !more ? vrec : rec_at(false, c0 + i + 1);
#pragma unroll
        for (int x = 0; x < PER; ++x) {
          put(p.kc, krec, x);
          if (more) load_chunk_b<D>(kbits, knext + kat + 32 * x * kbits, kx[x]);
          if (x + 1 < PER) decode_chunk_b(kbits, kx[x + 1 < PER ? x + 1 : 0], kpl, klut, v, lane);
        }
        if (!one) {
          decode_chunk_b(vbits, vx[0], vpl, vlut, v, lane);
#pragma unroll
          for (int x = 0; x < PER; ++x) {
            put(p.vc, vrec, x);
            if (more) load_chunk_b<D>(vbits, vnext + vat + 32 * x * vbits, vx[x]);
            if (x + 1 < PER) decode_chunk_b(vbits, vx[x + 1 < PER ? x + 1 : 0], vpl, vlut, v, lane);
          }
        }
        if (more) decode_chunk_b(kbits, kx[0], kpl, klut, v, lane);
        krec = knext;
        vrec = vnext;
      }
    }
  } else {
    // ---------------------------------------------------------------- softmax: a thread per token
    const int tok = 32 * warp + lane;
    const uint32_t lrow = (uint32_t)(32 * warp) << 16;
    int low = min(ms.lim[lane], ms.lim[32 + lane]);
#pragma unroll
    for (int m = 16; m; m >>= 1) low = min(low, __shfl_xor_sync(0xffffffffu, low, m));
    const SoftCap cap = make_cap(p.scap, p.iscap);
    const bool capped = p.scap > 0.f;
    float peak = -INFINITY;      // rows' (thread tid < 64) largest logit where references moved
    uint32_t bound0 = 0xFFFFFFFFu, bound1 = 0xFFFFFFFFu;
    bool sunk = false;           // a row's weights have become small and its reference may move down
    float lacc[2] = {0.f, 0.f};  // sums of rows lane and 32 + lane over this warp's tokens
    auto scale_at = [&](bool key, int i) {
      if constexpr (DENSE) return 1.f;
      const float n = __ldg(reinterpret_cast<const float*>(rec_at(key, c0 + i) + (key ? p.kc.off_norm : p.vc.off_norm)) + tok);
      return finite_or_nan(n);
    };
    float nk1 = scale_at(true, 0), nv1 = scale_at(false, 0);
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const float nk = nk1, nv = nv1 * ev;  // the token's scales
      if (i + 1 < n) {
        nk1 = scale_at(true, i + 1);
        nv1 = scale_at(false, i + 1);
      }
      mbar_wait_idle(&ms.s_full, i & 1, abort_f);
      tc_fence_after();
      const int at = i * kChunk + tok;
      const bool edge = (i + 1) * kChunk > low;
      // logits of rows 32 hh .. (log2 units, -inf where the row does not see the token)
      auto logits = [&](int hh, float (&t)[32]) {
        uint32_t a[32];
        tmem_ld32(tS + lrow + 32 * hh, a);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          const float4 f = *reinterpret_cast<const float4*>(&ms.qf[32 * hh + j]);
          t[j] = __uint_as_float(a[j]) * nk * f.x;
          t[j + 1] = __uint_as_float(a[j + 1]) * nk * f.y;
          t[j + 2] = __uint_as_float(a[j + 2]) * nk * f.z;
          t[j + 3] = __uint_as_float(a[j + 3]) * nk * f.w;
        }
        if (capped) {
#pragma unroll
          for (int j = 0; j < 32; ++j) t[j] = cap_logit(t[j], cap);
        }
        if (edge) {
#pragma unroll
          for (int j = 0; j < 32; ++j) t[j] = at < ms.lim[32 * hh + j] ? t[j] : -INFINITY;
        }
      };
      // weights against the references as they stand (the unscaled ones, rounded, are
      // kept for the sums); a logit that passes its reference by the margin (or
      // finds none yet) sends the record to the slow path.  The outputs of the
      // record before are in: the scores were issued behind them.
      uint32_t w[32];
      auto put = [&](int hh, int j, const float2 (&x)[4]) {  // rows 32 hh + j .. + 7
        uint32_t u[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          w[16 * hh + j / 2 + k] = DENSE ? pack2_bf16(x[k].x, x[k].y) : pack2_f16(x[k].x, x[k].y);
          const float2 y = mul2(x[k], f2(nv, nv));
          u[k] = DENSE ? w[16 * hh + j / 2 + k] : pack2_f16(y.x, y.y);
        }
        *reinterpret_cast<uint4*>(sm + C::P + sw128_off(tok, 4 * hh + j / 8)) = make_uint4(u[0], u[1], u[2], u[3]);
      };
      float over = -INFINITY;
      const bool plain = !edge && !cap.large;
      if (plain && !capped) {
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          uint32_t a[32];
          tmem_ld32(tS + lrow + 32 * hh, a);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 32; j += 8) {
            float2 x[4];
#pragma unroll
            for (int k = 0; k < 4; k += 2) {
              const float4 f = *reinterpret_cast<const float4*>(&ms.qf[32 * hh + j + 2 * k]);
              const float4 r = *reinterpret_cast<const float4*>(&ms.ref[32 * hh + j + 2 * k]);
              const float2 A = mul2(f2(__uint_as_float(a[j + 2 * k]), __uint_as_float(a[j + 2 * k + 1])), f2(nk, nk));
              const float2 B = mul2(f2(__uint_as_float(a[j + 2 * k + 2]), __uint_as_float(a[j + 2 * k + 3])), f2(nk, nk));
              x[k] = fma2(A, f2(f.x, f.y), f2(-r.x, -r.y));
              x[k + 1] = fma2(B, f2(f.z, f.w), f2(-r.z, -r.w));
              over = max3(max3(over, x[k].x, x[k].y), x[k + 1].x, x[k + 1].y);
              x[k] = f2(ex2(x[k].x), ex2(x[k].y));
              x[k + 1] = f2(ex2(x[k + 1].x), ex2(x[k + 1].y));
            }
            put(hh, j, x);
          }
        }
      } else if (plain) {
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          uint32_t a[32];
          tmem_ld32(tS + lrow + 32 * hh, a);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 32; j += 8) {
            float2 x[4];
#pragma unroll
            for (int k = 0; k < 4; k += 2) {
              const float4 f = *reinterpret_cast<const float4*>(&ms.qf[32 * hh + j + 2 * k]);
              const float4 r = *reinterpret_cast<const float4*>(&ms.ref[32 * hh + j + 2 * k]);
              const float2 A = mul2(f2(__uint_as_float(a[j + 2 * k]), __uint_as_float(a[j + 2 * k + 1])), f2(nk, nk));
              const float2 B = mul2(f2(__uint_as_float(a[j + 2 * k + 2]), __uint_as_float(a[j + 2 * k + 3])), f2(nk, nk));
              const float2 a2 = mul2(A, f2(f.x, f.y)), b2 = mul2(B, f2(f.z, f.w));
              x[k] = f2(cap_near(a2.x, cap) - r.x, cap_near(a2.y, cap) - r.y);
              x[k + 1] = f2(cap_near(b2.x, cap) - r.z, cap_near(b2.y, cap) - r.w);
              over = max3(max3(over, x[k].x, x[k].y), x[k + 1].x, x[k + 1].y);
              x[k] = f2(ex2(x[k].x), ex2(x[k].y));
              x[k + 1] = f2(ex2(x[k + 1].x), ex2(x[k + 1].y));
            }
            put(hh, j, x);
          }
        }
      }
      if (bar_soft_or(!plain || over > kPfMargin || sunk)) {
        // new references for the rows that passed theirs; their outputs and sums rescaled
#pragma unroll 1
        for (int hh = 0; hh < 2; ++hh) {
          float t[32];
          logits(hh, t);
          ms.red[warp][32 * hh + lane] = transpose_reduce32<true>(t, lane);
        }
        bar_soft();
        float sc = 1.f, mn = 0.f;
        if (tid < 64) {
          const float mx = fmaxf(fmaxf(ms.red[0][tid], ms.red[1][tid]), fmaxf(ms.red[2][tid], ms.red[3][tid]));
          const float mo = ms.ref[tid];
          peak = fmaxf(peak, mx);
          const bool up = mx > mo + kPfMargin;
          const bool down = !DENSE && mx < mo + kPfLow && mx > -INFINITY && mo > peak - kPfFloor;
          mn = !(up || down) ? mo : fmaxf(mx - kPfTop, peak - kPfFloor);
          sc = mo > -INFINITY ? ex2(mo - mn) : mn > -INFINITY ? 0.f : 1.f;
          const uint32_t stays = __ballot_sync(0xffffffffu, !(mn > peak - kPfFloor));
          if (lane == 0) ms.bound[warp] = stays;
        }
        bar_soft();
        if (tid < 64) {
          ms.ref[tid] = mn;
          ms.red[0][tid] = sc;
        }
        bar_soft();
        bound0 = ms.bound[0];
        bound1 = ms.bound[1];
        lacc[0] *= ms.red[0][lane];
        lacc[1] *= ms.red[0][32 + lane];
        if (i > 0) {
#pragma unroll 1
          for (int j = 0; j < 2 * NBL; ++j) {  // block j / 2, rows 32 (j % 2) ..
            uint32_t o[32];
            tmem_ld32(tO + lrow + 32 * j, o);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * ms.red[0][32 * (j & 1) + k]);
            tmem_st32(tO + lrow + 32 * j, o);
          }
          tmem_st_wait();
        }
        bar_soft();  // the factors are read before the reductions' space is used again
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          float t[32];
          logits(hh, t);
#pragma unroll
          for (int j = 0; j < 32; j += 8) {
            float2 x[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 r = *reinterpret_cast<const float2*>(&ms.ref[32 * hh + j + 2 * k]);
              x[k] = f2(ex2(t[j + 2 * k] - (r.x > -INFINITY ? r.x : 0.f)), ex2(t[j + 2 * k + 1] - (r.y > -INFINITY ? r.y : 0.f)));
            }
            put(hh, j, x);
          }
        }
      }
      fence_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms.p_full);
      // the sums, of the weights as rounded, while the outputs are multiplied
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        float t[32];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const uint32_t v = w[16 * hh + j];
          const float2 x = DENSE ? f2(bf16_lo(v), bf16_hi(v)) : __half22float2(*reinterpret_cast<const __half2*>(&v));
          t[2 * j] = x.x;
          t[2 * j + 1] = x.y;
        }
        const float sum = transpose_reduce32<false>(t, lane);
        lacc[hh] += sum;
        if (!DENSE) {
          const uint32_t m = __ballot_sync(0xffffffffu, sum < exp2f(kPfLow));
          if (lane == 0) reinterpret_cast<uint32_t*>(&ms.small[i & 1][hh])[warp] = m;
        }
      }
      if (!DENSE && i > 0) {  // the record before: its words are behind this one's barrier
        const uint4 x = ms.small[(i - 1) & 1][0], y = ms.small[(i - 1) & 1][1];
        sunk = ((x.x & x.y & x.z & x.w & ~bound0) | (y.x & y.y & y.z & y.w & ~bound1)) != 0;
      }
    }
    mbar_wait_idle(&ms.o_done, (n - 1) & 1, abort_f);
    tc_fence_after();
    ms.red[warp][lane] = lacc[0];
    ms.red[warp][32 + lane] = lacc[1];
    bar_soft();
    const float un = DENSE ? 1.f : pow2i(-15) * (1.f / ev);
#pragma unroll 1
    for (int j = 0; j < 2 * NBL; ++j) {
      uint32_t o[32];
      tmem_ld32(tO + lrow + 32 * j, o);
      tmem_ld_wait();
      const int rb = 32 * (j & 1);
      float* dst = pp.ws_acc + ((wrow + rb) * S + sidx) * D + 128 * (j >> 1) + tok;
#pragma unroll
      for (int k = 0; k < 32; ++k)
        if (rb + k < rn) dst[(int64_t)k * S * D] = __uint_as_float(o[k]) * un;
    }
    if (tid < rn) {
      const float bad = __int_as_float(0x7fc00000);
      const float sum = (ms.red[0][tid] + ms.red[1][tid]) + (ms.red[2][tid] + ms.red[3][tid]);
      pp.ws_ml[(wrow + tid) * S + sidx] =
          *abort_f || sum != sum ? make_float2(bad, bad) : sum > 0.f ? make_float2(ms.ref[tid], sum) : make_float2(-INFINITY, 0.f);
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == kPwIssue) {
    volatile int drain = 0;  // every MMA has completed, whatever the abort flag says
    mbar_wait_idle(&ms.fin, 0, &drain);
    tc_fence_after();
    tmem_dealloc(ms.tbase, 512);
  }
}

template <int D>
__global__ void __launch_bounds__(kPwThreads, 1) prefill_wide_kernel(const __grid_constant__ PrefillParams pp) {
  pdl_start();
  extern __shared__ __align__(1024) unsigned char smraw[];
  unsigned char* sm = smraw + ((1024u - (smem_u32(smraw) & 1023u)) & 1023u);
  const int64_t U = (int64_t)pp.q.L * pp.q.B * pp.q.Hkv * pp.tiles;
  const int split = (int)(blockIdx.x / U), tile = (int)(blockIdx.x % U % pp.tiles);
  const int64_t unit = blockIdx.x % U / pp.tiles;
  if (split < pp.Sc) prefill_wide_body<D, false>(pp, sm, unit, tile, split);
  else prefill_wide_body<D, true>(pp, sm, unit, tile, split - pp.Sc);
}

template <int D>
cudaError_t prefill_wide_launch(const PrefillParams& pp, cudaStream_t s) {
  if (pp.Sc + pp.St == 0) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(prefill_wide_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, PwCfg<D>::SMEM);
  if (e != cudaSuccess) return e;
  const int64_t grid = (int64_t)pp.q.L * pp.q.B * pp.q.Hkv * pp.tiles * (pp.Sc + pp.St);
  prefill_wide_kernel<D><<<(unsigned)grid, kPwThreads, PwCfg<D>::SMEM, s>>>(pp);
  return cudaGetLastError();
}

}  // namespace tq
