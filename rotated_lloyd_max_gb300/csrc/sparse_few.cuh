// Attention over listed records and the ring for at most 16 query rows a list
// (query heads of a kv head x tokens of a block), head dims 64 and 128, codecs
// without side lists: the decode step of a long cache.
//
// The lists' entries, one list after the other, are cut into equal runs, and so are
// the rings' tiles behind them; a run is worked off by a team of four warps, which
// has parts of one or more lists, each a partial for the merge.  A CTA per SM holds
// four teams that share nothing but the lookup tables, so that one team's set-up,
// first loads and joining of its warps run under the others' records.  A warp takes
// 32 tokens of a record and copies its tokens of the next record but one into shared
// memory while it works (cp.async, two stages): no barrier between records.
//
// Tokens are the M dimension of the scores (K q~^T, rows as N), coordinates that of
// the outputs (V^T p), so that 8 rows fill the N of mma.sync and both operands A are
// decoded from the packed codes straight into registers: a lane holds d / 4
// neighbouring codes of four keys, and d / 8 codes of eight values, paired by token
// before the lookup (3-bit codes after it).  Every pair of codes is one lookup in a
// table with a copy per lane (no bank conflicts).
//
// Centroids and rotated queries are f16 (11 bits), logits take the key's scale and
// sums in f32.  A weight enters times its value's scale, relative to the running
// maxima of both and 2^14 above f16's 1: what lies within 2^-28 of the largest
// keeps 11 bits, so that a token with nearly all of a row's weight leaves the
// others theirs.  The ring's weights are two bf16 (16 bits) against exact values.
//
// 32 of 256 records (4 and 3 bits) + 144 tokens of 32 sequences, 8 kv heads of 4: 51.7 us, of which the
// merge 5; 145 MB at 2.8 TB/s.  Issue 63%, shared memory 55% and ALU 56% of what they can: the lookups.
#pragma once

#include "packed_run.cuh"
#include "prefill.cuh"

namespace tq {

// teams of a CTA: four of up to 8 rows; two of 16, whose accumulators take 255 registers a
// thread (four with 128 spill: 256 records of 32 sequences, 4 kv heads of 16: 433 us, 237 with two)
constexpr int few_teams(int rows) { return rows <= 8 ? 4 : 2; }
__device__ __forceinline__ void team_sync() { asm volatile("bar.sync %0, 128;" ::"r"(1 + (int)(threadIdx.x >> 7)) : "memory"); }

constexpr int kFewIds = 256;  // records that are listed at a time

template <int D, int KB, int VB, int NT>
struct FewCfg {
  static constexpr int KTAB = (1 << (2 * KB)) * 128, VTAB = (1 << (2 * VB)) * 128;
  // of a team:
  static constexpr int QF = 0, QFB = D / 16 * NT * 32 * 8;
  static constexpr int IDS = QF + QFB, MISC = IDS + kFewIds * 4;
  static constexpr int MISCB = 8 * NT * 8 + 64, ML = MISC + MISCB;
  static constexpr int STAGE = ML + 4 * 8 * NT * 8;  // two a warp: 32 keys, 32 values, their scales
  static constexpr int VAT = 32 * (D * KB / 8), NAT = VAT + 32 * (D * VB / 8), STAGEB = NAT + 256;
  static constexpr int RED = 4 * 8 * (D + D / 8) * 4;  // in the stages' place: the warps' outputs of eight rows
  static constexpr int TEAM = STAGE + (8 * STAGEB > RED ? 8 * STAGEB : RED);
  static constexpr int TEAMS = few_teams(8 * NT), THREADS = 128 * TEAMS, SMEM = KTAB + VTAB + TEAMS * TEAM;
  static_assert(STAGE % 16 == 0 && STAGEB % 16 == 0 && TEAM % 16 == 0 && SMEM <= 232448, "one CTA per SM");
};

// Where 16-byte chunk c of a row lies in a warp's 32 rows: rows of 64 bytes two to a line of 128, in which the
// chunks move on by two from line to line, so that the eight lanes of a key's and the sixteen of a value's
// access meet no bank twice; other rows one behind the other.
template <int ROW>
__device__ __forceinline__ int few_chunk(int i) {
  if constexpr (ROW == 64) {
    const int line = i >> 3;
    return line * 128 + (((i & 7) + 2 * line) & 7) * 16;
  }
  return 16 * i;
}

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// A warp's softmax state: rows 8 nt + 2 t + e, and its outputs: coordinates
// (d / 8) g + 2 mc (+ 1 for elements 2, 3), rows 2 t (+ 1 for odd elements).
template <int D, int NT>
struct FewState {
  float m[NT][2], l[NT][2];
  float acc[NT][D / 16][4];
  int ev;  // exponent of the largest value scale so far

  __device__ __forceinline__ void init() {
    ev = -100;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[nt][e] = -INFINITY;
        l[nt][e] = 0.f;
      }
#pragma unroll
      for (int mc = 0; mc < D / 16; ++mc)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[nt][mc][e] = 0.f;
    }
  }
  // x[mi][nt][2 half + e]: logits (log2 units) of token 16 mi + 8 half + g.  New maxima where a row's logits pass
  // the old one by more than 1 (weights of up to 2 spare a rescaling); grow: what the values' scales ask of the outputs.
  template <int MI>
  __device__ __forceinline__ void raise(const float (&x)[MI][NT][4], float grow) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float f[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float v = fmaxf(x[0][nt][e], x[0][nt][2 + e]);
#pragma unroll
        for (int mi = 1; mi < MI; ++mi) v = fmaxf(v, fmaxf(x[mi][nt][e], x[mi][nt][2 + e]));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
        const bool up = v > m[nt][e] + 1.f;
        f[e] = up ? ex2(m[nt][e] - v) : 1.f;
        if (up) m[nt][e] = v;
        l[nt][e] *= f[e];
        f[e] *= grow;
      }
#pragma unroll
      for (int mc = 0; mc < D / 16; ++mc)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[nt][mc][e] *= f[e & 1];
    }
  }
  __device__ __forceinline__ float ref(int nt, int e) const { return m[nt][e] > -INFINITY ? m[nt][e] : 0.f; }
  // logits less their rows' references become weights
  template <int MI>
  __device__ __forceinline__ void weigh(float (&x)[MI][NT][4]) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int mi = 0; mi < MI; ++mi) {
          x[mi][nt][e] = ex2(x[mi][nt][e]);
          x[mi][nt][2 + e] = ex2(x[mi][nt][2 + e]);
          l[nt][e] += x[mi][nt][e] + x[mi][nt][2 + e];
        }
  }
};

// The records of a split.
template <int D, int KB, int VB, int NT>
__device__ __forceinline__ void few_records(const PrefillParams& pp, const unsigned char* tables, unsigned char* sm, const int* ids, int n, int l, int b,
                                            int h, const float* qf, const int* lim, int low, FewState<D, NT>& st) {
  using C = FewCfg<D, KB, VB, NT>;
  constexpr int KS = D / 16, KR = D / 4, VR = D / 8, KNB = KR * KB, VNB = VR * VB;
  constexpr int KROW = D * KB / 8, VROW = D * VB / 8, VNW = Run<VNB>::NW;
  const QueryParams& p = pp.q;
  const int lane = threadIdx.x & 31, w4 = (threadIdx.x >> 5) & 3, g = lane >> 2, t = lane & 3;
  const uint32_t loff = lane * 4;
  const unsigned char *ktab = tables, *vtab = tables + C::KTAB;
  const ByteTable kbt = byte_table(ktab, loff, 128), vbt = byte_table(vtab, loff, 128);
  const uint2* qfrag = reinterpret_cast<const uint2*>(sm + C::QF) + lane;
  float nk[4], nv[4];
  // contiguous records follow one another behind a base; pages are looked up
  const int32_t* table = p.table ? p.table + (int64_t)b * p.table_stride : nullptr;
  const int64_t unit = table ? (int64_t)h : ((int64_t)b * p.Hkv + h) * p.rec_cap;
  const int kstep = (table ? p.Hkv : 1) * p.kc.rec_bytes, vstep = (table ? p.Hkv : 1) * p.vc.rec_bytes;
  const uint8_t* kbase = p.krec + l * p.krec_ls + unit * p.kc.rec_bytes + 32 * w4 * KROW + 16 * lane;
  const uint8_t* vbase = p.vrec + l * p.vrec_ls + unit * p.vc.rec_bytes + 32 * w4 * VROW + 16 * lane;
  const int norm = (lane < 8 ? p.kc.off_norm - 32 * w4 * KROW : p.vc.off_norm - 32 * w4 * VROW - 128) + 128 * w4;
  unsigned char* stages = sm + C::STAGE + w4 * 2 * C::STAGEB;
  // the warp's tokens of entry i into a stage
  auto ask = [&](int i, int s) {
    const int e = ids[i], c = table ? min(max(__ldg(table + e), 0), p.rec_cap - 1) : e;
    unsigned char* st_ = stages + s * C::STAGEB;
    const uint8_t *k = kbase + (int64_t)c * kstep, *v = vbase + (int64_t)c * vstep;
#pragma unroll
    for (int j = 0; j < 2 * KROW; j += 32)
      if (j + 32 <= 2 * KROW || j + lane < 2 * KROW) cp_async16(st_ + few_chunk<KROW>(j + lane), k + 16 * j);
#pragma unroll
    for (int j = 0; j < 2 * VROW; j += 32)
      if (j + 32 <= 2 * VROW || j + lane < 2 * VROW) cp_async16(st_ + C::VAT + few_chunk<VROW>(j + lane), v + 16 * j);
    if (lane < 16) cp_async16(st_ + C::NAT + 16 * lane, (lane < 8 ? k : v) + norm);
  };
  // a key's run of codes: token 8 i + g, run t; a value's: token 16 mt + 2 t + {0, 1, 8, 9}, run g
  const int kat = KROW == 64 ? (g >> 1) * 128 + (((g & 1) * 4 + t + 2 * (g >> 1)) & 7) * 16 : g * KROW;
  auto key_run = [&](const unsigned char* st_, int i, uint32_t (&w)[Run<KNB>::NW]) {
    Run<KNB> r;
    if constexpr (KROW == 64) r.fetch(st_ + kat + 512 * i, 0);
    else r.fetch(st_ + kat + 8 * i * KROW, KNB * t);
    r.get(KNB * t, w);
  };
  auto value_run = [&](const unsigned char* st_, int mt, int k, uint32_t (&w)[VNW]) {
    Run<VNB> r;
    if constexpr (VROW == 64)
      r.fetch(st_ + C::VAT + (8 * mt + t + 4 * (k >> 1)) * 128 + (((k & 1) * 4 + (g >> 1) + 2 * t) & 7) * 16 + (g & 1) * 8, 0);
    else r.fetch(st_ + C::VAT + (16 * mt + 2 * t + (k & 1) + 8 * (k >> 1)) * VROW, VNB * g);
    r.get(VNB * g, w);
  };
  const bool capped = p.scap > 0.f;
  float f[NT][2], rf[NT][2];  // logit factors and references of the lane's rows
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      f[nt][e] = qf[8 * nt + 2 * t + e];
      rf[nt][e] = 0.f;
    }
  bool none = true;  // a row has no reference yet
  float reach = 0.f, up = 0.f;  // scales that the exponent of the values' covers; 2^14 2^-(ev + 1)
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    if (s < n) ask(s, s);
    cp_async_commit();
  }
#pragma unroll 1
  for (int i = 0, s = 0; i < n; ++i, s ^= 1) {
    cp_async_wait<1>();
    __syncwarp();
    const unsigned char* stage = stages + s * C::STAGEB;
    // ---------------------------------------------------------------- scores
    float x[2][NT][4];
#pragma unroll
    for (int mi = 0; mi < 2; ++mi)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[mi][nt][e] = 0.f;
    {
      uint32_t w[4][Run<KNB>::NW];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        key_run(stage, k, w[k]);
        nk[k] = finite_or_nan(reinterpret_cast<const float*>(stage + C::NAT)[8 * k + g]);
      }
#pragma unroll
      for (int kk = 0; kk < KS; ++kk) {
        uint32_t a[2][4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int o = 4 * kk + 2 * e;
            uint32_t v;
            if constexpr (KB == 4) v = byte_lookup(kbt, w[k][o / 8], o % 8 / 2);
            else v = *reinterpret_cast<const uint32_t*>(ktab + pair_off(w[k], o * KB, 2 * KB, loff));
            a[k >> 1][(k & 1) + 2 * e] = v;
          }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint2 q = qfrag[(kk * NT + nt) * 32];
          mma_f16(x[0][nt], a[0], q.x, q.y);
          mma_f16(x[1][nt], a[1], q.x, q.y);
        }
      }
    }
    // ---------------------------------------------------------------- weights
    // against the references as they stand, unless a row has none, a logit passes its by more than 1, a value's
    // scale the exponent, a row does not see a token, or logits are capped
    const int token = ids[i] * kChunk + 32 * w4 + g;  // of k = 0
    const bool edge = (ids[i] + 1) * kChunk > low;
    float over = -INFINITY, big = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      nv[k] = reinterpret_cast<const float*>(stage + C::NAT)[32 + 8 * k + g];
      big = fmaxf(big, fabsf(nv[k]));
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float& v = x[k >> 1][nt][2 * (k & 1) + e];
          v = fmaf(v, nk[k] * f[nt][e], -rf[nt][e]);
          over = fmaxf(over, v);
        }
    }
    if (__any_sync(0xffffffffu, over > 1.f || big >= reach || edge || none)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float& v = x[k >> 1][nt][2 * (k & 1) + e];
            v += rf[nt][e];
            if (capped) v = soft_cap(v, p.scap, p.iscap);
            if (edge) v = token + 8 * k < lim[8 * nt + 2 * t + e] ? v : -INFINITY;
          }
      const int en = exp_of(__uint_as_float(__reduce_max_sync(0xffffffffu, big < INFINITY ? __float_as_uint(big) : 0u)));
      float grow = 1.f;
      if (en > st.ev) {
        grow = pow2i(st.ev - en);
        st.ev = en;
      }
      reach = pow2i(st.ev + 1);
      up = pow2i(13 - st.ev);
      st.raise(x, grow);
      none = capped;  // capped logits take this way always
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          none = none || st.m[nt][e] == -INFINITY;
          rf[nt][e] = capped ? 0.f : st.ref(nt, e);
#pragma unroll
          for (int k = 0; k < 4; ++k) x[k >> 1][nt][2 * (k & 1) + e] -= st.ref(nt, e);
        }
    }
    st.weigh(x);
#pragma unroll
    for (int k = 0; k < 4; ++k) nv[k] *= up;
    // ---------------------------------------------------------------- values
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      uint32_t b0[NT], b1[NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        b0[nt] = transpose8(pack2_f16(x[mt][nt][0] * nv[2 * mt], x[mt][nt][1] * nv[2 * mt]));
        b1[nt] = transpose8(pack2_f16(x[mt][nt][2] * nv[2 * mt + 1], x[mt][nt][3] * nv[2 * mt + 1]));
      }
      if constexpr (VB == 3) {
        // a field of two 3-bit codes would have to be put together for two tokens: cheaper to look up each
        // token's pairs of neighbours and to pair the results (8 instructions for two operands; 12)
        uint32_t r[4][VNW];
#pragma unroll
        for (int k = 0; k < 4; ++k) value_run(stage, mt, k, r[k]);
#pragma unroll
        for (int mc = 0; mc < KS; ++mc) {
          uint32_t y[4], a[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) y[k] = *reinterpret_cast<const uint32_t*>(vtab + pair_off(r[k], mc * 6, 6, loff));
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            a[2 * k] = __byte_perm(y[2 * k], y[2 * k + 1], 0x5410);
            a[2 * k + 1] = __byte_perm(y[2 * k], y[2 * k + 1], 0x7632);
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_f16(st.acc[nt][mc], a, b0[nt], b1[nt]);
        }
      } else {
        uint32_t z[4][VNW];  // even and odd coordinates of tokens 2 t, 2 t + 1; of 2 t + 8, 2 t + 9
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t r0[VNW], r1[VNW];
          value_run(stage, mt, 2 * k, r0);
          value_run(stage, mt, 2 * k + 1, r1);
          v_pair_words<VB, VNW>(r0, r1, z[2 * k], z[2 * k + 1]);
        }
#pragma unroll
        for (int mc = 0; mc < KS; ++mc) {
          uint32_t a[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if constexpr (VB == 4) a[k] = byte_lookup(vbt, z[k][mc / 4], mc % 4);
            else a[k] = *reinterpret_cast<const uint32_t*>(vtab + pair_off(z[k], mc * 2 * VB, 2 * VB, loff));
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_f16(st.acc[nt][mc], a, b0[nt], b1[nt]);
        }
      }
    }
    __syncwarp();  // the stage has been read
    if (i + 2 < n) ask(i + 2, s);
    cp_async_commit();
  }
  cp_async_wait<0>();
}

// The ring's tokens [k0, k1) of a split: a warp takes 16 at a time, whose keys and values are asked for together.
template <int D, int NT>
__device__ __forceinline__ void few_ring(const PrefillParams& pp, const uint2* qfrag, int k0, int k1, int len, int l, int b,
                                         int h, int start, const float* qf, const int* lim, int low, FewState<D, NT>& st) {
  constexpr int KS = D / 16, KR = D / 4, VR = D / 8;
  const QueryParams& p = pp.q;
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3, g = lane >> 2, t = lane & 3;
  const int64_t ring = l * p.tail_ls + (int64_t)(b * p.Hkv + h) * p.tail_cap * D;
  const uint16_t *kt = p.ktail + ring, *vt = p.vtail + ring;
  // clamped to the last token: its values are finite, its weights zero
  auto row = [&](int tok) {
    uint32_t s = (uint32_t)start + (uint32_t)min(tok, len - 1);  // (up to twice the capacity: 32 bits)
    if (s >= (uint32_t)p.tail_cap) s -= (uint32_t)p.tail_cap;
    return (int64_t)s * D;
  };
#pragma unroll 1
  for (int a0 = k0 + 16 * warp; a0 < k1; a0 += 64) {
    uint4 kw[2][KS / 2], vw[4][VR / 8];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4* r = reinterpret_cast<const uint4*>(kt + row(a0 + 8 * i + g) + KR * t);
#pragma unroll
      for (int k = 0; k < KS / 2; ++k) kw[i][k] = __ldg(r + k);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {  // tokens 2 t + {0, 1, 8, 9}
      const uint4* r = reinterpret_cast<const uint4*>(vt + row(a0 + 2 * t + (k & 1) + 8 * (k >> 1)) + VR * g);
#pragma unroll
      for (int j = 0; j < VR / 8; ++j) vw[k][j] = __ldg(r + j);
    }
    float x[1][NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[0][nt][e] = 0.f;
#pragma unroll
    for (int k = 0; k < KS / 2; ++k) {
      const uint32_t a[2][4] = {{kw[0][k].x, kw[1][k].x, kw[0][k].y, kw[1][k].y}, {kw[0][k].z, kw[1][k].z, kw[0][k].w, kw[1][k].w}};
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint2 q = qfrag[((2 * k + j) * NT + nt) * 32 + lane];
          mma_bf16(x[0][nt], a[j], q.x, q.y);
        }
    }
    const bool edge = a0 + 16 > low;
    float over = -INFINITY;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float f = qf[8 * nt + 2 * t + e];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float& v = x[0][nt][2 * k + e];
          v *= f;
          if (p.scap > 0.f) v = soft_cap(v, p.scap, p.iscap);
          if (edge) v = a0 + 8 * k + g < lim[8 * nt + 2 * t + e] ? v : -INFINITY;
          over = fmaxf(over, v - st.m[nt][e]);
        }
      }
    if (__any_sync(0xffffffffu, over > 1.f)) st.raise(x, 1.f);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int k = 0; k < 2; ++k) x[0][nt][2 * k + e] -= st.ref(nt, e);
    st.weigh(x);
    uint32_t bh[2][NT], bl[2][NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float u = x[0][nt][2 * k], v = x[0][nt][2 * k + 1];
        const uint32_t hi = pack2_bf16(u, v);
        bh[k][nt] = transpose8(hi);
        bl[k][nt] = transpose8(pack2_bf16(u - bf16_lo(hi), v - bf16_hi(hi)));
      }
#pragma unroll
    for (int mc = 0; mc < KS; ++mc) {
      auto at = [&](int k) { return mc % 4 == 0 ? vw[k][mc / 4].x : mc % 4 == 1 ? vw[k][mc / 4].y : mc % 4 == 2 ? vw[k][mc / 4].z : vw[k][mc / 4].w; };
      const uint32_t a[4] = {__byte_perm(at(0), at(1), 0x5410), __byte_perm(at(0), at(1), 0x7632),
                             __byte_perm(at(2), at(3), 0x5410), __byte_perm(at(2), at(3), 0x7632)};
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        mma_bf16(st.acc[nt][mc], a, bh[0][nt], bh[1][nt]);
        mma_bf16(st.acc[nt][mc], a, bl[0][nt], bl[1][nt]);
      }
    }
  }
}

// One list's part of a team's run: entries [k0, k1) of it, or (dense) tiles of 128 ring tokens.
// split: the partial's place of the list's `slots`; the first one marks those behind the list's last one as empty.
template <int D, int KB, int VB, int NT>
__device__ __forceinline__ void few_segment(const PrefillParams& pp, const unsigned char* tables, unsigned char* sm, bool dense, int64_t x, int k0, int k1,
                                            int split, int last, int slots) {
  using C = FewCfg<D, KB, VB, NT>;
  constexpr int R = 8 * NT, E = D / 32, KR = D / 4;
  const QueryParams& p = pp.q;
  int* ids = reinterpret_cast<int*>(sm + C::IDS);
  float* qf = reinterpret_cast<float*>(sm + C::MISC);  // logit factor of a row
  int* lim = reinterpret_cast<int*>(qf + R);           // tokens it sees (dense: of the ring)
  int* head = lim + R;                                 // records of the segment
  float2* wml = reinterpret_cast<float2*>(sm + C::ML); // the warps' statistics
  float* red = reinterpret_cast<float*>(sm + C::STAGE);
  constexpr int WARPS = 4, T = 128;
  const int tid = threadIdx.x & (T - 1), lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int h = (int)(x % p.Hkv), j = (int)(x / p.Hkv % pp.tiles), lb = (int)(x / p.Hkv / pp.tiles), b = lb % p.B, l = lb / p.B;
  const CacheLen cl = cache_len(p, lb);
  const int tb = query_len(p, b);
  const int r0 = j * pp.q_block * p.G, rn = min(pp.q_block, tb - j * pp.q_block) * p.G;
  if (rn <= 0) return;
  const int S = pp.Sc + pp.St;
  const int64_t wrow = ((int64_t)lb * p.Hkv + h) * pp.rows + r0;
  const int base = dense ? cl.n * kChunk : 0, place = (dense ? pp.Sc : 0) + split;
  if (split == 0)  // places that no part of this list fills
    for (int i = tid; i < rn * (slots - 1 - last); i += T)
      pp.ws_ml[(wrow + i % rn) * S + (dense ? pp.Sc : 0) + last + 1 + i / rn] = make_float2(-INFINITY, 0.f);
  int t0 = 0, t1 = 0, n = 0;
  team_sync();  // the segment before is done with what lies in shared memory
  if (dense) {
    t0 = k0 * kChunk;
    t1 = min(min(k1 * kChunk, cl.len), row_limit(p, cl, tb, r0 + rn - 1) - base);
  } else if (warp == 0) {  // the entries that name a record, in their order
    const int cnt = cl.n > 0 ? min(max(__ldg(pp.list_count + x), 0), pp.list_stride) : 0;
    const int c1 = min(k1, cnt);
    int at = 0;
    for (int c = k0; c < c1; c += 32) {
      const int v = c + lane < c1 ? __ldg(pp.list + x * pp.list_stride + c + lane) : -1;
      const bool on = v >= 0 && v < cl.n;
      const uint32_t m = __ballot_sync(0xffffffffu, on);
      if (on) ids[at + __popc(m & ((1u << lane) - 1u))] = v;
      at += __popc(m);
    }
    if (lane == 0) *head = at;
  }
  // ---------------------------------------------------------------- queries: a warp a row
  for (int r = warp; r < R; r += WARPS) {
    const int row = r0 + r;
    float v[E];
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = 0.f;
    if (r < rn) {
      const uint16_t* qp = p.q + l * p.q_ls + b * p.q_bs + (int64_t)(row / p.G) * p.q_ts +
                           (int64_t)(h * p.G + row % p.G) * D + lane * E;
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(qp + e));
        v[e] = bf16_lo(w);
        v[e + 1] = bf16_hi(w);
      }
    }
    float f = p.sscale, sc = 1.f;
    if (!dense) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int c = lane * E + e;
        if ((p.kc.signs[c >> 5] >> (c & 31)) & 1u) v[e] = -v[e];
      }
      fwht_regs<E>(v);
      fwht_lanes<E>(v, lane, 32);
      float mx = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        v[e] *= inv_sqrt_dim<D>();
        mx = fmaxf(mx, fabsf(v[e]));
      }
      mx = warp_max(mx);
      const int s = mx > 0.f ? 13 - exp_of(mx) : 0;  // largest in [2^13, 2^14)
      sc = pow2i(s);
      f *= pow2i(-15 - s);
    }
    if (lane == 0) {
      qf[r] = f;
      lim[r] = r < rn ? row_limit(p, cl, tb, row) - base : 0x7FFFFFFF;
    }
#pragma unroll
    for (int e = 0; e < E; e += 2) {  // coordinate c: lane c / KR's word of k-step (c % KR) / 4
      const int c = lane * E + e, kk = c % KR / 4;
      reinterpret_cast<uint32_t*>(sm + C::QF)[((kk * NT + (r >> 3)) * 32 + (r & 7) * 4 + c / KR) * 2 + (c & 2) / 2] =
          dense ? pack2_bf16(v[e], v[e + 1]) : pack2_f16(v[e] * sc, v[e + 1] * sc);
    }
  }
  team_sync();
  if (!dense) n = *head;
  if (dense ? t0 >= t1 : n == 0) {
    if (tid < rn) pp.ws_ml[(wrow + tid) * S + place] = make_float2(-INFINITY, 0.f);
    return;
  }
  int low = 0x7FFFFFFF;
#pragma unroll
  for (int r = 0; r < R; ++r) low = min(low, lim[r]);
  FewState<D, NT> st;
  st.init();
  if (dense) {
    int start = p.tail_start ? p.tail_start[lb] % p.tail_cap : 0;
    if (start < 0) start += p.tail_cap;
    few_ring<D, NT>(pp, reinterpret_cast<const uint2*>(sm + C::QF), t0, t1, cl.len, l, b, h, start, qf, lim, low, st);
  } else {
    few_records<D, KB, VB, NT>(pp, tables, sm, ids, n, l, b, h, qf, lim, low, st);
  }
  // ---------------------------------------------------------------- the warps' partials: one of the segment
  const float un = dense ? 1.f : pow2i(-15) * pow2i(st.ev - 13);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float s = st.l[nt][e];
#pragma unroll
      for (int m = 4; m < 32; m <<= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
      if (g == 0) wml[warp * R + 8 * nt + 2 * t + e] = make_float2(st.m[nt][e], s);
    }
  constexpr int RS = D + D / 8;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    team_sync();  // stages, or the rows before, are done with
    // element (row r, coordinate c) of a warp at r RS + c + 4 (c / 32) + r / 2: 32 stores, 32 banks
#pragma unroll
    for (int mc = 0; mc < D / 16; ++mc)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int c = D / 8 * g + 2 * mc + (e >> 1), r = 2 * t + (e & 1);
        red[warp * 8 * RS + r * RS + c + 4 * (c >> 5) + (r >> 1)] = st.acc[nt][mc][e] * un;
      }
    team_sync();
    for (int i = tid; i < 8 * D; i += T) {
      const int r = i / D, c = i % D, row = 8 * nt + r;
      if (row >= rn) break;
      float M = -INFINITY, W = 0.f, v = 0.f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) M = fmaxf(M, wml[w * R + row].x);
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        const float2 ml = wml[w * R + row];
        // a NaN sum stays one, whatever the maximum is
        const float f = ml.x > -INFINITY ? ex2(ml.x - M) : ml.y != ml.y ? 1.f : 0.f;
        W = fmaf(f, ml.y, W);
        v = fmaf(f, red[w * 8 * RS + r * RS + c + 4 * (c >> 5) + (r >> 1)], v);
      }
      pp.ws_acc[((wrow + row) * S + place) * D + c] = v;
      if (c == 0) pp.ws_ml[(wrow + row) * S + place] = W != W ? make_float2(W, W) : make_float2(M, W);
    }
  }
}

template <int D, int KB, int VB, int NT>
__global__ void __launch_bounds__(128 * few_teams(8 * NT), 1) sparse_few_kernel(const __grid_constant__ PrefillParams pp) {
  using C = FewCfg<D, KB, VB, NT>;
  const QueryParams& p = pp.q;
  pdl_start();
  extern __shared__ __align__(128) unsigned char sm[];
  {  // pair tables: entry i at 128 i, a copy of four bytes a lane
    constexpr int KM = (1 << KB) - 1, VM = (1 << VB) - 1;
    for (int i = threadIdx.x; i < (1 << (2 * KB)) * 8; i += C::THREADS) {
      const int e = i >> 3;
      const uint32_t v = pack2_f16(p.kc.centroids[e & KM] * kTableScale, p.kc.centroids[e >> KB] * kTableScale);
      reinterpret_cast<uint4*>(sm)[i] = make_uint4(v, v, v, v);
    }
    for (int i = threadIdx.x; i < (1 << (2 * VB)) * 8; i += C::THREADS) {
      const int e = i >> 3;
      const uint32_t v = pack2_f16(p.vc.centroids[e & VM] * kTableScale, p.vc.centroids[e >> VB] * kTableScale);
      reinterpret_cast<uint4*>(sm + C::KTAB)[i] = make_uint4(v, v, v, v);
    }
  }
  __syncthreads();
  // the team's run of all lists' entries (or of all rings' tiles), list by list; the teams of an SM take
  // runs far apart, so that records and ring meet there
  const int team = threadIdx.x >> 7, slot = team * (int)gridDim.x + (int)blockIdx.x;
  const bool dense = slot >= pp.rec_runs;
  if (slot >= pp.rec_runs + pp.ring_runs) return;
  const int64_t U = (int64_t)p.L * p.B * p.Hkv * pp.tiles;
  const int per = dense ? pp.tps : pp.cps, len = dense ? pp.ring : pp.list_stride, slots = dense ? pp.St : pp.Sc;
  const int64_t u0 = (int64_t)(slot - (dense ? pp.rec_runs : 0)) * per, u1 = min(u0 + per, U * len);
  for (int64_t u = u0; u < u1;) {
    const int64_t x = u / len, first = x * len;  // the list, and where its entries begin
    const int k0 = (int)(u - first), k1 = (int)min((int64_t)len, u1 - first);
    const int c = (int)(first / per);  // the run that has its first entry
    few_segment<D, KB, VB, NT>(pp, sm, sm + C::KTAB + C::VTAB + team * C::TEAM, dense, x, k0, k1, (int)(u / per) - c,
                               (int)((first + len - 1) / per) - c, slots);
    u = first + k1;
  }
}

template <int D, int KB, int VB, int NT>
cudaError_t sparse_few_launch_t(const PrefillParams& pp, cudaStream_t s) {
  auto kern = sparse_few_kernel<D, KB, VB, NT>;
  constexpr int smem = FewCfg<D, KB, VB, NT>::SMEM;
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  const int runs = pp.rec_runs + pp.ring_runs;
  constexpr int teams = few_teams(8 * NT);
  kern<<<(unsigned)(runs <= teams * sm_count() ? min(runs, sm_count()) : cdiv(runs, teams)), 128 * teams, smem, s>>>(pp);
  return cudaGetLastError();
}
template <int D, int KB, int VB>
cudaError_t sparse_few_launch_n(const PrefillParams& pp, cudaStream_t s) {
  return pp.q_block * pp.q.G <= 8 ? sparse_few_launch_t<D, KB, VB, 1>(pp, s) : sparse_few_launch_t<D, KB, VB, 2>(pp, s);
}
template <int D, int KB>
cudaError_t sparse_few_launch(const PrefillParams& pp, cudaStream_t s) {
  switch (pp.q.vc.bits) {
    case 1: return sparse_few_launch_n<D, KB, 1>(pp, s);
    case 2: return sparse_few_launch_n<D, KB, 2>(pp, s);
    case 3: return sparse_few_launch_n<D, KB, 3>(pp, s);
    case 4: return sparse_few_launch_n<D, KB, 4>(pp, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace tq
