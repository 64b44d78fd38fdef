// Attention of several query tokens per sequence over records and ring: what
// its kernels (prefill_umma.cuh, prefill_umma_wide.cuh) and the merge of
// their context splits (prefill_merge.cu) share.
//
// The query rows of a kv head are its query heads x new tokens, row = token *
// G + head, so that a tile of rows shares the keys it reads whatever the group
// size.  Packed codes become f16 operands in shared memory (centroids x 2^15,
// so that side-list values up to 1 fit and no centroid is subnormal).  Rounding
// to f16 (11 bits) of rotated queries, centroids, scales and weights is finer
// than the bf16 output's 8; softmax statistics and outputs accumulate in f32.
// O stays in the rotated basis; the merge of the splits turns it back once.
#pragma once

#include "attn_mass.cuh"

namespace tq {

struct PrefillParams {
  QueryParams q;
  int Sc, St, cps, tps;  // splits over records / ring tokens; records, ring tokens per split
  int rows, tiles;       // query rows of a unit, row tiles
  float* ws_acc;         // partial outputs and statistics (layouts: the kernels)
  float2* ws_ml;
  uint16_t* out;
  int64_t o_ls, o_bs, o_ts;
  float inv_sqrt_d;
  // listed records (tq_sparse_attn; q_block 0: every record).  A block of q_block
  // tokens shares a list; its rows make sub row tiles, tiles = blocks * sub.
  const int32_t* list;
  const int32_t* list_count;
  int list_stride, q_block, sub;
  bool ring_first;  // the ring's CTAs before the records' (head dims 64 and 128)
  // few rows: runs of the lists' entries (cps each) and of the rings' tiles of 128 tokens (tps each, ring a list)
  int rec_runs, ring_runs, ring;
};

// The records of a row tile's split: c0, c0 + 1, .., or (LISTED) the entries c0,
// c0 + 1, .. of its list, of which those that name no record stand for the run's
// first that does (its values are finite, as weights of zero need them) with no token seen.
struct RecordRun {
  const int32_t* list;
  int c0, n, stand;  // first record or entry; records of the sequence; what entries that name none stand for
};
// the first of entries c0 .. c1 - 1 that names a record; -1 where there is none.  By whole warps.
__device__ __forceinline__ int first_entry(const RecordRun& r, int c1) {
  const int lane = threadIdx.x & 31;
  for (int c = r.c0; c < c1; c += 32) {
    const int v = c + lane < c1 ? __ldg(r.list + c + lane) : -1;
    const uint32_t m = __ballot_sync(0xffffffffu, v >= 0 && v < r.n);
    if (m) return __shfl_sync(0xffffffffu, v, __ffs((int)m) - 1);
  }
  return -1;
}
template <bool LISTED>
__device__ __forceinline__ int run_entry(const RecordRun& r, int i) {
  return LISTED ? __ldg(r.list + r.c0 + i) : r.c0 + i;
}
template <bool LISTED>
__device__ __forceinline__ int run_record(const RecordRun& r, int i) {
  const int e = run_entry<LISTED>(r, i);
  return LISTED && (e < 0 || e >= r.n) ? r.stand : e;
}
// of entry i's 128 tokens, those below `lim` (a row's limit in the sequence), counted from the record's first
__device__ __forceinline__ int listed_seen(const RecordRun& r, int i, int lim) {
  const int e = run_entry<true>(r, i);
  return e < 0 || e >= r.n ? 0 : lim - e * kChunk;
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

// The soft cap of a logit in log2 units, C tanh(t / C) = C - 2 C / (1 + 2^(t k)),
// k = 2 log2(e) / C: off by at most 2^-21 C (about half an ulp of each of 2^x, the
// sum and the quotient), under 2^-13 for C up to 256, where a weight keeps 11
// bits.  Larger caps go through tanhf.  (1024 tokens over 32768 cached with a cap
// of 20: 952 us, at an earlier stage 970 against 3085 through tanhf; without a cap 550.)
struct SoftCap {
  float k, c, m2c, ic;
  bool large;
};
__device__ __forceinline__ SoftCap make_cap(float C, float iC) {
  return SoftCap{2.885390081777927f * iC, C, -2.f * C, iC, C > 256.f};
}
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float cap_near(float t, const SoftCap& s) {
  return fmaf(s.m2c, rcp_approx(1.f + ex2(t * s.k)), s.c);
}
__device__ __forceinline__ float cap_logit(float t, const SoftCap& s) {
  return s.large ? soft_cap(t, s.c, s.ic) : cap_near(t, s);
}

}  // namespace tq
