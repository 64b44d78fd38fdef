// Attention of several query tokens per sequence on the fifth-generation
// tensor cores (tcgen05, accumulators in tensor memory), head dims 64 and 128.
//
// A CTA keeps 256 query rows (two M = 128 tiles; row = token * G + head, so any
// group size fills them) and walks a run of 128-token tiles: records, or the
// ring's tokens.  Scores S = Q~ K^T (A and B from shared memory) and outputs
// O += P V (P from tensor memory, V from shared memory) accumulate in f32:
// columns 0-255 hold S of the two tiles, which the softmax replaces by P in
// half as many, columns 256.. hold O.
//
// Operands of the records are f16: q~ 2^s (s per row), and centroid * scale
// with the token's scale folded in, n 2^-(E+1) with E the exponent of the largest
// scale of the CTA's run (read ahead; values below 2^-24 of the largest round to
// zero), so that a logit needs one multiply-add and a weight none.  A key's scale
// is a sum of two f16: rounded to one, it would be off by up to 2^-12 in all of
// the key's coordinates alike and move a logit of 12 by 3e-3, where the products'
// own roundings average out (outputs' error 2.0e-3, not 2.6e-3, for 5% of the
// time; scaling the f32 scores instead took 23%).  The ring's operands are bf16 as
// they are.
//
// The softmax subtracts a reference that stays while a tile's largest weight lies
// between 2^kPfLow and 2^kPfMargin, so that scores are read once and O is hardly
// ever rescaled (by the warps that own the rows; a warp that rescales holds the
// whole CTA up for about 3000 cycles), and else moves to where that weight is
// 2^kPfTop. Weights are f16: 11 bits down to 2^-14, to within 2^-25 below, so that
// f16 drops at most 128 2^-25 of a tile, 2^-16 of the row's largest weight.  The
// reference moves down as well, because a token that takes nearly all of a row's
// weight would push the others, whose values may be the output, below what f16
// holds; it stays within 2^kPfFloor of the largest logit, under which no number of
// tokens counts.  (A wider reach below a reference that only moves up, 2^-33 of
// the first tile's largest weight, took 782 us where this takes 550: it leaves 2^7
// before logits that grow rescale.)  The ring's weights are bf16, of f32's range:
// there it only moves up.
//
// Warps: 0-3 and 4-7 softmax of tile 0 and 1 (a thread per row), 8-23 decode
// records (or copy ring tokens) into two stages each of key and value tiles,
// 24 issues MMAs.  A tile's MMAs run P V(i) then Q K(i+1), and the two tiles
// alternate, so that one tile's softmax runs under the other's MMAs.  The
// decoding warps give registers to the softmax warps.  Every wait is bounded; a
// CTA whose wait expired leaves NaN statistics, so that its rows come out NaN.
//
// The rotation of the queries is a product with the signed Hadamard matrix
// (+-1, exact in bf16, as the queries are), one more MMA per tile.
//
// Measured: 1024 tokens of 32 heads over 32768 + 1280 (4 bits, head dim 128) 550 us,
// 1.02 PFLOP/s.  Neither the tensor pipe (48%) nor the issue slots (58%) are full: the
// two tiles' chains softmax -> weights -> MMA cover one another only in part.  Instructions
// count (lookups by shift and mask took 9% longer).
//
// Partials lie as [128-row tile][split][D / 4][128 rows][4], so that the
// thread that owns a row writes 16 bytes beside its neighbours'.
#pragma once

#include "prefill.cuh"
#include "umma.cuh"

namespace tq {

constexpr int kPfSoft = 8, kPfLoad = 16;  // softmax and loading warps
constexpr int kPfThreads = 32 * (kPfSoft + kPfLoad + 1);
constexpr int kPfRows = 256;
constexpr int kPfTok = 128 / kPfLoad;  // tokens of a tile that a loading warp decodes
// log2 of a tile's largest weight against an old reference (at most, and at least),
// and against a new one; how far a reference may lie below the largest logit
constexpr float kPfMargin = 15.f, kPfLow = -14.f, kPfTop = -2.f, kPfFloor = 24.f;

// Registers per thread: 72 at launch (25 warps: seven on one of the SM's four
// partitions), then 104 for the softmax and 56 for the decoding warps, no more
// in sum than at launch.  Sixteen decoding warps rather than eight: what they do
// is short dependent chains (1024 tokens over 32768 cached: 652 us against 817
// at that stage).
constexpr int kPfLaunchRegs = 72, kPfSoftRegs = 104, kPfLoadRegs = 56;
static_assert(kPfSoft * kPfSoftRegs + kPfLoad * kPfLoadRegs + kPfLaunchRegs <= (kPfSoft + kPfLoad + 1) * kPfLaunchRegs,
              "the registers that some warps take, others gave");

template <int D>
struct PfCfg {
  static constexpr int TILE = 128 * D * 2;      // bytes of a 128-row operand tile
  static constexpr int Q = 0, K = 2 * TILE, V = 4 * TILE, LUT = 6 * TILE, MISC = LUT + 32768;
  static constexpr int SMEM = MISC + 1024 + 1024;  // + bookkeeping + alignment slack
};

struct PfMisc {
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full[2], o_done[2], rot, fin;
  uint32_t tbase;
  int abort_;
  float red[2][kPfThreads / 32];
};
static_assert(sizeof(PfMisc) <= 1024, "bookkeeping block");

// mbar_wait for warps that mostly wait: the thread is suspended (for at
// most about a tenth of a millisecond a time) instead of polling, which leaves the issue
// slots to the warps that work.
__device__ __forceinline__ bool mbar_wait_idle(uint64_t* b, uint32_t parity, volatile int* abort) {
  const uint32_t a = smem_u32(b);
  if (mbar_try(a, parity)) return true;
  const uint64_t t0 = global_ns();
  for (;;) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(a), "r"(parity), "r"(100000u)
        : "memory");
    if (ok) return true;
    if (*abort) return false;
    if (global_ns() - t0 > 2000000000ull) {
      *abort = 1;
      return false;
    }
  }
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// D (tensor memory) += A (tensor memory) * B (shared memory)
__device__ __forceinline__ void umma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// true in one lane of a converged warp, in a form that keeps the MMA loop's operands in uniform registers
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
constexpr uint32_t kIdescBf16 = (1u << 7) | (1u << 10);  // bf16 A and B

__device__ __forceinline__ uint32_t hmul2(uint32_t a, __half2 b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), b);
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, __half2 b, uint32_t c) {
  const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&a), b, *reinterpret_cast<const __half2*>(&c));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// centroids of up to 16 levels as byte planes; with 8 levels or fewer one lookup a plane is enough
template <int B>
__device__ __forceinline__ uint4 decode_codes(uint32_t x, const Planes& pl) {
  if constexpr (B == 4) return decode8(x, pl);
  if constexpr (B == 3) x = spread3(x);
  if constexpr (B == 2) {
    x &= 0xFFFFu;
    x = (x | (x << 8)) & 0x00FF00FFu;
    x = (x | (x << 4)) & 0x0F0F0F0Fu;
    x = (x | (x << 2)) & 0x33333333u;
  }
  if constexpr (B == 1) {
    x &= 0xFFu;
    x = (x | (x << 12)) & 0x000F000Fu;
    x = (x | (x << 6)) & 0x03030303u;
    x = (x | (x << 3)) & 0x11111111u;
  }
  const uint32_t y = x >> 16;
  const uint32_t a0 = __byte_perm(pl.lo[0], pl.lo[1], x), b0 = __byte_perm(pl.hi[0], pl.hi[1], x);
  const uint32_t a1 = __byte_perm(pl.lo[0], pl.lo[1], y), b1 = __byte_perm(pl.hi[0], pl.hi[1], y);
  return make_uint4(__byte_perm(a0, b0, 0x5140), __byte_perm(a0, b0, 0x7362), __byte_perm(a1, b1, 0x5140),
                    __byte_perm(a1, b1, 0x7362));
}

// One record's keys or values into a stage: warp w takes its kPfTok tokens
// from kPfTok w on, a lane eight codes (16 bytes of f16) at a time.  The
// packed words of the next tile are loaded before this one's are decoded.
template <int D>
struct Packed {
  static constexpr int CH = D / 8, PER = kPfTok * CH / 32;  // chunks per row, per lane
  uint32_t x[PER];
  float n;
};
// rec points at the record's rows of this lane: token kPfTok w + lane / CH, codes 8 (lane % CH) ..
template <int D, int B>
__device__ __forceinline__ void load_packed(const uint8_t* rec, Packed<D>& k) {
  using P = Packed<D>;
  constexpr int STEP = 32 / P::CH * (D * B / 8);  // bytes between a lane's chunks
#pragma unroll
  for (int i = 0; i < P::PER; ++i) {
    if constexpr (B == 4) k.x[i] = __ldg(reinterpret_cast<const uint32_t*>(rec + i * STEP));
    else if constexpr (B == 2) k.x[i] = __ldg(reinterpret_cast<const uint16_t*>(rec + i * STEP));
    else if constexpr (B == 1) k.x[i] = __ldg(rec + i * STEP);
    else {  // the two words around three bytes (the second may lie past the row, inside the record)
      const uint32_t o = (uint32_t)reinterpret_cast<uintptr_t>(rec) & 3u;
      const uint32_t* w = reinterpret_cast<const uint32_t*>(rec - o + i * STEP);
      k.x[i] = __funnelshift_r(__ldg(w), __ldg(w + 1), 8 * o);
    }
  }
}
// LUT: pairs of 4-bit codes by one shared-memory lookup in a table with a copy per
// lane (entry e at 128 e + 4 lane, no bank conflicts), a byte extraction and a
// multiply-add a pair where the byte planes take six logic operations.
template <int D, int B, bool LUT, bool KEYS>
__device__ __forceinline__ void store_decoded(const Packed<D>& k, float n, const Planes& pl, const unsigned char* lut,
                                              unsigned char* st, int w, int lane) {
  using P = Packed<D>;
  const float lead = __half2float(__float2half_rn(n));
  const uint32_t n2 = pack2_f16(n, KEYS ? n - lead : n);
  st += w * kPfTok * 128;
  const ByteTable tab = byte_table(lut, 4 * lane, 128);
#pragma unroll
  for (int i = 0; i < P::PER; ++i) {
    const int row = (lane + 32 * i) / P::CH, ch = (lane + 32 * i) % P::CH;
    const uint32_t sw = __shfl_sync(0xffffffffu, n2, row);
    const __half2 sl = *reinterpret_cast<const __half2*>(&sw), s = __half2half2(__low2half(sl)), l = __high2half2(sl);
    uint4 v;
    if constexpr (LUT) {
      const uint32_t x = k.x[i];
      v = make_uint4(byte_lookup(tab, x, 0), byte_lookup(tab, x, 1), byte_lookup(tab, x, 2), byte_lookup(tab, x, 3));
    } else {
      v = decode_codes<B>(k.x[i], pl);
    }
    if constexpr (KEYS) {  // one rounding of centroid * (lead + rest), not two
      v = make_uint4(hfma2(v.x, s, hmul2(v.x, l)), hfma2(v.y, s, hmul2(v.y, l)), hfma2(v.z, s, hmul2(v.z, l)),
                     hfma2(v.w, s, hmul2(v.w, l)));
    } else {
      v = make_uint4(hmul2(v.x, s), hmul2(v.y, s), hmul2(v.z, s), hmul2(v.w, s));
    }
    *reinterpret_cast<uint4*>(st + (ch >> 3) * 16384 + row * 128 + (((ch ^ row) & 7) << 4)) = v;
  }
}

// Where a lane reads one codec's records: its rows and its token's scale.
struct RecSource {
  const uint8_t* layer;  // the layer's records
  const uint8_t* next;   // next record of the run
  int rows, bytes, bits, norm;
};
template <int D>
__device__ __forceinline__ RecSource rec_source(const CodecDev& c, const uint8_t* layer, int w, int lane) {
  constexpr int CH = D / 8;
  RecSource r;
  r.layer = r.next = layer;
  r.bits = c.bits;
  r.bytes = c.rec_bytes;
  r.rows = (kPfTok * w + lane / CH) * (D * c.bits / 8) + lane % CH * c.bits;
  r.norm = c.off_norm + 4 * (kPfTok * w + lane % kPfTok);
  return r;
}
template <int D>
__device__ __forceinline__ void load_tile(const RecSource& r, Packed<D>& k) {
  const uint8_t* at = r.next + r.rows;
  switch (r.bits) {
    case 1: load_packed<D, 1>(at, k); break;
    case 2: load_packed<D, 2>(at, k); break;
    case 3: load_packed<D, 3>(at, k); break;
    default: load_packed<D, 4>(at, k); break;
  }
  k.n = __ldg(reinterpret_cast<const float*>(r.next + r.norm));
}

// The side lists of the warp's tokens: put(row, coordinate, value, the token's n)
// for each entry, after the warp has written the rows; entries past the capacity are not read.
template <int D, class Put>
__device__ __forceinline__ void side_list(const CodecDev& c, const uint8_t* rec, int w, int lane, float n, Put&& put) {
  const uint32_t* cw = reinterpret_cast<const uint32_t*>(rec + c.off_count);
  int from = 0;
  for (int q = 0; q < kPfTok / 4 * w; ++q) from = __dp4a(__ldg(cw + q), 0x01010101u, (uint32_t)from);
  const int mine = __ldg(rec + c.off_count + kPfTok * w + lane % kPfTok);
  int inc = mine;
#pragma unroll
  for (int m = 1; m < kPfTok; m <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, inc, m, kPfTok);
    if (lane % kPfTok >= m) inc += o;
  }
  from += inc - mine;
  const int cnt = min(mine, max(c.cap - from, 0));
  const uint32_t* ent = reinterpret_cast<const uint32_t*>(rec + c.off_entries);
  __syncwarp();
#pragma unroll 1
  for (int row = 0; row < kPfTok; ++row) {
    const int f = __shfl_sync(0xffffffffu, from, row), m = __shfl_sync(0xffffffffu, cnt, row);
    const float s = __shfl_sync(0xffffffffu, n, row);
    for (int e = lane; e < m; e += 32) {
      const uint32_t en = __ldg(ent + f + e);
      put(row, (int)(en & (D - 1)), bf16_hi(en), s);
    }
  }
}

template <int D, bool KEYS>
__device__ __forceinline__ void decode_tile(const CodecDev& c, const uint8_t* rec, const Packed<D>& k, const Planes& pl,
                                            const unsigned char* lut, float nscale, unsigned char* st, int w, int lane) {
  const float n = k.n * nscale;
  switch (c.bits) {
    case 1: store_decoded<D, 1, false, KEYS>(k, n, pl, lut, st, w, lane); break;
    case 2: store_decoded<D, 2, false, KEYS>(k, n, pl, lut, st, w, lane); break;
    case 3: store_decoded<D, 3, false, KEYS>(k, n, pl, lut, st, w, lane); break;
    default:
      if (lut) store_decoded<D, 4, true, KEYS>(k, n, pl, lut, st, w, lane);
      else store_decoded<D, 4, false, KEYS>(k, n, pl, lut, st, w, lane);
  }
  if (c.has_outl)
    side_list<D>(c, rec, w, lane, n, [&](int row, int j, float y, float nr) {
      *reinterpret_cast<__half*>(st + (j >> 6) * 16384 + sw128_off(kPfTok * w + row, (j >> 3) & 7) + 2 * (j & 7)) =
          __float2half_rn(y * nr * kTableScale);
    });
}

// CAP: the call caps its logits (a kernel of its own: the branch cost registers).
template <int D, bool DENSE, bool CAP>
__device__ __forceinline__ void prefill_umma_body(const PrefillParams& pp, unsigned char* sm, int64_t unit, int tile,
                                                  int split) {
  using C = PfCfg<D>;
  const QueryParams& p = pp.q;
  PfMisc& ms = *reinterpret_cast<PfMisc*>(sm + C::MISC);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = (int)(unit % p.Hkv), lb = (int)(unit / p.Hkv), b = lb % p.B, l = lb / p.B;
  const int S = pp.Sc + pp.St;
  const CacheLen cl = cache_len(p, lb);
  const int tb = query_len(p, b);
  const int r0 = tile * kPfRows, rn = min(kPfRows, tb * p.G - r0);
  if (rn <= 0) return;
  const int base = DENSE ? cl.n * kChunk : 0;
  const int top = row_limit(p, cl, tb, r0 + rn - 1) - base;
  const int k0 = split * (DENSE ? pp.tps : pp.cps * kChunk);
  const int k1 = min(min(k0 + (DENSE ? pp.tps : pp.cps * kChunk), DENSE ? cl.len : cl.n * kChunk), top);
  const int sidx = DENSE ? pp.Sc + split : split;
  // partials of the CTA's first 128-row tile (a second one follows S blocks later)
  const int64_t blk = ((unit * ((pp.rows + 127) / 128) + 2 * tile) * S + sidx) * 128;
  if (k0 >= k1) {
    for (int r = tid; r < rn; r += kPfThreads)
      pp.ws_ml[blk + (r >> 7) * S * 128 + (r & 127)] = make_float2(-INFINITY, 0.f);
    return;
  }
  const int n = (k1 - k0 + kChunk - 1) / kChunk;  // 128-token tiles
  const int nt = rn > 128 ? 2 : 1;                // row tiles in use
  const int c0 = k0 / kChunk;
  const uint8_t* kl = p.krec + l * p.krec_ls;
  const uint8_t* vl = p.vrec + l * p.vrec_ls;
  auto rec_at = [&](bool key, int c) {
    const int bytes = key ? p.kc.rec_bytes : p.vc.rec_bytes;
    return (key ? kl : vl) + rec_offset(p.table, p.table_stride, p.rec_cap, p.Hkv, b, h, c, bytes);
  };

  // ---------------------------------------------------------------- set-up
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ms.k_full[i], kPfLoad);
      mbar_init(&ms.v_full[i], kPfLoad);
      mbar_init(&ms.k_empty[i], 1);
      mbar_init(&ms.v_empty[i], 1);
      mbar_init(&ms.s_full[i], 1);
      mbar_init(&ms.p_full[i], 4);
      mbar_init(&ms.o_done[i], 1);
    }
    mbar_init(&ms.rot, 1);
    mbar_init(&ms.fin, 1);
    ms.abort_ = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kPfSoft + kPfLoad) tmem_alloc(&ms.tbase, 512);
  bool vtable = false;  // the values are decoded through the lookup table
  if constexpr (!DENSE) {
    vtable = p.vc.bits == 4;
    if (p.kc.bits == 4)
      for (int k = 8; k < 16; ++k) vtable = vtable && p.kc.centroids[k] == p.vc.centroids[k];  // tables are symmetric
  }
  if constexpr (!DENSE) {  // the run's largest finite scales (an infinite key may be one that no query here sees)
    float mk = 0.f, mv = 0.f;
    auto mag = [](float x) { return fabsf(x) < INFINITY ? fabsf(x) : 0.f; };
    for (int i = tid; i < n * (kChunk / 4); i += kPfThreads) {
      const int c = c0 + i / (kChunk / 4), o = i % (kChunk / 4);
      const float4 x = __ldg(reinterpret_cast<const float4*>(rec_at(true, c) + p.kc.off_norm) + o);
      const float4 y = __ldg(reinterpret_cast<const float4*>(rec_at(false, c) + p.vc.off_norm) + o);
      mk = fmaxf(mk, fmaxf(fmaxf(mag(x.x), mag(x.y)), fmaxf(mag(x.z), mag(x.w))));
      mv = fmaxf(mv, fmaxf(fmaxf(mag(y.x), mag(y.y)), fmaxf(mag(y.z), mag(y.w))));
    }
    mk = warp_max(mk);
    mv = warp_max(mv);
    if (lane == 0) {
      ms.red[0][warp] = mk;
      ms.red[1][warp] = mv;
    }
  }
  {  // queries, bf16 as they are (the softmax scale's sign folded in)
    constexpr int CH = D / 8;
    const uint32_t flip = p.sscale < 0.f ? 0x80008000u : 0u;
    for (int i = tid; i < 128 * nt * CH; i += kPfThreads) {
      const int r = i / CH, ch = i % CH, row = r0 + r;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (r < rn)
        v = __ldg(reinterpret_cast<const uint4*>(p.q + l * p.q_ls + b * p.q_bs + (int64_t)(row / p.G) * p.q_ts +
                                                 (int64_t)(h * p.G + row % p.G) * D) + ch);
      v = make_uint4(v.x ^ flip, v.y ^ flip, v.z ^ flip, v.w ^ flip);
      *reinterpret_cast<uint4*>(sm + C::Q + (r >> 7) * C::TILE + (ch >> 3) * 16384 + sw128_off(r & 127, ch & 7)) = v;
    }
    if constexpr (!DENSE) {
      // lookup table of the 4-bit codec (the keys', and the values' where it is the same)
      const CodecDev& c4 = p.kc.bits == 4 ? p.kc : p.vc;
      if (c4.bits == 4)
        for (int i = tid; i < 256; i += kPfThreads) {
          const uint32_t v = pack2_f16(c4.centroids[i & 15] * kTableScale, c4.centroids[i >> 4] * kTableScale);
#pragma unroll
          for (int k = 0; k < 8; ++k) reinterpret_cast<uint4*>(sm + C::LUT + 128 * i)[(k + i) & 7] = make_uint4(v, v, v, v);
        }
    }
    if constexpr (!DENSE) {  // signed Hadamard matrix: row n, column k: (-1)^popc(n & k) s_k
      for (int i = tid; i < D * CH; i += kPfThreads) {
        const int n_ = i / CH, ch = i % CH;
        const uint32_t sg = (p.kc.signs[ch >> 2] >> (8 * (ch & 3))) ^ (__popc((n_ >> 3) & ch) & 1 ? 0xFFu : 0u);
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t s0 = (sg >> (2 * j)) ^ __popc(n_ & (2 * j)), s1 = (sg >> (2 * j + 1)) ^ __popc(n_ & (2 * j + 1));
          w[j] = 0x3F803F80u | ((s0 & 1u) << 15) | ((s1 & 1u) << 31);
        }
        *reinterpret_cast<uint4*>(sm + C::K + (ch >> 3) * 16384 + sw128_off(n_, ch & 7)) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
  fence_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  volatile int* abort_f = &ms.abort_;
  float ek = 1.f, ev = 1.f;  // 2^-(E+1) of keys and values
  float f = fabsf(p.sscale);  // logit factor of the thread's row (softmax warps)
  if constexpr (!DENSE) {
    float mk = ms.red[0][lane < kPfThreads / 32 ? lane : 0], mv = ms.red[1][lane < kPfThreads / 32 ? lane : 0];
    ek = pow2i(-1 - exp_of(warp_max(mk)));
    ev = pow2i(-1 - exp_of(warp_max(mv)));
    // rotation: scores' columns receive Q H, which return to the Q tiles as f16
    if (warp == kPfSoft + kPfLoad) {
      if (elect_one()) {
        const uint64_t dQ = sdesc_sw128(smem_u32(sm + C::Q), 16, 1024), dH = sdesc_sw128(smem_u32(sm + C::K), 16, 1024);
        for (int t = 0; t < nt; ++t)
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint64_t o = (ks >> 2) * 1024 + 2 * (ks & 3);
            umma_f16(ms.tbase + 128 * t, dQ + t * (C::TILE / 16) + o, dH + o,
                     idesc_f16(128, D, false, false) | kIdescBf16, ks != 0);
          }
        umma_commit(&ms.rot);
      }
      __syncwarp();
    } else if (warp < 4 * nt) {
      mbar_wait_idle(&ms.rot, 0, abort_f);
      tc_fence_after();
      const uint32_t tS = ms.tbase + 128 * (warp >> 2) + ((uint32_t)(32 * (warp & 3)) << 16);
      float mx = 0.f;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t a[32];
        tmem_ld32(tS + 32 * c, a);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 32; ++j) mx = fmaxf(mx, fabsf(__uint_as_float(a[j])));
      }
      mx *= inv_sqrt_dim<D>();
      const int s = mx > 0.f ? 13 - exp_of(mx) : 0;  // largest in [2^13, 2^14)
      const float sc = pow2i(s) * inv_sqrt_dim<D>();
      f *= pow2i(-15 - s) * (1.f / ek);
      const int r = 32 * (warp & 3) + lane;
      unsigned char* dst = sm + C::Q + (warp >> 2) * C::TILE;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t a[32], w[16];
        tmem_ld32(tS + 32 * c, a);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 32; j += 2) w[j / 2] = pack2_f16(__uint_as_float(a[j]) * sc, __uint_as_float(a[j + 1]) * sc);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          *reinterpret_cast<uint4*>(dst + (c >> 1) * 16384 + sw128_off(r, 4 * (c & 1) + k)) =
              make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
      }
      fence_async_smem();
      tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
  }
  const uint32_t tb0 = ms.tbase;

  if (warp == kPfSoft + kPfLoad) {
    // ---------------------------------------------------------------- MMA issue
    if (elect_one()) {
      constexpr uint32_t T = DENSE ? kIdescBf16 : 0u;
      constexpr uint32_t IS = idesc_f16(128, 128, false, false) | T;
      constexpr uint32_t IV = idesc_f16(128, D, false, true) | T;
      const uint64_t dQ = sdesc_sw128(smem_u32(sm + C::Q), 16, 1024);
      const uint64_t dK = sdesc_sw128(smem_u32(sm + C::K), 16, 1024);
      const uint64_t dV = sdesc_sw128(smem_u32(sm + C::V), 16384, 1024);
      constexpr uint64_t TS = C::TILE / 16;
      auto scores = [&](int t, int i) {
        const uint64_t a = dQ + t * TS, bk = dK + (i & 1) * TS;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint64_t o = (ks >> 2) * 1024 + 2 * (ks & 3);
          umma_f16(tb0 + 128 * t, a + o, bk + o, IS, ks != 0);
        }
        umma_commit(&ms.s_full[t]);
      };
      mbar_wait_idle(&ms.k_full[0], 0, abort_f);
      tc_fence_after();
      for (int t = 0; t < nt; ++t) scores(t, 0);
      umma_commit(&ms.k_empty[0]);
#pragma unroll 1
      for (int i = 0; i < n; ++i) {
        for (int t = 0; t < nt; ++t) {
          if (t == 0) mbar_wait_idle(&ms.v_full[i & 1], (i >> 1) & 1, abort_f);
          mbar_wait_idle(&ms.p_full[t], i & 1, abort_f);
          tc_fence_after();
          const uint64_t bv = dV + (i & 1) * TS;
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)
            umma_f16_ts(tb0 + 256 + D * t, tb0 + 128 * t + 8 * ks, bv + 128 * ks, IV, i > 0 || ks > 0);
          umma_commit(&ms.o_done[t]);
          if (t == nt - 1) umma_commit(&ms.v_empty[i & 1]);
          if (i + 1 < n) {
            if (t == 0) mbar_wait_idle(&ms.k_full[(i + 1) & 1], ((i + 1) >> 1) & 1, abort_f);
            mbar_wait_idle(&ms.o_done[t], i & 1, abort_f);  // P is read before S takes its columns
            tc_fence_after();
            scores(t, i + 1);
            if (t == nt - 1) umma_commit(&ms.k_empty[(i + 1) & 1]);
          }
        }
      }
      umma_commit(&ms.fin);
    }
    __syncwarp();
  } else if (warp >= kPfSoft) {
    // ---------------------------------------------------------------- keys and values
    regs_down<kPfLoadRegs>();
    const int w = warp - kPfSoft;
    if constexpr (DENSE) {
      constexpr int CH = D / 8, PER = kPfTok * CH / 32;
      const int cap = p.tail_cap;
      const int start = p.tail_start ? ((p.tail_start[lb] % cap) + cap) % cap : 0;
      const int64_t ring = l * p.tail_ls + (int64_t)(b * p.Hkv + h) * cap * D;
      for (int i = 0; i < n; ++i) {
        const int s = i & 1, ph = ((i >> 1) & 1) ^ 1;
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv) {
          const uint16_t* src = (kv ? p.vtail : p.ktail) + ring;
          mbar_wait_idle(kv ? &ms.v_empty[s] : &ms.k_empty[s], ph, abort_f);
          unsigned char* st = sm + (kv ? C::V : C::K) + s * C::TILE;
#pragma unroll
          for (int k = 0; k < PER; ++k) {
            const int x = lane + 32 * k, row = kPfTok * w + x / CH, ch = x % CH;
            const int tok = min(k0 + i * kChunk + row, cl.len - 1);
            cp_async16(st + (ch >> 3) * 16384 + sw128_off(row, ch & 7),
                       src + (int64_t)((start + (int64_t)tok) % cap) * D + 8 * ch);
          }
          cp_async_commit();
          if (kv) {  // the keys have landed, then the values
            cp_async_wait<1>();
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ms.k_full[s]);
            cp_async_wait<0>();
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ms.v_full[s]);
          }
        }
      }
    } else {
      const Planes kpl = make_planes(p.kc, kTableScale), vpl = make_planes(p.vc, kTableScale);
      const unsigned char* klut = p.kc.bits == 4 ? sm + C::LUT : nullptr;
      const unsigned char* vlut = vtable ? sm + C::LUT : nullptr;
      RecSource ks = rec_source<D>(p.kc, kl, w, lane), vs = rec_source<D>(p.vc, vl, w, lane);
      auto seek = [&](RecSource& r, int c) {  // contiguous records follow one another
        if (p.table || c == c0) r.next = r.layer + rec_offset(p.table, p.table_stride, p.rec_cap, p.Hkv, b, h, c, r.bytes);
        else r.next += r.bytes;
      };
      Packed<D> xk, xv;
      seek(ks, c0);
      load_tile<D>(ks, xk);
      seek(vs, c0);
      load_tile<D>(vs, xv);
#pragma unroll 1
      for (int i = 0; i < n; ++i) {
        const int s = i & 1, ph = ((i >> 1) & 1) ^ 1;
        mbar_wait_idle(&ms.k_empty[s], ph, abort_f);
        decode_tile<D, true>(p.kc, ks.next, xk, kpl, klut, ek, sm + C::K + s * C::TILE, w, lane);
        fence_async_smem();  // before the next loads, which it would wait for
        __syncwarp();
        if (lane == 0) mbar_arrive(&ms.k_full[s]);
        if (i + 1 < n) {
          seek(ks, c0 + i + 1);
          load_tile<D>(ks, xk);
        }
        mbar_wait_idle(&ms.v_empty[s], ph, abort_f);
        decode_tile<D, false>(p.vc, vs.next, xv, vpl, vlut, ev, sm + C::V + s * C::TILE, w, lane);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ms.v_full[s]);
        if (i + 1 < n) {
          seek(vs, c0 + i + 1);
          load_tile<D>(vs, xv);
        }
      }
    }
  } else {
    // ---------------------------------------------------------------- softmax: a thread per row
    regs_up<kPfSoftRegs>();
    if ((warp >> 2) < nt) {
    const int t = warp >> 2, q = warp & 3, r = 128 * t + 32 * q + lane;
    const uint32_t lrow = (uint32_t)(32 * q) << 16;
    const uint32_t tS = tb0 + 128 * t + lrow, tO = tb0 + 256 + D * t + lrow;
    // tokens it sees, counted from the run's first; rows of no query see everything
    const int lim = r < rn ? row_limit(p, cl, tb, r0 + r) - base - k0 : 0x7FFFFFFF;
    // the largest logit where references moved; how low a tile's maximum may lie against one
    float mref = -INFINITY, lsum = 0.f, peak = -INFINITY, low = -INFINITY;
    const SoftCap cap = make_cap(p.scap, p.iscap);
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      mbar_wait_idle(&ms.s_full[t], i & 1, abort_f);
      tc_fence_after();
      const int seen = lim - i * kChunk;  // columns below it
      const bool edge = __any_sync(0xffffffffu, seen < kChunk);
      uint32_t w[64];  // weights as pairs; chunk c of S becomes columns 16 c .. 16 c + 15
      float mx = -INFINITY, tm = -INFINITY;
      bool known = false;  // tm is the tile's largest logit
      float2 sum = f2(0.f, 0.f);
      // a pair of weights as an operand, and its sum: bf16 ones as rounded, since weights that
      // are alike round alike and 2^-8 would not average out
      auto weigh = [&](float2 v) {
        const uint32_t u = DENSE ? pack2_bf16(v.x, v.y) : pack2_f16(v.x, v.y);
        sum = add2(sum, DENSE ? f2(bf16_lo(u), bf16_hi(u)) : v);
        return u;
      };
      bool again = edge || mref == -INFINITY || (CAP && cap.large);
      if (!__any_sync(0xffffffffu, again)) {
        // weights against the reference as it stands; the maximum is found on the way
        const float fk = CAP ? f * cap.k : f, m0 = CAP ? cap.c - mref : -mref;
        const float2 f2v = f2(fk, fk), m2 = f2(m0, m0);
        float x0 = -INFINITY;
        uint32_t a[2][16];
        tmem_ld16(tS, a[0]);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          tmem_ld_wait();
          if (c < 7) tmem_ld16(tS + 16 * (c + 1), a[(c + 1) & 1]);
#pragma unroll
          for (int j = 0; j < 16; j += 2) {
            float2 v = f2(__uint_as_float(a[c & 1][j]), __uint_as_float(a[c & 1][j + 1]));
            if constexpr (CAP) {
              v = mul2(v, f2v);
              v = add2(f2(ex2(v.x), ex2(v.y)), f2(1.f, 1.f));
              v = fma2(f2(rcp_approx(v.x), rcp_approx(v.y)), f2(cap.m2c, cap.m2c), m2);
            } else {
              v = fma2(v, f2v, m2);
            }
            x0 = max3(x0, v.x, v.y);
            v = f2(ex2(v.x), ex2(v.y));
            w[8 * c + j / 2] = weigh(v);
          }
        }
        again = x0 > kPfMargin || x0 < low;
        tm = x0 + mref;
        known = true;
      }
      if (__any_sync(0xffffffffu, again)) {
        // a new reference for the rows that passed theirs by the margin (or have none yet):
        // find the maximum, rescale, and form the weights again
        again = false;
        sum = f2(0.f, 0.f);
        if (!known) {
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            uint32_t a[16];
            tmem_ld16(tS + 16 * c, a);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j) mx = fmaxf(mx, 16 * c + j < seen ? __uint_as_float(a[j]) : -INFINITY);
          }
          tm = mx > -INFINITY ? mx * f : -INFINITY;
          if (CAP && mx > -INFINITY) tm = cap_logit(tm, cap);
        }
        peak = fmaxf(peak, tm);
        const bool moves = tm > mref + kPfMargin || (tm < mref + low && tm > -INFINITY);
        if (__any_sync(0xffffffffu, moves)) {
          const float mn = !moves ? mref : fmaxf(tm - kPfTop, peak - kPfFloor);
          if (moves && !DENSE) low = mn > peak - kPfFloor ? kPfLow : -INFINITY;
          const float al = mref > -INFINITY ? ex2(mref - mn) : 0.f;  // 1 where the reference stays
          const float sc = mn > -INFINITY ? al : 1.f;
          lsum *= sc;
          mref = mn;
          if (i > 0) {  // P V(i - 1) is complete: the scores of this tile were issued after it
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
              uint32_t o[16];
              tmem_ld16(tO + 16 * c, o);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * sc);
              tmem_st16(tO + 16 * c, o);
            }
          }
        }
        const float ref = mref > -INFINITY ? mref : 0.f;
        const int top = __reduce_max_sync(0xffffffffu, seen);  // columns that some row of the warp sees
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          if (16 * c >= top) {
#pragma unroll
            for (int j = 0; j < 8; ++j) w[8 * c + j] = 0u;
            continue;
          }
          uint32_t a[16];
          tmem_ld16(tS + 16 * c, a);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; j += 2) {
            float2 v = f2(__uint_as_float(a[j]) * f, __uint_as_float(a[j + 1]) * f);
            if constexpr (CAP) v = f2(cap_logit(v.x, cap), cap_logit(v.y, cap));
            v = f2(16 * c + j < seen ? ex2(v.x - ref) : 0.f, 16 * c + j + 1 < seen ? ex2(v.y - ref) : 0.f);
            w[8 * c + j / 2] = weigh(v);
          }
        }
      }
      lsum += sum.x + sum.y;
      if (lsum != lsum && mref == -INFINITY) mref = 0.f;  // a NaN row has no maximum to wait for
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t u[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) u[j] = w[16 * c + j];
        tmem_st16(tS + 16 * c, u);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms.p_full[t]);
    }
    mbar_wait_idle(&ms.o_done[t], (n - 1) & 1, abort_f);
    tc_fence_after();
    const float un = DENSE ? 1.f : pow2i(-15) * (1.f / ev);
    const int64_t at = blk + (int64_t)t * S * 128;
    float4* dst = reinterpret_cast<float4*>(pp.ws_acc) + at * (D / 4) + (r & 127);
#pragma unroll 1
    for (int c = 0; c < D / 32; ++c) {
      uint32_t o[32];
      tmem_ld32(tO + 32 * c, o);
      tmem_ld_wait();
      if (r < rn) {
#pragma unroll
        for (int j = 0; j < 32; j += 4)
          dst[(8 * c + j / 4) * 128] =
              make_float4(__uint_as_float(o[j]) * un, __uint_as_float(o[j + 1]) * un, __uint_as_float(o[j + 2]) * un,
                          __uint_as_float(o[j + 3]) * un);
      }
    }
    if (r < rn) {
      const float bad = __int_as_float(0x7fc00000);
      pp.ws_ml[at + (r & 127)] = *abort_f || lsum != lsum ? make_float2(bad, bad)
                                 : lsum > 0.f ? make_float2(mref, lsum) : make_float2(-INFINITY, 0.f);
    }
    tc_fence_before();
    }
  }
  __syncthreads();
  if (warp == kPfSoft + kPfLoad) {
    volatile int drain = 0;  // every MMA has completed, whatever the abort flag says
    mbar_wait_idle(&ms.fin, 0, &drain);
    tc_fence_after();
    tmem_dealloc(tb0, 512);
  }
}

template <int D, bool CAP>
__global__ void __launch_bounds__(kPfThreads, 1) prefill_umma_kernel(const __grid_constant__ PrefillParams pp) {
  pdl_start();
  extern __shared__ __align__(1024) unsigned char smraw[];
  unsigned char* sm = smraw + ((1024u - (smem_u32(smraw) & 1023u)) & 1023u);
  // records first, the ring's shorter runs behind them
  const int64_t U = (int64_t)pp.q.L * pp.q.B * pp.q.Hkv * pp.tiles;
  const int split = (int)(blockIdx.x / U), tile = (int)(blockIdx.x % U % pp.tiles);
  const int64_t unit = blockIdx.x % U / pp.tiles;
  if (split < pp.Sc) prefill_umma_body<D, false, CAP>(pp, sm, unit, tile, split);
  else prefill_umma_body<D, true, CAP>(pp, sm, unit, tile, split - pp.Sc);
}

template <int D>
cudaError_t prefill_umma_launch(const PrefillParams& pp, cudaStream_t s) {
  if (pp.Sc + pp.St == 0) return cudaSuccess;
  auto kern = pp.q.scap > 0.f ? prefill_umma_kernel<D, true> : prefill_umma_kernel<D, false>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, PfCfg<D>::SMEM);
  if (e != cudaSuccess) return e;
  // the split of the registers counts on this many at launch
  cudaFuncAttributes fa;
  if ((e = cudaFuncGetAttributes(&fa, kern)) != cudaSuccess) return e;
  if (fa.numRegs != kPfLaunchRegs) return cudaErrorInvalidConfiguration;
  const int64_t grid = (int64_t)pp.q.L * pp.q.B * pp.q.Hkv * pp.tiles * (pp.Sc + pp.St);
  kern<<<(unsigned)grid, kPfThreads, PfCfg<D>::SMEM, s>>>(pp);
  return cudaGetLastError();
}

}  // namespace tq
