// The C ABI of the append, the several-query attention, the accumulated
// weights and the eviction by them (include/tq.h): host-side validation, split
// planning and dispatch, by the rules of abi.cu (every argument is checked
// before anything is launched).
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "attn_mass_few.cuh"
#include "prefill.cuh"

using namespace tq;

namespace tq {

#define TQ_DECL_DIM(d)                                                        \
  cudaError_t launch_attn_mass_d##d(const MassParams& mp, int NT, cudaStream_t s); \
  cudaError_t launch_attn_mass_few_d##d(const MassParams& mp, cudaStream_t s); \
  cudaError_t launch_prefill_d##d(const PrefillParams& pp, cudaStream_t s);   \
  int prefill_rows_d##d();
TQ_DECL_DIM(64)
TQ_DECL_DIM(128)
TQ_DECL_DIM(256)
TQ_DECL_DIM(512)
#undef TQ_DECL_DIM
cudaError_t launch_prefill_merge(const PrefillParams& pp, cudaStream_t s);
cudaError_t launch_attn_mass_umma_d64(const MassParams& mp, cudaStream_t s);
cudaError_t launch_attn_mass_umma_d128(const MassParams& mp, cudaStream_t s);
cudaError_t launch_attn_mass_add(const MassParams& mp, cudaStream_t s);

}  // namespace tq

namespace {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline size_t pad256(size_t x) { return (x + 255) / 256 * 256; }
inline bool dim_ok(int d) { return d == 64 || d == 128 || d == 256 || d == 512; }
inline bool strides_ok(int64_t a, int64_t b, int64_t c) {
  return a >= 0 && b >= 0 && c >= 0 && a % 8 == 0 && b % 8 == 0 && c % 8 == 0;
}

// Tokens of a sequence.  Indices are 32-bit, and kernels count past the last
// token by less than 2^20: to the end of the last split (fewer than 128 records
// behind, the split counts being at most 128) or of a block's last batch (8192).
constexpr int64_t kMostTokens = (1ll << 31) - (1 << 20);

// what a call writes must not overlap itself: along every axis longer than one
// a step is at least a row of `row` elements
inline bool rows_apart(int64_t ls, int64_t bs, int64_t ts, int L, int B, int T, int64_t row) {
  return (L == 1 || ls >= row) && (B == 1 || bs >= row) && (T == 1 || ts >= row);
}
// nor one layer the next
inline bool layers_apart(int L, int64_t ls, int64_t layer) { return L == 1 || ls >= layer; }

// ----------------------------------------------------------------- append
tq_status append_params(const tq_append_args* a, AppendParams* p) {
  if (!a) return TQ_ERR_INVALID_ARG;
  std::memset(p, 0, sizeof(*p));
  const int d = a->head_dim;
  if (!dim_ok(d)) return TQ_ERR_UNSUPPORTED;
  if (a->n_layers <= 0 || a->batch <= 0 || a->t_q <= 0 || a->n_q_heads < 0 || a->n_kv_heads <= 0 ||
      a->n_q_heads > 16384 || a->n_kv_heads > 16384)
    return TQ_ERR_INVALID_ARG;
  if (!a->k || !a->k_tail || !a->tail_len || !a->tail_len_out || a->tail_cap <= 0) return TQ_ERR_INVALID_ARG;
  if ((a->v == nullptr) != (a->v_tail == nullptr) || (a->q != nullptr) != (a->n_q_heads > 0) ||
      (a->q != nullptr) != (a->q_out != nullptr))
    return TQ_ERR_INVALID_ARG;
  for (const void* x : {a->q, a->k, a->v, (const void*)a->q_out, (const void*)a->k_tail, (const void*)a->v_tail})
    if (!aligned(x, 16)) return TQ_ERR_INVALID_ARG;
  if (a->v_tail && a->v_tail == a->k_tail) return TQ_ERR_INVALID_ARG;  // both would write one slot
  for (const void* x : {(const void*)a->tail_start, (const void*)a->tail_len, (const void*)a->tail_len_out,
                        (const void*)a->q_lens, (const void*)a->positions, (const void*)a->inv_freq,
                        (const void*)a->mass, (const void*)a->n_chunks})
    if (!aligned(x, 4)) return TQ_ERR_INVALID_ARG;
  if (!strides_ok(a->q_layer_stride, a->q_batch_stride, a->q_token_stride) ||
      !strides_ok(a->kv_layer_stride, a->kv_batch_stride, a->kv_token_stride) ||
      !strides_ok(a->q_out_layer_stride, a->q_out_batch_stride, a->q_out_token_stride) ||
      a->tail_layer_stride < 0 || a->tail_layer_stride % 8)
    return TQ_ERR_INVALID_ARG;
  if (a->q && !rows_apart(a->q_out_layer_stride, a->q_out_batch_stride, a->q_out_token_stride, a->n_layers, a->batch,
                          a->t_q, (int64_t)a->n_q_heads * d))
    return TQ_ERR_INVALID_ARG;
  if (!layers_apart(a->n_layers, a->tail_layer_stride, (int64_t)a->batch * a->n_kv_heads * a->tail_cap * d))
    return TQ_ERR_INVALID_ARG;
  if (a->q_out == a->q && a->q &&
      (a->q_out_layer_stride != a->q_layer_stride || a->q_out_batch_stride != a->q_batch_stride ||
       a->q_out_token_stride != a->q_token_stride))
    return TQ_ERR_INVALID_ARG;
  if (a->rot_dim < 0 || a->rot_start < 0 || a->rot_dim > d || a->rot_start > d - a->rot_dim)
    return TQ_ERR_INVALID_ARG;
  if (a->rot_dim % 16 || a->rot_start % 8) return TQ_ERR_UNSUPPORTED;
  if (a->rot_dim > 0) {
    if (a->n_axes < 1 || a->n_axes > TQ_MAX_AXES || !a->positions || !a->inv_freq || !std::isfinite(a->rot_scale))
      return TQ_ERR_INVALID_ARG;
    for (int i = 0; i < a->rot_dim / 2; ++i)
      if (a->pair_axis[i] >= a->n_axes) return TQ_ERR_INVALID_ARG;
  }
  if (a->mass && (a->mass_cap <= 0 || a->mass_layer_stride < 0 ||
                  !layers_apart(a->n_layers, a->mass_layer_stride, (int64_t)a->batch * a->n_kv_heads * a->mass_cap)))
    return TQ_ERR_INVALID_ARG;
  p->L = a->n_layers;
  p->B = a->batch;
  p->T = a->t_q;
  p->Hq = a->n_q_heads;
  p->Hkv = a->n_kv_heads;
  p->D = d;
  p->heads = a->n_q_heads + a->n_kv_heads * (a->v ? 2 : 1);
  p->q = (const uint16_t*)a->q;
  p->k = (const uint16_t*)a->k;
  p->v = (const uint16_t*)a->v;
  p->q_ls = a->q_layer_stride;
  p->q_bs = a->q_batch_stride;
  p->q_ts = a->q_token_stride;
  p->kv_ls = a->kv_layer_stride;
  p->kv_bs = a->kv_batch_stride;
  p->kv_ts = a->kv_token_stride;
  p->q_out = (uint16_t*)a->q_out;
  p->o_ls = a->q_out_layer_stride;
  p->o_bs = a->q_out_batch_stride;
  p->o_ts = a->q_out_token_stride;
  p->q_lens = a->q_lens;
  p->positions = a->positions;
  p->rot_start = a->rot_start;
  p->rot_dim = a->rot_dim;
  p->adjacent = a->pair_adjacent != 0;
  p->inv_freq = a->inv_freq;
  std::memcpy(p->pair_axis, a->pair_axis, sizeof(p->pair_axis));
  p->rot_scale = a->rot_scale;
  p->k_tail = (uint16_t*)a->k_tail;
  p->v_tail = (uint16_t*)a->v_tail;
  p->tail_ls = a->tail_layer_stride;
  p->tail_cap = a->tail_cap;
  p->tail_start = a->tail_start;
  p->tail_len = a->tail_len;
  p->tail_len_out = a->tail_len_out;
  p->in_place = a->tail_len == a->tail_len_out;
  p->mass = a->mass;
  p->mass_ls = a->mass_layer_stride;
  p->mass_cap = a->mass_cap;
  p->n_chunks = a->n_chunks;
  // about 1024 two-chunk units a CTA: up to 8 tokens with all their heads, or
  // fewer heads of one token where the call has too few tokens for the SMs
  const int uph = d / 16;
  const int64_t lb = (int64_t)p->L * p->B;
  p->tile = (int)std::max<int64_t>(1, std::min<int64_t>(std::min(8, p->T), 1024 / std::max(1, p->heads * uph)));
  p->tiles = (int)cdiv(p->T, p->tile);
  p->group = p->heads;
  const int64_t want = cdiv(2 * sm_count(), std::max<int64_t>(1, lb * p->tiles));
  if (want > 1) p->group = (int)std::max<int64_t>(std::max(1, 64 / uph), cdiv(p->heads, want));
  p->group = std::min(p->group, p->heads);
  p->units = make_fast_div((uint32_t)(p->group * uph));
  if (lb * p->tiles > 0x7FFFFFFFll) return TQ_ERR_UNSUPPORTED;
  return TQ_OK;
}

// ----------------------------------------------------------------- queries
// values: whether the call reads them (tq_attn_mass does not)
tq_status query_params(const tq_query_args* a, const tq_codec* kcod, const tq_codec* vcod, bool values,
                       QueryParams* p) {
  if (!a) return TQ_ERR_INVALID_ARG;
  std::memset(p, 0, sizeof(*p));
  const int d = a->head_dim;
  if (!dim_ok(d)) return TQ_ERR_UNSUPPORTED;
  if (a->n_layers <= 0 || a->n_layers > 65535 || a->batch <= 0 || a->t_q <= 0 || a->n_q_heads <= 0 ||
      a->n_kv_heads <= 0 || a->n_q_heads % a->n_kv_heads)
    return TQ_ERR_INVALID_ARG;
  if ((int64_t)a->batch * a->n_kv_heads > 65535) return TQ_ERR_UNSUPPORTED;
  if ((int64_t)a->t_q * (a->n_q_heads / a->n_kv_heads) > (1 << 28)) return TQ_ERR_UNSUPPORTED;
  if (!a->q || !aligned(a->q, 16) || !strides_ok(a->q_layer_stride, a->q_batch_stride, a->q_token_stride))
    return TQ_ERR_INVALID_ARG;
  if (values && (!a->out || !aligned(a->out, 16) ||
                 !strides_ok(a->out_layer_stride, a->out_batch_stride, a->out_token_stride) ||
                 !rows_apart(a->out_layer_stride, a->out_batch_stride, a->out_token_stride, a->n_layers, a->batch,
                             a->t_q, (int64_t)a->n_q_heads * d)))
    return TQ_ERR_INVALID_ARG;
  if (!std::isfinite(a->scale) || !std::isfinite(a->softcap) || a->softcap < 0.f) return TQ_ERR_INVALID_ARG;
  if (a->max_chunks < 0 || a->max_tail < 0 || a->splits < 0) return TQ_ERR_INVALID_ARG;
  for (const void* x : {(const void*)a->q_lens, (const void*)a->n_chunks, (const void*)a->tail_start,
                        (const void*)a->tail_len, (const void*)a->block_table})
    if (!aligned(x, 4)) return TQ_ERR_INVALID_ARG;
  if (a->k_rec) {
    if (!a->n_chunks || (values && !a->v_rec)) return TQ_ERR_INVALID_ARG;
    tq_status st = resolve_codec_dev(kcod, &p->kc);
    if (st != TQ_OK) return st;
    if (p->kc.d != d) return TQ_ERR_INVALID_ARG;
    if (values) {
      st = resolve_codec_dev(vcod, &p->vc);
      if (st != TQ_OK) return st;
      if (p->vc.d != d) return TQ_ERR_INVALID_ARG;
      p->shared_kv = a->v_rec == a->k_rec;
      if (p->shared_kv && std::memcmp(kcod, vcod, sizeof(tq_codec)) != 0) return TQ_ERR_INVALID_ARG;
    }
    if (!aligned(a->k_rec, 16) || a->k_rec_layer_stride % 16 || a->rec_cap <= 0) return TQ_ERR_INVALID_ARG;
    if (values && (!aligned(a->v_rec, 16) || a->v_rec_layer_stride % 16)) return TQ_ERR_INVALID_ARG;
    if (a->block_table && a->table_stride <= 0) return TQ_ERR_INVALID_ARG;
    if (a->max_chunks > (a->block_table ? a->table_stride : a->rec_cap)) return TQ_ERR_INVALID_ARG;
  } else if (a->v_rec || a->n_chunks || a->block_table || a->max_chunks) {
    return TQ_ERR_INVALID_ARG;
  }
  if (a->k_tail) {
    if (!a->tail_len || (values && !a->v_tail) || !aligned(a->k_tail, 16) || a->tail_layer_stride % 8 ||
        a->tail_cap <= 0 || a->max_tail > a->tail_cap || (values && !aligned(a->v_tail, 16)))
      return TQ_ERR_INVALID_ARG;
  } else if (a->v_tail || a->tail_len || a->tail_start || a->max_tail) {
    return TQ_ERR_INVALID_ARG;
  }
  if ((int64_t)a->max_chunks * TQ_CHUNK + a->max_tail > kMostTokens) return TQ_ERR_UNSUPPORTED;
  p->L = a->n_layers;
  p->B = a->batch;
  p->T = a->t_q;
  p->Hq = a->n_q_heads;
  p->Hkv = a->n_kv_heads;
  p->G = a->n_q_heads / a->n_kv_heads;
  p->D = d;
  const double log2e = 1.4426950408889634074;
  p->sscale = (float)((double)a->scale * log2e);
  p->scap = a->softcap > 0.f ? (float)((double)a->softcap * log2e) : 0.f;
  p->iscap = a->softcap > 0.f ? (float)(1.0 / ((double)a->softcap * log2e)) : 0.f;
  p->causal = a->causal != 0;
  p->q = (const uint16_t*)a->q;
  p->q_ls = a->q_layer_stride;
  p->q_bs = a->q_batch_stride;
  p->q_ts = a->q_token_stride;
  p->q_lens = a->q_lens;
  p->krec = (const uint8_t*)a->k_rec;
  p->vrec = (const uint8_t*)a->v_rec;
  p->krec_ls = a->k_rec_layer_stride;
  p->vrec_ls = a->v_rec_layer_stride;
  p->rec_cap = a->rec_cap;
  p->table = a->block_table;
  p->table_stride = a->table_stride;
  p->rec_limit = a->block_table ? a->table_stride : a->rec_cap;
  p->ktail = (const uint16_t*)a->k_tail;
  p->vtail = (const uint16_t*)a->v_tail;
  p->tail_ls = a->tail_layer_stride;
  p->tail_cap = a->tail_cap;
  p->n_chunks = a->n_chunks;
  p->tail_start = a->tail_start;
  p->tail_len = a->tail_len;
  p->max_chunks = a->max_chunks;
  p->max_tail = a->max_tail;
  return TQ_OK;
}

struct PrefillPlan {
  PrefillParams pp;
  size_t ml_off, bytes;
};

tq_status prefill_plan(const tq_query_args* a, const tq_codec* kcod, const tq_codec* vcod, PrefillPlan* pl) {
  PrefillParams& pp = pl->pp;
  std::memset(&pp, 0, sizeof(pp));
  const tq_status st = query_params(a, kcod, vcod, true, &pp.q);
  if (st != TQ_OK) return st;
  const int d = pp.q.D;
  const int bm = d == 64 ? prefill_rows_d64() : d == 128 ? prefill_rows_d128() : d == 256 ? prefill_rows_d256() : prefill_rows_d512();
  pp.rows = pp.q.T * pp.q.G;
  pp.tiles = (int)cdiv(pp.rows, bm);
  const int64_t units = (int64_t)pp.q.L * pp.q.B * pp.q.Hkv;
  const int64_t sms = sm_count(), U = units * pp.tiles;
  // One CTA per SM.  The split count that minimises, in 128-token tiles' time:
  // waves of records' CTAs with six tiles' worth of set-up and epilogue each,
  // the ring's CTAs in the last wave's idle SMs or after it, and the partials'
  // traffic (about 0.03 tiles per CTA).
  const int64_t ring = cdiv(pp.q.max_tail, TQ_CHUNK), most = std::max<int64_t>(pp.q.max_chunks, ring);
  double best = 1e300;
  for (int64_t s = 1; s <= std::min<int64_t>(most, 128); ++s) {
    if (a->splits > 0 && s != std::min<int64_t>(a->splits, std::min<int64_t>(most, 128))) continue;
    const int64_t per = cdiv(most, s);
    const int64_t sc = cdiv(pp.q.max_chunks, per), st = cdiv(ring, per);
    const int64_t waves = cdiv(U * sc, sms);
    const double one = (double)(sc ? cdiv(pp.q.max_chunks, sc) : 0) + 6, rest = (double)(st ? cdiv(ring, st) : 0) + 6;
    const double idle = (double)(waves * sms - U * sc) * one, dense = (double)(U * st) * rest;
    double cost = (double)waves * one + 0.03 * (double)(U * (sc + st));
    if (dense > 0.9 * idle) cost += std::max(rest, (dense - 0.9 * idle) / (double)sms);
    if (cost < best) {
      best = cost;
      pp.cps = (int)per;
      pp.Sc = (int)sc;
      pp.tps = (int)(TQ_CHUNK * per);
      pp.St = (int)st;
    }
  }
  // the grids of the attention and of the merge of its splits
  const int64_t merges = d <= 128 ? 16 * units * cdiv(pp.rows, 128) : cdiv(units * pp.rows, 4);
  if (U * (pp.Sc + pp.St) > 0x7FFFFFFFll || merges > 0x7FFFFFFFll) return TQ_ERR_UNSUPPORTED;
  pp.out = (uint16_t*)a->out;
  pp.o_ls = a->out_layer_stride;
  pp.o_bs = a->out_batch_stride;
  pp.o_ts = a->out_token_stride;
  pp.inv_sqrt_d = (float)(1.0 / std::sqrt((double)d));
  // partials: every row, or at head dims 64 and 128 whole tiles of 128 rows
  const size_t parts = (size_t)(units * (d <= 128 ? cdiv(pp.rows, 128) * 128 : pp.rows)) * (pp.Sc + pp.St);
  pl->ml_off = pad256(parts * d * 4);
  pl->bytes = pl->ml_off + pad256(parts * 8) + 256;
  return TQ_OK;
}

struct MassPlan {
  MassParams mp;
  bool few;  // at most eight query rows: the logits are kept
  bool umma; // many rows at head dims 64 and 128: tcgen05, blocks of 128 rows
  int NT;    // else rows per block / 8
  size_t ml, frag, fragd, qsc, qrot, logits, bytes;
};

tq_status mass_plan(const tq_query_args* a, const tq_codec* kcod, MassPlan* pl) {
  std::memset(pl, 0, sizeof(*pl));
  MassParams& mp = pl->mp;
  const tq_status st = query_params(a, kcod, nullptr, false, &mp.q);
  if (st != TQ_OK) return st;
  const QueryParams& q = mp.q;
  const bool outl = q.krec && q.kc.has_outl;
  mp.rows = q.T * q.G;
  const int64_t units = (int64_t)q.L * q.B * q.Hkv, sms = sm_count();
  const int bits = q.krec ? q.kc.bits : 1;
  pl->few = mp.rows <= 8;
  // Up to 8 rows the logits are kept (8 sequences of 32768, 8 kv heads: 8 rows 95 us, 461
  // with the scores formed twice).  A tile of 128 rows costs the tensor cores what
  // 40 rows cost mma.sync (a quarter of the rate), beside a set-up of its own: 18 rows of 2 kv heads
  // over 4096 take 25 us on mma.sync and 29 on tcgen05, 36 rows 40 and 29, 54 rows 46 and 31;
  // over 32768 with 8 kv heads, 12 rows 116 and 69, 40 rows 218 and 69, 48 rows 221 and 69.
  pl->umma = mp.rows > 40 && q.D <= 128;
  const int64_t ring = cdiv(q.max_tail, TQ_CHUNK);
  if (pl->few) {
    mp.nrb = 1;
    mp.pitch = mp.rows <= 1 ? 1 : mp.rows <= 2 ? 2 : mp.rows <= 4 ? 4 : 8;
    attn_mass_few_layout(mp, q.D, bits, outl);
    // CTAs per SM by shared memory (four at the widest table); the split count
    // that minimises waves x records per split, three records' worth of set-up included
    const int64_t slots = sms * std::max<int64_t>(1, std::min<int64_t>(5, max_dynamic_smem() / (mp.sm_total + 1024)));
    const int64_t most = std::max<int64_t>(q.max_chunks, ring);
    int64_t best = INT64_MAX, per = 1;
    for (int64_t s = 1; s <= std::min<int64_t>(most, 512); ++s) {
      if (a->splits > 0 && s != std::min<int64_t>(a->splits, std::min<int64_t>(most, 512))) continue;
      const int64_t c = cdiv(most, s);
      const int64_t cost = cdiv(units * (cdiv(q.max_chunks, c) + cdiv(ring, c)), slots) * (c + 3);
      if (cost < best) {
        best = cost;
        per = c;
      }
    }
    mp.cps = (int)per;
    mp.Sc = (int)cdiv(q.max_chunks, per);
    mp.tps = (int)(TQ_CHUNK * per);
    mp.St = (int)cdiv(ring, per);
  } else if (pl->umma) {
    // one CTA per SM: the split count that minimises waves x tiles per split in
    // both passes (row tiles are CTAs in the first and a loop in the second),
    // six tiles' worth of set-up per row tile included
    mp.nrb = (int)cdiv(mp.rows, 128);
    const int64_t most = std::max<int64_t>(std::max<int64_t>(q.max_chunks, ring), 1);
    int64_t best = INT64_MAX, per = 1;
    for (int64_t s = cdiv(most, kMassUmmaPer); s <= most; ++s) {
      if (a->splits > 0 && s != std::max(cdiv(most, kMassUmmaPer), std::min<int64_t>(a->splits, most))) continue;
      const int64_t c = cdiv(most, s), ctas = units * (cdiv(q.max_chunks, c) + cdiv(ring, c));
      const int64_t cost = cdiv(ctas * mp.nrb, sms) * (c + 6) + cdiv(ctas, sms) * mp.nrb * (c + 6);
      if (cost < best) {
        best = cost;
        per = c;
      }
      if (s > 512) break;
    }
    mp.cps = (int)per;
    mp.Sc = (int)cdiv(q.max_chunks, per);
    mp.tps = (int)(TQ_CHUNK * per);
    mp.St = (int)cdiv(ring, per);
  } else {
    pl->NT = outl ? 2 : mp.rows <= 32 ? 4 : 8;
    mp.nrb = (int)cdiv(mp.rows, 8 * pl->NT);
    // Eight CTAs per SM for the first pass (splits x row blocks), of which shared
    // memory holds one (head dim 512, 170 KB) to four at a time; at most 32 records or
    // ring tiles of 128 tokens a split (their sums sit in shared memory).  The second
    // pass has a CTA a split, which walks the row blocks: few where those are many
    // (32 tokens of one kv head of 64, head dim 512, over 32768: 1280 CTAs, then 40; 4.6 ms).
    const int64_t want = a->splits > 0 ? a->splits : cdiv(8 * sms, units * mp.nrb);
    if (q.max_chunks > 0) {
      mp.cps = (int)std::min<int64_t>(32, cdiv(q.max_chunks, std::min<int64_t>(want, q.max_chunks)));
      mp.Sc = (int)cdiv(q.max_chunks, mp.cps);
    }
    if (q.max_tail > 0) {
      const int64_t per = std::min<int64_t>(32, cdiv(ring, std::min<int64_t>(want, ring)));
      mp.tps = (int)(TQ_CHUNK * per);
      mp.St = (int)cdiv(q.max_tail, mp.tps);
    }
    attn_mass_layout(mp, q.D, bits, pl->NT, outl);
  }
  const int S = mp.Sc + mp.St;
  if ((int64_t)S * mp.nrb > 0x7FFFFFFFll) return TQ_ERR_UNSUPPORTED;
  if (mp.sm_total > max_dynamic_smem()) return TQ_ERR_UNSUPPORTED;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += pad256(bytes);
    return at;
  };
  if (pl->few) {
    pl->ml = take((size_t)units * S * 8 * 8);
    pl->logits = take((size_t)units * (q.max_chunks * (size_t)TQ_CHUNK + (size_t)mp.St * mp.tps) * mp.pitch * 4);
  } else if (pl->umma) {
    pl->ml = take((size_t)units * mp.nrb * S * 128 * 8);
  } else {
    const int R = 8 * pl->NT;
    const size_t blocks = (size_t)units * mp.nrb, frags = blocks * (q.D / 16) * pl->NT * 32;
    pl->ml = take(blocks * R * S * 8);
    pl->frag = take(frags * 16);
    pl->fragd = take(frags * 8);
    pl->qsc = take(blocks * R * 4);
    pl->qrot = take(outl ? blocks * R * q.D * 4 : 0);
  }
  pl->bytes = off + 256;
  return TQ_OK;
}

// ----------------------------------------------------------------- eviction
tq_status evict_mass_params(const tq_evict_mass_args* a, const tq_codec* kcod, const tq_codec* vcod,
                            EvictMassParams* p) {
  if (!a) return TQ_ERR_INVALID_ARG;
  std::memset(p, 0, sizeof(*p));
  tq_status st = resolve_codec_dev(kcod, &p->kc);
  if (st != TQ_OK) return st;
  const bool shared = a->v_rec == a->k_rec;
  if (shared) {
    if (vcod && std::memcmp(kcod, vcod, sizeof(tq_codec)) != 0) return TQ_ERR_INVALID_ARG;
    p->vc = p->kc;
  } else {
    st = resolve_codec_dev(vcod, &p->vc);
    if (st != TQ_OK) return st;
  }
  if (p->kc.d != p->vc.d) return TQ_ERR_INVALID_ARG;
  if (a->n_layers <= 0 || a->batch <= 0 || a->n_kv_heads <= 0) return TQ_ERR_INVALID_ARG;
  if ((int64_t)a->batch * a->n_kv_heads > 65535 || (int64_t)a->n_layers * a->batch * a->n_kv_heads > 65535)
    return TQ_ERR_UNSUPPORTED;
  if (!a->k_rec || !a->v_rec || !a->k_dst || !a->v_dst || !a->mass || !a->mass_dst || !a->n_chunks || !a->n_chunks_dst)
    return TQ_ERR_INVALID_ARG;
  for (const void* x : {(const void*)a->k_rec, (const void*)a->v_rec, (const void*)a->k_dst, (const void*)a->v_dst})
    if (!aligned(x, 16)) return TQ_ERR_INVALID_ARG;
  for (const void* x : {(const void*)a->mass, (const void*)a->mass_dst, (const void*)a->n_chunks,
                        (const void*)a->n_chunks_dst, (const void*)a->tail_len, (const void*)a->kept,
                        (const void*)a->block_table, (const void*)a->dst_table})
    if (!aligned(x, 4)) return TQ_ERR_INVALID_ARG;
  const bool in_place = a->k_dst == a->k_rec;
  if (in_place) {  // all of it or nothing
    if (a->v_dst != a->v_rec || a->mass_dst != a->mass || a->n_chunks_dst != a->n_chunks) return TQ_ERR_INVALID_ARG;
  } else if (a->v_dst == a->v_rec || a->mass_dst == a->mass || a->n_chunks_dst == a->n_chunks ||
             (a->v_dst == a->k_dst) != shared) {
    return TQ_ERR_INVALID_ARG;
  }
  if (a->rec_cap <= 0 || (a->block_table && a->table_stride <= 0) || a->k_rec_layer_stride % 16 ||
      a->v_rec_layer_stride % 16 || a->max_chunks < 0 || a->max_tail < 0 || a->keep_chunks < 1 || a->sink < 0 ||
      a->recent < 0)
    return TQ_ERR_INVALID_ARG;
  const int limit = a->block_table ? a->table_stride : a->rec_cap;
  if (a->max_chunks > limit) return TQ_ERR_INVALID_ARG;
  if ((int64_t)a->sink + a->recent > (int64_t)TQ_CHUNK * a->keep_chunks) return TQ_ERR_INVALID_ARG;
  const int64_t most = (int64_t)TQ_CHUNK * a->max_chunks + a->max_tail;
  if (most > kMostTokens || (int64_t)TQ_CHUNK * a->keep_chunks > 0x7FFFFFFFll - a->max_tail) return TQ_ERR_UNSUPPORTED;
  if (a->mass_cap < most || a->mass_layer_stride < 0 ||
      !layers_apart(a->n_layers, a->mass_layer_stride, (int64_t)a->batch * a->n_kv_heads * a->mass_cap))
    return TQ_ERR_INVALID_ARG;
  const int kept = std::min(a->keep_chunks, std::max(a->max_chunks, 1));  // records that can remain
  // a layer's records follow one another (pages: at least its own blocks are there)
  auto records_apart = [&](const int32_t* table, int cap, int64_t k_ls, int64_t v_ls) {
    const int64_t heads = (table ? 1 : (int64_t)a->batch * cap) * a->n_kv_heads;
    return layers_apart(a->n_layers, k_ls, heads * p->kc.rec_bytes) &&
           (shared || layers_apart(a->n_layers, v_ls, heads * p->vc.rec_bytes));
  };
  if (in_place) {  // the source is written
    if (!records_apart(a->block_table, a->rec_cap, a->k_rec_layer_stride, a->v_rec_layer_stride))
      return TQ_ERR_INVALID_ARG;
  } else {
    if (a->dst_cap <= 0 || (a->dst_table && a->dst_table_stride <= 0) || a->k_dst_layer_stride % 16 ||
        a->v_dst_layer_stride % 16 || a->mass_dst_layer_stride < 0 ||
        !layers_apart(a->n_layers, a->mass_dst_layer_stride, (int64_t)a->batch * a->n_kv_heads * a->mass_dst_cap))
      return TQ_ERR_INVALID_ARG;
    if (!records_apart(a->dst_table, a->dst_cap, a->k_dst_layer_stride, a->v_dst_layer_stride)) return TQ_ERR_INVALID_ARG;
    if ((a->dst_table ? a->dst_table_stride : a->dst_cap) < std::min(a->keep_chunks, a->max_chunks) ||
        a->mass_dst_cap < (int64_t)TQ_CHUNK * std::min(a->keep_chunks, a->max_chunks) + a->max_tail)
      return TQ_ERR_INVALID_ARG;
  }
  p->L = a->n_layers;
  p->B = a->batch;
  p->Hkv = a->n_kv_heads;
  p->shared = shared;
  p->k_rec = (const uint8_t*)a->k_rec;
  p->v_rec = (const uint8_t*)a->v_rec;
  p->k_ls = a->k_rec_layer_stride;
  p->v_ls = a->v_rec_layer_stride;
  p->rec_cap = a->rec_cap;
  p->table = a->block_table;
  p->table_stride = a->table_stride;
  p->rec_limit = limit;
  p->k_dst = (uint8_t*)a->k_dst;
  p->v_dst = (uint8_t*)a->v_dst;
  p->kd_ls = in_place ? a->k_rec_layer_stride : a->k_dst_layer_stride;
  p->vd_ls = in_place ? a->v_rec_layer_stride : a->v_dst_layer_stride;
  p->dst_cap = in_place ? a->rec_cap : a->dst_cap;
  p->dst_table = in_place ? a->block_table : a->dst_table;
  p->dst_table_stride = in_place ? a->table_stride : a->dst_table_stride;
  p->mass = a->mass;
  p->mass_dst = a->mass_dst;
  p->mass_ls = a->mass_layer_stride;
  p->mass_dst_ls = in_place ? a->mass_layer_stride : a->mass_dst_layer_stride;
  p->mass_cap = a->mass_cap;
  p->mass_dst_cap = in_place ? a->mass_cap : a->mass_dst_cap;
  p->n_chunks = a->n_chunks;
  p->n_chunks_dst = a->n_chunks_dst;
  p->tail_len = a->tail_len;
  p->max_chunks = a->max_chunks;
  p->max_tail = a->max_tail;
  p->keep = a->keep_chunks;
  p->slots = kept;
  p->sink = a->sink;
  p->recent = a->recent;
  p->in_place = in_place;
  p->kept = a->kept;
  return TQ_OK;
}

size_t evict_mass_bytes(const EvictMassParams& p) {
  return pad256((size_t)p.L * p.B * 4) + pad256((size_t)p.L * p.B * p.Hkv * p.slots * TQ_CHUNK * 4) + 256;
}

}  // namespace

extern "C" {

tq_status tq_append(const tq_append_args* a, void* stream) {
  AppendParams p;
  const tq_status st = append_params(a, &p);
  if (st != TQ_OK) return st;
  cudaStream_t s = (cudaStream_t)stream;
  if (launch_append(p, s) != cudaSuccess) return TQ_ERR_CUDA;
  if (p.in_place && launch_append_commit(p, s) != cudaSuccess) return TQ_ERR_CUDA;
  return TQ_OK;
}

size_t tq_prefill_attn_workspace_size(const tq_query_args* a, const tq_codec* k_codec, const tq_codec* v_codec) {
  PrefillPlan pl;
  return prefill_plan(a, k_codec, v_codec, &pl) == TQ_OK ? pl.bytes : 0;
}

tq_status tq_prefill_attn(const tq_query_args* a, const tq_codec* k_codec, const tq_codec* v_codec, void* workspace,
                          size_t workspace_bytes, void* stream) {
  PrefillPlan pl;
  const tq_status st = prefill_plan(a, k_codec, v_codec, &pl);
  if (st != TQ_OK) return st;
  if (!workspace || !aligned(workspace, 256)) return TQ_ERR_INVALID_ARG;
  if (workspace_bytes < pl.bytes) return TQ_ERR_WORKSPACE;
  PrefillParams& pp = pl.pp;
  pp.ws_acc = (float*)workspace;
  pp.ws_ml = (float2*)((char*)workspace + pl.ml_off);
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e;
  switch (pp.q.D) {
    case 64: e = launch_prefill_d64(pp, s); break;
    case 128: e = launch_prefill_d128(pp, s); break;
    case 256: e = launch_prefill_d256(pp, s); break;
    default: e = launch_prefill_d512(pp, s); break;
  }
  if (e != cudaSuccess) return TQ_ERR_CUDA;
  return launch_prefill_merge(pp, s) == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

size_t tq_attn_mass_workspace_size(const tq_query_args* a, const tq_codec* k_codec) {
  MassPlan pl;
  return mass_plan(a, k_codec, &pl) == TQ_OK ? pl.bytes : 0;
}

tq_status tq_attn_mass(const tq_query_args* a, const tq_codec* k_codec, float* mass, int64_t mass_layer_stride,
                       int32_t mass_cap, float decay, void* workspace, size_t workspace_bytes, void* stream) {
  MassPlan pl;
  const tq_status st = mass_plan(a, k_codec, &pl);
  if (st != TQ_OK) return st;
  MassParams& mp = pl.mp;
  if (!mass || !aligned(mass, 4) || mass_layer_stride < 0 ||
      !layers_apart(mp.q.L, mass_layer_stride, (int64_t)mp.q.B * mp.q.Hkv * mass_cap) ||
      mass_cap < (int64_t)TQ_CHUNK * mp.q.max_chunks + mp.q.max_tail || !std::isfinite(decay) || decay < 0.f)
    return TQ_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256)) return TQ_ERR_INVALID_ARG;
  if (workspace_bytes < pl.bytes) return TQ_ERR_WORKSPACE;
  if (mp.Sc + mp.St == 0) return TQ_OK;  // no token to weigh
  char* ws = (char*)workspace;
  mp.ml = (float2*)(ws + pl.ml);
  mp.logits = (float*)(ws + pl.logits);
  mp.frag = (uint4*)(ws + pl.frag);
  mp.fragd = (uint2*)(ws + pl.fragd);
  mp.qsc = (float*)(ws + pl.qsc);
  mp.qrot = (float*)(ws + pl.qrot);
  mp.mass = mass;
  mp.mass_ls = mass_layer_stride;
  mp.mass_cap = mass_cap;
  mp.decay = decay;
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e;
  if (pl.few) {
    switch (mp.q.D) {
      case 64: e = launch_attn_mass_few_d64(mp, s); break;
      case 128: e = launch_attn_mass_few_d128(mp, s); break;
      case 256: e = launch_attn_mass_few_d256(mp, s); break;
      default: e = launch_attn_mass_few_d512(mp, s); break;
    }
    if (e != cudaSuccess) return TQ_ERR_CUDA;
    return launch_attn_mass_add(mp, s) == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
  }
  for (mp.pass = 0; mp.pass < 2; ++mp.pass) {
    switch (pl.umma ? -mp.q.D : mp.q.D) {
      case -64: e = launch_attn_mass_umma_d64(mp, s); break;
      case -128: e = launch_attn_mass_umma_d128(mp, s); break;
      case 64: e = launch_attn_mass_d64(mp, pl.NT, s); break;
      case 128: e = launch_attn_mass_d128(mp, pl.NT, s); break;
      case 256: e = launch_attn_mass_d256(mp, pl.NT, s); break;
      default: e = launch_attn_mass_d512(mp, pl.NT, s); break;
    }
    if (e != cudaSuccess) return TQ_ERR_CUDA;
  }
  return TQ_OK;
}

size_t tq_evict_mass_workspace_size(const tq_evict_mass_args* a, const tq_codec* k_codec, const tq_codec* v_codec) {
  EvictMassParams p;
  if (evict_mass_params(a, k_codec, v_codec, &p) != TQ_OK) return 0;
  return evict_mass_bytes(p);
}

tq_status tq_evict_mass(const tq_evict_mass_args* a, const tq_codec* k_codec, const tq_codec* v_codec, void* workspace,
                        size_t workspace_bytes, void* stream) {
  EvictMassParams p;
  const tq_status st = evict_mass_params(a, k_codec, v_codec, &p);
  if (st != TQ_OK) return st;
  if (!workspace || !aligned(workspace, 256)) return TQ_ERR_INVALID_ARG;
  if (workspace_bytes < evict_mass_bytes(p)) return TQ_ERR_WORKSPACE;
  p.counts = (int32_t*)workspace;
  p.list = (int32_t*)((char*)workspace + pad256((size_t)p.L * p.B * 4));
  return launch_evict_mass(p, (cudaStream_t)stream) == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

}  // extern "C"
