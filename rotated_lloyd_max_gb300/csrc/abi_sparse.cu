// The C ABI of the append with norms, the bounds of keys, the selection of
// records and the attention over listed ones (include/tq.h): validation, split
// planning and dispatch, by the rules of abi.cu and abi_cache.cu.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "prefill.cuh"

using namespace tq;

namespace tq {

#define TQ_DECL_DIM(d) cudaError_t launch_prefill_listed_d##d(const PrefillParams& pp, cudaStream_t s);
TQ_DECL_DIM(64)
TQ_DECL_DIM(128)
TQ_DECL_DIM(256)
TQ_DECL_DIM(512)
#undef TQ_DECL_DIM
#define TQ_DECL_BITS(d, k) cudaError_t launch_sparse_few_d##d##_k##k(const PrefillParams& pp, cudaStream_t s);
TQ_DECL_BITS(64, 1)
TQ_DECL_BITS(64, 2)
TQ_DECL_BITS(64, 3)
TQ_DECL_BITS(64, 4)
TQ_DECL_BITS(128, 1)
TQ_DECL_BITS(128, 2)
TQ_DECL_BITS(128, 3)
TQ_DECL_BITS(128, 4)
#undef TQ_DECL_BITS
int prefill_rows_d64();
int prefill_rows_d128();
int prefill_rows_d256();
int prefill_rows_d512();
cudaError_t launch_prefill_merge(const PrefillParams& pp, cudaStream_t s);
cudaError_t launch_merge_rows(const PrefillParams& pp, cudaStream_t s);

}  // namespace tq

namespace {

// Rows of a list on mma.sync at most, two of its tiles (32 of 256 records of 32 sequences, 4 kv heads of 16: 39 us, 90
// on tcgen05; one sequence of 8 kv heads of 16: 17 and 27).
constexpr int kFewRows = 16;
constexpr int kFewRecords = 256;  // records of a team's part of a list there at most
// A tile of 128 ring tokens and a list's part, in records (8 sequences over 16 records + 4096 tokens: 47 us, 51 with a
// tile as one record, 50 as four; 32 of 256 records + 144: 51.5 us, 57.5 with a part as three).
constexpr double kFewTile = 2, kFewPart = 1.5;
constexpr int64_t kMostInt = 0x7FFFFFFF;

// ----------------------------------------------------------------- bounds
// where bounds or records lie: contiguous or a pool
bool records_ok(int rec_cap, const int32_t* table, int table_stride, int max_chunks) {
  return rec_cap > 0 && (!table || table_stride > 0) && max_chunks <= (table ? table_stride : rec_cap);
}

tq_status bounds_params(const tq_codec* kcod, const tq_bounds_args* a, BoundsParams* p) {
  if (!a) return TQ_ERR_INVALID_ARG;
  std::memset(p, 0, sizeof(*p));
  const tq_status st = resolve_codec_dev(kcod, &p->c);
  if (st != TQ_OK) return st;
  if (a->n_layers <= 0 || a->batch <= 0 || a->n_kv_heads <= 0 || a->max_chunks < 0 || a->max_new < 1)
    return TQ_ERR_INVALID_ARG;
  if (!a->k_rec || !a->bounds || !a->n_chunks || !aligned(a->k_rec, 16) || !aligned(a->bounds, 16))
    return TQ_ERR_INVALID_ARG;
  for (const void* x : {(const void*)a->block_table, (const void*)a->n_chunks, (const void*)a->first})
    if (!aligned(x, 4)) return TQ_ERR_INVALID_ARG;
  if (a->k_rec_layer_stride % 16 || a->bounds_layer_stride % 8 ||
      !records_ok(a->rec_cap, a->block_table, a->table_stride, a->max_chunks))
    return TQ_ERR_INVALID_ARG;
  const int64_t heads = (a->block_table ? 1 : (int64_t)a->batch) * a->rec_cap * a->n_kv_heads;
  if (!layers_apart(a->n_layers, a->bounds_layer_stride, heads * 2 * p->c.d)) return TQ_ERR_INVALID_ARG;
  if ((int64_t)a->max_chunks * TQ_CHUNK > kMostTokens) return TQ_ERR_UNSUPPORTED;
  p->L = a->n_layers;
  p->B = a->batch;
  p->Hkv = a->n_kv_heads;
  p->rec = (const uint8_t*)a->k_rec;
  p->rec_ls = a->k_rec_layer_stride;
  p->rec_cap = a->rec_cap;
  p->table = a->block_table;
  p->table_stride = a->table_stride;
  p->rec_limit = a->block_table ? a->table_stride : a->rec_cap;
  p->n_chunks = a->n_chunks;
  p->first = a->first;
  p->max_chunks = a->max_chunks;
  p->max_new = std::min(a->max_new, std::max(a->max_chunks, 1));
  p->bounds = (uint16_t*)a->bounds;
  p->bounds_ls = a->bounds_layer_stride;
  if ((double)a->n_layers * a->batch * a->n_kv_heads * p->max_new > 2000000000.0) return TQ_ERR_UNSUPPORTED;
  p->by_new = make_fast_div((uint32_t)p->max_new);
  p->by_heads = make_fast_div((uint32_t)p->Hkv);
  p->by_batch = make_fast_div((uint32_t)p->B);
  return TQ_OK;
}

// ----------------------------------------------------------------- selection
struct SelectPlan {
  SelectParams p;
  size_t limits, exact, bytes;
};

tq_status select_plan(const tq_select_args* a, SelectPlan* pl) {
  SelectParams& p = pl->p;
  std::memset(pl, 0, sizeof(*pl));
  if (!a) return TQ_ERR_INVALID_ARG;
  const int d = a->head_dim;
  if (!dim_ok(d)) return TQ_ERR_UNSUPPORTED;
  if (a->n_layers <= 0 || a->batch <= 0 || a->t_q <= 0 || a->n_q_heads <= 0 || a->n_kv_heads <= 0 ||
      a->n_q_heads % a->n_kv_heads)
    return TQ_ERR_INVALID_ARG;
  if (!a->q || !aligned(a->q, 16) || !strides_ok(a->q_layer_stride, a->q_batch_stride, a->q_token_stride))
    return TQ_ERR_INVALID_ARG;
  if (!a->bounds || !aligned(a->bounds, 16) || a->bounds_layer_stride % 8 || !a->n_chunks || !a->list || !a->count)
    return TQ_ERR_INVALID_ARG;
  for (const void* x : {(const void*)a->q_lens, (const void*)a->block_table, (const void*)a->n_chunks,
                        (const void*)a->tail_len, (const void*)a->list, (const void*)a->count})
    if (!aligned(x, 4)) return TQ_ERR_INVALID_ARG;
  if (a->max_chunks < 0 || a->max_tail < 0 || (!a->tail_len && a->max_tail) ||
      !records_ok(a->rec_cap, a->block_table, a->table_stride, a->max_chunks))
    return TQ_ERR_INVALID_ARG;
  if (a->q_block < 1 || a->keep < 1 || a->sink < 0 || a->recent < 0 || (int64_t)a->sink + a->recent > a->keep)
    return TQ_ERR_INVALID_ARG;
  if (a->max_chunks > TQ_SELECT_MAX_CHUNKS || (int64_t)a->max_chunks * TQ_CHUNK + a->max_tail > kMostTokens)
    return TQ_ERR_UNSUPPORTED;
  QueryParams& q = p.q;
  q.L = a->n_layers;
  q.B = a->batch;
  q.T = a->t_q;
  q.Hq = a->n_q_heads;
  q.Hkv = a->n_kv_heads;
  q.G = a->n_q_heads / a->n_kv_heads;
  q.D = d;
  if ((int64_t)q.T * q.G > (1 << 28)) return TQ_ERR_UNSUPPORTED;
  q.causal = a->causal != 0;
  q.q = (const uint16_t*)a->q;
  q.q_ls = a->q_layer_stride;
  q.q_bs = a->q_batch_stride;
  q.q_ts = a->q_token_stride;
  q.q_lens = a->q_lens;
  q.rec_cap = a->rec_cap;
  q.table = a->block_table;
  q.table_stride = a->table_stride;
  q.rec_limit = a->block_table ? a->table_stride : a->rec_cap;
  q.n_chunks = a->n_chunks;
  q.tail_len = a->tail_len;
  q.max_chunks = a->max_chunks;
  q.max_tail = q.tail_cap = a->max_tail;
  p.bounds = (const uint16_t*)a->bounds;
  p.bounds_ls = a->bounds_layer_stride;
  p.qb = std::min(a->q_block, a->t_q);
  p.blocks = (int)cdiv(a->t_q, p.qb);
  p.group = make_fast_div((uint32_t)q.G);
  p.keep = a->keep;
  p.sink = a->sink;
  p.recent = a->recent;
  p.list = a->list;
  p.count = a->count;
  p.tile = 128;  // 16 records a warp (select_records.cu)
  p.tiles = (int)std::max<int64_t>(1, cdiv(q.max_chunks, p.tile));
  const double lists = (double)q.L * q.B * q.Hkv * p.blocks;
  // A list's rows are cut into at most 64 parts, of 32 rows or more, and few lists share their parts among CTAs: two
  // blocks of 4096 rows of 512 take 29 us, 76 with 16 parts, 1076 with one.  Two CTAs an SM: with four, 1024 tokens of
  // 32 heads take 36 us instead of 34.
  const int rows = p.qb * q.G;
  p.part = (int)cdiv(cdiv(rows, 64), 32) * 32;
  p.parts = (int)cdiv(rows, p.part);
  p.share = (int)cdiv(p.parts, std::max<int64_t>(1, (int64_t)(2.0 * sm_count() / (lists * p.tiles))));
  p.shares = (int)cdiv(p.parts, p.share);
  if (lists * p.tiles * p.shares > 2147483647.0) return TQ_ERR_UNSUPPORTED;
  const size_t n = (size_t)lists;
  pl->limits = pad256(n * p.parts * q.max_chunks * 4);
  pl->exact = pl->limits + pad256(n * p.tiles * p.shares * 4);
  pl->bytes = pl->exact + pad256(n * q.max_chunks * 8) + 256;
  return TQ_OK;
}

// ----------------------------------------------------------------- attention
struct SparsePlan {
  PrefillParams pp;
  bool few;  // mma.sync
  size_t ml_off, bytes;
};

tq_status sparse_plan(const tq_query_args* a, const tq_record_lists* r, const tq_codec* kcod, const tq_codec* vcod,
                      SparsePlan* pl) {
  PrefillParams& pp = pl->pp;
  std::memset(pl, 0, sizeof(*pl));
  if (!a || !r) return TQ_ERR_INVALID_ARG;
  const tq_status st = query_params(a, kcod, vcod, true, &pp.q);
  if (st != TQ_OK) return st;
  if (!a->k_rec || !r->list || !r->count || !aligned(r->list, 4) || !aligned(r->count, 4) || r->list_stride < 1 ||
      r->q_block < 1)
    return TQ_ERR_INVALID_ARG;
  if (r->list_stride > kMostTokens / TQ_CHUNK) return TQ_ERR_UNSUPPORTED;
  const QueryParams& q = pp.q;
  const int d = q.D;
  pp.rows = q.T * q.G;
  pp.q_block = std::min(r->q_block, q.T);
  pp.list = r->list;
  pp.list_count = r->count;
  pp.list_stride = r->list_stride;
  const int blocks = (int)cdiv(q.T, pp.q_block), rows = pp.q_block * q.G;
  pl->few = d <= 128 && rows <= kFewRows && !q.kc.has_outl && !q.vc.has_outl;
  const int bm = pl->few ? rows : d == 64 ? prefill_rows_d64() : d == 128 ? prefill_rows_d128() : d == 256 ? prefill_rows_d256() : prefill_rows_d512();
  pp.sub = (int)cdiv(rows, bm);
  const int64_t tiles = (int64_t)blocks * pp.sub;
  const int64_t units = (int64_t)q.L * q.B * q.Hkv, U = units * tiles, sms = sm_count();
  if (tiles > 0x3FFFFFFF || U > kMostInt) return TQ_ERR_UNSUPPORTED;
  pp.tiles = (int)tiles;
  const int64_t keep = r->list_stride, ring = cdiv(q.max_tail, TQ_CHUNK), most = std::max(keep, ring);
  if (pl->few) {
    // A run for each team of an SM (sparse_few.cuh), shared between records and ring.  A run's time,
    // in records: its entries, kFewTile for a tile of 128 ring tokens, and kFewPart for every
    // list it has a part of (query set-up, first loads, joining the warps).  Of the
    // entries per run that fill the teams, or fit the lists' ends, the best are taken.
    const int64_t slots = (rows <= 8 ? 4 : 2) * sms;
    auto most_parts = [](int64_t len, int64_t n) -> int64_t {  // runs that share a list of len, n a run
      return len == 0 ? 0 : n % len == 0 ? 1 : len % n == 0 ? len / n : (len - 1) / n + 2;
    };
    auto parts_of = [](int64_t len, int64_t n) -> int64_t {  // lists that a run has a part of
      return len == 0 ? 0 : n % len == 0 ? n / len : len % n == 0 ? 1 : (n - 1) / len + 2;
    };
    double best = 1e300;
    auto consider = [&](int64_t per) {
      per = std::max<int64_t>(1, std::min<int64_t>(per, keep > kFewRecords ? kFewRecords : std::min(U * keep, kMostInt)));
      const int64_t ctas = cdiv(U * keep, per), waves = cdiv(ctas, slots);
      const int64_t left = std::max<int64_t>(waves * slots - ctas, std::max<int64_t>(1, slots / 16));
      int64_t tiles_per = std::max<int64_t>(1, cdiv(U * ring, left));
      if (tiles_per > ring && ring) tiles_per = std::min(cdiv(tiles_per, ring), kMostInt / ring) * ring;
      const double a1 = (double)waves * ((double)per + kFewPart * (double)parts_of(keep, per));
      const double b1 = ring ? kFewTile * (double)tiles_per + kFewPart * (double)parts_of(ring, tiles_per) : 0;
      const double cost = std::max(a1, b1) + 0.05 * (a1 + b1);
      if (cost < best) {
        best = cost;
        pp.cps = (int)per;
        pp.tps = (int)tiles_per;
      }
    };
    if (a->splits > 0) {
      consider(cdiv(keep, std::min<int64_t>(a->splits, keep)));
    } else {
      const double share = (keep + kFewPart) / (keep + kFewPart + (ring ? kFewTile * ring + kFewPart : 0));
      const int64_t even = std::max<int64_t>(1, (int64_t)((double)(U * keep) / (share * (double)slots)) + 1);
      for (const int64_t per : {even, even + 1, even + even / 8, 2 * cdiv(even, 2)}) consider(per);
      if (even >= keep)
        for (int64_t k = even / keep; k <= even / keep + 1; ++k) consider(k * keep);
      else
        for (int64_t k = std::max<int64_t>(1, keep / even); k >= std::max<int64_t>(1, keep / even - 1); --k) consider(cdiv(keep, k));
    }
    pp.ring = (int)ring;
    pp.Sc = (int)most_parts(keep, pp.cps);
    pp.St = (int)most_parts(ring, pp.tps);
    // (the last CTA's teams count past the runs)
    if (cdiv(U * keep, pp.cps) + cdiv(U * ring, pp.tps) > kMostInt - 4) return TQ_ERR_UNSUPPORTED;
    pp.rec_runs = (int)cdiv(U * keep, pp.cps);
    pp.ring_runs = (int)cdiv(U * ring, pp.tps);
  } else {
    // The split count that minimises, in the time of a record's tile, waves of records'
    // CTAs with their set-up and epilogue, the ring's CTAs (whose tiles need no decoding)
    // in the last wave's idle slots or after it, and the partials' traffic.  Where the ring's
    // outlast those slots they go first, at head dims 64 and 128 (1024 tokens of 32 heads over 32 records
    // 150 us, 153 behind; at 256 and 512 they stay behind: 512 tokens of 64 heads of 512 over 32
    // records + 2048 1071 us, 1122 first; 512 of 16 heads of 256 208 us, 226).
    const double setup = d <= 128 ? 4 : 3, ringtile = 0.45;
    const double part = d <= 128 ? 0.03 * std::min(rows, bm) / bm : 0.015;
    double best = 1e300;
    for (int64_t s = 1; s <= std::min<int64_t>(most, 128); ++s) {
      if (a->splits > 0 && s != std::min<int64_t>(a->splits, std::min<int64_t>(most, 128))) continue;
      const int64_t per = cdiv(most, s);
      const int64_t sc = cdiv(keep, per), sr = cdiv(ring, per);
      const int64_t waves = cdiv(U * sc, sms);
      const double one = (double)cdiv(keep, sc) + setup, rest = ringtile * (double)(sr ? cdiv(ring, sr) : 0) + setup;
      const double idle = (double)(waves * sms - U * sc) * one, dense = (double)(U * sr) * rest;
      double cost = (double)waves * one + part * (double)(U * (sc + sr));
      if (dense > 0.9 * idle) cost += std::max(rest, (dense - 0.9 * idle) / (double)sms);
      if (cost < best) {
        best = cost;
        pp.ring_first = d <= 128 && dense > 0.9 * idle;
        pp.cps = (int)per;
        pp.Sc = (int)sc;
        pp.tps = (int)(TQ_CHUNK * per);
        pp.St = (int)sr;
      }
    }
    if (U * (pp.Sc + pp.St) > kMostInt) return TQ_ERR_UNSUPPORTED;
  }
  const int64_t padded = cdiv(pp.rows, 128) * 128;
  const bool by_tile = !pl->few && d <= 128;  // partials in tiles of 128 of a unit's rows
  const int64_t merges = by_tile ? units * padded / 8 : units * pp.rows;
  if (merges > kMostInt) return TQ_ERR_UNSUPPORTED;
  pp.out = (uint16_t*)a->out;
  pp.o_ls = a->out_layer_stride;
  pp.o_bs = a->out_batch_stride;
  pp.o_ts = a->out_token_stride;
  pp.inv_sqrt_d = (float)(1.0 / std::sqrt((double)d));
  const size_t parts = (size_t)(units * (by_tile ? padded : pp.rows)) * (pp.Sc + pp.St);
  pl->ml_off = pad256(parts * d * 4);
  pl->bytes = pl->ml_off + pad256(parts * 8) + 256;
  return TQ_OK;
}

cudaError_t launch_few(const PrefillParams& pp, cudaStream_t s) {
  switch (pp.q.D + pp.q.kc.bits) {
    case 65: return launch_sparse_few_d64_k1(pp, s);
    case 66: return launch_sparse_few_d64_k2(pp, s);
    case 67: return launch_sparse_few_d64_k3(pp, s);
    case 68: return launch_sparse_few_d64_k4(pp, s);
    case 129: return launch_sparse_few_d128_k1(pp, s);
    case 130: return launch_sparse_few_d128_k2(pp, s);
    case 131: return launch_sparse_few_d128_k3(pp, s);
    case 132: return launch_sparse_few_d128_k4(pp, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

extern "C" {

tq_status tq_norm_append(const tq_append_args* a, const tq_head_norm* n, void* stream) {
  AppendParams p;
  const tq_status st = append_params(a, &p);
  if (st != TQ_OK) return st;
  if (!n || (!n->q_weight && !n->k_weight) || (n->q_weight && !a->q) || !aligned(n->q_weight, 16) ||
      !aligned(n->k_weight, 16) || n->q_head_stride < 0 || n->k_head_stride < 0 || n->q_head_stride % 4 ||
      n->k_head_stride % 4 || !std::isfinite(n->eps) || n->eps < 0.f)
    return TQ_ERR_INVALID_ARG;
  const HeadNorm norm = {n->q_weight, n->k_weight, n->q_head_stride, n->k_head_stride, n->eps};
  // With many tokens eight a CTA, all their heads, since a CTA's angles and first loads are a chain of 2 to 3 us: 4864
  // tokens of 48 heads of 128 24 us, 29 with the two tokens a CTA of the plain append; but 1024 tokens 11.1 and 8.5.
  const int64_t eights = (int64_t)p.L * p.B * cdiv(p.T, 8);
  if (eights >= 2 * sm_count()) {
    p.tile = 8;
    p.tiles = (int)cdiv(p.T, 8);
    p.group = p.heads;
  }
  cudaStream_t s = (cudaStream_t)stream;
  if (launch_norm_append(p, norm, s) != cudaSuccess) return TQ_ERR_CUDA;
  if (p.in_place && launch_append_commit(p, s) != cudaSuccess) return TQ_ERR_CUDA;
  return TQ_OK;
}

tq_status tq_key_bounds(const tq_codec* k_codec, const tq_bounds_args* a, void* stream) {
  BoundsParams p;
  const tq_status st = bounds_params(k_codec, a, &p);
  if (st != TQ_OK) return st;
  return launch_key_bounds(p, (cudaStream_t)stream) == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

size_t tq_select_records_workspace_size(const tq_select_args* a) {
  SelectPlan pl;
  return select_plan(a, &pl) == TQ_OK ? pl.bytes : 0;
}

tq_status tq_select_records(const tq_select_args* a, void* workspace, size_t workspace_bytes, void* stream) {
  SelectPlan pl;
  const tq_status st = select_plan(a, &pl);
  if (st != TQ_OK) return st;
  if (!workspace || !aligned(workspace, 256)) return TQ_ERR_INVALID_ARG;
  if (workspace_bytes < pl.bytes) return TQ_ERR_WORKSPACE;
  char* ws = (char*)workspace;
  pl.p.scores = (float*)ws;
  pl.p.limits = (float*)(ws + pl.limits);
  pl.p.exact = (uint64_t*)(ws + pl.exact);
  return launch_select_records(pl.p, (cudaStream_t)stream) == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

size_t tq_sparse_attn_workspace_size(const tq_query_args* a, const tq_record_lists* lists, const tq_codec* k_codec,
                                     const tq_codec* v_codec) {
  SparsePlan pl;
  return sparse_plan(a, lists, k_codec, v_codec, &pl) == TQ_OK ? pl.bytes : 0;
}

tq_status tq_sparse_attn(const tq_query_args* a, const tq_record_lists* lists, const tq_codec* k_codec,
                         const tq_codec* v_codec, void* workspace, size_t workspace_bytes, void* stream) {
  SparsePlan pl;
  const tq_status st = sparse_plan(a, lists, k_codec, v_codec, &pl);
  if (st != TQ_OK) return st;
  if (!workspace || !aligned(workspace, 256)) return TQ_ERR_INVALID_ARG;
  if (workspace_bytes < pl.bytes) return TQ_ERR_WORKSPACE;
  PrefillParams& pp = pl.pp;
  pp.ws_acc = (float*)workspace;
  pp.ws_ml = (float2*)((char*)workspace + pl.ml_off);
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e;
  if (pl.few) {
    e = launch_few(pp, s);
  } else {
    switch (pp.q.D) {
      case 64: e = launch_prefill_listed_d64(pp, s); break;
      case 128: e = launch_prefill_listed_d128(pp, s); break;
      case 256: e = launch_prefill_listed_d256(pp, s); break;
      default: e = launch_prefill_listed_d512(pp, s); break;
    }
  }
  if (e != cudaSuccess) return TQ_ERR_CUDA;
  e = pl.few || pp.q.D > 128 ? launch_merge_rows(pp, s) : launch_prefill_merge(pp, s);
  return e == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

}  // extern "C"
