// Eviction by accumulated attention weight: of the 128 n compressed tokens of
// a stream (layer, sequence, kv head) the 128 n' of the largest weight stay,
// in their order, and their records are compacted.
//
// mass_select_kernel finds the threshold by a radix selection over the
// weights' bits, mapped to integers of the same order: three passes of 11, 11
// and 10 bits, each a histogram of the keys that share the digits found so far.
// A cluster of CTAs holds one stream: every CTA keeps the keys of its run of
// tokens in shared memory (they are read from memory once), histograms meet
// through distributed shared memory, and ballots give each remaining token
// its rank, so that ties fall to the lower index and the list comes out in
// order without a sort.
//
// mass_compact_kernel moves what remains: scales and code rows (16 bytes a
// thread, or 8 where a row is no multiple of 16), side lists re-based, weights
// behind their tokens.  The destination index of a token is never above its
// source index.  In place, a cluster therefore walks one stream in waves of
// ascending records: all its CTAs gather a wave into registers, meet at the
// cluster barrier, and write it; what a wave overwrites no later wave reads.
// Out of place nothing orders the records and a CTA takes one each.  Both
// are bound by memory: every remaining record is read and written once.
//
// 256 streams of 32768 tokens to 8192 each, 4-bit keys and 3-bit values: 188 us,
// 59 of them the selection (two waves of one CTA per SM; keys read again from L2
// with two CTAs per SM: 8 us longer), 123 the moves (rows of 64 and 48 bytes and
// scales of 4 gathered at random take 32-byte sectors: 780 MB, 115 us).
#include <cooperative_groups.h>

#include <algorithm>
#include <type_traits>

#include "cache_params.h"
#include "tq_common.cuh"

namespace cg = cooperative_groups;

namespace tq {

constexpr int kSelThreads = 1024, kSelWarps = kSelThreads / 32;
constexpr int kSelBins = 2048;
constexpr int kBatch = 8;
constexpr int kMoveThreads = 256;
constexpr int kMoveUnits = 8;   // 16-byte units a thread may hold: 128 rows of 256 bytes at most
constexpr int kMoveCluster = 8;

// order-preserving image of a weight; NaN below every number, -0 equal to 0
__device__ __forceinline__ uint32_t mass_key(float m) {
  if (m != m) return 0u;
  const uint32_t u = __float_as_uint(m + 0.f);
  return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}

struct SelShared {
  uint32_t hist[2][kSelBins], total[kSelBins], more[kSelBins];
  uint32_t warp_sum[kSelWarps];
  uint32_t digit, left;
  uint32_t gt[kSelWarps], eq[kSelWarps];
  uint32_t cta_gt, cta_eq;
};

// CACHED: the CTA's keys stay in shared memory (otherwise, where a cluster of eight
// cannot keep them, each pass reads the weights again).  CLUSTER: several CTAs hold
// a stream; their histograms meet slice by slice, CTA r summing the r-th slice of
// the bins over all of them.
template <bool CACHED, bool CLUSTER>
__global__ void __launch_bounds__(kSelThreads, 1) mass_select_kernel(const __grid_constant__ EvictMassParams p) {
  __shared__ SelShared sh;
  extern __shared__ uint32_t keys[];
  pdl_start();
  cg::cluster_group cl = cg::this_cluster();
  const int C = CLUSTER ? (int)cl.num_blocks() : 1, rank = CLUSTER ? (int)cl.block_rank() : 0;
  const int64_t stream = blockIdx.x / C;
  const int h = stream % p.Hkv, lb = stream / p.Hkv, l = lb / p.B, b = lb % p.B;
  const int n = min(max(p.n_chunks[lb], 0), min(p.max_chunks, p.rec_limit));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (h == 0 && rank == 0 && tid == 0) p.counts[lb] = n;
  const int N = n * kChunk, K = min(n, p.keep) * kChunk;
  int32_t* list = p.list + stream * (int64_t)p.slots * kChunk;
  int32_t* kept = p.kept ? p.kept + stream * (int64_t)p.keep * kChunk : nullptr;
  auto keep_token = [&](uint32_t at, int token) {
    list[at] = token;
    if (kept) kept[at] = token;
  };
  if (n <= p.keep) {  // everything stays
    for (int i = rank * kSelThreads + tid; i < N; i += C * kSelThreads) keep_token(i, i);
    return;
  }
  const float* mass = p.mass + l * p.mass_ls + ((int64_t)b * p.Hkv + h) * p.mass_cap;
  const int slice = (n + C - 1) / C * kChunk;
  const int first = min(rank * slice, N), count = min(slice, N - first);
  auto load_key = [&](int i) -> uint32_t {
    const int at = first + i;
    return at < p.sink || at >= N - p.recent ? 0xFFFFFFFFu : mass_key(mass[at]);
  };
  auto key_at = [&](int i) -> uint32_t { return CACHED ? keys[i] : load_key(i); };
  uint32_t prefix = 0, mask = 0, want = K;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : 2048;
    uint32_t* hist = sh.hist[pass & 1];
    if (pass == 0) {
      // the leading digits of weights are few (their exponents): four copies of
      // the histogram, a quarter of the lanes each, keep the atomics from queueing
      uint32_t* all = sh.hist[0];  // hist[0], hist[1], total, more lie one behind another
      for (int i = tid; i < 4 * kSelBins; i += kSelThreads) all[i] = 0;
      __syncthreads();
      for (int i0 = tid; i0 < count; i0 += kBatch * kSelThreads) {  // a batch's loads in flight together
        uint32_t key[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
          if (i0 + k * kSelThreads < count) key[k] = load_key(i0 + k * kSelThreads);
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
          if (i0 + k * kSelThreads < count) {
            if (CACHED) keys[i0 + k * kSelThreads] = key[k];
            atomicAdd(&all[(lane & 3) * kSelBins + (key[k] >> 21)], 1u);
          }
      }
      __syncthreads();
      for (int i = tid; i < kSelBins; i += kSelThreads)
        all[i] += (all[kSelBins + i] + all[2 * kSelBins + i]) + all[3 * kSelBins + i];
    } else {
      for (int i = tid; i < kSelBins; i += kSelThreads) hist[i] = 0;
      __syncthreads();
#pragma unroll 8
      for (int i = tid; i < count; i += kSelThreads) {
        const uint32_t key = key_at(i);
        if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & (bins - 1)], 1u);
      }
    }
    if constexpr (CLUSTER) {  // the slice's totals go back to every CTA's second copy
      cl.sync();
      const int per = kSelBins / C;
      for (int i = tid; i < per; i += kSelThreads) {
        uint32_t sum = 0;
        for (int r = 0; r < C; ++r) sum += cl.map_shared_rank(hist, r)[rank * per + i];
        for (int r = 0; r < C; ++r) cl.map_shared_rank(sh.total, r)[rank * per + i] = sum;
      }
      cl.sync();
    } else {
      __syncthreads();
    }
    // thread t holds bins 2t, 2t + 1; the digit is the largest whose count of
    // keys at or above it reaches `want`
    const uint32_t* tot = CLUSTER ? sh.total : hist;
    const uint32_t b0 = tot[2 * tid], b1 = tot[2 * tid + 1], mine = b0 + b1;
    uint32_t up = mine;  // inclusive sum over this lane and those above it
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const uint32_t o = __shfl_down_sync(0xffffffffu, up, m);
      if (lane + m < 32) up += o;
    }
    if (lane == 0) sh.warp_sum[warp] = up;
    __syncthreads();
    uint32_t above = up - mine;
    {
      const uint32_t others = lane > warp ? sh.warp_sum[lane] : 0u;  // 32 warps
      above += __reduce_add_sync(0xffffffffu, others);
    }
    if (above < want && above + mine >= want) {
      const bool upper = above + b1 >= want;
      sh.digit = 2 * tid + (upper ? 1 : 0);
      sh.left = want - above - (upper ? 0 : b1);
    }
    __syncthreads();
    prefix |= sh.digit << shift;
    mask |= (uint32_t)(bins - 1) << shift;
    want = sh.left;
  }
  // prefix is the smallest key that stays, `want` of its ties do
  const int run = (count + kSelThreads - 1) / kSelThreads * 32;  // tokens of a warp, contiguous
  const int w0 = min(warp * run, count), w1 = min(w0 + run, count);
  uint32_t gt = 0, eq = 0;
#pragma unroll 8
  for (int i = w0 + lane; i < w1; i += 32) {
    const uint32_t key = key_at(i);
    gt += key > prefix;
    eq += key == prefix;
  }
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  if (lane == 0) {
    sh.gt[warp] = gt;
    sh.eq[warp] = eq;
  }
  __syncthreads();
  // before this warp's run: the warps in front, and the CTAs in front
  uint32_t gt0 = __reduce_add_sync(0xffffffffu, lane < warp ? sh.gt[lane] : 0u);
  uint32_t eq0 = __reduce_add_sync(0xffffffffu, lane < warp ? sh.eq[lane] : 0u);
  if constexpr (CLUSTER) {
    if (tid == kSelThreads - 1) {
      sh.cta_gt = gt0 + sh.gt[warp];
      sh.cta_eq = eq0 + sh.eq[warp];
    }
    cl.sync();
    for (int r = 0; r < rank; ++r) {
      gt0 += *cl.map_shared_rank(&sh.cta_gt, r);
      eq0 += *cl.map_shared_rank(&sh.cta_eq, r);
    }
  }
#pragma unroll 4
  for (int i0 = w0; i0 < w1; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t key = i < w1 ? key_at(i) : 0u;
    const bool g = i < w1 && key > prefix, e = i < w1 && key == prefix;
    const uint32_t bg = __ballot_sync(0xffffffffu, g), be = __ballot_sync(0xffffffffu, e);
    const uint32_t lower = (1u << lane) - 1u;
    const uint32_t gb = gt0 + __popc(bg & lower), eb = eq0 + __popc(be & lower);
    if (g || (e && eb < want)) keep_token(gb + min(eb, want), first + i);
    gt0 += __popc(bg);
    eq0 += __popc(be);
  }
  if constexpr (CLUSTER) cl.sync();  // no CTA leaves while another reads its counters
}

// ----------------------------------------------------------------- compaction
struct MoveShared {
  int64_t at[kChunk];   // byte offset of each slot's source record
  int src[kChunk];      // its slot there
  int off[kChunk + 1];  // side list: entries before each slot in the destination
  int from[kChunk];     // and before it in the source
  int warp_sum[4];
};

// One destination record: gathered into registers (entries into shared
// memory), then, after `meet` (the cluster's barrier in place), written.
template <int UNIT, bool OUTL, class Src, class Meet>
__device__ __forceinline__ void move_record(const CodecDev& c, const uint8_t* base, Src&& src_of, uint8_t* dst,
                                            const int32_t* list, bool live, int r, bool in_place, MoveShared& sh,
                                            uint32_t* ent, Meet&& meet) {
  using V = typename std::conditional<UNIT == 16, uint4, uint2>::type;
  const int tid = threadIdx.x;
  const int row = c.off_norm / kChunk, upr = row / UNIT, units = kChunk * upr;
  bool moves = false;
  if (live && tid < kChunk) {
    const int s = list[r * kChunk + tid];
    sh.at[tid] = src_of(s / kChunk);
    sh.src[tid] = s % kChunk;
    moves = s != r * kChunk + tid;
  }
  // in place, a record whose tokens all stay where they are is left alone
  const bool go = __syncthreads_or(moves) || (live && !in_place);
  const bool lists = OUTL && c.has_outl;
  V buf[kMoveUnits * 16 / UNIT];
  float scale = 0.f;
  if (go) {
#pragma unroll
    for (int k = 0; k < kMoveUnits * 16 / UNIT; ++k) {
      const int u = tid + k * kMoveThreads;
      if (u < units) {
        const int slot = u / upr, part = u % upr;
        buf[k] = *reinterpret_cast<const V*>(base + sh.at[slot] + sh.src[slot] * row + part * UNIT);
      }
    }
    if (tid < kChunk) scale = *reinterpret_cast<const float*>(base + sh.at[tid] + c.off_norm + 4 * sh.src[tid]);
    if (lists) {
      int cnt = 0;
      if (tid < kChunk) {
        const uint8_t* cs = base + sh.at[tid] + c.off_count;
        const int s = sh.src[tid];
        int before = 0;
        for (int w = 0; w < kChunk / 4; ++w) {  // entries of the slots in front
          uint32_t v = reinterpret_cast<const uint32_t*>(cs)[w];
          const int inside = s - 4 * w;
          if (inside < 4) v &= inside > 0 ? (1u << (8 * inside)) - 1u : 0u;
          before = __dp4a(v, 0x01010101u, (uint32_t)before);
        }
        cnt = min((int)cs[s], max(c.cap - before, 0));
        sh.from[tid] = before;
        int inc = cnt;
        for (int m = 1; m < 32; m <<= 1) {
          const int o = __shfl_up_sync(0xffffffffu, inc, m);
          if ((tid & 31) >= m) inc += o;
        }
        sh.off[tid + 1] = inc;
        if ((tid & 31) == 31) sh.warp_sum[tid >> 5] = inc;
      }
      __syncthreads();
      if (tid < kChunk) {
        int add = 0;
        for (int w = 0; w < (tid >> 5); ++w) add += sh.warp_sum[w];
        sh.off[tid + 1] = min(sh.off[tid + 1] + add, c.cap);  // entries past the capacity are dropped
        if (tid == 0) sh.off[0] = 0;
      }
      __syncthreads();
      for (int slot = tid >> 5; slot < kChunk; slot += kMoveThreads / 32) {
        const int o = sh.off[slot], m = sh.off[slot + 1] - o;
        const uint32_t* es = reinterpret_cast<const uint32_t*>(base + sh.at[slot] + c.off_entries) + sh.from[slot];
        for (int e = tid & 31; e < m; e += 32) ent[o + e] = es[e];
      }
      __syncthreads();
    }
  }
  meet();
  if (go) {
#pragma unroll
    for (int k = 0; k < kMoveUnits * 16 / UNIT; ++k) {
      const int u = tid + k * kMoveThreads;
      if (u < units) *reinterpret_cast<V*>(dst + u * UNIT) = buf[k];
    }
    if (tid < kChunk) reinterpret_cast<float*>(dst + c.off_norm)[tid] = scale;
    if (lists) {
      if (tid < kChunk) dst[c.off_count + tid] = (uint8_t)(sh.off[tid + 1] - sh.off[tid]);
      uint32_t* ed = reinterpret_cast<uint32_t*>(dst + c.off_entries);
      for (int e = tid; e < sh.off[kChunk]; e += kMoveThreads) ed[e] = ent[e];
    }
  }
  __syncthreads();  // the bookkeeping block is free again
}

template <int UNIT, bool OUTL, bool INPLACE>
__global__ void __launch_bounds__(kMoveThreads) mass_compact_kernel(const __grid_constant__ EvictMassParams p) {
  __shared__ MoveShared sh;
  extern __shared__ uint32_t ent[];
  const int job = blockIdx.z;  // 0: keys, 1: values, 2: weights
  pdl_wait();
  const int64_t stream = blockIdx.y;
  const int h = stream % p.Hkv, lb = stream / p.Hkv, l = lb / p.B, b = lb % p.B;
  const int n = p.counts[lb], left = min(n, p.keep);
  const int32_t* list = p.list + stream * (int64_t)p.slots * kChunk;
  const int tid = threadIdx.x;
  if (job == 0 && h == 0 && blockIdx.x == 0 && tid == 0) p.n_chunks_dst[lb] = left;
  if (INPLACE && n <= p.keep) return;  // nothing moves (the whole cluster leaves)
  if (job == 1 && p.shared) return;
  const int C = INPLACE ? kMoveCluster : 1;
  if (job == 2) {
    const int len = p.tail_len ? min(max(p.tail_len[lb], 0), p.max_tail) : 0;
    const float* m = p.mass + l * p.mass_ls + ((int64_t)b * p.Hkv + h) * p.mass_cap;
    float* d = p.mass_dst + l * p.mass_dst_ls + ((int64_t)b * p.Hkv + h) * p.mass_dst_cap;
    const int live = left * kChunk, all = live + len, was = n * kChunk;
    auto source = [&](int i) { return i < live ? list[i] : was + (i - live); };
    constexpr int PER = 8;
    const int64_t step = (int64_t)gridDim.x * kMoveThreads * PER;  // past 32 bits from 2^20 records on
    for (int64_t i0 = 0; i0 < all; i0 += step) {
      const int64_t at = i0 + (int64_t)blockIdx.x * PER * kMoveThreads + tid;
      float v[PER];
#pragma unroll
      for (int k = 0; k < PER; ++k) {
        const int64_t i = at + k * kMoveThreads;
        v[k] = i < all ? m[source((int)i)] : 0.f;
      }
      if constexpr (INPLACE) cg::this_cluster().sync();
#pragma unroll
      for (int k = 0; k < PER; ++k) {
        const int64_t i = at + k * kMoveThreads;
        if (i < all) d[i] = v[k];
      }
    }
    if (INPLACE)
      for (int i = all + blockIdx.x * kMoveThreads + tid; i < was + len; i += C * kMoveThreads) d[i] = 0.f;
    return;
  }
  const CodecDev& c = job == 0 ? p.kc : p.vc;
  const uint8_t* base = (job == 0 ? p.k_rec + l * p.k_ls : p.v_rec + l * p.v_ls);
  uint8_t* dbase = (job == 0 ? p.k_dst + l * p.kd_ls : p.v_dst + l * p.vd_ls);
  auto src_of = [&](int r) { return rec_offset(p.table, p.table_stride, p.rec_cap, p.Hkv, b, h, r, c.rec_bytes); };
  for (int r0 = INPLACE ? 0 : (int)blockIdx.x; r0 < left; r0 += INPLACE ? C : (int)gridDim.x) {
    const int r = INPLACE ? r0 + (int)blockIdx.x : r0;
    const bool live = r < left;
    uint8_t* dst =
        dbase + rec_offset(p.dst_table, p.dst_table_stride, p.dst_cap, p.Hkv, b, h, live ? r : 0, c.rec_bytes);
    move_record<UNIT, OUTL>(c, base, src_of, dst, list, live, r, INPLACE, sh, ent, [&] {
      if constexpr (INPLACE) cg::this_cluster().sync();
    });
  }
}

// Out of place without side lists nothing ties the tokens of a record together:
// a warp takes 32 of them, a lane each for its source and scale, and the lanes
// together for the code rows, with every load of a task in flight at once and no
// barrier.
template <int UNIT>
__global__ void __launch_bounds__(kMoveThreads) mass_move_kernel(const __grid_constant__ EvictMassParams p) {
  using V = typename std::conditional<UNIT == 16, uint4, uint2>::type;
  pdl_wait();
  const int64_t stream = blockIdx.y;
  const int h = stream % p.Hkv, lb = stream / p.Hkv, l = lb / p.B, b = lb % p.B;
  const int n = p.counts[lb], left = min(n, p.keep);
  const int32_t* list = p.list + stream * (int64_t)p.slots * kChunk;
  const int tid = threadIdx.x, lane = tid & 31;
  if (h == 0 && blockIdx.x == 0 && tid == 0) p.n_chunks_dst[lb] = left;
  const int i0 = (blockIdx.x * kMoveThreads + tid) & ~31;  // the warp's first token
  const int live = left * kChunk;
  // weights: the remaining tokens' and the ring's behind them
  const int len = p.tail_len ? min(max(p.tail_len[lb], 0), p.max_tail) : 0;
  const float* m = p.mass + l * p.mass_ls + ((int64_t)b * p.Hkv + h) * p.mass_cap;
  float* d = p.mass_dst + l * p.mass_dst_ls + ((int64_t)b * p.Hkv + h) * p.mass_dst_cap;
  const int i = i0 + lane;
  if (i0 >= live) {
    if (i < live + len) d[i] = m[n * kChunk + (i - live)];
    return;
  }
  const int src = list[i];
  const float w = m[src];
  const int sc = src / kChunk, slot = src % kChunk, r = i0 / kChunk;
  auto move = [&](const CodecDev& c, const uint8_t* base, uint8_t* dbase) {
    const uint8_t* rec = base + rec_offset(p.table, p.table_stride, p.rec_cap, p.Hkv, b, h, sc, c.rec_bytes);
    uint8_t* dst = dbase + rec_offset(p.dst_table, p.dst_table_stride, p.dst_cap, p.Hkv, b, h, r, c.rec_bytes);
    const int row = c.off_norm / kChunk, upr = row / UNIT;
    const int inv = (65536 + upr - 1) / upr;  // u / upr = u inv >> 16 for u < 1024
    const float scale = *reinterpret_cast<const float*>(rec + c.off_norm + 4 * slot);
    const uint64_t from = (uint64_t)(rec + slot * row);
    const int first = (i0 % kChunk) * row;
    for (int k0 = 0; k0 < upr; k0 += 4) {
      V v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int u = lane + 32 * (k0 + k), q = u * inv >> 16;
        const uint64_t a = __shfl_sync(0xffffffffu, from, q & 31);
        if (k0 + k < upr) v[k] = *reinterpret_cast<const V*>(a + (u - q * upr) * UNIT);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (k0 + k < upr) *reinterpret_cast<V*>(dst + first + (lane + 32 * (k0 + k)) * UNIT) = v[k];
    }
    reinterpret_cast<float*>(dst + c.off_norm)[i % kChunk] = scale;
  };
  move(p.kc, p.k_rec + l * p.k_ls, p.k_dst + l * p.kd_ls);
  if (!p.shared) move(p.vc, p.v_rec + l * p.v_ls, p.v_dst + l * p.vd_ls);
  d[i] = w;
}

template <int UNIT>
static cudaError_t move_launch(const EvictMassParams& p, cudaStream_t s) {
  const int64_t tokens = (int64_t)p.slots * kChunk + p.max_tail;
  const dim3 grid((unsigned)((tokens + kMoveThreads - 1) / kMoveThreads), p.L * p.B * p.Hkv);
  return launch_after(mass_move_kernel<UNIT>, grid, kMoveThreads, 0, s, 1, p);
}

template <int UNIT, bool OUTL, bool INPLACE>
static cudaError_t compact_launch(const EvictMassParams& p, cudaStream_t s) {
  auto kern = mass_compact_kernel<UNIT, OUTL, INPLACE>;
  int cap = 0;
  if (OUTL) cap = std::min(std::max(p.kc.has_outl ? p.kc.cap : 0, p.vc.has_outl ? p.vc.cap : 0), kChunk * 255);
  const int smem = 4 * cap;
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  return launch_after(kern, dim3(INPLACE ? kMoveCluster : p.slots, p.L * p.B * p.Hkv, 3), kMoveThreads, smem, s,
                      INPLACE ? kMoveCluster : 1, p);
}

template <int UNIT, bool OUTL>
static cudaError_t compact_pick(const EvictMassParams& p, cudaStream_t s) {
  if (p.in_place) return compact_launch<UNIT, OUTL, true>(p, s);
  if constexpr (OUTL) return compact_launch<UNIT, OUTL, false>(p, s);
  else return move_launch<UNIT>(p, s);
}

cudaError_t launch_evict_mass(const EvictMassParams& p, cudaStream_t s) {
  // One CTA a stream, or several (a cluster of at most 8) where the streams do
  // not fill the SMs and a CTA keeps 4096 tokens, or where one CTA's shared
  // memory does not hold the keys.  (256 streams of 32768 tokens: 8 CTAs each
  // took 217 us, mostly for meetings of the histograms.)
  const int64_t streams = (int64_t)p.L * p.B * p.Hkv;
  auto bytes = [&](int c) { return (int64_t)((p.max_chunks + c - 1) / c) * kChunk * 4; };
  int C = 1;
  while (C < 8 && ((p.max_chunks > 32 * C && streams * C < sm_count()) || bytes(C) > 192 * 1024)) C *= 2;
  const bool cached = bytes(C) <= 192 * 1024;
  const int smem = cached ? (int)bytes(C) : 0;
  auto kern = C > 1 ? (cached ? mass_select_kernel<true, true> : mass_select_kernel<false, true>)
                    : mass_select_kernel<true, false>;
  if (smem + (int)sizeof(SelShared) > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(streams * C));
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = C;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = C > 1 ? 1 : 0;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p);
  if (e != cudaSuccess) return e;
  const bool outl = p.kc.has_outl || p.vc.has_outl;
  const bool wide = p.kc.off_norm / kChunk % 16 == 0 && p.vc.off_norm / kChunk % 16 == 0;
  if (outl) return wide ? compact_pick<16, true>(p, s) : compact_pick<8, true>(p, s);
  return wide ? compact_pick<16, false>(p, s) : compact_pick<8, false>(p, s);
}

}  // namespace tq
