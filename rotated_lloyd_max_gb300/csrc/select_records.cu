// Records chosen for blocks of queries by an upper bound of their logits.
//
// Scores.  sum_j max(q_j lo_j, q_j hi_j) = q+ . hi + q- . lo with q+ = max(q, 0),
// q- = min(q, 0): a product of bf16 operands over 2 d, records as M and query rows
// as N of mma.sync, so that a record's bounds are read once and straight from
// memory (a lane's eight neighbouring coordinates serve two k-steps, the order of
// the reduction being free); the products are exact, the sums f32.  A record's
// score is the maximum over the rows.
//
// Selection.  A radix selection finds the need-th largest f32 score x.  No f32
// score is further than e from its exact value (below), so that records above
// x + 2 e are chosen, those below x - 2 e are not, and only where the records in
// between are more than the places left are they formed again: bf16 products
// are exact in f32, and a sum kept as two f32 has twice the bits.  So the list
// depends on neither the order of the sums nor the split of the work.  The largest
// of them are found by comparing pairs, or, of more than 64, by a selection as
// before over 64-bit keys, whose ties a bit a record puts in order: the time grows with the
// records however many tie (16384 of them: 53 us with queries of zeros, 0.5 ms where exact sums are formed).
//
// e = 2^-22 a step of the tensor core's 2 d / 16, of the largest sum of a row's
// |terms|: measured, its f32 accumulation (16 products and the accumulator, cut off
// below the largest) is off by at most 2.5 2^-24 of that sum after one step and
// 1.5 2^-24 a step after 64.
#include "attn_mass.cuh"

namespace tq {

constexpr int kSelThreads = 256;
constexpr int kPickThreads = 512;

// what a list covers
struct SelList {
  int l, b, h, t0, rows, m;  // first token, query rows, records it may read
};
__device__ __forceinline__ void select_place(const SelectParams& p, int64_t list, SelList& s) {
  s.h = (int)(list % p.q.Hkv);
  const int64_t x = list / p.q.Hkv;
  const int lb = (int)(x / p.blocks);
  s.t0 = (int)(x % p.blocks) * p.qb;
  s.b = lb % p.q.B;
  s.l = lb / p.q.B;
}
// from the sequence's counters as they are
__device__ __forceinline__ void select_extent(const SelectParams& p, SelList& s, int chunks, int tail, int queries) {
  const QueryParams& q = p.q;
  CacheLen cl;
  cl.n = min(max(chunks, 0), min(q.max_chunks, q.rec_limit));
  cl.len = min(max(tail, 0), q.max_tail);
  cl.total = cl.n * kChunk + cl.len;
  const int tb = min(max(queries, 0), q.T), nt = min(p.qb, tb - s.t0);
  s.rows = max(nt, 0) * q.G;
  s.m = 0;
  if (nt > 0) {
    const int limit = row_limit(q, cl, tb, (s.t0 + nt - 1) * q.G);
    s.m = max(0, min(cl.n, (limit + kChunk - 1) / kChunk));
  }
}
__device__ __forceinline__ SelList select_list(const SelectParams& p, int64_t list) {
  SelList s;
  select_place(p, list, s);
  const int lb = s.l * p.q.B + s.b;
  select_extent(p, s, __ldg(p.q.n_chunks + lb), p.q.tail_len ? __ldg(p.q.tail_len + lb) : 0,
                p.q.q_lens ? __ldg(p.q.q_lens + s.b) : p.q.T);
  return s;
}
// query row r of a list: head r % G of token t0 + r / G
__device__ __forceinline__ const uint16_t* query_row(const SelectParams& p, const SelList& s, int r) {
  const int tok = (int)fast_div((uint32_t)r, p.group), head = r - tok * p.q.G;
  return p.q.q + s.l * p.q.q_ls + s.b * p.q.q_bs + (int64_t)(s.t0 + tok) * p.q.q_ts + (int64_t)(s.h * p.q.G + head) * p.q.D;
}
__device__ __forceinline__ const uint16_t* bounds_row(const SelectParams& p, const SelList& s, int r) {
  return p.bounds + s.l * p.bounds_ls +
         rec_offset(p.q.table, p.q.table_stride, p.q.rec_cap, p.q.Hkv, s.b, s.h, r, 2 * p.q.D);
}
// all ones in the halves of a bf16 pair that are negative: one byte permutation that spreads the signs
__device__ __forceinline__ uint32_t sign_mask2(uint32_t w) {
  uint32_t r;
  asm("prmt.b32 %0, %1, 0, 0xBB99;" : "=r"(r) : "r"(w));
  return r;
}
// the negative halves (LOW) or the others, zero in their place
template <bool LOW>
__device__ __forceinline__ uint4 halves_of(const uint4& q) {
  const uint32_t x = sign_mask2(q.x), y = sign_mask2(q.y), z = sign_mask2(q.z), w = sign_mask2(q.w);
  return LOW ? make_uint4(q.x & x, q.y & y, q.z & z, q.w & w) : make_uint4(q.x & ~x, q.y & ~y, q.z & ~z, q.w & ~w);
}
// by halves, the sign bit where a bf16 is not finite (an exponent of ones carries into it)
__device__ __forceinline__ uint32_t infinite2(uint32_t w) { return ((w & 0x7FFF7FFFu) + 0x00800080u) & 0x80008000u; }
// by halves, the magnitude; what is not finite counts as 0
__device__ __forceinline__ uint32_t finite_abs2(uint32_t w) {
  w &= 0x7FFF7FFFu;
  return w & ~sign_mask2(w + 0x00800080u);
}
__device__ __forceinline__ uint4 max8(const uint4& a, const uint4& b) {
  return make_uint4(__vmaxu2(a.x, b.x), __vmaxu2(a.y, b.y), __vmaxu2(a.z, b.z), __vmaxu2(a.w, b.w));
}
__device__ __forceinline__ uint4 abs4(const uint4& v) {
  return make_uint4(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu, v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu);
}
// twice the error of an f32 score whose terms' magnitudes add up to at most `size`: 4 2^-24 a step (above)
__device__ __forceinline__ float score_error2(int D, float size) { return size * ((float)D * 5.9604644775390625e-8f); }

// Where query rows r0 .. lie as fragments: lane (g, t) of k-step pair k holds coordinates
// 32 k + 8 t .. + 7 of row g.  [n-tile][pair][lane]; rows from nr on are zeros.  Asked for, not waited for.
template <int D, int T>
__device__ __forceinline__ void query_fragments(const SelectParams& p, const SelList& s, int r0, int nr, uint4* frag) {
  constexpr int KP = D / 32;
  for (int i = threadIdx.x; i < (nr + 7) / 8 * KP * 32; i += T) {
    const int ln = i & 31, k = (i >> 5) % KP, r = i / (32 * KP) * 8 + (ln >> 2);
    if (r < nr) cp_async16(frag + i, reinterpret_cast<const uint4*>(query_row(p, s, r0 + r)) + 4 * k + (ln & 3));
    else frag[i] = make_uint4(0, 0, 0, 0);
  }
  cp_async_commit();
}
// the largest finite one of a score fragment's rows below nr; rows 2 t, 2 t + 1 of an n-tile in c[0], c[1] (c[2], c[3])
__device__ __forceinline__ void keep_best(float (&best)[2], const float (&c)[4], int at, int nr) {
#pragma unroll
  for (int e = 0; e < 4; ++e)
    best[e >> 1] = fmaxf(best[e >> 1], at + (e & 1) < nr && c[e] < INFINITY ? c[e] : -INFINITY);  // NaN is neither
}
// c += bounds x queries over 32 coordinates: u, v the bounds of records g, g + 8
__device__ __forceinline__ void score_step(float (&c)[4], const uint4& u, const uint4& v, const uint4& w) {
  const uint32_t a0[4] = {u.x, v.x, u.y, v.y}, a1[4] = {u.z, v.z, u.w, v.w};
  mma_bf16(c, a0, w.x, w.y);
  mma_bf16(c, a1, w.z, w.w);
}

// Scores of p.tile = 128 records a CTA, 16 a warp, against the list's query rows, which
// lie in shared memory (64 KB of them at a time).  Up to head dim 128 a warp's bounds stay
// in registers; the wider ones are read again (from L1) for every 8 NT rows.  The sum of
// |terms| is bounded by that of |q_j| and the CTA's largest |bound| of coordinate j,
// formed the same way.  A part's largest score of each record is kept, so that the exact
// sums ask only the parts that may hold it.  1024 tokens of 32 heads in blocks of 64, 256
// records: 21 us of the call's 33, 13 to 16 of them in mma.sync's loop (256 CTAs, two on
// most SMs); 4096 tokens over 1024 records 306 us, 224 TFLOP/s.
template <int D>
struct ScoreCfg {
  static constexpr bool HELD = D <= 128;
  static constexpr int ROWS = 65536 / (2 * D), NT = HELD ? 2 : 4;  // query rows in shared memory; n-tiles at a time
  static constexpr int SMEM = 65536;
};
template <int D>
__global__ void __launch_bounds__(kSelThreads, 2) select_scores_kernel(const __grid_constant__ SelectParams p) {
  using C = ScoreCfg<D>;
  constexpr int KP = D / 32, NT = C::NT;  // pairs of k-steps of one half (q+ . hi or q- . lo)
  extern __shared__ __align__(16) uint4 frag[];
  __shared__ uint4 top[kSelThreads / 32][D / 8];  // the warps' largest |bound| by coordinate
  __shared__ float red[kSelThreads / 32];
  pdl_start();
  const int64_t at = blockIdx.x / p.shares, list = at / p.tiles;
  const int tile = (int)(at % p.tiles);
  const SelList s = select_list(p, list);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int c0 = tile * p.tile, c1 = min(c0 + p.tile, s.m), c = c0 + 16 * warp;
  const int first = (int)(blockIdx.x % p.shares) * p.share * p.part, end = min(first + p.share * p.part, s.rows);
  if (c0 >= c1 || s.m <= p.keep || first >= end) return;  // nothing here, or all of them are chosen
  query_fragments<D, kSelThreads>(p, s, first, min(C::ROWS, end - first), frag);
  const uint4* rows[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) rows[i] = reinterpret_cast<const uint4*>(bounds_row(p, s, min(c + 8 * i + g, c1 - 1))) + t;
  auto bound = [&](int i, int half, int k) { return __ldg(rows[i] + (half ? 0 : D / 8) + 4 * k); };  // hi, then lo
  uint4 held[C::HELD ? KP : 1][2][2];
  if constexpr (C::HELD) {
#pragma unroll
    for (int k = 0; k < KP; ++k)
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int i = 0; i < 2; ++i) held[k][half][i] = bound(i, half, k);
  }
#pragma unroll
  for (int k = 0; k < KP; ++k) {  // coordinates 32 k + 8 t .. of all the warp's records
    uint4 m = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint4 x;
        if constexpr (C::HELD) x = held[k][half][i];
        else x = bound(i, half, k);
        m = max8(m, make_uint4(finite_abs2(x.x), finite_abs2(x.y), finite_abs2(x.z), finite_abs2(x.w)));
      }
#pragma unroll
    for (int j = 4; j < 32; j <<= 1)
      m = max8(m, make_uint4(__shfl_xor_sync(0xffffffffu, m.x, j), __shfl_xor_sync(0xffffffffu, m.y, j),
                             __shfl_xor_sync(0xffffffffu, m.z, j), __shfl_xor_sync(0xffffffffu, m.w, j)));
    if (g == 0) top[warp][4 * k + t] = m;
  }
  float best[2] = {-INFINITY, -INFINITY}, size[2] = {0.f, 0.f};
  int left = p.part;  // rows to the end of a part
  float* scores = p.scores + (list * p.parts + first / p.part) * p.q.max_chunks + c + g;
  for (int r0 = first; r0 < end; r0 += C::ROWS) {
    const int nr = min(C::ROWS, end - r0);
    if (r0 != first) {
      __syncthreads();
      query_fragments<D, kSelThreads>(p, s, r0, nr, frag);
    }
    cp_async_wait<0>();
    __syncthreads();
    if (r0 == first) {  // of all the warps'
      if (threadIdx.x < D / 2) {
        uint32_t m = 0u;
        for (int w = 0; w < kSelThreads / 32; ++w) m = __vmaxu2(m, reinterpret_cast<const uint32_t*>(top[w])[threadIdx.x]);
        reinterpret_cast<uint32_t*>(top[0])[threadIdx.x] = m;
      }
      __syncthreads();
    }
    if (c < c1) {
      for (int n0 = 0; n0 < nr; n0 += 8 * NT) {
        const uint4* fr = frag + n0 / 8 * KP * 32 + lane;
        float acc[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[nt][e] = 0.f;
#pragma unroll C::HELD ? KP : 2
        for (int k = 0; k < KP; ++k) {
          uint4 x[2][2];
#pragma unroll
          for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              if constexpr (C::HELD) x[half][i] = held[k][half][i];
              else x[half][i] = bound(i, half, k);
            }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if (nt && n0 + 8 * nt >= nr) break;
            const uint4 q = fr[(nt * KP + k) * 32];
            score_step(acc[nt], x[0][0], x[0][1], halves_of<false>(q));
            score_step(acc[nt], x[1][0], x[1][1], halves_of<true>(q));
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) keep_best(best, acc[nt], n0 + 8 * nt + 2 * t, nr);
        left -= 8 * NT;
        if (left == 0 || r0 + n0 + 8 * NT >= end) {  // parts are a multiple of 8 NT rows
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            best[i] = fmaxf(best[i], __shfl_xor_sync(0xffffffffu, best[i], 1));
            best[i] = fmaxf(best[i], __shfl_xor_sync(0xffffffffu, best[i], 2));
            if (t == 0 && c + 8 * i + g < c1) scores[8 * i] = best[i];
            best[i] = -INFINITY;
          }
          left = p.part;
          scores += p.q.max_chunks;
        }
      }
    }
    // the rows' sizes, a warp every eighth n-tile
    for (int n0 = 8 * warp; n0 < nr; n0 += 8 * (kSelThreads / 32)) {
      const uint4* fr = frag + n0 / 8 * KP * 32 + lane;
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
      for (int k = 0; k < KP; ++k) {
        const uint4 m = top[0][4 * k + t];
        score_step(acc, m, m, abs4(fr[k * 32]));
      }
      keep_best(size, acc, n0 + 2 * t, nr);
    }
  }
  const float sz = warp_max(size[0]);
  if (lane == 0) red[warp] = sz;
  __syncthreads();
  if (threadIdx.x == 0) {
    float m = 0.f;
    for (int w = 0; w < kSelThreads / 32; ++w) m = fmaxf(m, red[w]);
    p.limits[blockIdx.x] = m;
  }
}

// a float's order as an unsigned number's, and back
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t u = __float_as_uint(x);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k); }
__device__ __forceinline__ uint64_t order_key(double x) {
  const uint64_t u = (uint64_t)__double_as_longlong(x);
  return u >> 63 ? ~u : u | (1ull << 63);
}

// a + x, the rounding error added to c
__device__ __forceinline__ void add_exact(float& a, float& c, float x) {
  const float s = __fadd_rn(a, x), bb = __fsub_rn(s, a);
  c = __fadd_rn(c, __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(x, bb)));
  a = s;
}

// (x, its rounding errors) of two sums in one, the larger part first
__device__ __forceinline__ float2 join_exact(float2 a, float2 b) {
  float s = a.x, c = __fadd_rn(a.y, b.y);
  add_exact(s, c, b.x);
  const float h = __fadd_rn(s, c);
  return make_float2(h, __fadd_rn(c, __fsub_rn(s, h)));
}

// Records up to which the warps search for the threshold in registers; beyond that its bytes are counted, which
// takes four rounds of shared memory's atomics (2048 lists of 256 records 56 us by search, 68 by counting).
constexpr int kSearch = 256;
// Candidates up to which each sum is compared with all the others; beyond that the border is searched for, whose rounds
// cost about as much as 64 comparisons (32, 64, 128, 256 candidates: 11.2, 14.3, 22.0, 35.7 us by pairs, 13.6, 14.3, 16.0,
// 19.4 by search; 16384: 45.5 ms and 0.46).
constexpr int kPairs = 64;
struct PickMisc {
  uint32_t hist[256];
  uint32_t warp[32];
  uint32_t x, prefix, left, above, cand, items;
  uint32_t item[512];  // candidates' parts that may hold their best row: index << 6 | part
};

// The left-th largest of n numbers, eight bits at a time: key(i, k) says whether number i counts, and sets it.
// left becomes how many of those that equal it are among the left largest.  By all T threads.
template <int T, class K>
__device__ __forceinline__ uint32_t nth_largest(PickMisc& ms, int n, uint32_t& left, K key) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t prefix = 0u;
  for (int sh = 24; sh >= 0; sh -= 8) {
    if (tid < 256) ms.hist[tid] = 0u;
    __syncthreads();
    for (int i = tid; i < n; i += T) {
      uint32_t k;
      if (key(i, k) && (sh == 24 || (k >> (sh + 8)) == prefix)) atomicAdd(&ms.hist[(k >> sh) & 255u], 1u);
    }
    __syncthreads();
    // numbers in bins from this thread's upwards: thread t looks at bin 255 - t
    const uint32_t mine = tid < 256 ? ms.hist[255 - tid] : 0u;
    uint32_t inc = mine;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
      const uint32_t o = __shfl_up_sync(0xffffffffu, inc, k);
      if (lane >= k) inc += o;
    }
    if (lane == 31) ms.warp[warp] = inc;
    __syncthreads();
    for (int w = 0; w < warp; ++w) inc += ms.warp[w];
    if (tid < 256 && inc >= left && inc - mine < left) {
      ms.prefix = prefix << 8 | (uint32_t)(255 - tid);
      ms.left = left - (inc - mine);
    }
    __syncthreads();
    prefix = ms.prefix;
    left = ms.left;
  }
  return prefix;
}

// The list of one block from its keys (smem, one a record; later other uses), of T threads.  e2: twice the error of a
// score.  cand: room for every record; bits: a bit a record.  Starts and ends with every thread past its use of keys.
template <int T>
__device__ __forceinline__ void pick_list(const SelectParams& p, const SelList& s, int64_t list, uint32_t* keys,
                                          uint32_t* cand, uint32_t* bits, PickMisc& ms, float e2) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int32_t* out = p.list + list * p.keep;
  const int M = p.q.max_chunks, words = (s.m + 31) / 32;
  // records that the scores decide on
  const int a = min(p.sink, s.m), z = max(a, s.m - p.recent), need = p.keep - a - (s.m - z);
  for (int w = tid; w < words; w += T) {
    const int lo = a - 32 * w, hi = z - 32 * w;  // chosen: bits below lo, and from hi to m
    uint32_t v = lo >= 32 ? ~0u : lo > 0 ? (1u << lo) - 1u : 0u;
    v |= hi >= 32 ? 0u : hi > 0 ? ~0u << hi : ~0u;
    if (s.m - 32 * w < 32) v &= (1u << (s.m - 32 * w)) - 1u;
    bits[w] = v;
  }
  if (tid == 0) ms.above = ms.cand = 0u;
  if (need > 0) {
    uint32_t x;
    __syncthreads();
    if (z - a <= kSearch) {
      // ---------------------------------------------------------- the largest number that need keys reach, four bits at a
      // time below what all keys have in common: every warp holds all keys and tries one of 16 numbers.  Where one is
      // reached by just `need` keys, the least of those is it.
      static_assert(T == 512, "16 warps");
      uint32_t k[kSearch / 32], most = 0u, least = 0xFFFFFFFFu;
#pragma unroll
      for (int i = 0; i < kSearch / 32; ++i) {
        const int j = a + 32 * i + lane;
        k[i] = j < z ? keys[j] : 0u;
        most = max(most, k[i]);
        least = min(least, j < z ? k[i] : 0xFFFFFFFFu);
      }
      most = __reduce_max_sync(0xffffffffu, most);
      least = __reduce_min_sync(0xffffffffu, least);
      x = least;
      if (most != least) {
        int sh = (31 - __clz((int)(most ^ least))) & ~3;
        x = sh == 28 ? 0u : least >> (sh + 4) << (sh + 4);
        for (; sh >= 0; sh -= 4) {
          const uint32_t trial = x | (uint32_t)warp << sh;
          int n[2] = {0, 0};
#pragma unroll
          for (int i = 0; i < kSearch / 64; i += 2) {
            n[0] += k[i] >= trial;
            n[1] += k[i + 1] >= trial;
          }
          if (z - a > kSearch / 2) {
#pragma unroll
            for (int i = kSearch / 64; i < kSearch / 32; i += 2) {
              n[0] += k[i] >= trial;
              n[1] += k[i + 1] >= trial;
            }
          }
          const int reach = (int)__reduce_add_sync(0xffffffffu, (unsigned)(n[0] + n[1]));
          if (reach == need) {
            least = 0xFFFFFFFFu;
#pragma unroll
            for (int i = 0; i < kSearch / 32; ++i) least = min(least, k[i] >= trial ? k[i] : 0xFFFFFFFFu);
            least = __reduce_min_sync(0xffffffffu, least);
            if (lane == 0) ms.x = least;
          }
          const int votes = __syncthreads_count(lane == 0 ? reach >= need : reach == need);
          if (votes >= 31) {
            x = ms.x;
            break;
          }
          x |= (uint32_t)(votes - 1) << sh;  // the numbers reached are the lower ones
        }
      }
    } else {
      uint32_t left = (uint32_t)need;
      x = nth_largest<T>(ms, z - a, left, [&](int i, uint32_t& k) {
        k = keys[a + i];
        return true;
      });
    }
    // ------------------------------------------------------------ records that f32 cannot tell from it
    const uint32_t lo = order_key(key_value(x) - e2), hi = order_key(key_value(x) + e2);
    for (int i = a + tid; i < z; i += T) {
      const uint32_t k = keys[i];
      if (k > hi) {
        atomicOr(&bits[i >> 5], 1u << (i & 31));
        atomicAdd(&ms.above, 1u);
      } else if (k >= lo) {
        cand[atomicAdd(&ms.cand, 1u)] = (uint32_t)i;
      }
    }
    __syncthreads();
    const int nc = (int)ms.cand, places = need - (int)ms.above;
    if (nc > places) {
      // ---------------------------------------------------------- their scores with twice the bits
      unsigned long long* exact = reinterpret_cast<unsigned long long*>(p.exact) + list * M;
      for (int i = tid; i < nc; i += T) exact[i] = 0ull;
      __syncthreads();
      const int D = p.q.D, sub = lane & 7, grp = tid >> 3;  // eight lanes a (candidate, row), four of them at a time
      constexpr int NG = T / 8;
      // T candidates' parts at a time (a list has 64 at most); none where every product is zero (queries of zeros, which
      // would make candidates of all records): their sums are alike as they are.
      const int lg = 32 - __clz(p.parts - 1);
      for (int c0 = 0; c0 < nc && e2 != 0.f; c0 += T >> lg) {
        if (tid == 0) ms.items = 0u;
        __syncthreads();
        {
          const int i = c0 + (tid >> lg), part = tid & ((1 << lg) - 1);
          if (i < nc && part < p.parts && part * p.part < s.rows &&
              (p.parts == 1 ||
               !(__ldcg(p.scores + (list * p.parts + part) * M + cand[i]) < key_value(keys[cand[i]]) - e2)))
            ms.item[atomicAdd(&ms.items, 1u)] = (uint32_t)i << 6 | (uint32_t)part;
        }
        __syncthreads();
        const int ni = (int)ms.items, per = min(p.part, s.rows);
        // pair i = item i / per, row i % per of its part; from one round to the next both move by fixed steps
        const int stepi = 4 * NG / per, stepr = 4 * NG - stepi * per;
        int it[4], row[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          it[u] = (u * NG + grp) / per;
          row[u] = u * NG + grp - it[u] * per;
        }
        for (;;) {
          const uint4 *q[4], *bnd[4];
          bool far[4];
          int c[4];
          if (__all_sync(0xffffffffu, it[0] >= ni)) break;  // (the others are further)
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const uint32_t e = ms.item[min(it[u], ni - 1)];
            const int r = (int)(e & 63u) * p.part + row[u];
            c[u] = (int)(e >> 6);
            far[u] = it[u] >= ni || r >= s.rows;
            q[u] = reinterpret_cast<const uint4*>(query_row(p, s, far[u] ? 0 : r));
            bnd[u] = reinterpret_cast<const uint4*>(bounds_row(p, s, (int)cand[c[u]]));
          }
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            if (__all_sync(0xffffffffu, far[u])) continue;
            float2 part[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
            uint32_t none = 0u;  // a bound that is not finite: 0 times it is no number in the scores either
            for (int k = sub; k < D / 8; k += 8) {
              const uint4 qv = __ldg(q[u] + k), lv = __ldg(bnd[u] + k), hv = __ldg(bnd[u] + D / 8 + k);
              const uint32_t qw[4] = {qv.x, qv.y, qv.z, qv.w}, lw[4] = {lv.x, lv.y, lv.z, lv.w}, hw[4] = {hv.x, hv.y, hv.z, hv.w};
#pragma unroll
              for (int w = 0; w < 4; ++w) {
                none |= infinite2(lw[w]) | infinite2(hw[w]);
                const uint32_t pick = sign_mask2(qw[w]), bw = (lw[w] & pick) | (hw[w] & ~pick);
                add_exact(part[0].x, part[0].y, bf16_lo(qw[w]) * bf16_lo(bw));
                add_exact(part[1].x, part[1].y, bf16_hi(qw[w]) * bf16_hi(bw));
              }
            }
            if (none) part[0].x = INFINITY;
            float2 sum = join_exact(part[0], part[1]);
#pragma unroll
            for (int k = 1; k < 8; k <<= 1)
              sum = join_exact(sum, make_float2(__shfl_xor_sync(0xffffffffu, sum.x, k), __shfl_xor_sync(0xffffffffu, sum.y, k)));
            sum = join_exact(sum, make_float2(0.f, 0.f));
            // the order of the pairs (sum to the nearest f32, what is left) is that of the sums
            if (!far[u] && sub == 0 && fabsf(sum.x) < INFINITY)
              atomicMax(exact + c[u], (unsigned long long)order_key(sum.x + 0.f) << 32 | order_key(sum.y + 0.f));
          }
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            it[u] += stepi;
            row[u] += stepr;
            if (row[u] >= per) {
              row[u] -= per;
              ++it[u];
            }
          }
        }
        __syncthreads();
      }
      __syncthreads();
      // (the maxima were formed in L2: no line of L1 is asked for them)
      if (nc <= kPairs && e2 != 0.f) {
        for (int i = tid; i < nc; i += T) {
          const unsigned long long k = __ldcg(exact + i);
          const uint32_t r = cand[i];
          int before = 0;
          for (int j = 0; j < nc; ++j) {
            const unsigned long long o = __ldcg(exact + j);
            before += o > k || (o == k && cand[j] < r);
          }
          if (before < places) atomicOr(&bits[r >> 5], 1u << (r & 31));
        }
      } else {
        // the places-th largest sum; of the records that have it, the lowest
        uint32_t left = (uint32_t)places, high = 0u, low = 0u;
        if (e2 != 0.f) {
          high = nth_largest<T>(ms, nc, left, [&](int i, uint32_t& k) {
            k = (uint32_t)(__ldcg(exact + i) >> 32);
            return true;
          });
          low = nth_largest<T>(ms, nc, left, [&](int i, uint32_t& k) {
            const unsigned long long v = __ldcg(exact + i);
            k = (uint32_t)v;
            return (uint32_t)(v >> 32) == high;
          });
        }
        const unsigned long long border = (unsigned long long)high << 32 | low;
        static_assert(TQ_SELECT_MAX_CHUNKS <= 32 * T, "a word of ties a thread");
        uint32_t* ties = keys;  // whose keys have served
        if (tid < words) ties[tid] = 0u;
        __syncthreads();
        for (int i = tid; i < nc; i += T) {
          const unsigned long long k = e2 != 0.f ? __ldcg(exact + i) : 0ull;
          if (k >= border) atomicOr((k > border ? bits : ties) + (cand[i] >> 5), 1u << (cand[i] & 31));
        }
        __syncthreads();
        uint32_t v = tid < words ? ties[tid] : 0u, inc = __popc(v);
        const uint32_t mine = inc;
#pragma unroll
        for (int k = 1; k < 32; k <<= 1) {
          const uint32_t o = __shfl_up_sync(0xffffffffu, inc, k);
          if (lane >= k) inc += o;
        }
        if (lane == 31) ms.warp[warp] = inc;
        __syncthreads();
        for (int w = 0; w < warp; ++w) inc += ms.warp[w];
        for (uint32_t at = inc - mine; v && at < left; ++at) {
          bits[tid] |= v & (0u - v);
          v &= v - 1u;
        }
      }
    } else {
      for (int i = tid; i < nc; i += T) atomicOr(&bits[cand[i] >> 5], 1u << (cand[i] & 31));
    }
  }
  __syncthreads();
  // ---------------------------------------------------------------- the chosen ones in ascending order
  uint32_t base = 0;
  for (int w0 = 0; w0 < words; w0 += T / 32) {  // a warp a word, a lane a record
    const int w = w0 + warp;
    const uint32_t v = w < words ? bits[w] : 0u;
    if (w0) __syncthreads();
    if (lane == 0) ms.warp[warp] = __popc(v);
    __syncthreads();
    uint32_t before = 0, all = 0;
#pragma unroll
    for (int k = 0; k < T / 32; ++k) {
      const uint32_t n = ms.warp[k];
      if (k < warp) before += n;
      all += n;
    }
    if ((v >> lane) & 1u) out[base + before + __popc(v & ((1u << lane) - 1u))] = 32 * w + lane;
    base += all;
  }
}

// what of a list needs no scores: all of it where it takes every record (returns true), else the count
template <int T>
__device__ __forceinline__ bool list_is_all(const SelectParams& p, const SelList& s, int64_t list) {
  int32_t* out = p.list + list * p.keep;
  if (threadIdx.x == 0) p.count[list] = min(s.m, p.keep);
  if (s.m > p.keep) return false;
  for (int i = threadIdx.x; i < p.keep; i += T) out[i] = i < s.m ? i : -1;
  return true;
}

__global__ void __launch_bounds__(kPickThreads) select_pick_kernel(const __grid_constant__ SelectParams p) {
  extern __shared__ __align__(16) uint32_t keys[];  // [max_chunks], then candidates [max_chunks], then chosen records' bits
  __shared__ PickMisc ms;
  pdl_wait();
  const int64_t list = blockIdx.x;
  const SelList s = select_list(p, list);
  if (list_is_all<kPickThreads>(p, s, list)) return;
  const int M = p.q.max_chunks, lane = threadIdx.x & 31, Mp = (M + 3) & ~3;
  const float* score = p.scores + list * p.parts * M;
  const int parts = (s.rows + p.part - 1) / p.part, shares = (parts + p.share - 1) / p.share;
  for (int i = threadIdx.x; i < s.m; i += kPickThreads) {
    float best = -INFINITY;
    for (int k0 = 0; k0 < parts; k0 += 8) {
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = k0 + k < parts ? __ldcg(score + (int64_t)(k0 + k) * M + i) : -INFINITY;
#pragma unroll
      for (int k = 0; k < 8; ++k) best = fmaxf(best, v[k]);
    }
    keys[i] = order_key(best);
  }
  float bm = 0.f;
  const int used = (s.m + p.tile - 1) / p.tile * p.shares;
  for (int i = lane; i < used; i += 32)
    if (i % p.shares < shares) bm = fmaxf(bm, __ldcg(p.limits + list * p.tiles * p.shares + i));
  const float e2 = score_error2(p.q.D, warp_max(bm));
  pick_list<kPickThreads>(p, s, list, keys, keys + Mp, keys + 2 * Mp, ms, e2);
}

// Scores and list in one CTA, for up to 256 records and eight query rows a list: 16
// warps take 16 records each, whose bounds are on their way at once.
constexpr int kOneThreads = 512, kOneRecords = 256;
template <int D>
__global__ void __launch_bounds__(kOneThreads, 2) select_one_kernel(const __grid_constant__ SelectParams p) {
  constexpr int KP = D / 32;
  __shared__ __align__(16) uint4 frag[KP * 32];
  __shared__ __align__(16) uint32_t keys[2 * kOneRecords + kOneRecords / 32];
  __shared__ PickMisc ms;
  __shared__ float red[kOneThreads / 32];
  const int64_t list = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int c = 16 * warp;
  constexpr int AHEAD = 2;  // k-step pairs whose bounds are loaded ahead
  uint4 x[AHEAD][2][2];
  const uint4* rows[2];
  SelList s;
  select_place(p, list, s);
  const int lb = s.l * p.q.B + s.b;
  const int n0 = __ldg(p.q.n_chunks + lb), l0 = p.q.tail_len ? __ldg(p.q.tail_len + lb) : 0;
  const int t0 = p.q.q_lens ? __ldg(p.q.q_lens + s.b) : p.q.T;
  // the first ones are on their way before the sequence's counts are known: up to max_chunks they lie in the buffer
  // (a table's entries are taken as blocks of the pool, whatever they hold)
  if (c < p.q.max_chunks) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      rows[i] = reinterpret_cast<const uint4*>(bounds_row(p, s, min(c + 8 * i + g, p.q.max_chunks - 1))) + t;
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int i = 0; i < 2; ++i) x[k][half][i] = __ldg(rows[i] + (half ? 0 : D / 8) + 4 * k);
  }
  select_extent(p, s, n0, l0, t0);
  if (list_is_all<kOneThreads>(p, s, list)) return;
  const bool work = c < s.m;
  query_fragments<D, kOneThreads>(p, s, 0, s.rows, frag);
  cp_async_wait<0>();
  __syncthreads();
  float best[2] = {-INFINITY, -INFINITY}, size[2] = {0.f, 0.f};
  if (work) {
    float acc[4] = {0.f, 0.f, 0.f, 0.f}, sz[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < KP; ++k) {
      const uint4 q = frag[k * 32 + lane];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const uint4 u = x[k % AHEAD][half][0], v = x[k % AHEAD][half][1];
        if (k + AHEAD < KP) {
#pragma unroll
          for (int i = 0; i < 2; ++i) x[k % AHEAD][half][i] = __ldg(rows[i] + (half ? 0 : D / 8) + 4 * (k + AHEAD));
        }
        const uint4 w = half ? halves_of<true>(q) : halves_of<false>(q);
        score_step(acc, u, v, w);
        score_step(sz, abs4(u), abs4(v), abs4(w));  // |terms|: |lo| where q is negative, |hi| where it is not
      }
    }
    keep_best(best, acc, 2 * t, s.rows);
    keep_best(size, sz, 2 * t, s.rows);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      best[i] = fmaxf(best[i], __shfl_xor_sync(0xffffffffu, best[i], 1));
      best[i] = fmaxf(best[i], __shfl_xor_sync(0xffffffffu, best[i], 2));
      if (t == 0) keys[c + 8 * i + g] = order_key(best[i]);
      if (c + 8 * i + g >= s.m) size[i] = 0.f;
    }
  }
  const float sw = warp_max(fmaxf(size[0], size[1]));
  if (lane == 0) red[warp] = sw;
  __syncthreads();
  const float e2 = score_error2(D, warp_max(red[lane & 15]));
  pick_list<kOneThreads>(p, s, list, keys, keys + kOneRecords, keys + 2 * kOneRecords, ms, e2);
}

template <int D>
static cudaError_t scores_launch(const SelectParams& p, int64_t lists, cudaStream_t s) {
  const cudaError_t e = cudaFuncSetAttribute(select_scores_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, ScoreCfg<D>::SMEM);
  if (e != cudaSuccess) return e;
  select_scores_kernel<D><<<(unsigned)(lists * p.tiles * p.shares), kSelThreads, ScoreCfg<D>::SMEM, s>>>(p);
  return cudaGetLastError();
}

static bool select_in_one(const SelectParams& p) { return p.q.max_chunks <= kOneRecords && p.qb * p.q.G <= 8; }

cudaError_t launch_select_records(const SelectParams& p, cudaStream_t s) {
  const int64_t lists = (int64_t)p.q.L * p.q.B * p.q.Hkv * p.blocks;
  if (select_in_one(p)) {
    switch (p.q.D) {
      case 64: select_one_kernel<64><<<(unsigned)lists, kOneThreads, 0, s>>>(p); break;
      case 128: select_one_kernel<128><<<(unsigned)lists, kOneThreads, 0, s>>>(p); break;
      case 256: select_one_kernel<256><<<(unsigned)lists, kOneThreads, 0, s>>>(p); break;
      case 512: select_one_kernel<512><<<(unsigned)lists, kOneThreads, 0, s>>>(p); break;
      default: return cudaErrorInvalidValue;
    }
    return cudaGetLastError();
  }
  cudaError_t e;
  switch (p.q.D) {
    case 64: e = scores_launch<64>(p, lists, s); break;
    case 128: e = scores_launch<128>(p, lists, s); break;
    case 256: e = scores_launch<256>(p, lists, s); break;
    case 512: e = scores_launch<512>(p, lists, s); break;
    default: return cudaErrorInvalidValue;
  }
  if (e != cudaSuccess) return e;
  const int smem = (p.q.max_chunks + 3) / 4 * 32 + (p.q.max_chunks + 31) / 32 * 4;
  if (smem > 48 * 1024) {
    e = cudaFuncSetAttribute(select_pick_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  return launch_after(select_pick_kernel, dim3((unsigned)lists), kPickThreads, smem, s, 1, p);
}

}  // namespace tq
