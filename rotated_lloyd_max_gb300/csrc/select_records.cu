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
// depends on neither the order of the sums nor the split of the work.
//
// e: the tensor core adds 16 products and the accumulator with a relative error
// of at most 2^-21 of the largest partial sum (f32 accumulation with truncated
// alignment is within 2^-22); 2 d / 16 such steps, partial sums at most
// |q|_1 max|bound|: e = d 2^-24 |q|_1 max|bound|, of the list's largest |q|_1 and
// bound.
#include "attn_mass.cuh"

namespace tq {

constexpr int kSelThreads = 128;  // scores: four warps, 16 records a warp at a time
constexpr int kPickThreads = 256;

// what a list covers
struct SelList {
  int l, b, h, t0, rows, m;  // first token, query rows, records it may read
};
__device__ __forceinline__ SelList select_list(const SelectParams& p, int64_t list) {
  SelList s;
  const QueryParams& q = p.q;
  s.h = (int)(list % q.Hkv);
  const int64_t x = list / q.Hkv;
  const int j = (int)(x % p.blocks);
  const int lb = (int)(x / p.blocks);
  s.b = lb % q.B;
  s.l = lb / q.B;
  const int tb = query_len(q, s.b);
  s.t0 = j * p.qb;
  const int nt = min(p.qb, tb - s.t0);
  s.rows = max(nt, 0) * q.G;
  s.m = 0;
  if (nt > 0) {
    const CacheLen cl = cache_len(q, lb);
    const int limit = row_limit(q, cl, tb, (s.t0 + nt - 1) * q.G);
    s.m = max(0, min(cl.n, (limit + kChunk - 1) / kChunk));
  }
  return s;
}
// query row r of a list: head r % G of token t0 + r / G
__device__ __forceinline__ const uint16_t* query_row(const SelectParams& p, const SelList& s, int r) {
  return p.q.q + s.l * p.q.q_ls + s.b * p.q.q_bs + (int64_t)(s.t0 + r / p.q.G) * p.q.q_ts +
         (int64_t)(s.h * p.q.G + r % p.q.G) * p.q.D;
}
__device__ __forceinline__ const uint16_t* bounds_row(const SelectParams& p, const SelList& s, int r) {
  return p.bounds + s.l * p.bounds_ls +
         rec_offset(p.q.table, p.q.table_stride, p.q.rec_cap, p.q.Hkv, s.b, s.h, r, 2 * p.q.D);
}
// the negative of a bf16 pair's halves, the others zero
__device__ __forceinline__ uint32_t negative_halves(uint32_t w) { return w & (((w & 0x80008000u) >> 15) * 0xFFFFu); }
__device__ __forceinline__ uint32_t abs_max2(uint32_t a, uint32_t w) {
  const __nv_bfloat162 r = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&a), __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w)));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// NT: n-tiles of eight query rows at a time
template <int D, int NT>
__global__ void __launch_bounds__(kSelThreads) select_scores_kernel(const __grid_constant__ SelectParams p) {
  constexpr int KP = D / 32;  // pairs of k-steps of one half (q+ . hi or q- . lo)
  extern __shared__ __align__(16) uint4 frag[];  // [n-tile][KP][half][lane]
  __shared__ float red[2][kSelThreads / 32];
  pdl_start();
  const int64_t list = blockIdx.x / p.tiles;
  const int tile = (int)(blockIdx.x % p.tiles);
  const SelList s = select_list(p, list);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int c0 = tile * p.tile, c1 = min(c0 + p.tile, s.m);
  if (c0 >= c1 || s.m <= p.keep) return;  // all of them are chosen
  float qmax = 0.f;
  uint32_t bmax = 0u;
  for (int r0 = 0; r0 < s.rows; r0 += 8 * NT) {
    const int nr = min(8 * NT, s.rows - r0);
    if (r0) __syncthreads();
    // fragments: lane (g, t) of k-step pair k holds coordinates 32 k + 8 t .. + 7 of row g
    for (int i = tid; i < NT * KP * 32; i += kSelThreads) {
      const int ln = i & 31, k = (i >> 5) % KP, nt = i / (32 * KP), r = 8 * nt + (ln >> 2);
      uint4 v = make_uint4(0, 0, 0, 0);
      if (r < nr) v = __ldg(reinterpret_cast<const uint4*>(query_row(p, s, r0 + r)) + 4 * k + (ln & 3));
      const uint4 n = make_uint4(negative_halves(v.x), negative_halves(v.y), negative_halves(v.z), negative_halves(v.w));
      frag[(nt * KP + k) * 64 + ln] = make_uint4(v.x ^ n.x, v.y ^ n.y, v.z ^ n.z, v.w ^ n.w);
      frag[(nt * KP + k) * 64 + 32 + ln] = n;
    }
    for (int r = warp; r < nr; r += kSelThreads / 32) {  // 1-norms of the finite rows
      const uint16_t* q = query_row(p, s, r0 + r);
      float a = 0.f;
      for (int j = 2 * lane; j < D; j += 64) {
        const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(q + j));
        a += fabsf(bf16_lo(w)) + fabsf(bf16_hi(w));
      }
      a = warp_sum(a);
      if (a < INFINITY) qmax = fmaxf(qmax, a);
    }
    __syncthreads();
    for (int c = c0 + 16 * warp; c < c1; c += 16 * (kSelThreads / 32)) {
      const uint4* rows[2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
        rows[i] = reinterpret_cast<const uint4*>(bounds_row(p, s, min(c + 8 * i + g, c1 - 1))) + t;
      float acc[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[nt][e] = 0.f;
#pragma unroll 4
      for (int k = 0; k < KP; ++k)
#pragma unroll
        for (int half = 0; half < 2; ++half) {  // hi with q+, lo with q-
          const int at = (half ? 0 : D / 8) + 4 * k;
          const uint4 x = __ldg(rows[0] + at), y = __ldg(rows[1] + at);
          if (r0 == 0) {
            bmax = abs_max2(abs_max2(abs_max2(abs_max2(bmax, x.x), x.y), x.z), x.w);
            bmax = abs_max2(abs_max2(abs_max2(abs_max2(bmax, y.x), y.y), y.z), y.w);
          }
          const uint32_t a0[4] = {x.x, y.x, x.y, y.y}, a1[4] = {x.z, y.z, x.w, y.w};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const uint4 q = frag[(nt * KP + k) * 64 + 32 * half + lane];
            mma_bf16(acc[nt], a0, q.x, q.y);
            mma_bf16(acc[nt], a1, q.z, q.w);
          }
        }
      float best[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (8 * nt + 2 * t + (e & 1) < nr && fabsf(acc[nt][e]) < INFINITY) best[e >> 1] = fmaxf(best[e >> 1], acc[nt][e]);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        best[i] = fmaxf(best[i], __shfl_xor_sync(0xffffffffu, best[i], 1));
        best[i] = fmaxf(best[i], __shfl_xor_sync(0xffffffffu, best[i], 2));
        const int r = c + 8 * i + g;
        if (t == 0 && r < c1) {
          float* at = p.scores + list * p.q.max_chunks + r;
          *at = r0 ? fmaxf(*at, best[i]) : best[i];
        }
      }
    }
  }
  float b = fmaxf(bf16_lo(bmax), bf16_hi(bmax));
  b = warp_max(b);
  qmax = warp_max(qmax);
  if (lane == 0) {
    red[0][warp] = qmax;
    red[1][warp] = b;
  }
  __syncthreads();
  if (tid == 0)
    p.limits[list * p.tiles + tile] = make_float2(fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3])),
                                                  fmaxf(fmaxf(red[1][0], red[1][1]), fmaxf(red[1][2], red[1][3])));
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

struct PickMisc {
  uint32_t hist[256];
  uint32_t warp[kPickThreads / 32];
  uint32_t prefix, left, above, cand;
};

__global__ void __launch_bounds__(kPickThreads) select_pick_kernel(const __grid_constant__ SelectParams p) {
  extern __shared__ __align__(16) uint32_t keys[];  // [max_chunks], then candidates [max_chunks], then chosen records' bits
  __shared__ PickMisc ms;
  pdl_wait();
  const int64_t list = blockIdx.x;
  const SelList s = select_list(p, list);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int32_t* out = p.list + list * p.keep;
  const int take = min(s.m, p.keep);
  if (tid == 0) p.count[list] = take;
  for (int i = tid; i < p.keep; i += kPickThreads)
    if (i >= take || s.m <= p.keep) out[i] = i < take ? i : -1;
  if (s.m <= p.keep) return;
  const int M = p.q.max_chunks, words = (s.m + 31) / 32;
  uint32_t* cand = keys + M;
  uint32_t* bits = cand + M;
  // records that the scores decide on
  const int a = min(p.sink, s.m), z = max(a, s.m - p.recent), need = p.keep - a - (s.m - z);
  for (int w = tid; w < words; w += kPickThreads) {
    uint32_t v = 0u;
    for (int i = 0; i < 32; ++i) {
      const int r = 32 * w + i;
      if (r < a || (r >= z && r < s.m)) v |= 1u << i;
    }
    bits[w] = v;
  }
  const float* score = p.scores + list * M;
  for (int i = a + tid; i < z; i += kPickThreads) keys[i] = order_key(__ldcg(score + i));
  if (tid == 0) {
    ms.prefix = 0u;
    ms.left = (uint32_t)need;
    ms.above = ms.cand = 0u;
  }
  if (need > 0) {
    // ------------------------------------------------------------ the need-th largest key, eight bits at a time
    for (int sh = 24; sh >= 0; sh -= 8) {
      ms.hist[tid] = 0u;
      __syncthreads();
      const uint32_t prefix = ms.prefix, left = ms.left;
      for (int i = a + tid; i < z; i += kPickThreads)
        if (sh == 24 || (keys[i] >> (sh + 8)) == prefix) atomicAdd(&ms.hist[(keys[i] >> sh) & 255u], 1u);
      __syncthreads();
      // keys in bins from this thread's upwards: thread t looks at bin 255 - t
      const uint32_t mine = ms.hist[255 - tid];
      uint32_t inc = mine;
#pragma unroll
      for (int k = 1; k < 32; k <<= 1) {
        const uint32_t o = __shfl_up_sync(0xffffffffu, inc, k);
        if (lane >= k) inc += o;
      }
      if (lane == 31) ms.warp[warp] = inc;
      __syncthreads();
      for (int w = 0; w < warp; ++w) inc += ms.warp[w];
      if (inc >= left && inc - mine < left) {
        ms.prefix = prefix << 8 | (uint32_t)(255 - tid);
        ms.left = left - (inc - mine);
      }
      __syncthreads();
    }
    // ------------------------------------------------------------ records that f32 cannot tell from it
    float q1 = 0.f, bm = 0.f;
    const int used = (s.m + p.tile - 1) / p.tile;
    for (int i = lane; i < used; i += 32) {
      const float2 v = __ldcg(p.limits + list * p.tiles + i);
      q1 = fmaxf(q1, v.x);
      bm = fmaxf(bm, v.y);
    }
    float e = warp_max(q1) * warp_max(bm) * ((float)p.q.D * 1.1920929e-7f);  // 2 e: d 2^-23
    if (!(e < INFINITY)) e = 0.f;
    const float x = key_value(ms.prefix);
    const uint32_t lo = order_key(x - e), hi = order_key(x + e);
    for (int i = a + tid; i < z; i += kPickThreads) {
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
      uint64_t* exact = p.exact + list * M;
      for (int i = tid; i < nc; i += kPickThreads) exact[i] = order_key(-(double)INFINITY);
      __syncthreads();
      const int D = p.q.D, sub = lane & 7;  // eight lanes a candidate and row
      const int64_t pairs = (int64_t)nc * s.rows;
      for (int64_t i0 = warp * 4; i0 < pairs; i0 += kPickThreads / 8) {
        const int64_t i = i0 + (lane >> 3);
        const bool on = i < pairs;
        const int c = on ? (int)(i / s.rows) : 0, r = on ? (int)(i % s.rows) : 0;
        const uint4* q = reinterpret_cast<const uint4*>(query_row(p, s, r));
        const uint4* bnd = reinterpret_cast<const uint4*>(bounds_row(p, s, (int)cand[c]));
        float sum[2] = {0.f, 0.f}, err[2] = {0.f, 0.f};
        for (int k = sub; k < D / 8; k += 8) {
          const uint4 qv = __ldg(q + k), lv = __ldg(bnd + k), hv = __ldg(bnd + D / 8 + k);
          const uint32_t qw[4] = {qv.x, qv.y, qv.z, qv.w}, lw[4] = {lv.x, lv.y, lv.z, lv.w}, hw[4] = {hv.x, hv.y, hv.z, hv.w};
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const uint32_t n = (qw[w] & 0x80008000u) >> 15, pick = n * 0xFFFFu, bw = (lw[w] & pick) | (hw[w] & ~pick);
            add_exact(sum[0], err[0], bf16_lo(qw[w]) * bf16_lo(bw));
            add_exact(sum[1], err[1], bf16_hi(qw[w]) * bf16_hi(bw));
          }
        }
        double v = ((double)sum[0] + (double)sum[1]) + ((double)err[0] + (double)err[1]);
#pragma unroll
        for (int k = 1; k < 8; k <<= 1) v += __shfl_xor_sync(0xffffffffu, v, k);
        if (on && sub == 0 && fabs(v) < (double)INFINITY)
          atomicMax(reinterpret_cast<unsigned long long*>(exact + c), (unsigned long long)order_key(v));
      }
      __syncthreads();
      for (int i = tid; i < nc; i += kPickThreads) {
        // the maxima were formed in L2: no line of L1 is asked for them
        const uint64_t k = __ldcg(reinterpret_cast<const unsigned long long*>(exact) + i);
        const uint32_t r = cand[i];
        int before = 0;
        for (int j = 0; j < nc; ++j) {
          const uint64_t o = __ldcg(reinterpret_cast<const unsigned long long*>(exact) + j);
          before += o > k || (o == k && cand[j] < r);
        }
        if (before < places) atomicOr(&bits[r >> 5], 1u << (r & 31));
      }
    } else {
      for (int i = tid; i < nc; i += kPickThreads) atomicOr(&bits[cand[i] >> 5], 1u << (cand[i] & 31));
    }
  }
  __syncthreads();
  // ---------------------------------------------------------------- the chosen ones in ascending order
  uint32_t base = 0;
  for (int w0 = 0; w0 < words; w0 += kPickThreads) {
    const int w = w0 + tid;
    uint32_t v = w < words ? bits[w] : 0u, inc = __popc(v);
    const uint32_t mine = inc;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
      const uint32_t o = __shfl_up_sync(0xffffffffu, inc, k);
      if (lane >= k) inc += o;
    }
    __syncthreads();
    if (lane == 31) ms.warp[warp] = inc;
    __syncthreads();
    uint32_t before = 0, all = 0;
    for (int k = 0; k < kPickThreads / 32; ++k) {
      if (k < warp) before += ms.warp[k];
      all += ms.warp[k];
    }
    uint32_t at = base + before + inc - mine;
    for (; v; v &= v - 1) out[at++] = 32 * w + __ffs(v) - 1;
    base += all;
  }
}

template <int D, int NT>
static cudaError_t scores_launch(const SelectParams& p, int64_t lists, cudaStream_t s) {
  const int smem = NT * (D / 32) * 64 * 16;
  auto kern = select_scores_kernel<D, NT>;
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  kern<<<(unsigned)(lists * p.tiles), kSelThreads, smem, s>>>(p);
  return cudaGetLastError();
}
template <int D>
static cudaError_t scores_launch_d(const SelectParams& p, int64_t lists, cudaStream_t s) {
  return p.qb * p.q.G <= 8 ? scores_launch<D, 1>(p, lists, s) : scores_launch<D, 4>(p, lists, s);
}

cudaError_t launch_select_records(const SelectParams& p, cudaStream_t s) {
  const int64_t lists = (int64_t)p.q.L * p.q.B * p.q.Hkv * p.blocks;
  cudaError_t e;
  switch (p.q.D) {
    case 64: e = scores_launch_d<64>(p, lists, s); break;
    case 128: e = scores_launch_d<128>(p, lists, s); break;
    case 256: e = scores_launch_d<256>(p, lists, s); break;
    case 512: e = scores_launch_d<512>(p, lists, s); break;
    default: return cudaErrorInvalidValue;
  }
  if (e != cudaSuccess) return e;
  const int smem = p.q.max_chunks * 8 + (p.q.max_chunks + 31) / 32 * 4;
  if (smem > 48 * 1024) {
    e = cudaFuncSetAttribute(select_pick_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  return launch_after(select_pick_kernel, dim3((unsigned)lists), kPickThreads, smem, s, 1, p);
}

}  // namespace tq
