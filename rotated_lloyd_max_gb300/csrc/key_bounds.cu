// Bounds of a record's keys: per coordinate the smallest and the largest of the
// 128 decoded keys, rounded outward to bf16.
//
// H_d = H_16 x H_{d/16} over a split of the index bits.  A lane holds d / 4
// neighbouring codes of a token, four of them a k-step: the top two and the low two
// bits of the index are the sixteen columns of mma.sync's k, on which H_16 (+-2^-14,
// exact) works as operand A with eight tokens as N; the bits between count the
// k-steps, whose butterflies stay in registers.  So a lane ends with two outputs a
// k-step for two tokens each, and a running minimum and maximum of d / 8
// coordinates, which four lanes join at the end of a record.  Centroids enter as
// f16 hi + lo (22 bits, two MMAs), looked up in pairs in a table with 16 copies (no
// bank conflicts); sums are f32.  The table holds them times 2^14, so that lo parts keep
// their bits, and A takes the factor out again: sums times 2^14 would leave f32's range for
// keys above 2^114.  At head dim 512 a warp forms half of the outputs
// (the top k-step bit's sum or difference by the sign of A).
//
// A warp takes a record at a time as long as there is one for every warp (8192 of
// 3 bits at head dim 128: 53 us, 64 with four warps a record); those that are left
// (or all of a short call) are shared by the four warps of a CTA (256 records: 5.2 us,
// 7.0 a warp each; 512 of head dim 512: 26 and 39).  The instructions bound it, about 2.2
// a cycle and SM: lookups, butterflies, minima and maxima of 128 d values a record.
//
// Codecs with side lists go through f32 butterflies on the CUDA cores, a vector
// spread over d / 32 lanes as in the decoder, which replaces single coordinates easily.
#include "attn_mass.cuh"
#include "packed_run.cuh"

namespace tq {

// f32 to the next bf16 below (DOWN) or above; NaN and infinities as they are
template <bool DOWN>
__device__ __forceinline__ uint32_t bf16_outward(float x) {
  const uint32_t u = __float_as_uint(x), cut = u >> 16;
  if (x != x) return 0x7FC0u;
  return cut + ((u & 0xFFFFu) != 0 && (u >> 31) == (DOWN ? 1u : 0u) ? 1u : 0u);
}
// minimum and maximum that keep a NaN
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// the smaller (LOW) or larger of bf16 pairs; NaN where one is
template <bool LOW>
__device__ __forceinline__ uint32_t join2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162*>(&a), y = *reinterpret_cast<const __nv_bfloat162*>(&b);
  const __nv_bfloat162 r = LOW ? __hmin2_nan(x, y) : __hmax2_nan(x, y);
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ float min3(float a, float b, float c) {
  float r;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// f32 to the next bf16 below (DOWN) or above, as bits; a NaN where `bad`
template <bool DOWN>
__device__ __forceinline__ uint16_t bound_bits(float x, bool bad) {
  return (uint16_t)(bad ? 0x7FC0u : bf16_outward<DOWN>(x));
}

__device__ __forceinline__ void mma_f16_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};\n"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

constexpr float kBoundsTable = 16384.f;

template <int D, int B>
struct BoundsCfg {
  static constexpr int TAB = (1 << (2 * B)) * 128;  // pair table: entry i at 128 i, 16 copies of (hi, lo)
  static constexpr int SMEM = TAB + 4 * 4 * D;      // and the warps' bounds, bf16 [2][D]
};

// tasks: records, or at head dim 512 halves of their outputs; the first `solo` of them a warp each
template <int D, int B>
__global__ void __launch_bounds__(kThreads, D <= 128 ? 4 : 3)
    key_bounds_mma_kernel(const __grid_constant__ BoundsParams p, uint32_t tasks, uint32_t solo) {
  constexpr int KK = D / 16, RUN = D / 4, STEP = RUN < 32 ? RUN : 32, NS = RUN / STEP, NB = STEP * B;
  constexpr int HALVES = D == 512 ? 2 : 1, ACC = KK / HALVES, ROW = D * B / 8;
  extern __shared__ __align__(128) unsigned char sm[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  for (int i = tid; i < (1 << (2 * B)) * 16; i += kThreads) {
    const int e = i >> 4;
    const float x = p.c.centroids[e & ((1 << B) - 1)] * kBoundsTable, y = p.c.centroids[e >> B] * kBoundsTable;
    uint32_t hi, lo;
    split_f16x2(x, y, hi, lo);
    reinterpret_cast<uint2*>(sm)[i] = make_uint2(hi, lo);
  }
  __syncthreads();
  const uint32_t loff = (lane & 15) * 8;
  const ByteTable tab = byte_table(sm, loff, 128);
  uint16_t* mine = reinterpret_cast<uint16_t*>(sm + BoundsCfg<D, B>::TAB) + warp * 2 * D;  // [2][D]
  // H_16 / kBoundsTable: rows g, g + 8 (t' = row / 4, j' = row % 4), columns (t, j): the sign is the parity of t & t' and j & j'
  uint32_t h16[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = g + 8 * (i & 1), j = 2 * (i >> 1);
    const uint32_t s0 = __popc(t & (row >> 2)) + __popc(j & row & 3), s1 = __popc(t & (row >> 2)) + __popc((j + 1) & row & 3);
    h16[i] = 0x04000400u | (s0 & 1u) << 15 | (s1 & 1u) << 31;  // +-1 / kBoundsTable
  }
  struct Task {
    uint32_t q;
    int64_t out;  // place of its bounds
    const uint8_t* rec;
  };
  // the first task from k.q on that names a record; false where there is none before `end`
  auto seek = [&](Task& k, uint32_t stride, uint32_t end) {
    for (; k.q < end; k.q += stride) {
      const uint32_t x = HALVES == 1 ? k.q : k.q >> 1, unit = fast_div(x, p.by_new), lb = fast_div(unit, p.by_heads);
      const int h = (int)(unit - lb * p.Hkv), l = (int)fast_div(lb, p.by_batch), b = (int)lb - l * p.B;
      const int n = min(max(__ldg(p.n_chunks + lb), 0), min(p.max_chunks, p.rec_limit));
      const int64_t r = (int64_t)(p.first ? max(__ldg(p.first + lb), 0) : 0) + (x - unit * p.max_new);
      if (r >= n) continue;
      const int64_t at = rec_offset(p.table, p.table_stride, p.rec_cap, p.Hkv, b, h, (int)r, 1);
      k.rec = p.rec + l * p.rec_ls + at * p.c.rec_bytes;
      k.out = l * p.bounds_ls + at * 2 * D;
      return true;
    }
    return false;
  };
#pragma unroll 1
  for (int team = 0; team < 2; ++team) {  // warps alone, then four together
    const uint32_t stride = team ? gridDim.x : 4 * gridDim.x, end = team ? tasks : solo;
    const int tiles = team ? kChunk / 32 : kChunk / 8, first = team ? warp * tiles : 0;
    Task cur, nxt;
    cur.q = team ? solo + blockIdx.x : 4 * blockIdx.x + warp;
    bool more = seek(cur, stride, end);
    Run<NB> run;
    float2 nn = f2(0.f, 0.f);
    if (more) {
      run.load(cur.rec + (8 * first + g) * ROW, t * RUN * B);
      nn = __ldg(reinterpret_cast<const float2*>(cur.rec + p.c.off_norm) + 4 * first + t);
    }
    for (; more; cur = nxt) {
      nxt.q = cur.q + stride;
      nxt.rec = cur.rec;
      more = seek(nxt, stride, end);
      const int half = HALVES == 1 ? 0 : (int)(cur.q & 1);
      const uint8_t* rec = cur.rec;
      uint32_t sign = 0u;  // of A for the k-steps of the upper half
      if (HALVES == 2 && half) sign = 0x80008000u;
      float lo[ACC][2], hi[ACC][2];
#pragma unroll
      for (int k = 0; k < ACC; ++k)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          lo[k][e] = INFINITY;
          hi[k][e] = -INFINITY;
        }
      bool bad = false;
      const uint8_t* row = rec + (8 * first + g) * ROW;
#pragma unroll 1
      for (int i = 0; i < tiles; ++i) {
        float acc[ACC][4];
        const float2 f = f2(nn.x * p.c.inv_sqrt_d, nn.y * p.c.inv_sqrt_d);
        bad = bad || !(fabsf(nn.x) < INFINITY) || !(fabsf(nn.y) < INFINITY);
        const bool last = i + 1 == tiles;
        const uint8_t* next = last ? nxt.rec + (8 * first + g) * ROW : row + 8 * ROW;
        nn = __ldg(reinterpret_cast<const float2*>((last ? nxt.rec : rec) + p.c.off_norm) + 4 * (last ? first : first + i + 1) + t);
#pragma unroll
        for (int s = 0; s < NS; ++s) {
          uint32_t w[Run<NB>::NW];
          run.get((t * RUN + s * STEP) * B, w);
          run.load(s + 1 < NS ? row : next, (t * RUN + (s + 1 < NS ? s + 1 : 0) * STEP) * B);
          const bool upper = HALVES == 2 && s >= NS / 2;
          const uint32_t a[4] = {h16[0] ^ (upper ? sign : 0u), h16[1] ^ (upper ? sign : 0u), h16[2] ^ (upper ? sign : 0u),
                                 h16[3] ^ (upper ? sign : 0u)};
#pragma unroll
          for (int k = 0; k < STEP / 4; ++k) {
            const uint2 e0 = pair_at<B>(tab, sm, w, 4 * k, loff), e1 = pair_at<B>(tab, sm, w, 4 * k + 2, loff);
            const int kk = s * (STEP / 4) + k;
            if (kk < ACC) mma_f16_first(acc[kk % ACC], a, e0.x, e1.x);
            else mma_f16(acc[kk % ACC], a, e0.x, e1.x);
            mma_f16(acc[kk % ACC], a, e0.y, e1.y);
          }
        }
        // the k-steps' bits
#pragma unroll
        for (int m = 1; m < ACC; m <<= 1)
#pragma unroll
          for (int k = 0; k < ACC; ++k)
            if (!(k & m)) {
#pragma unroll
              for (int e = 0; e < 4; e += 2) {
                const float2 x = f2(acc[k][e], acc[k][e + 1]), y = f2(acc[k | m][e], acc[k | m][e + 1]);
                const float2 u = add2(x, y), v = fma2(y, f2(-1.f, -1.f), x);
                acc[k][e] = u.x;
                acc[k][e + 1] = u.y;
                acc[k | m][e] = v.x;
                acc[k | m][e + 1] = v.y;
              }
            }
#pragma unroll
        for (int k = 0; k < ACC; ++k)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float2 y = mul2(f2(acc[k][2 * e], acc[k][2 * e + 1]), f);
            lo[k][e] = min3(lo[k][e], y.x, y.y);
            hi[k][e] = max3(hi[k][e], y.x, y.y);
          }
        row = next;
      }
      // over the four lanes of a quad (tokens), of which lane t keeps k-steps = t modulo 4: half of them go over at
      // a time; then to the keys' signs and bf16
      bad = __any_sync(0xffffffffu, bad);
      if (team) __syncthreads();  // the bounds of the record before are written
      else __syncwarp();
#pragma unroll
      for (int m = 1; m < 4; m <<= 1)
#pragma unroll
        for (int k = 0; k < ACC; ++k)
          if (m == 1 ? !(k & 1) : (k & 3) < 2) {  // after the first round, what a lane keeps lies in even places
            if (m == 2 && (k & 1)) continue;
            const int o = k + m;
            const bool up = (t & m) != 0;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float x = __shfl_xor_sync(0xffffffffu, up ? lo[k][e] : lo[o][e], m);
              const float y = __shfl_xor_sync(0xffffffffu, up ? hi[k][e] : hi[o][e], m);
              lo[k][e] = fminf(up ? lo[o][e] : lo[k][e], x);
              hi[k][e] = fmaxf(up ? hi[o][e] : hi[k][e], y);
            }
          }
#pragma unroll
      for (int k0 = 0; k0 < ACC; k0 += 4) {
        const int k = k0 + t;  // the k-step that lane t keeps in place k0
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int o = g + 8 * e, c = (o >> 2) * RUN + 4 * (half * ACC + k) + (o & 3);
          float x = lo[k0][e], y = hi[k0][e];
          if ((p.c.signs[c >> 5] >> (c & 31)) & 1u) {
            const float z = x;
            x = -y;
            y = -z;
          }
          mine[c] = bound_bits<true>(x, bad);
          mine[D + c] = bound_bits<false>(y, bad);
        }
      }
      uint16_t* out = p.bounds + cur.out;
      // coordinates come in runs of 4 ACC at steps of RUN: 16-byte chunks
      constexpr int CH = 4 * ACC / 8;  // chunks of a run
      auto chunk = [&](int i) { return (i / CH) * (RUN / 8) + half * CH + i % CH; };
      if (!team) {
        __syncwarp();
        for (int i = lane; i < 8 * CH; i += 32) {
          const int c = chunk(i);
          reinterpret_cast<uint4*>(out)[c] = reinterpret_cast<const uint4*>(mine)[c];
        }
      } else {
        __syncthreads();
        for (int i = tid; i < 8 * CH; i += kThreads) {
          const int c = chunk(i);
          uint4 v = reinterpret_cast<const uint4*>(sm + BoundsCfg<D, B>::TAB)[c];
#pragma unroll
          for (int w = 1; w < 4; ++w) {
            const uint4 x = reinterpret_cast<const uint4*>(sm + BoundsCfg<D, B>::TAB)[w * (D / 4) + c];
            v = c < D / 8 ? make_uint4(join2<true>(v.x, x.x), join2<true>(v.y, x.y), join2<true>(v.z, x.z), join2<true>(v.w, x.w))
                          : make_uint4(join2<false>(v.x, x.x), join2<false>(v.y, x.y), join2<false>(v.z, x.z), join2<false>(v.w, x.w));
          }
          reinterpret_cast<uint4*>(out)[c] = v;
        }
      }
    }
    __syncthreads();
  }
}

template <int D, int B>
__global__ void __launch_bounds__(kThreads) key_bounds_kernel(const __grid_constant__ BoundsParams p) {
  constexpr int L = D / 32, VPW = 32 / L, VPC = 4 * VPW, RB = D * B / 8;
  __shared__ float lut[16];
  __shared__ int pre[kChunk];
  __shared__ float part[2][4][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, lg = lane % L, vi = lane / L;
  const int64_t unit = blockIdx.x / p.max_new;
  const int h = (int)(unit % p.Hkv), lb = (int)(unit / p.Hkv), b = lb % p.B, l = lb / p.B;
  const int n = min(max(p.n_chunks[lb], 0), min(p.max_chunks, p.rec_limit));
  const int64_t r = (int64_t)(p.first ? max(p.first[lb], 0) : 0) + blockIdx.x % p.max_new;
  if (r >= n) return;
  const uint8_t* rec = p.rec + l * p.rec_ls +
                       rec_offset(p.table, p.table_stride, p.rec_cap, p.Hkv, b, h, (int)r, p.c.rec_bytes);
  if (threadIdx.x < 16) lut[threadIdx.x] = p.c.centroids[threadIdx.x & ((1 << B) - 1)];
  if (warp == 0) {  // where a slot's entries begin
    int run = 0;
    for (int k = 0; k < kChunk; k += 32) {
      const int v = rec[p.c.off_count + k + lane];
      int inc = v;
#pragma unroll
      for (int m = 1; m < 32; m <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, inc, m);
        if (lane >= m) inc += o;
      }
      pre[k + lane] = run + inc - v;
      run += __shfl_sync(0xffffffffu, inc, 31);
    }
  }
  __syncthreads();
  float lo[32], hi[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    lo[i] = INFINITY;
    hi[i] = -INFINITY;
  }
#pragma unroll 1
  for (int slot = warp * VPW + vi; slot < kChunk; slot += VPC) {
    const uint32_t* src = reinterpret_cast<const uint32_t*>(rec + slot * RB + lg * 4 * B);
    uint32_t w[B];
#pragma unroll
    for (int q = 0; q < B; ++q) w[q] = __ldg(src + q);
    float f = __ldg(reinterpret_cast<const float*>(rec + p.c.off_norm) + slot) * p.c.inv_sqrt_d;
    f = fmaf(f, 0.f, f);  // NaN where it is not finite
    float x[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const int bit = i * B;
      uint32_t code = w[bit >> 5] >> (bit & 31);
      if ((bit & 31) + B > 32) code |= w[(bit >> 5) + 1] << (32 - (bit & 31));
      x[i] = lut[code & ((1u << B) - 1u)];
    }
    {
      const int e0 = pre[slot], e1 = min(e0 + rec[p.c.off_count + slot], p.c.cap);
      const uint32_t* ent = reinterpret_cast<const uint32_t*>(rec + p.c.off_entries);
      for (int e = e0; e < e1; ++e) {
        const uint32_t v = __ldg(ent + e);
        const int idx = (int)(v & (D - 1));
        if ((idx >> 5) == lg) {
          const float val = bf16_hi(v);
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] = i == (idx & 31) ? val : x[i];
        }
      }
      __syncwarp();
    }
    fwht_regs<32>(x);
    fwht_lanes<32>(x, lane, L);
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const float y = x[i] * f;
      lo[i] = min_nan(lo[i], y);
      hi[i] = max_nan(hi[i], y);
    }
  }
  // over the warp's vectors, then the four warps
#pragma unroll
  for (int m = L; m < 32; m <<= 1)
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      lo[i] = min_nan(lo[i], __shfl_xor_sync(0xffffffffu, lo[i], m));
      hi[i] = max_nan(hi[i], __shfl_xor_sync(0xffffffffu, hi[i], m));
    }
  if (vi == 0) {
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      part[0][warp][32 * lg + i] = lo[i];
      part[1][warp][32 * lg + i] = hi[i];
    }
  }
  __syncthreads();
  uint16_t* out = p.bounds + l * p.bounds_ls + rec_offset(p.table, p.table_stride, p.rec_cap, p.Hkv, b, h, (int)r, 2 * D);
  for (int j = threadIdx.x; j < D; j += kThreads) {
    float a = min_nan(min_nan(part[0][0][j], part[0][1][j]), min_nan(part[0][2][j], part[0][3][j]));
    float z = max_nan(max_nan(part[1][0][j], part[1][1][j]), max_nan(part[1][2][j], part[1][3][j]));
    if ((p.c.signs[j >> 5] >> (j & 31)) & 1u) {  // the coordinate's sign turns them around
      const float o = a;
      a = -z;
      z = -o;
    }
    out[j] = (uint16_t)bf16_outward<true>(a);
    out[D + j] = (uint16_t)bf16_outward<false>(z);
  }
}

template <int D, int B>
static cudaError_t bounds_launch(const BoundsParams& p, cudaStream_t s) {
  const int64_t records = (int64_t)p.L * p.B * p.Hkv * p.max_new;
  if (p.c.has_outl) {
    key_bounds_kernel<D, B><<<(unsigned)records, kThreads, 0, s>>>(p);
    return cudaGetLastError();
  }
  auto kern = key_bounds_mma_kernel<D, B>;
  constexpr int smem = BoundsCfg<D, B>::SMEM;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int64_t tasks = records * (D == 512 ? 2 : 1), grid = min(tasks, (int64_t)sm_count() * (D <= 128 ? 4 : 3));
  kern<<<(unsigned)grid, kThreads, smem, s>>>(p, (uint32_t)tasks, (uint32_t)(tasks / (4 * grid) * (4 * grid)));
  return cudaGetLastError();
}

cudaError_t launch_key_bounds(const BoundsParams& p, cudaStream_t s) {
  switch (p.c.d * 10 + p.c.bits) {
#define TQ_CASE(D_) \
  case D_ * 10 + 1: return bounds_launch<D_, 1>(p, s); \
  case D_ * 10 + 2: return bounds_launch<D_, 2>(p, s); \
  case D_ * 10 + 3: return bounds_launch<D_, 3>(p, s); \
  case D_ * 10 + 4: return bounds_launch<D_, 4>(p, s);
    TQ_CASE(64) TQ_CASE(128) TQ_CASE(256) TQ_CASE(512)
#undef TQ_CASE
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace tq
