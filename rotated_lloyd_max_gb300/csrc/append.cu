// Rotary positions with several axes on queries and keys, fused with the
// append of keys and values to the ring.
//
// A pair (x0, x1) of a head turns by a = position * inv_freq.  The angle is
// reduced exactly: inv_freq / 2 pi is held as a 64-bit fraction of a turn, and
// position * fraction modulo 2^64 is the angle's fraction of a turn (integer
// arithmetic wraps where the turn does), off by at most |position| 2^-54 turns
// (the f64 product's rounding; 2^-34 turns at a position of a million), where
// f32 angles would be off by |a| 2^-24.  sincospif takes it from there.
//
// Every input is read once and every output written once: bound by memory.
// The (cos, sin) of a token's pairs are shared by all its heads, so a CTA
// takes a few tokens with all their heads (fewer heads where there are too few
// tokens to fill the SMs) and keeps the table in shared memory.  A thread
// moves units of two 16-byte chunks, the two halves of eight pairs, so that
// the rotation needs no exchange and may run in place.  Four prompts of up to 4099
// tokens, 48 heads of 128: 54 us, 5.6 TB/s.  One token: 3.0 us from a graph, a launch
// and one chain behind it (lengths, inv_freq, angle, barrier, and only then the loads);
// with the counters in place, which a second launch moves, 3.7 us.
#include "cache_params.h"
#include "tq_common.cuh"

namespace tq {

constexpr int kAppendThreads = 256;

__device__ __forceinline__ int append_len(const AppendParams& p, int b) {
  return p.q_lens ? min(max(p.q_lens[b], 0), p.T) : p.T;
}
// tokens of (l, b) that enter the ring: all T_b or none
__device__ __forceinline__ bool append_fits(const AppendParams& p, int len, int tb) {
  return len >= 0 && len <= p.tail_cap && tb <= p.tail_cap - len;
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
// eight pairs: a holds the first members, b the second
__device__ __forceinline__ void turn_halves(uint4& a, uint4& b, const float2* cs) {
  uint32_t* x = reinterpret_cast<uint32_t*>(&a);
  uint32_t* y = reinterpret_cast<uint32_t*>(&b);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 c = *reinterpret_cast<const float4*>(cs + 2 * i);
    const float x0 = bf16_lo(x[i]), x1 = bf16_hi(x[i]), y0 = bf16_lo(y[i]), y1 = bf16_hi(y[i]);
    x[i] = pack_bf16(x0 * c.x - y0 * c.y, x1 * c.z - y1 * c.w);
    y[i] = pack_bf16(y0 * c.x + x0 * c.y, y1 * c.z + x1 * c.w);
  }
}
// four pairs of neighbours in one chunk
__device__ __forceinline__ void turn_adjacent(uint4& a, const float2* cs) {
  uint32_t* x = reinterpret_cast<uint32_t*>(&a);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float x0 = bf16_lo(x[i]), x1 = bf16_hi(x[i]);
    x[i] = pack_bf16(x0 * cs[i].x - x1 * cs[i].y, x1 * cs[i].x + x0 * cs[i].y);
  }
}

template <int D>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int UPH = D / 16;  // two-chunk units per head
  extern __shared__ __align__(16) float2 table[];  // [tile][rot_dim / 2] cos, sin (times rot_scale)
  const int lb = blockIdx.x / p.tiles, t0 = (blockIdx.x % p.tiles) * p.tile;
  const int l = lb / p.B, b = lb % p.B;
  const int h0 = blockIdx.y * p.group, nh = min(p.group, p.heads - h0);
  const int tb = append_len(p, b);
  const int cap = p.tail_cap;
  const int len = p.tail_len[lb];
  const bool fits = append_fits(p, len, tb);
  if (blockIdx.y == 0 && t0 == 0 && threadIdx.x == 0 && !p.in_place) p.tail_len_out[lb] = fits ? len + tb : len;
  const int nt = min(p.tile, tb - t0);
  if (nt <= 0) return;
  const int start = p.tail_start ? ((p.tail_start[lb] % cap) + cap) % cap : 0;
  const int half = p.rot_dim >> 1;
  for (int i = threadIdx.x; i < half; i += kAppendThreads) {
    double turns = (double)p.inv_freq[i] * 0.15915494309189533577;
    turns -= floor(turns);
    // turns in [0, 1]; the product below only needs it modulo 1
    const uint64_t frac = turns < 1.0 ? (uint64_t)(turns * 18446744073709551616.0) : 0ull;
    const int32_t* pos = p.positions + ((int64_t)p.pair_axis[i] * p.B + b) * p.T + t0;
    for (int t = 0; t < nt; ++t) {
      const int64_t part = (int64_t)((uint64_t)(int64_t)pos[t] * frac);
      float s, c;
      sincospif((float)(int32_t)(part >> 32) * 4.656612873077393e-10f, &s, &c);  // 2^-31: half turns
      table[t * half + i] = f2(c * p.rot_scale, s * p.rot_scale);
    }
  }
  if (p.mass && fits && blockIdx.y == 0) {
    const int64_t first = (int64_t)kChunk * (p.n_chunks ? max(p.n_chunks[lb], 0) : 0) + len + t0;
    float* m = p.mass + l * p.mass_ls + (int64_t)b * p.Hkv * p.mass_cap;
    for (int i = threadIdx.x; i < nt * p.Hkv; i += kAppendThreads) {
      const int64_t at = first + i % nt;
      if (at < p.mass_cap) m[(int64_t)(i / nt) * p.mass_cap + at] = 0.f;
    }
  }
  __syncthreads();
  const uint16_t* q = p.q + l * p.q_ls + b * p.q_bs;
  const uint16_t* k = p.k + l * p.kv_ls + b * p.kv_bs;
  const uint16_t* v = p.v + l * p.kv_ls + b * p.kv_bs;
  uint16_t* qo = p.q_out + l * p.o_ls + b * p.o_bs;
  const int64_t ring0 = l * p.tail_ls + (int64_t)b * p.Hkv * cap * D;
  const int first = (int)((start + (int64_t)(fits ? len : 0)) % cap);
  const int per = p.group * UPH;
  for (int i = threadIdx.x; i < nt * per; i += kAppendThreads) {
    const int t = fast_div(i, p.units), r = i - t * per;
    const int hh = r / UPH, u = r % UPH;
    if (hh >= nh) continue;
    const int h = h0 + hh, tok = t0 + t;
    const uint16_t* src;
    uint16_t* dst;
    bool turns = true;
    if (h < p.Hq) {
      src = q + (int64_t)tok * p.q_ts + (int64_t)h * D;
      dst = qo + (int64_t)tok * p.o_ts + (int64_t)h * D;
    } else {
      if (!fits) continue;
      const bool value = h >= p.Hq + p.Hkv;
      const int kv = h - p.Hq - (value ? p.Hkv : 0);
      const int slot = (int)(((int64_t)first + tok) % cap);
      const int64_t at = ring0 + ((int64_t)kv * cap + slot) * D;
      src = (value ? v : k) + (int64_t)tok * p.kv_ts + (int64_t)kv * D;
      dst = (value ? p.v_tail : p.k_tail) + at;
      turns = !value;
    }
    int c0 = u, c1 = u + UPH;  // chunks of eight coordinates
    bool pairs = false;
    if (turns && !p.adjacent) {
      const int rc = half >> 3, a = p.rot_start >> 3;
      pairs = u < rc;
      if (pairs) {
        c0 = a + u;
        c1 = c0 + rc;
      } else {  // the chunks that do not turn, in two runs around the rotated ones
        const int rest = UPH - rc;
        c0 = u - rc;
        c1 = c0 + rest;
        if (c0 >= a) c0 += 2 * rc;
        if (c1 >= a) c1 += 2 * rc;
      }
    }
    uint4 x = *reinterpret_cast<const uint4*>(src + 8 * c0), y = *reinterpret_cast<const uint4*>(src + 8 * c1);
    const float2* cs = table + t * half;
    if (pairs) {
      turn_halves(x, y, cs + 8 * u);
    } else if (turns && p.adjacent) {
      const int r0 = 8 * c0 - p.rot_start, r1 = 8 * c1 - p.rot_start;
      if (r0 >= 0 && r0 < p.rot_dim) turn_adjacent(x, cs + (r0 >> 1));
      if (r1 >= 0 && r1 < p.rot_dim) turn_adjacent(y, cs + (r1 >> 1));
    }
    *reinterpret_cast<uint4*>(dst + 8 * c0) = x;
    *reinterpret_cast<uint4*>(dst + 8 * c1) = y;
  }
}

__global__ void append_commit_kernel(const __grid_constant__ AppendParams p) {
  for (int lb = blockIdx.x * blockDim.x + threadIdx.x; lb < p.L * p.B; lb += gridDim.x * blockDim.x) {
    const int len = p.tail_len[lb], tb = append_len(p, lb % p.B);
    if (append_fits(p, len, tb)) p.tail_len_out[lb] = len + tb;
  }
}

cudaError_t launch_append(const AppendParams& p, cudaStream_t s) {
  const dim3 grid((unsigned)((int64_t)p.L * p.B * p.tiles), (p.heads + p.group - 1) / p.group);
  const int smem = p.tile * (p.rot_dim / 2) * (int)sizeof(float2);
  switch (p.D) {
    case 64: append_kernel<64><<<grid, kAppendThreads, smem, s>>>(p); break;
    case 128: append_kernel<128><<<grid, kAppendThreads, smem, s>>>(p); break;
    case 256: append_kernel<256><<<grid, kAppendThreads, smem, s>>>(p); break;
    case 512: append_kernel<512><<<grid, kAppendThreads, smem, s>>>(p); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

cudaError_t launch_append_commit(const AppendParams& p, cudaStream_t s) {
  const int n = p.L * p.B;
  append_commit_kernel<<<(n + 127) / 128, 128, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace tq
