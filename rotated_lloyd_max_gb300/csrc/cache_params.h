// Kernel parameter blocks of the append, the eviction by accumulated weight
// and the several-query calls, shared between the C ABI (abi_cache.cu) and the
// kernels.  Host-visible plain structs.
#pragma once

#include "../../include/tq.h"
#include "tq_params.h"

namespace tq {

struct AppendParams {
  int L, B, T, Hq, Hkv, D;
  int heads;          // heads of a token this launch handles: queries, keys, values (unless shared)
  int group;          // heads per CTA
  int tile, tiles;    // tokens per CTA; token tiles per (layer, sequence)
  FastDiv units;      // division by group * (d / 16)
  const uint16_t *q, *k, *v;
  int64_t q_ls, q_bs, q_ts, kv_ls, kv_bs, kv_ts;
  uint16_t* q_out;
  int64_t o_ls, o_bs, o_ts;
  const int32_t* q_lens;
  const int32_t* positions;
  int rot_start, rot_dim, adjacent;
  const float* inv_freq;
  uint8_t pair_axis[256];
  float rot_scale;
  uint16_t *k_tail, *v_tail;
  int64_t tail_ls;
  int tail_cap;
  const int32_t* tail_start;
  const int32_t* tail_len;
  int32_t* tail_len_out;
  int in_place;       // tail_len_out == tail_len: a launch of its own moves the counters
  float* mass;
  int64_t mass_ls;
  int mass_cap;
  const int32_t* n_chunks;
};

struct EvictMassParams {
  int L, B, Hkv;
  CodecDev kc, vc;
  int shared;
  const uint8_t *k_rec, *v_rec;
  int64_t k_ls, v_ls;
  int rec_cap;
  const int32_t* table;
  int table_stride, rec_limit;
  uint8_t *k_dst, *v_dst;
  int64_t kd_ls, vd_ls;
  int dst_cap;
  const int32_t* dst_table;
  int dst_table_stride;
  const float* mass;
  float* mass_dst;
  int64_t mass_ls, mass_dst_ls;
  int mass_cap, mass_dst_cap;
  const int32_t* n_chunks;
  int32_t* n_chunks_dst;
  const int32_t* tail_len;
  int max_chunks, max_tail, keep, sink, recent;
  int slots;       // records a stream can keep: min(keep, max_chunks)
  int in_place;
  int32_t* kept;   // caller's list or null
  // workspace
  int32_t* list;   // [streams][128 slots] source index of each remaining token
  int32_t* counts; // [L * B] records before
};

struct QueryParams {
  int L, B, T, Hq, Hkv, G, D;
  float sscale;       // softmax scale * log2(e)
  float scap, iscap;  // logit soft cap * log2(e) and its reciprocal; 0, 0 = no cap
  int causal;
  const uint16_t* q;
  int64_t q_ls, q_bs, q_ts;
  const int32_t* q_lens;
  const uint8_t *krec, *vrec;
  int64_t krec_ls, vrec_ls;
  int rec_cap;
  const int32_t* table;
  int table_stride, rec_limit;
  CodecDev kc, vc;
  int shared_kv;
  const uint16_t *ktail, *vtail;
  int64_t tail_ls;
  int tail_cap;
  const int32_t* n_chunks;
  const int32_t* tail_start;
  const int32_t* tail_len;
  int max_chunks, max_tail;
};

cudaError_t launch_append(const AppendParams& p, cudaStream_t s);
cudaError_t launch_append_commit(const AppendParams& p, cudaStream_t s);
cudaError_t launch_evict_mass(const EvictMassParams& p, cudaStream_t s);

#ifdef __CUDACC__
// Programmatic dependent launch between the kernels of one call: the second is
// launched while the first runs and waits on the device for its end, which
// hides a launch's latency (1 to 2 us of the short calls).  Every thread of the
// second kernel waits before anything else, so that its end is never before the
// first one's.  pdl_start: from here
// on the next kernel may be made resident; pdl_wait: the kernel before has
// ended and what it wrote is visible.
__device__ __forceinline__ void pdl_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Lookup of a byte (two 4-bit codes) in a shared-memory table.  The entry's
// address is one byte extraction and one multiply-add, whose factor sits in a
// register that the compiler does not see through: shift, mask and sum in its
// place would take three operations of the ALU pipe, which the decoding fills.
struct ByteTable {
  uint32_t at, step;  // the lane's copy of entry 0; bytes from entry to entry
};
__device__ __forceinline__ ByteTable byte_table(const void* table, uint32_t lane_off, uint32_t step) {
  ByteTable t;
  t.at = (uint32_t)__cvta_generic_to_shared(table) + lane_off;
  asm volatile("mov.u32 %0, %1;" : "=r"(t.step) : "r"(step));
  return t;
}
__device__ __forceinline__ uint32_t byte_entry(const ByteTable& t, uint32_t x, int k) {
  return __byte_perm(x, 0, 0x4440 + k) * t.step + t.at;
}
__device__ __forceinline__ uint32_t byte_lookup(const ByteTable& t, uint32_t x, int k) {
  uint32_t r;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(r) : "r"(byte_entry(t, x, k)));
  return r;
}
__device__ __forceinline__ uint2 byte_lookup2(const ByteTable& t, uint32_t x, int k) {
  uint2 r;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(byte_entry(t, x, k)));
  return r;
}

template <class... Args>
inline cudaError_t launch_after(void (*kern)(Args...), dim3 grid, int block, int smem, cudaStream_t s, int cluster,
                                const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}
#endif

// abi.cu
int sm_count();
int max_dynamic_smem();
tq_status resolve_codec_dev(const tq_codec* c, CodecDev* o);

}  // namespace tq
