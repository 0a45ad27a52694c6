// msa_cache.h — the cache of a densely attended layer: launchers of its decode
// attention (msa_dense_decode.cu), of the attention weight a prompt's queries
// give every key (msa_attn_weights.cu) and of the eviction by accumulated
// weight (msa_evict.cu).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <atomic>

#include <cuda_runtime.h>

#include "../../include/msa.h"

namespace msa {

struct DevError;

// Host-side check of a paged description (msa_api.cu).
msa_status_t check_paged(const msa_shape_t* s, const msa_paged_t* pg);

// DevError::where of these kernels.
constexpr int32_t kSiteDenseDecode = 241;   // lengths, pages and waits of the dense paged decode
constexpr int32_t kSiteAttnWeights = 251;   // key weights of a prompt's queries
constexpr int32_t kSiteEvictSelect = 261;   // a length outside its bounds
constexpr int32_t kSiteEvictMove = 271;     // lengths, kept indices and pages of the move

// CTAs of the dense paged decode and of the key weights (one per SM of a B200;
// fewer on a smaller device).  A constant, so that the workspace size needs no device.
constexpr int kDecodeCtas = 148;

// A kernel's dynamic shared memory allowed once per device (`done`: a bit per
// device; the call takes 1 us).
template <typename K>
int allow_smem(K* kernel, int bytes, std::atomic<uint64_t>* done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return (int)e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0ull;
  if (bit != 0 && (done->load(std::memory_order_acquire) & bit) != 0) return 0;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done->fetch_or(bit, std::memory_order_release);
  return (int)e;
}

// A launch whose grid may start before the one ahead of it in the stream has
// ended (it waits for that with griddepcontrol.wait).
template <typename... P, typename... A>
int launch_after(void (*kernel)(P...), dim3 grid, int threads, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return (int)cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

struct DenseDecodeArgs {
  const void* q;              // bf16 [batch, H, d]
  const void* k_pages;        // bf16 [num_pages * 128, G, d]
  const void* v_pages;
  void* out;                  // bf16 [batch, H, d]
  float* lse;                 // [batch, H] or null
  float* weights;             // [batch, G, max_blocks * 128] or null
  float decay;
  float sm_scale;
  int32_t batch, H, G, d;
  const int32_t* seqlens;     // [batch]
  const int32_t* block_table; // [batch, max_blocks]
  int32_t max_blocks, max_seqlen;
  int64_t num_pages;
  DevError* err;              // written by the join
  // workspace slices (dense_decode_layout)
  DevError* errors;           // [CTA]
  float2* stats;              // [batch, H]: m (the largest score in units of log2, or up to 8 below it) and sum of 2^(score - m)
  float2* part_ml;            // [CTA, 2, H]
  float* part_o;              // [CTA, 2, H, d]
  float* logits;              // scores of every key (with weights only)
};
struct DenseDecodeLayout {
  size_t errors, stats, part_ml, part_o, logits, total;
};
DenseDecodeLayout dense_decode_layout(int32_t batch, int32_t H, int32_t d, int32_t max_seqlen, bool with_weights);
int launch_dense_decode(const DenseDecodeArgs& a, void* stream);

struct AttnWeightsArgs {
  const void* q;              // bf16 [total_q, H, d]
  const void* k;              // bf16 [total_k, G, d]
  const float* lse;           // [total_q, H]
  float* weights;             // [batch, G, width]
  int64_t width;
  float decay, sm_scale;
  int32_t batch, H, G, d;
  const int32_t *cu_q, *cu_k;
  int64_t total_q, total_k;
  DevError* err;              // written by the join
  // workspace slices (attn_weights_layout)
  DevError* errors;           // [CTA]
  void* open;                 // [CTA]: the key block that a CTA leaves to be joined
  float* part;                // [CTA, 2, 256]
};
struct AttnWeightsLayout {
  size_t errors, open, part, total;
};
AttnWeightsLayout attn_weights_layout();
int launch_attn_weights(const AttnWeightsArgs& a, void* stream);

struct EvictSelectArgs {
  const float* weights;       // [batch, G, width]
  int64_t width;              // a multiple of 128
  const int32_t* seqlens;
  int32_t batch, G, per_group, max_seqlen, budget, n_sink, n_recent;
  int32_t* kept;              // [batch, per_group ? G : 1, budget]
  int32_t* new_lens;          // [batch]
  void* work;                 // evict_select_work_bytes of workspace, right behind the header of err
  DevError* err;              // written in any case
};
// Workspace behind the header (0 where registers hold a sequence's keys).
size_t evict_select_work_bytes(int32_t batch, int32_t rankings, int32_t max_seqlen);
int launch_evict_select(const EvictSelectArgs& a, void* stream);

struct EvictMoveArgs {
  const int32_t *src_lens, *src_table, *dst_lens, *dst_table;
  const int32_t* kept;        // [batch, per_group ? G : 1, kept_width]
  int32_t batch, src_blocks, src_max, dst_blocks, dst_max, kept_width, per_group, G, d, d_idx;
  int64_t num_pages;
  void *k, *v, *k_idx;        // pages, read and written
  const float* weights;       // [batch, G, src_blocks * 128] or null
  float* weights_out;         // [batch, G, dst_blocks * 128] or null
  uint32_t* flags;            // [num_pages] of workspace
  DevError* err;
};
int launch_evict_move(const EvictMoveArgs& a, void* stream);

}  // namespace msa
