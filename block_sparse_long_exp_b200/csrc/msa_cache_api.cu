// C entry points of a densely attended layer's cache (declared in
// include/msa.h): argument checks, workspace layout and launches.
#include <cuda_runtime.h>

#include <climits>

#include "msa_internal.h"
#include "msa_cache.h"

using namespace msa;

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool ws_ok(const void* ws, size_t have, size_t need) { return ws != nullptr && aligned(ws, 256) && have >= need; }

// Keys past a sequence's end count as scores of -inf, which the kernels multiply with the scale in units of log2: a scale
// of 0 or below (a denormal one is 0 there) would turn them into NaN, one past the largest number a score of 0.
bool scale_ok(float s) { return s >= 0x1p-126f && s * 1.4426950408889634f <= 0x1.fffffep127f; }

bool decay_ok(float d) { return d >= 0.f && d <= 1.f; }

bool clear_error(void* ws, void* stream) {
  return cudaMemsetAsync(ws, 0, sizeof(DevError), reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess;
}

}  // namespace

extern "C" {

size_t msa_dense_attn_decode_paged_workspace_size(const msa_shape_t* shape, const msa_paged_t* pages,
                                                  int32_t with_weights) {
  if (check_paged(shape, pages) != MSA_OK) return 0;
  return dense_decode_layout(pages->batch, shape->H, shape->d, pages->max_seqlen, with_weights != 0).total;
}

msa_status_t msa_dense_attn_decode_paged(const msa_shape_t* shape, const msa_paged_t* pages, const void* q,
                                         const void* k_pages, const void* v_pages, void* out, float* lse,
                                         float* weights, float decay, void* ws, size_t ws_bytes, void* stream) {
  const msa_status_t st = check_paged(shape, pages);
  if (st != MSA_OK) return st;
  if (!q || !k_pages || !v_pages || !out) return MSA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(out, 16))
    return MSA_ERR_INVALID_ARG;
  if (!scale_ok(shape->sm_scale) || (weights != nullptr && !decay_ok(decay))) return MSA_ERR_INVALID_ARG;
  const DenseDecodeLayout L =
      dense_decode_layout(pages->batch, shape->H, shape->d, pages->max_seqlen, weights != nullptr);
  if (!ws_ok(ws, ws_bytes, L.total)) return MSA_ERR_WORKSPACE;
  uint8_t* base = static_cast<uint8_t*>(ws);
  DenseDecodeArgs a{};
  a.q = q; a.k_pages = k_pages; a.v_pages = v_pages; a.out = out; a.lse = lse;
  a.weights = weights; a.decay = decay; a.sm_scale = shape->sm_scale;
  a.batch = pages->batch; a.H = shape->H; a.G = shape->G; a.d = shape->d;
  a.seqlens = pages->seqlens; a.block_table = pages->block_table;
  a.max_blocks = pages->max_blocks; a.max_seqlen = pages->max_seqlen; a.num_pages = pages->num_pages;
  a.err = reinterpret_cast<DevError*>(ws);
  a.errors = reinterpret_cast<DevError*>(base + L.errors);
  a.stats = reinterpret_cast<float2*>(base + L.stats);
  a.part_ml = reinterpret_cast<float2*>(base + L.part_ml);
  a.part_o = reinterpret_cast<float*>(base + L.part_o);
  a.logits = reinterpret_cast<float*>(base + L.logits);
  return launch_dense_decode(a, stream) == 0 ? MSA_OK : MSA_ERR_CUDA;
}

size_t msa_attn_weights_workspace_size(const msa_shape_t* shape, const msa_varlen_t* seqs) {
  if (check_shape(shape) != MSA_OK || check_seqs(seqs) != MSA_OK) return 0;
  return attn_weights_layout().total;
}

msa_status_t msa_attn_weights(const msa_shape_t* shape, const msa_varlen_t* seqs, const void* q, const void* k,
                              const float* lse, float* weights, int64_t width, float decay, void* ws, size_t ws_bytes,
                              void* stream) {
  msa_status_t st = check_shape(shape);
  if (st != MSA_OK) return st;
  st = check_seqs(seqs);
  if (st != MSA_OK) return st;
  if (width < seqs->max_k_len || !scale_ok(shape->sm_scale) || !decay_ok(decay)) return MSA_ERR_INVALID_ARG;
  if (seqs->total_q > 0 && (!q || !k || !lse || !weights)) return MSA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(lse, 16)) return MSA_ERR_INVALID_ARG;
  const AttnWeightsLayout L = attn_weights_layout();
  if (!ws_ok(ws, ws_bytes, L.total)) return MSA_ERR_WORKSPACE;
  if (seqs->total_q == 0) return clear_error(ws, stream) ? MSA_OK : MSA_ERR_CUDA;
  uint8_t* base = static_cast<uint8_t*>(ws);
  AttnWeightsArgs a{};
  a.q = q; a.k = k; a.lse = lse; a.weights = weights; a.width = width; a.decay = decay;
  a.sm_scale = shape->sm_scale; a.batch = seqs->batch; a.H = shape->H; a.G = shape->G; a.d = shape->d;
  a.cu_q = seqs->cu_q; a.cu_k = seqs->cu_k; a.total_q = seqs->total_q; a.total_k = seqs->total_k;
  a.err = static_cast<DevError*>(ws);
  a.errors = reinterpret_cast<DevError*>(base + L.errors);
  a.open = base + L.open;
  a.part = reinterpret_cast<float*>(base + L.part);
  return launch_attn_weights(a, stream) == 0 ? MSA_OK : MSA_ERR_CUDA;
}

size_t msa_evict_select_workspace_size(const msa_shape_t* shape, const msa_paged_t* pages, int32_t per_group) {
  if (check_paged(shape, pages) != MSA_OK) return 0;
  return kWsHeader + evict_select_work_bytes(pages->batch, per_group != 0 ? shape->G : 1, pages->max_seqlen);
}

msa_status_t msa_evict_select(const msa_shape_t* shape, const msa_paged_t* pages, const float* weights,
                              int32_t budget, int32_t n_sink, int32_t n_recent, int32_t per_group, int32_t* kept,
                              int32_t* new_lens, void* ws, size_t ws_bytes, void* stream) {
  const msa_status_t st = check_paged(shape, pages);
  if (st != MSA_OK) return st;
  if (!weights || !kept || !new_lens || !aligned(weights, 16)) return MSA_ERR_INVALID_ARG;
  if (budget < 1 || n_sink < 0 || n_recent < 0 || (int64_t)n_sink + n_recent > budget) return MSA_ERR_INVALID_ARG;
  if (!ws_ok(ws, ws_bytes, msa_evict_select_workspace_size(shape, pages, per_group))) return MSA_ERR_WORKSPACE;
  if ((int64_t)pages->batch * shape->G * 8 > INT32_MAX) return MSA_ERR_UNSUPPORTED;      // CTAs of one launch
  EvictSelectArgs a{};
  a.weights = weights; a.width = (int64_t)pages->max_blocks * kBk; a.seqlens = pages->seqlens;
  a.batch = pages->batch; a.G = shape->G; a.per_group = per_group != 0; a.max_seqlen = pages->max_seqlen;
  a.budget = budget; a.n_sink = n_sink; a.n_recent = n_recent;
  a.kept = kept; a.new_lens = new_lens;
  a.work = static_cast<uint8_t*>(ws) + kWsHeader;
  a.err = static_cast<DevError*>(ws);
  return launch_evict_select(a, stream) == 0 ? MSA_OK : MSA_ERR_CUDA;
}

size_t msa_evict_move_workspace_size(const msa_shape_t* shape, const msa_paged_t* pages) {
  if (check_paged(shape, pages) != MSA_OK) return 0;
  return kWsHeader + align_up(sizeof(uint32_t) * (size_t)pages->num_pages, 256);
}

msa_status_t msa_evict_move(const msa_shape_t* shape, const msa_paged_t* pages, const msa_paged_t* new_pages,
                            const int32_t* kept, int32_t kept_width, int32_t per_group, void* k_pages, void* v_pages,
                            void* k_idx_pages, const float* weights, float* weights_out, void* ws, size_t ws_bytes,
                            void* stream) {
  msa_status_t st = check_paged(shape, pages);
  if (st != MSA_OK) return st;
  st = check_paged(shape, new_pages);
  if (st != MSA_OK) return st;
  if (new_pages->batch != pages->batch || new_pages->num_pages != pages->num_pages) return MSA_ERR_INVALID_ARG;
  if (!kept || kept_width < 1 || !k_pages || !v_pages) return MSA_ERR_INVALID_ARG;
  if (!aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(k_idx_pages, 16)) return MSA_ERR_INVALID_ARG;
  if ((weights == nullptr) != (weights_out == nullptr)) return MSA_ERR_INVALID_ARG;
  if (weights != nullptr) {                       // rows go out while others are still read
    const uintptr_t row = (uintptr_t)pages->batch * shape->G * kBk * sizeof(float);
    const uintptr_t in = reinterpret_cast<uintptr_t>(weights), to = reinterpret_cast<uintptr_t>(weights_out);
    if (in < to + row * new_pages->max_blocks && to < in + row * pages->max_blocks) return MSA_ERR_INVALID_ARG;
  }
  // the groups share the index keys: tokens kept by group have none of their own
  if (per_group != 0 && shape->G > 1 && k_idx_pages != nullptr) return MSA_ERR_INVALID_ARG;
  if (!ws_ok(ws, ws_bytes, msa_evict_move_workspace_size(shape, pages))) return MSA_ERR_WORKSPACE;
  EvictMoveArgs a{};
  a.src_lens = pages->seqlens; a.src_table = pages->block_table;
  a.dst_lens = new_pages->seqlens; a.dst_table = new_pages->block_table;
  a.kept = kept; a.batch = pages->batch; a.src_blocks = pages->max_blocks; a.src_max = pages->max_seqlen;
  a.dst_blocks = new_pages->max_blocks; a.dst_max = new_pages->max_seqlen; a.kept_width = kept_width;
  a.per_group = per_group != 0; a.G = shape->G; a.d = shape->d; a.d_idx = shape->d_idx;
  a.num_pages = pages->num_pages;
  a.k = k_pages; a.v = v_pages; a.k_idx = k_idx_pages; a.weights = weights; a.weights_out = weights_out;
  a.flags = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(ws) + kWsHeader);
  a.err = static_cast<DevError*>(ws);
  return launch_evict_move(a, stream) == 0 ? MSA_OK : MSA_ERR_CUDA;
}

}  // extern "C"
