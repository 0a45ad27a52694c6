// C entry points of a densely attended layer's cache (declared in
// include/msa.h): argument checks, workspace layout and launches.
#include <cuda_runtime.h>

#include <climits>
#include <cmath>

#include "msa_internal.h"
#include "msa_cache.h"

using namespace msa;

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool ws_ok(const void* ws, size_t have, size_t need) { return ws != nullptr && aligned(ws, 256) && have >= need; }

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
  if (weights != nullptr && !decay_ok(decay)) return MSA_ERR_INVALID_ARG;
  const DenseDecodeLayout L =
      dense_decode_layout(pages->batch, shape->H, shape->d, pages->max_seqlen, weights != nullptr);
  if (!ws_ok(ws, ws_bytes, L.total)) return MSA_ERR_WORKSPACE;
  if (!clear_error(ws, stream)) return MSA_ERR_CUDA;
  uint8_t* base = static_cast<uint8_t*>(ws);
  DenseDecodeArgs a{};
  a.q = q; a.k_pages = k_pages; a.v_pages = v_pages; a.out = out; a.lse = lse;
  a.weights = weights; a.decay = decay; a.sm_scale = shape->sm_scale;
  a.batch = pages->batch; a.H = shape->H; a.G = shape->G; a.d = shape->d;
  a.seqlens = pages->seqlens; a.block_table = pages->block_table;
  a.max_blocks = pages->max_blocks; a.max_seqlen = pages->max_seqlen; a.num_pages = pages->num_pages;
  a.err = reinterpret_cast<DevError*>(ws);
  a.seq_start = reinterpret_cast<int32_t*>(base + L.seq_start);
  a.stats = reinterpret_cast<float2*>(base + L.stats);
  a.part_ml = reinterpret_cast<float2*>(base + L.part_ml);
  a.part_o = reinterpret_cast<float*>(base + L.part_o);
  a.logits = reinterpret_cast<float*>(base + L.logits);
  return launch_dense_decode(a, stream) == 0 ? MSA_OK : MSA_ERR_CUDA;
}

}  // extern "C"
