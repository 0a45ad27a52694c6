// Eviction from a densely attended layer's paged cache by accumulated
// attention weight (include/msa.h: msa_evict_select, msa_evict_move).
//
// select: the tokens of a sequence that stay under a budget, in their order.
//   A token's score becomes a 32-bit key of the same order (NaN lowest; the
//   first n_sink and last n_recent tokens highest), and the budget-th largest
//   key T is found by its bits: 11, 11 and 10 at a time, a histogram of the keys
//   that share the bits found so far.  Kept: the keys above T and, of those
//   equal to T, the first ones.  Counts are whole numbers, so the result does
//   not depend on the order of the atomics.  A cluster of 1 to 8 CTAs has one
//   (sequence, ranking): each CTA counts its part of the tokens in its own
//   shared memory and adds up the others' histograms from there; the histograms
//   also give each part's number of kept tokens, so that every CTA knows where
//   its tokens go.  Bound by latency (a few passes over shared memory with a
//   cluster barrier after each) up to some 100,000 tokens, by the one pass over
//   the weights in HBM beyond.
// move: the rows of the kept tokens gathered into other pages; reads and writes
//   each kept byte once (HBM).  Out of place: a page of the source may be shared
//   with another sequence, and the rows can go in any order.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "msa_common.cuh"
#include "msa_cache.h"
#include "msa_gather.h"
#include "msa_internal.h"

namespace cg = cooperative_groups;

namespace msa {
namespace {

// ----------------------------------------------------------------- select ---

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelTile = kSelThreads * 4;        // tokens per step of a CTA
constexpr int kKeysInSmem = 40960;               // keys a CTA keeps in shared memory (160 KB)
constexpr int kMaxCluster = 8;
constexpr uint32_t kForced = 0xffffffffu;        // above +inf's key

struct SelCtl {
  uint32_t hist[3][2048];
  uint32_t warp_sum[kSelWarps];
  uint32_t bin, above;        // the bin the budget ends in, keys above it
  uint32_t gt, eq;            // this CTA's keys above and equal to the threshold
};

// 32-bit key in the order of the scores; NaN lowest, -0 as 0.
__device__ __forceinline__ uint32_t order_key(uint32_t u) {
  if ((u & 0x7fffffffu) > 0x7f800000u) return 0u;
  if (u == 0x80000000u) u = 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
// f32 -> f64 and back without flushing denormals (the build flushes by default).
__device__ __forceinline__ double widen(float x) {
  double y;
  asm("cvt.f64.f32 %0, %1;" : "=d"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float narrow(double x) {
  float y;
  asm("cvt.rn.f32.f64 %0, %1;" : "=f"(y) : "d"(x));
  return y;
}

// Exclusive sum over the block in thread order (all threads call; two barriers).
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* warp_sum, uint32_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  __syncthreads();                               // the sums of the scan before are read
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  uint32_t w = warp_sum[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += x;
  }
  *total = __shfl_sync(0xffffffffu, w, 31);
  const uint32_t before = __shfl_sync(0xffffffffu, w, warp == 0 ? 0 : warp - 1);
  return incl - v + (warp == 0 ? 0u : before);
}

__global__ void __launch_bounds__(kSelThreads, 1)
evict_select_kernel(const float* __restrict__ weights, int G, int per_group, int64_t width,
                    const int32_t* __restrict__ seqlens, int max_seqlen, int budget, int n_sink, int n_recent,
                    int32_t* __restrict__ kept, int32_t* __restrict__ new_lens, uint32_t* __restrict__ ws_keys,
                    int64_t ws_stride, DevError* err) {
  extern __shared__ uint8_t smem_raw[];
  SelCtl* ctl = reinterpret_cast<SelCtl*>(smem_raw);
  uint32_t* smem_keys = reinterpret_cast<uint32_t*>(smem_raw + sizeof(SelCtl));
  cg::cluster_group cluster = cg::this_cluster();
  const int cs = cluster.num_blocks(), rank = cluster.block_rank();
  const int R = per_group ? G : 1;
  const int row = blockIdx.x / cs;                // (sequence, ranking)
  const int b = row / R, r = row - b * R;
  const int tid = threadIdx.x;
  const int raw_len = seqlens[b];
  const int L = (raw_len < 0 || raw_len > max_seqlen) ? 0 : raw_len;
  int32_t* dst = kept + (int64_t)row * budget;
  if (rank == 0 && tid == 0) {
    if (r == 0) new_lens[b] = L < budget ? L : budget;
    if (L != raw_len) report_error(err, MSA_ERR_DEVICE_CHECK, kSiteEvictSelect, b, raw_len);
  }
  if (L <= budget) {                              // every token stays (the whole cluster takes this way)
    for (int64_t i = rank * kSelThreads + tid; i < budget; i += cs * kSelThreads) dst[i] = i < L ? (int32_t)i : -1;
    return;
  }

  for (int i = tid; i < 3 * 2048; i += kSelThreads) (&ctl->hist[0][0])[i] = 0u;
  __syncthreads();

  // this CTA's tokens [j0, j1)
  const int per = ((L + cs - 1) / cs + 3) / 4 * 4;
  const int j0 = min(rank * per, L), j1 = min(j0 + per, L);
  const int n = j1 - j0;
  uint32_t* keys = n <= kKeysInSmem ? smem_keys : ws_keys + (int64_t)row * ws_stride + j0;

  // ---- keys, and the histogram of their top 11 bits
  const float* w0 = weights + ((int64_t)b * G + r) * width + j0;   // 16-byte aligned: width % 128 == 0, j0 % 4 == 0
  for (int i = tid * 4; i < n; i += kSelTile) {
    uint32_t u[4];
    if (R == G) {
      const float4 v = *reinterpret_cast<const float4*>(w0 + i);   // the row reaches past L to its width
      u[0] = __float_as_uint(v.x); u[1] = __float_as_uint(v.y); u[2] = __float_as_uint(v.z); u[3] = __float_as_uint(v.w);
    } else {
      double s[4] = {0.0, 0.0, 0.0, 0.0};
#pragma unroll 4
      for (int g = 0; g < G; ++g) {
        const float4 v = *reinterpret_cast<const float4*>(w0 + (int64_t)g * width + i);
        s[0] += widen(v.x); s[1] += widen(v.y); s[2] += widen(v.z); s[3] += widen(v.w);
      }
#pragma unroll
      for (int x = 0; x < 4; ++x) u[x] = __float_as_uint(narrow(s[x]));
    }
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int j = j0 + i + x;
      const uint32_t key = (j < n_sink || j >= L - n_recent) ? kForced : order_key(u[x]);
      if (i + x < n) {
        keys[i + x] = key;
        atomicAdd(&ctl->hist[0][key >> 21], 1u);
      }
    }
  }

  // ---- the threshold, 11 + 11 + 10 bits
  uint32_t need = budget, top = 0;                // keys still to take; the bits found so far
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int nbin = pass == 2 ? 1024 : 2048;
    if (pass > 0) {
      const int shift = pass == 1 ? 21 : 10, down = pass == 1 ? 10 : 0;
      for (int i = tid; i < n; i += kSelThreads) {
        const uint32_t key = keys[i];
        if ((key >> shift) == top) atomicAdd(&ctl->hist[pass][(key >> down) & (nbin - 1)], 1u);
      }
    }
    cluster.sync();
    // bins from the top: thread t has 2 t and 2 t + 1 from there
    uint32_t c0 = 0, c1 = 0;
    const int b0 = nbin - 1 - 2 * tid;
    if (b0 > 0) {
      for (int k = 0; k < cs; ++k) {
        const uint32_t* h = cluster.map_shared_rank(&ctl->hist[pass][0], k);
        const uint2 v = *reinterpret_cast<const uint2*>(h + b0 - 1);
        c0 += v.y;
        c1 += v.x;
      }
    }
    uint32_t total;
    const uint32_t before = block_scan(c0 + c1, ctl->warp_sum, &total);
    if (before < need && need <= before + c0 + c1) {
      const bool first = need <= before + c0;
      ctl->bin = first ? b0 : b0 - 1;
      ctl->above = first ? before : before + c0;
    }
    __syncthreads();
    top = pass == 2 ? (top << 10 | ctl->bin) : (top << 11 | ctl->bin);
    need -= ctl->above;
  }
  // keys above `top` all stay, and the first `need` of those equal to it

  // ---- how many of this CTA's keys are above and equal
  uint32_t mine = 0;
  {
    const uint32_t d[3] = {top >> 21, (top >> 10) & 2047u, top & 1023u};
    for (int pass = 0; pass < 3; ++pass)
      for (int i = tid; i < (pass == 2 ? 1024 : 2048); i += kSelThreads)
        if ((uint32_t)i > d[pass]) mine += ctl->hist[pass][i];
    uint32_t total;
    block_scan(mine, ctl->warp_sum, &total);
    if (tid == 0) {
      ctl->gt = total;
      ctl->eq = ctl->hist[2][d[2]];
    }
  }
  cluster.sync();
  uint32_t gt = 0, eq = 0;                        // of the CTAs before this one
  for (int k = 0; k < rank; ++k) {
    const SelCtl* other = cluster.map_shared_rank(ctl, k);
    gt += other->gt;
    eq += other->eq;
  }

  // ---- the kept tokens in order
  for (int base = 0; base < n; base += kSelTile) {
    const int i = base + tid * 4;
    uint32_t f = 0;                               // above | equal << 16 of the thread's four
    uint32_t key[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      key[x] = i + x < n ? keys[i + x] : 0u;
      if (i + x < n) f += key[x] > top ? 1u : (key[x] == top ? 0x10000u : 0u);
    }
    uint32_t total;
    const uint32_t before = block_scan(f, ctl->warp_sum, &total);
    uint32_t g0 = gt + (before & 0xffffu), e0 = eq + (before >> 16);
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      if (i + x >= n) break;
      if (key[x] > top) {
        dst[g0 + min(e0, need)] = j0 + i + x;
        ++g0;
      } else if (key[x] == top) {
        if (e0 < need) dst[g0 + e0] = j0 + i + x;
        ++e0;
      }
    }
    gt += total & 0xffffu;
    eq += total >> 16;
  }
  cluster.sync();                                 // the others read this CTA's counts
}

// ------------------------------------------------------------------- move ---

constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 32;                     // rows of a new page per CTA
constexpr uint32_t kSourceBit = 0x80000000u;

struct MoveArgs {
  const int32_t* src_lens;
  const int32_t* src_table;
  const int32_t* dst_lens;
  const int32_t* dst_table;
  const int32_t* kept;                            // [batch, R, kept_width]
  int32_t batch, src_blocks, src_max, dst_blocks, dst_max, kept_width, R, G, row_words, idx_words;
  int64_t num_pages;
  uint4 *k, *v, *k_idx;
  const float* weights;
  float* weights_out;
  uint32_t* flags;                                // [num_pages], zeroed
  DevError* err;
};

__device__ __forceinline__ int bounded_len(int L, int most) { return (L < 0 || L > most) ? 0 : L; }

// Marks every page of the sources and counts every page of the destinations,
// so that the move can tell a page that is both, or twice a destination.
__global__ void __launch_bounds__(256) evict_mark_kernel(const MoveArgs a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the move waits for this grid's end
  const int64_t src = (int64_t)a.batch * a.src_blocks, dst = (int64_t)a.batch * a.dst_blocks;
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < src + dst; i += gridDim.x * 256ll) {
    const bool from = i < src;
    const int64_t x = from ? i : i - src;
    const int nb = from ? a.src_blocks : a.dst_blocks;
    const int b = (int)(x / nb), j = (int)(x - (int64_t)b * nb);
    const int L = from ? bounded_len(a.src_lens[b], a.src_max)
                       : bounded_len(a.dst_lens[b], a.dst_max < a.kept_width ? a.dst_max : a.kept_width);
    if ((int64_t)j * kBk >= L) continue;
    const int page = from ? a.src_table[x] : a.dst_table[x];
    if (page < 0 || page >= a.num_pages) continue;                // the move reports it
    if (from) atomicOr(&a.flags[page], kSourceBit);
    else atomicAdd(&a.flags[page], 1u);
  }
}

__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const MoveArgs a, int chunks) {
  __shared__ int64_t src_row[4][kMoveRows];       // row of the pages; -1: nothing to copy
  __shared__ int32_t from[4][kMoveRows];          // position in the source; -1: none
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int b = blockIdx.x / chunks, i0 = (blockIdx.x - b * chunks) * kMoveRows;
  const int tid = threadIdx.x;
  const int raw_src = a.src_lens[b], raw_dst = a.dst_lens[b];
  const int most = a.dst_max < a.kept_width ? a.dst_max : a.kept_width;
  const int L = bounded_len(raw_src, a.src_max), N = bounded_len(raw_dst, most);
  if (i0 == 0 && tid == 0) {
    if (L != raw_src) report_error(a.err, MSA_ERR_DEVICE_CHECK, kSiteEvictMove, b, raw_src);
    if (N != raw_dst) report_error(a.err, MSA_ERR_DEVICE_CHECK, kSiteEvictMove, b, raw_dst);
  }
  const int rows = min(kMoveRows, N - i0);
  if (rows > 0) {
    const int dst_blk = i0 / kBk;                 // dst_max is within dst_blocks pages
    const int page = a.dst_table[(int64_t)b * a.dst_blocks + dst_blk];
    bool page_ok = page >= 0 && page < a.num_pages;
    if (page_ok) page_ok = a.flags[page] == 1u;   // a destination once, no source
    if (!page_ok && tid == 0) report_error(a.err, MSA_ERR_DEVICE_CHECK, kSiteEvictMove, b, dst_blk);
    if (tid < a.R * kMoveRows) {
      const int r = tid / kMoveRows, x = tid - r * kMoveRows;
      int j = -1;
      int64_t row = -1;
      if (x < rows) {
        j = a.kept[((int64_t)b * a.R + r) * a.kept_width + i0 + x];
        if (j < 0 || j >= L) {
          report_error(a.err, MSA_ERR_DEVICE_CHECK, kSiteEvictMove, b, i0 + x);
          j = -1;
        } else {
          const int p = a.src_table[(int64_t)b * a.src_blocks + j / kBk];
          if (p < 0 || p >= a.num_pages) report_error(a.err, MSA_ERR_DEVICE_CHECK, kSiteEvictMove, b, j / kBk);
          else row = gather_src_row(p, j % kBk, kBk);
        }
      }
      from[r][x] = j;
      src_row[r][x] = row;
    }
    __syncthreads();
    if (page_ok) {
      const int64_t dst0 = gather_src_row(page, i0 % kBk, kBk);
      // words of a row, a power of two; with R == G a group's words come from its own token
      auto copy = [&](uint4* pages, int words, int pieces) {
        const int sh = 31 - __clz(words), psh = sh - (31 - __clz(pieces));
        const int n = rows << sh;
        for (int w0 = tid; w0 < n; w0 += 8 * kMoveThreads) {
          uint4 t[8];
          bool have[8];
#pragma unroll
          for (int y = 0; y < 8; ++y) {
            const int w = w0 + y * kMoveThreads;
            have[y] = false;
            if (w < n) {
              const int x = w >> sh, col = w & (words - 1);
              const int64_t row = src_row[col >> psh][x];
              have[y] = row >= 0;
              if (have[y]) t[y] = __ldcs(pages + (row << sh) + col);
            }
          }
#pragma unroll
          for (int y = 0; y < 8; ++y) {
            const int w = w0 + y * kMoveThreads;
            if (have[y]) __stcs(pages + (dst0 << sh) + w, t[y]);
          }
        }
      };
      copy(a.k, a.row_words, a.R);
      copy(a.v, a.row_words, a.R);
      if (a.k_idx != nullptr) copy(a.k_idx, a.idx_words, 1);
    }
  }
  if (a.weights_out != nullptr) {
    const int64_t sw = (int64_t)a.src_blocks * kBk, dw = (int64_t)a.dst_blocks * kBk;
    for (int y = tid; y < a.G * kMoveRows; y += kMoveThreads) {
      const int g = y / kMoveRows, x = y - g * kMoveRows;
      float w = 0.f;
      if (x < rows) {
        const int j = from[a.R == 1 ? 0 : g][x];
        if (j >= 0) w = a.weights[((int64_t)b * a.G + g) * sw + j];
      }
      a.weights_out[((int64_t)b * a.G + g) * dw + i0 + x] = w;
    }
  }
}

// CTAs per (sequence, ranking): one for every 8192 tokens, up to 8.
int cluster_of(int32_t max_seqlen) {
  int cs = 1;
  while (cs < kMaxCluster && max_seqlen > cs * 8192) cs *= 2;
  return cs;
}

}  // namespace

size_t evict_select_keys_bytes(int32_t batch, int32_t rankings, int32_t max_seqlen) {
  const int cs = cluster_of(max_seqlen);
  if ((max_seqlen + cs - 1) / cs + 3 <= kKeysInSmem) return 0;
  return sizeof(uint32_t) * (size_t)batch * rankings * (((size_t)max_seqlen + 3) / 4 * 4);
}

int launch_evict_select(const EvictSelectArgs& a, void* stream) {
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int cs = cluster_of(a.max_seqlen);
  const int R = a.per_group ? a.G : 1;
  const int64_t per = ((int64_t)(a.max_seqlen + cs - 1) / cs + 3) / 4 * 4;
  const int smem = (int)sizeof(SelCtl) + (int)sizeof(uint32_t) * (int)(per < kKeysInSmem ? per : kKeysInSmem);
  cudaError_t e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)sizeof(SelCtl) + 4 * kKeysInSmem);
  if (e != cudaSuccess) return (int)e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((int64_t)a.batch * R * cs));
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = cs;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  ProfScope p("evict_select", stream);
  return (int)cudaLaunchKernelEx(&cfg, evict_select_kernel, a.weights, (int)a.G, (int)a.per_group, a.width, a.seqlens,
                                 (int)a.max_seqlen, (int)a.budget, (int)a.n_sink, (int)a.n_recent, a.kept, a.new_lens,
                                 a.keys, (int64_t)((a.max_seqlen + 3) / 4 * 4), a.err);
}

int launch_evict_move(const EvictMoveArgs& m, void* stream) {
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  MoveArgs a{};
  a.src_lens = m.src_lens; a.src_table = m.src_table; a.dst_lens = m.dst_lens; a.dst_table = m.dst_table;
  a.kept = m.kept; a.batch = m.batch; a.src_blocks = m.src_blocks; a.src_max = m.src_max;
  a.dst_blocks = m.dst_blocks; a.dst_max = m.dst_max; a.kept_width = m.kept_width;
  a.R = m.per_group ? m.G : 1;
  a.G = m.G; a.row_words = m.G * m.d / 8; a.idx_words = m.d_idx / 8; a.num_pages = m.num_pages;
  a.k = static_cast<uint4*>(m.k); a.v = static_cast<uint4*>(m.v); a.k_idx = static_cast<uint4*>(m.k_idx);
  a.weights = m.weights; a.weights_out = m.weights_out; a.flags = m.flags; a.err = m.err;
  {
    const int64_t n = (int64_t)a.batch * ((int64_t)a.src_blocks + a.dst_blocks);
    const int64_t want = (n + 255) / 256;
    ProfScope p("evict_mark", stream);
    evict_mark_kernel<<<(unsigned)(want < 1184 ? want : 1184), 256, 0, st>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return (int)e;
  }
  // weights_out is written to its whole width, rows only up to the new lengths
  const int64_t last = a.weights_out != nullptr ? (int64_t)a.dst_blocks * kBk : a.dst_max;
  const int64_t chunks = (last + kMoveRows - 1) / kMoveRows;
  if (chunks * a.batch > 0x7fffffffLL) return (int)cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(chunks * a.batch));
  cfg.blockDim = dim3(kMoveThreads);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  ProfScope p("evict_move", stream);
  return (int)cudaLaunchKernelEx(&cfg, evict_move_kernel, a, (int)chunks);
}

}  // namespace msa
