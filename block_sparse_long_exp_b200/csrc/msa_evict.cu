// Eviction from a densely attended layer's paged cache by accumulated
// attention weight (include/msa.h: msa_evict_select, msa_evict_move).
//
// select: the tokens of a sequence that stay under a budget, in their order.
//   A token's score becomes a 32-bit key of the same order (NaN lowest; the
//   first n_sink and last n_recent tokens highest), and the budget-th largest
//   key T is found by its bits: 11, 11 and 10 at a time, a histogram of the keys
//   that share the bits found so far.  Kept: the keys above T and, of those
//   equal to T, the first ones.  Counts are whole numbers, so the result does
//   not depend on the order of the atomics.  Up to 65,536 tokens a CTA, or a
//   cluster of them that add up their histograms from one another's shared
//   memory, has a (sequence, ranking), the keys in registers, and what it takes is
//   the latency of some fifteen barriers; beyond, a CTA has 4096 tokens and the
//   steps are launches.  Bound by those launches up to some 300,000 tokens in
//   all, then by the weights from HBM.  On a B200: 8 x 5K tokens 8.9 us in a
//   graph (13.5 called one by one), 2 x 1M 34 us.
// move: the rows of the kept tokens gathered into other pages; reads and writes
//   each kept byte once (HBM).  Out of place: a page of the source may be shared
//   with another sequence, and the rows can go in any order.  On a B200: 4 x 64K
//   rows (G 4, d 128) 188 us, 6.1 TB/s; 8 x 4K by group 29.3 us.
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
constexpr int kSelPart = kSelThreads * 8;        // tokens of a CTA at most: 4 or 8 a thread, in its registers
constexpr uint32_t kForced = 0xffffffffu;        // above +inf's key

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
// A finite f32 times 2^-896 as an f64: sign, exponent field and fraction moved
// to their places (0 and denormals too: the fields mean the same one scale
// down).  A conversion instruction would run at an eighth of the rate.
__device__ __forceinline__ double scaled_down(uint32_t u) {
  return __hiloint2double((int)((u & 0x80000000u) | ((u & 0x7fffffffu) >> 3)), (int)(u << 29));
}
// Its way back, rounded to nearest even: the f32's bits.  A sum in between is
// the f64 sum times 2^-896: multiples of 2^-149 keep all their bits there.
__device__ __forceinline__ uint32_t scaled_up(double s) {
  const uint32_t hi = (uint32_t)__double2hiint(s), lo = (uint32_t)__double2loint(s);
  uint32_t u = ((hi & 0x7fffffffu) << 3) | (lo >> 29);
  const uint32_t rest = lo & 0x1fffffffu;
  u += (rest > 0x10000000u || (rest == 0x10000000u && (u & 1u))) ? 1u : 0u;
  return (hi & 0x80000000u) | min(u, 0x7f800000u);
}

// Scores (as bits) of N tokens in a row: the sum over GS groups' weights in 64
// bits, rounded once to 32.
template <int GS, int N>
__device__ __forceinline__ void token_scores(const float* __restrict__ w, int64_t width, uint32_t (&u)[N]) {
  uint4 v[GS][N / 4];
#pragma unroll
  for (int g = 0; g < GS; ++g)
#pragma unroll
    for (int q = 0; q < N / 4; ++q) v[g][q] = *reinterpret_cast<const uint4*>(w + g * width + 4 * q);
  auto at = [&](int g, int i) {
    const uint4 q = v[g][i / 4];
    return i % 4 == 0 ? q.x : i % 4 == 1 ? q.y : i % 4 == 2 ? q.z : q.w;
  };
  if constexpr (GS == 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) u[i] = at(0, i);
  } else {
    uint32_t most = 0;                           // the largest size: from 0x7f800000 on an infinity or NaN is among them
#pragma unroll
    for (int i = 0; i < N; ++i) {
      double s = scaled_down(at(0, i));
#pragma unroll
      for (int g = 1; g < GS; ++g) s += scaled_down(at(g, i));
      u[i] = scaled_up(s);
#pragma unroll
      for (int g = 0; g < GS; ++g) most = max(most, at(g, i) & 0x7fffffffu);
    }
    if (most >= 0x7f800000u) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        double s = widen(__uint_as_float(at(0, i)));
#pragma unroll
        for (int g = 1; g < GS; ++g) s += widen(__uint_as_float(at(g, i)));
        u[i] = __float_as_uint(narrow(s));
      }
    }
  }
}

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Exclusive sum over the block of WARPS warps in thread order (all threads call; two barriers).
template <int WARPS>
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
  uint32_t w = lane < WARPS ? warp_sum[lane] : 0u;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += x;
  }
  *total = __shfl_sync(0xffffffffu, w, 31);
  const uint32_t before = __shfl_sync(0xffffffffu, w, warp == 0 ? 0 : warp - 1);
  return incl - v + (warp == 0 ? 0u : before);
}

// Counts N bins a thread (whole warps call).  A warp of one bin (weights that
// are all zero, the tokens kept in any case) adds once.
template <int N>
__device__ __forceinline__ void count_bins(uint32_t* hist, const uint32_t (&bin)[N], const bool (&in)[N]) {
  uint32_t lo = 0xffffffffu, hi = 0u, c = 0;
#pragma unroll
  for (int x = 0; x < N; ++x)
    if (in[x]) {
      lo = min(lo, bin[x]);
      hi = max(hi, bin[x]);
      ++c;
    }
  c = __reduce_add_sync(0xffffffffu, c);
  if (c == 0) return;
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  if (lo == hi) {
    if ((threadIdx.x & 31) == 0) atomicAdd(&hist[lo], c);
    return;
  }
#pragma unroll
  for (int x = 0; x < N; ++x)
    if (in[x]) atomicAdd(&hist[bin[x]], 1u);
}

// Of 32 counts, a lane each, the lane in which the `need` first ones end, from the top; *above: those before it.
__device__ __forceinline__ int find_lane(uint32_t c, uint32_t need, uint32_t* above) {
  const int lane = threadIdx.x & 31;
  uint32_t incl = c;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t x = __shfl_down_sync(0xffffffffu, incl, o);
    if (lane + o < 32) incl += x;
  }
  const int at = __ffs(__ballot_sync(0xffffffffu, incl - c < need && need <= incl)) - 1;
  *above = __shfl_sync(0xffffffffu, incl - c, at);
  return at;
}

struct SelCtl {
  union {
    struct {
      uint32_t hist[3][2048];
      uint32_t sum[2048];     // a cluster's histogram
    };
    int32_t list[kSelPart];   // afterwards: the CTA's kept tokens in their order
  };
  uint32_t warp_sum[kSelWarps];
  uint32_t gt, eq;            // this CTA's keys above and equal to the threshold
};

// A CTA, or a cluster of them, per (sequence, ranking).
template <bool kCluster, int GS, int PER>
__global__ void __launch_bounds__(kSelThreads, 1)
evict_select_kernel(const float* __restrict__ weights, int G, int64_t width, const int32_t* __restrict__ seqlens,
                    int batch, int max_seqlen, int budget, int n_sink, int n_recent, int32_t* __restrict__ kept,
                    int32_t* __restrict__ new_lens, DevError* err) {
  __shared__ SelCtl ctl;
  cg::cluster_group cluster = cg::this_cluster();
  const int cs = kCluster ? cluster.num_blocks() : 1, rank = kCluster ? cluster.block_rank() : 0;
  const int R = GS == 1 ? G : 1;
  const int row = blockIdx.x / cs, b = row / R, r = row - b * R;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto bounded = [&](int n) { return n < 0 || n > max_seqlen ? 0 : n; };
  const int L = bounded(seqlens[b]);
  int32_t* dst = kept + (int64_t)row * budget;
  if (rank == 0 && tid == 0 && r == 0) new_lens[b] = L < budget ? L : budget;
  if (blockIdx.x == 0) {                          // the first bad length, or none
    int bad = batch;
    for (int i = tid; i < batch; i += kSelThreads)
      if (bounded(seqlens[i]) != seqlens[i]) bad = min(bad, i);
    bad = __reduce_min_sync(0xffffffffu, bad);
    if (lane == 0) ctl.warp_sum[warp] = bad;
    __syncthreads();
    if (warp == 0) {
      bad = __reduce_min_sync(0xffffffffu, lane < kSelWarps ? (int)ctl.warp_sum[lane] : batch);
      if (lane == 0)
        *err = bad < batch ? DevError{MSA_ERR_DEVICE_CHECK, kSiteEvictSelect, bad, seqlens[bad]} : DevError{0, 0, 0, 0};
    }
    __syncthreads();
  }
  if (L <= budget) {                              // every token stays (the whole cluster takes this way)
    for (int64_t i = rank * kSelThreads + tid; i < budget; i += cs * kSelThreads) dst[i] = i < L ? (int32_t)i : -1;
    return;
  }

  // ---- this CTA's tokens [j0, j0 + n), PER in a row to a thread
  const int per = ((L + cs - 1) / cs + PER - 1) / PER * PER;
  const int j0 = min(rank * per, L), n = min(per, L - j0);
  const int i0 = tid * PER;
  uint32_t key[PER];
#pragma unroll
  for (int x = 0; x < PER; ++x) key[x] = 0u;
  if (i0 < n) token_scores<GS>(weights + ((int64_t)b * G + r) * width + j0 + i0, width, key);   // rows reach past L to their width
  for (int i = tid; i < 3 * 2048; i += kSelThreads) (&ctl.hist[0][0])[i] = 0u;
  __syncthreads();
#pragma unroll
  for (int x = 0; x < PER; ++x) {
    const int j = j0 + i0 + x;
    key[x] = (j < n_sink || j >= L - n_recent) ? kForced : order_key(key[x]);
  }

  // ---- the threshold, 11 + 11 + 10 bits: keys still to take, and the bits found so far
  uint32_t need = budget, top = 0;
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    constexpr int kShift[3] = {0, 21, 10}, kDown[3] = {21, 10, 0};
    uint32_t* hist = ctl.hist[pass];
    uint32_t bins[PER];
    bool in[PER];
#pragma unroll
    for (int x = 0; x < PER; ++x) {
      bins[x] = key[x] >> kDown[pass] & (pass == 2 ? 1023u : 2047u);
      in[x] = i0 + x < n && (pass == 0 || key[x] >> kShift[pass] == top);
    }
    count_bins(hist, bins, in);
    // a thread has two bins; every warp finds the bin from the warps' sums
    uint2 c = make_uint2(0u, 0u);
    if constexpr (kCluster) {
      cluster.sync();
      for (int k = 0; k < cs; ++k) {
        const uint2 v = reinterpret_cast<const uint2*>(cluster.map_shared_rank(hist, k))[tid];
        c.x += v.x;
        c.y += v.y;
      }
      reinterpret_cast<uint2*>(ctl.sum)[tid] = c;
      hist = ctl.sum;
    } else {
      __syncthreads();
      c = reinterpret_cast<const uint2*>(hist)[tid];
    }
    const uint32_t w = __reduce_add_sync(0xffffffffu, c.x + c.y);
    if (lane == 0) ctl.warp_sum[warp] = w;
    __syncthreads();
    uint32_t above, more;
    const int at = find_lane(ctl.warp_sum[lane], need, &above);
    const uint2 d = reinterpret_cast<const uint2*>(hist)[32 * at + lane];
    const int bl = find_lane(d.x + d.y, need - above, &more);
    need -= above + more;
    const uint32_t upper = __shfl_sync(0xffffffffu, d.y, bl);
    const bool high = need <= upper;              // the upper of the lane's two bins
    if (!high) need -= upper;
    top = top << (pass == 2 ? 10 : 11) | (64 * at + 2 * bl + (high ? 1 : 0));
  }
  // keys above `top` all stay, and the first `need` of those equal to it

  uint32_t f = 0;                                 // above | equal << 16 of the thread's tokens
#pragma unroll
  for (int x = 0; x < PER; ++x)
    if (i0 + x < n) f += key[x] > top ? 1u : (key[x] == top ? 0x10000u : 0u);
  uint32_t total;
  const uint32_t before = block_scan<kSelWarps>(f, ctl.warp_sum, &total);
  uint32_t eq0 = 0, first = 0;                    // equal keys of the CTAs before this one; kept tokens of theirs
  if constexpr (kCluster) {
    if (tid == 0) {
      ctl.gt = total & 0xffffu;
      ctl.eq = total >> 16;
    }
    cluster.sync();                               // (and every histogram is read)
    for (int k = 0; k < rank; ++k) {
      const SelCtl* other = cluster.map_shared_rank(&ctl, k);
      first += other->gt;
      eq0 += other->eq;
    }
    first += min(eq0, need);
  }
  const uint32_t left = need - min(eq0, need);    // equal keys that this CTA may keep
  // the list is put in order in shared memory (every histogram is read) and goes out in whole lines
  uint32_t gt = before & 0xffffu, eq = before >> 16;
#pragma unroll
  for (int x = 0; x < PER; ++x) {
    if (i0 + x < n) {
      if (key[x] > top) {
        ctl.list[gt + min(eq, left)] = j0 + i0 + x;
        ++gt;
      } else if (key[x] == top) {
        if (eq < left) ctl.list[gt + eq] = j0 + i0 + x;
        ++eq;
      }
    }
  }
  __syncthreads();
  const int here = (int)((total & 0xffffu) + min(total >> 16, left));
  for (int i = tid; i < here; i += kSelThreads) dst[first + i] = ctl.list[i];
  if constexpr (kCluster) cluster.sync();         // the others read this CTA's counts
}

// -------------------------------------------------- select, long sequences ---
//
// The same search with a CTA per 4096 tokens of every (sequence, ranking), the
// histograms in global memory and a launch per step: the keys and the histogram
// of their top 11 bits; of the next 11; of the last 10; each part's numbers of
// kept tokens; the kept tokens.  Every CTA finds the step's bin by itself.

constexpr int kLongThreads = 512;
constexpr int kLongPart = 4096;                   // tokens per CTA
constexpr int kLongPer = kLongPart / kLongThreads;

struct LongRow {
  uint32_t top, need;         // the bits found so far; keys still to take among those that share them
};
struct LongArgs {
  const float* weights;
  int64_t width;
  const int32_t* seqlens;
  int32_t G, R, parts, max_seqlen, budget, n_sink, n_recent;
  int32_t* kept;
  int32_t* new_lens;
  uint32_t* keys;             // [rows, parts * 4096]
  uint32_t* hist;             // [3, rows, 2048], zeroed
  LongRow* found;             // [3, rows]
  uint2* counts;              // [rows, parts]: keys above and equal to the threshold
  int32_t rows;
  DevError* err;
};

// The bin in which the `need` largest keys of a histogram end, and the keys above it (all threads call).
template <int BINS>
__device__ __forceinline__ void find_bin(const uint32_t* __restrict__ hist, uint32_t need, uint32_t* warp_sum,
                                         uint32_t* out, uint32_t* bin, uint32_t* above) {
  constexpr int N = BINS / kLongThreads;          // thread t has the bins N t .. N t + N - 1 from the top
  uint32_t c[N], sum = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    c[i] = hist[BINS - 1 - (N * (int)threadIdx.x + i)];
    sum += c[i];
  }
  uint32_t total;
  uint32_t before = block_scan<kLongThreads / 32>(sum, warp_sum, &total);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (before < need && need <= before + c[i]) {
      out[0] = BINS - 1 - (N * threadIdx.x + i);
      out[1] = before;
    }
    before += c[i];
  }
  __syncthreads();
  *bin = out[0];
  *above = out[1];
}

// What the CTAs of every step share: their row and part of it.
struct LongPlace {
  int row, part, b, r, L, n;                      // n: tokens of the part
  bool cut;                                       // the sequence is longer than the budget
  __device__ LongPlace(const LongArgs& a) {
    row = blockIdx.x / a.parts;
    part = blockIdx.x - row * a.parts;
    b = row / a.R;
    r = row - b * a.R;
    const int raw = a.seqlens[b];
    L = (raw < 0 || raw > a.max_seqlen) ? 0 : raw;
    cut = L > a.budget;
    n = min(max(L - part * kLongPart, 0), kLongPart);
  }
};

// The histograms and the error word cleared, while the next kernel reads its weights.
__global__ void __launch_bounds__(kLongThreads) long_clear_kernel(const LongArgs a) {
  pdl_launch_dependents();
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.err = DevError{0, 0, 0, 0};
  uint4* h = reinterpret_cast<uint4*>(a.hist);
  for (int64_t i = blockIdx.x * kLongThreads + threadIdx.x; i < 3ll * a.rows * 512; i += gridDim.x * kLongThreads)
    h[i] = make_uint4(0u, 0u, 0u, 0u);
}

template <int GS>
__global__ void __launch_bounds__(kLongThreads) long_keys_kernel(const LongArgs a) {
  __shared__ uint32_t hist[2048];
  pdl_launch_dependents();
  const LongPlace p(a);
  const int tid = threadIdx.x;
  if (p.part == 0 && p.r == 0 && tid == 0) a.new_lens[p.b] = p.L < a.budget ? p.L : a.budget;
  if (!p.cut) {                                   // every token stays
    pdl_wait();
    if (p.part == 0 && p.r == 0 && tid == 0 && p.L != a.seqlens[p.b])
      report_error(a.err, MSA_ERR_DEVICE_CHECK, kSiteEvictSelect, p.b, a.seqlens[p.b]);
    int32_t* dst = a.kept + (int64_t)p.row * a.budget;
    for (int64_t i = p.part * kLongThreads + tid; i < a.budget; i += (int64_t)a.parts * kLongThreads)
      dst[i] = i < p.L ? (int32_t)i : -1;
    return;
  }
  for (int i = tid; i < 2048; i += kLongThreads) hist[i] = 0u;
  __syncthreads();
  const int j0 = p.part * kLongPart;
  const float* w0 = a.weights + ((int64_t)p.b * a.G + p.r) * a.width + j0;
  uint32_t* keys = a.keys + (int64_t)blockIdx.x * kLongPart;
#pragma unroll
  for (int s = 0; s < kLongPer / 4; ++s) {
    const int i = (s * kLongThreads + tid) * 4;
    uint32_t u[4] = {0u, 0u, 0u, 0u};
    if (i < p.n) token_scores<GS>(w0 + i, a.width, u);               // the row reaches past L to its width
    uint32_t bins[4];
    bool in[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int j = j0 + i + x;
      u[x] = (j < a.n_sink || j >= p.L - a.n_recent) ? kForced : order_key(u[x]);
      bins[x] = u[x] >> 21;
      in[x] = i + x < p.n;
    }
    count_bins(hist, bins, in);
    *reinterpret_cast<uint4*>(keys + i) = make_uint4(u[0], u[1], u[2], u[3]);   // past the part's end: not counted
  }
  __syncthreads();
  pdl_wait();                                     // every CTA: this grid's end stands for the ends before it
  uint32_t* sum = a.hist + (int64_t)p.row * 2048;
  for (int i = tid; i < 2048; i += kLongThreads)
    if (hist[i] != 0) atomicAdd(&sum[i], hist[i]);
}

template <int PASS>
__global__ void __launch_bounds__(kLongThreads) long_hist_kernel(const LongArgs a) {
  constexpr int kBins = PASS == 2 ? 1024 : 2048;
  __shared__ uint32_t hist[kBins];
  __shared__ uint32_t warp_sum[kLongThreads / 32], out[2];
  pdl_launch_dependents();
  const LongPlace p(a);
  const int tid = threadIdx.x;
  for (int i = tid; i < kBins; i += kLongThreads) hist[i] = 0u;
  pdl_wait();                                     // every CTA: this grid's end stands for the ends before it
  if (!p.cut || p.n == 0) return;
  uint4 k[kLongPer / 4];
  const uint4* keys = reinterpret_cast<const uint4*>(a.keys + (int64_t)blockIdx.x * kLongPart);
#pragma unroll
  for (int s = 0; s < kLongPer / 4; ++s) k[s] = keys[s * kLongThreads + tid];
  LongRow f = PASS == 1 ? LongRow{0u, (uint32_t)a.budget} : a.found[(int64_t)a.rows + p.row];
  uint32_t bin, above;
  find_bin<2048>(a.hist + ((int64_t)(PASS - 1) * a.rows + p.row) * 2048, f.need, warp_sum, out, &bin, &above);
  f.top = f.top << 11 | bin;
  f.need -= above;
  if (p.part == 0 && tid == 0) a.found[(int64_t)PASS * a.rows + p.row] = f;
  constexpr int kShift = PASS == 1 ? 21 : 10, kDown = PASS == 1 ? 10 : 0;
#pragma unroll
  for (int s = 0; s < kLongPer / 4; ++s) {
    const int i = (s * kLongThreads + tid) * 4;
    const uint32_t u[4] = {k[s].x, k[s].y, k[s].z, k[s].w};
    uint32_t bins[4];
    bool in[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      bins[x] = (u[x] >> kDown) & (kBins - 1);
      in[x] = i + x < p.n && (u[x] >> kShift) == f.top;
    }
    count_bins(hist, bins, in);
  }
  __syncthreads();
  uint32_t* sum = a.hist + ((int64_t)PASS * a.rows + p.row) * 2048;
  for (int i = tid; i < kBins; i += kLongThreads)
    if (hist[i] != 0) atomicAdd(&sum[i], hist[i]);
}

__global__ void __launch_bounds__(kLongThreads) long_count_kernel(const LongArgs a) {
  __shared__ uint32_t warp_sum[kLongThreads / 32], out[2];
  pdl_launch_dependents();
  const LongPlace p(a);
  const int tid = threadIdx.x;
  pdl_wait();
  if (!p.cut || p.n == 0) return;
  uint4 k[kLongPer / 4];
  const uint4* keys = reinterpret_cast<const uint4*>(a.keys + (int64_t)blockIdx.x * kLongPart);
#pragma unroll
  for (int s = 0; s < kLongPer / 4; ++s) k[s] = keys[s * kLongThreads + tid];
  LongRow f = a.found[2ll * a.rows + p.row];
  uint32_t bin, above;
  find_bin<1024>(a.hist + (2ll * a.rows + p.row) * 2048, f.need, warp_sum, out, &bin, &above);
  f.top = f.top << 10 | bin;
  f.need -= above;
  if (p.part == 0 && tid == 0) a.found[p.row] = f;
  uint32_t c = 0;                                 // above | equal << 16
#pragma unroll
  for (int s = 0; s < kLongPer / 4; ++s) {
    const int i = (s * kLongThreads + tid) * 4;
    const uint32_t u[4] = {k[s].x, k[s].y, k[s].z, k[s].w};
#pragma unroll
    for (int x = 0; x < 4; ++x)
      if (i + x < p.n) c += u[x] > f.top ? 1u : (u[x] == f.top ? 0x10000u : 0u);
  }
  uint32_t total;
  block_scan<kLongThreads / 32>(c, warp_sum, &total);
  if (tid == 0) a.counts[blockIdx.x] = make_uint2(total & 0xffffu, total >> 16);
}

__global__ void __launch_bounds__(kLongThreads) long_write_kernel(const LongArgs a) {
  __shared__ uint32_t warp_sum[kLongThreads / 32];
  __shared__ int32_t list[kLongPart];             // the part's kept tokens: they go out in whole lines
  const LongPlace p(a);
  const int tid = threadIdx.x;
  pdl_wait();
  if (!p.cut || p.n == 0) return;
  uint4 k[kLongPer / 4];                          // 8 tokens in a row
  const uint4* keys = reinterpret_cast<const uint4*>(a.keys + (int64_t)blockIdx.x * kLongPart + tid * kLongPer);
#pragma unroll
  for (int s = 0; s < kLongPer / 4; ++s) k[s] = keys[s];
  const LongRow f = a.found[p.row];
  uint32_t g = 0, e = 0;                          // of the parts before this one
  for (int i = tid; i < p.part; i += kLongThreads) {
    const uint2 c = a.counts[(int64_t)p.row * a.parts + i];
    g += c.x;
    e += c.y;
  }
  uint32_t gt, eq, total;
  block_scan<kLongThreads / 32>(g, warp_sum, &gt);
  block_scan<kLongThreads / 32>(e, warp_sum, &eq);
  uint32_t c = 0;
#pragma unroll
  for (int s = 0; s < kLongPer / 4; ++s) {
    const uint32_t u[4] = {k[s].x, k[s].y, k[s].z, k[s].w};
#pragma unroll
    for (int x = 0; x < 4; ++x)
      if (tid * kLongPer + 4 * s + x < p.n) c += u[x] > f.top ? 1u : (u[x] == f.top ? 0x10000u : 0u);
  }
  const uint32_t before = block_scan<kLongThreads / 32>(c, warp_sum, &total);
  const uint32_t taken = min(eq, f.need), left = f.need - taken;   // equal keys kept by the parts before, and still to keep
  uint32_t g1 = before & 0xffffu, e1 = before >> 16;
  const int j0 = p.part * kLongPart + tid * kLongPer;
#pragma unroll
  for (int s = 0; s < kLongPer / 4; ++s) {
    const uint32_t u[4] = {k[s].x, k[s].y, k[s].z, k[s].w};
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      if (tid * kLongPer + 4 * s + x < p.n) {
        if (u[x] > f.top) {
          list[g1 + min(e1, left)] = j0 + 4 * s + x;
          ++g1;
        } else if (u[x] == f.top) {
          if (e1 < left) list[g1 + e1] = j0 + 4 * s + x;
          ++e1;
        }
      }
    }
  }
  __syncthreads();
  int32_t* dst = a.kept + (int64_t)p.row * a.budget + gt + taken;
  const int here = (int)((total & 0xffffu) + min(total >> 16, left));
  for (int i = tid; i < here; i += kLongThreads) dst[i] = list[i];
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

__global__ void __launch_bounds__(256) evict_clear_kernel(uint32_t* flags, int64_t n, DevError* err) {
  pdl_launch_dependents();
  if (blockIdx.x == 0 && threadIdx.x == 0) *err = DevError{0, 0, 0, 0};
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < n; i += gridDim.x * 256ll) flags[i] = 0u;
}

// Marks every page of the sources and counts every page of the destinations,
// so that the move can tell a page that is both, or twice a destination.
__global__ void __launch_bounds__(256) evict_mark_kernel(const MoveArgs a) {
  pdl_launch_dependents();                        // the move waits for this grid's end
  pdl_wait();                                     // the flags are clear
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
  const int b = blockIdx.x / chunks, i0 = (blockIdx.x - b * chunks) * kMoveRows;
  const int tid = threadIdx.x;
  const int raw_src = a.src_lens[b], raw_dst = a.dst_lens[b];
  const int most = a.dst_max < a.kept_width ? a.dst_max : a.kept_width;
  const int L = bounded_len(raw_src, a.src_max), N = bounded_len(raw_dst, most);
  const int rows = min(kMoveRows, N - i0);
  const int dst_blk = i0 / kBk;                   // dst_max is within dst_blocks pages
  int page = -1, bad = -1;                        // the new page; a bad position's row or source block
  if (rows > 0) {
    page = a.dst_table[(int64_t)b * a.dst_blocks + dst_blk];
    if (tid < a.R * kMoveRows) {
      const int r = tid / kMoveRows, x = tid - r * kMoveRows;
      int j = -1;
      int64_t row = -1;
      if (x < rows) {
        j = a.kept[((int64_t)b * a.R + r) * a.kept_width + i0 + x];
        if (j < 0 || j >= L) {
          bad = i0 + x;
          j = -1;
        } else {
          const int p = a.src_table[(int64_t)b * a.src_blocks + j / kBk];
          if (p < 0 || p >= a.num_pages) bad = j / kBk;
          else row = gather_src_row(p, j % kBk, kBk);
        }
      }
      from[r][x] = j;
      src_row[r][x] = row;
    }
    __syncthreads();
  }
  pdl_wait();                                     // the pages are marked, and the error word is clear
  if (i0 == 0 && tid == 0) {
    if (L != raw_src) report_error(a.err, MSA_ERR_DEVICE_CHECK, kSiteEvictMove, b, raw_src);
    if (N != raw_dst) report_error(a.err, MSA_ERR_DEVICE_CHECK, kSiteEvictMove, b, raw_dst);
  }
  if (rows > 0) {
    if (bad >= 0) report_error(a.err, MSA_ERR_DEVICE_CHECK, kSiteEvictMove, b, bad);
    bool page_ok = page >= 0 && page < a.num_pages;
    if (page_ok) page_ok = a.flags[page] == 1u;   // a destination once, no source
    if (!page_ok && tid == 0) report_error(a.err, MSA_ERR_DEVICE_CHECK, kSiteEvictMove, b, dst_blk);
    if (page_ok) {
      const int64_t dst0 = gather_src_row(page, i0 % kBk, kBk);
      // (four loads a thread in flight: 4 x 64K tokens in 191 us; with the streaming hints 193, and 218 with eight.)
      // words of a row, a power of two; with R == G a group's words come from its own token
      auto copy = [&](uint4* pages, int words, int pieces) {
        const int sh = 31 - __clz(words), psh = sh - (31 - __clz(pieces));
        const int n = rows << sh;
        for (int w0 = tid; w0 < n; w0 += 4 * kMoveThreads) {
          uint4 t[4];
          bool have[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const int w = w0 + y * kMoveThreads;
            have[y] = false;
            if (w < n) {
              const int x = w >> sh, col = w & (words - 1);
              const int64_t row = src_row[col >> psh][x];
              have[y] = row >= 0;
              if (have[y]) t[y] = pages[(row << sh) + col];
            }
          }
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const int w = w0 + y * kMoveThreads;
            if (have[y]) pages[(dst0 << sh) + w] = t[y];
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

// One launch, with a cluster of up to eight CTAs per (sequence, ranking), or six
// with a CTA per 4096 tokens?  In a graph 10K tokens take 13.2 us and 13.6, 40K
// 18.1 and 14.0; called one by one from Python 14.4 us and 26.6, 20.2 and 26.6.
// More clusters than run at once lose both ways (16 x 40K: 35 us and 19).
constexpr int kMaxCluster = 8, kMostCtas = 96;
int cluster_of(int32_t max_seqlen) {
  int cs = 1;
  while (cs <= kMaxCluster && max_seqlen > cs * kSelPart) cs *= 2;
  return cs;
}
bool by_launches(int64_t rows, int32_t max_seqlen) {
  const int cs = cluster_of(max_seqlen);
  return cs > kMaxCluster || (cs > 1 && rows * cs > kMostCtas);
}

struct LongLayout {
  int32_t parts;
  size_t keys, hist, found, counts, total;        // offsets after the header
};
LongLayout long_layout(int64_t rows, int32_t max_seqlen) {
  LongLayout L{};
  L.parts = (int32_t)(((int64_t)max_seqlen + kLongPart - 1) / kLongPart);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = align_up(off + bytes, 256);
    return o;
  };
  L.hist = take(sizeof(uint32_t) * 3 * rows * 2048);
  L.found = take(sizeof(LongRow) * 3 * rows);
  L.counts = take(sizeof(uint2) * rows * L.parts);
  L.keys = take(sizeof(uint32_t) * rows * L.parts * (size_t)kLongPart);
  L.total = off;
  return L;
}

int launch_long_select(const EvictSelectArgs& s, cudaStream_t st) {
  const int R = s.per_group ? s.G : 1;
  const int64_t rows = (int64_t)s.batch * R;
  const LongLayout L = long_layout(rows, s.max_seqlen);
  uint8_t* base = reinterpret_cast<uint8_t*>(s.work);
  LongArgs a{};
  a.weights = s.weights; a.width = s.width; a.seqlens = s.seqlens;
  a.G = s.G; a.R = R; a.parts = L.parts; a.max_seqlen = s.max_seqlen; a.budget = s.budget;
  a.n_sink = s.n_sink; a.n_recent = s.n_recent; a.kept = s.kept; a.new_lens = s.new_lens;
  a.keys = reinterpret_cast<uint32_t*>(base + L.keys);
  a.hist = reinterpret_cast<uint32_t*>(base + L.hist);
  a.found = reinterpret_cast<LongRow*>(base + L.found);
  a.counts = reinterpret_cast<uint2*>(base + L.counts);
  a.rows = (int32_t)rows; a.err = s.err;
  const dim3 grid((unsigned)(rows * L.parts));
  const int64_t clear = (3 * rows * 512 + kLongThreads - 1) / kLongThreads;
  ProfScope p("evict_select", st);                // all six
  prof_count_launch(5);
  long_clear_kernel<<<(unsigned)(clear < 592 ? clear : 592), kLongThreads, 0, st>>>(a);
  int rc = (int)cudaGetLastError();
  auto* keys = R == s.G ? long_keys_kernel<1> : s.G == 2 ? long_keys_kernel<2> : long_keys_kernel<4>;
  if (rc == 0) rc = launch_after(keys, grid, kLongThreads, st, a);
  if (rc == 0) rc = launch_after(long_hist_kernel<1>, grid, kLongThreads, st, a);
  if (rc == 0) rc = launch_after(long_hist_kernel<2>, grid, kLongThreads, st, a);
  if (rc == 0) rc = launch_after(long_count_kernel, grid, kLongThreads, st, a);
  if (rc == 0) rc = launch_after(long_write_kernel, grid, kLongThreads, st, a);
  return rc;
}

}  // namespace

size_t evict_select_work_bytes(int32_t batch, int32_t rankings, int32_t max_seqlen) {
  const int64_t rows = (int64_t)batch * rankings;
  return by_launches(rows, max_seqlen) ? long_layout(rows, max_seqlen).total : 0;
}

int launch_evict_select(const EvictSelectArgs& a, void* stream) {
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int64_t rows = (int64_t)a.batch * (a.per_group ? a.G : 1);
  if (by_launches(rows, a.max_seqlen)) return launch_long_select(a, st);
  const int gs = a.per_group ? 1 : a.G;
  const int cs = cluster_of(a.max_seqlen);
  // 1K tokens: 5.8 us with four tokens a thread, 8.7 with eight
#define MSA_SELECT(C, P) \
  (gs == 1 ? evict_select_kernel<C, 1, P> : gs == 2 ? evict_select_kernel<C, 2, P> : evict_select_kernel<C, 4, P>)
  auto* kernel = cs > 1 ? MSA_SELECT(true, 8) : a.max_seqlen > 4 * kSelThreads ? MSA_SELECT(false, 8) : MSA_SELECT(false, 4);
#undef MSA_SELECT
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * cs));
  cfg.blockDim = dim3(kSelThreads);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = cs;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cs > 1 ? 1 : 0;
  ProfScope p("evict_select", stream);
  return (int)cudaLaunchKernelEx(&cfg, kernel, a.weights, a.G, a.width, a.seqlens, a.batch, a.max_seqlen, a.budget,
                                 a.n_sink, a.n_recent, a.kept, a.new_lens, a.err);
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
    const int64_t want = (a.num_pages + 255) / 256;
    prof_count_launch(1);
    evict_clear_kernel<<<(unsigned)(want < 1184 ? want : 1184), 256, 0, st>>>(a.flags, a.num_pages, a.err);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return (int)e;
  }
  {
    const int64_t n = (int64_t)a.batch * ((int64_t)a.src_blocks + a.dst_blocks);
    const int64_t want = (n + 255) / 256;
    ProfScope p("evict_mark", stream);
    const int rc = launch_after(evict_mark_kernel, dim3((unsigned)(want < 1184 ? want : 1184)), 256, st, a);
    if (rc != 0) return rc;
  }
  // weights_out is written to its whole width, rows only up to the new lengths
  const int64_t last = a.weights_out != nullptr ? (int64_t)a.dst_blocks * kBk : a.dst_max;
  const int64_t chunks = (last + kMoveRows - 1) / kMoveRows;
  if (chunks * a.batch > 0x7fffffffLL) return (int)cudaErrorInvalidValue;
  ProfScope p("evict_move", stream);
  return launch_after(evict_move_kernel, dim3((unsigned)(chunks * a.batch)), kMoveThreads, st, a, (int)chunks);
}

}  // namespace msa
