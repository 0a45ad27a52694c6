// Dense attention of one new token per sequence over a paged KV cache, split
// over the cache's length and joined (include/msa.h:
// msa_dense_attn_decode_paged).
//
// For head h of group g and the keys j < L of its sequence
//   s_j = <q_h, k_j>,  out_h = sum_j e_j v_j / l,  e_j = 2^(c s_j - m),  l = sum_j e_j,
// with c = sm_scale log2(e) and m a 32-bit number no more than 8 below the largest
// c s_j so far (a larger one takes its place and rescales the sums by 2^(m_old -
// m_new), exact in m; letting e_j reach 2^8 spares most of that).  Parts of the keys
// have (m, l, o) of their own and join by the same rescaling.
//
// The step is bound by HBM: every cached key and value is read once and meets
// H / G query heads, 16 operations a byte at most.  On a B200 (H 64, G 4, d 128):
// 32 caches of 1..8192 tokens 53 to 55 us (283 MB; 43 at the rate of a copy), one of
// 1M 308 to 321 us in a row (6.7 to 7.0 TB/s); the loads alone take 306.  At H 32, G 4,
// d 64, 32 caches of 8192 tokens take 48 us (41 at the rate of a copy).
//   split : the caches are cut into tiles of 64 / G tokens with all G groups
//           (16 KB of keys and as much of values at d = 128, contiguous in the
//           page), and the tiles of all sequences, in order, into equal runs,
//           one per CTA and SM: a ragged batch is balanced to one tile.  One
//           warp streams the run through a ring of stages by TMA; eight warps
//           compute, four per tile (a warp has one group and 16 tokens of it),
//           so that two tiles are in work at once.
//   math  : mma.sync on 16 query rows x 16 tokens; tcgen05's smallest tile would
//           hold 128 rows, and the products take a quarter of the loads' time.
//           The softmax weights enter the second product as two bf16 terms
//           (value and remainder, 2^-17 in all): one bf16 would add an error as
//           large as the output's own rounding.
//   join  : a sequence that lies in one CTA's run is written at once; of the
//           others each CTA leaves (m, l, o), and dense_join_kernel adds them
//           in the order of the CTAs, the same from run to run.
//   weights: the scores are kept in 32 bits (a 16-bit score would be off by
//           2^-9 of its size, so its weight by per cents) and read again once m
//           and l are known: 8 H bytes a token next to the 4 G d of K and V.
//           Reading K again would cost 2 G d.  2 x 262K..400K tokens: 301 to
//           308 us, 16 x 1K..16K (H 32, G 2) 54.  The pass has a CTA per 512 tokens
//           of max_seqlen and leaves where a sequence has ended: 16 x 2K tokens take 31
//           us under a max_seqlen of 2K and 39 under one of 128K.
#include <cuda_runtime.h>

#include <atomic>

#include "msa_common.cuh"
#include "msa_cache.h"
#include "msa_internal.h"

namespace msa {
namespace {

constexpr int kSets = 2;                          // tiles in work at once
constexpr int kComputeWarps = 4 * kSets;
constexpr int kDecThreads = 32 * (kComputeWarps + 1);
constexpr int kTileTok = 16;                      // tokens of a warp in a tile
constexpr float kSlack = 8.f;                     // how far above m a score may be, in units of log2
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <int D>
__host__ __device__ constexpr int stage_bytes() { return 2 * 64 * D * 2; }          // keys and values of one tile
// 128 KB in flight per SM.  The loads alone, without the products: 1 x 1M tokens in 430 us with 64 KB, 306 us with
// 128 KB and 342 us with 192 KB, where more requests meet in L2 than it takes in order.
template <int D>
__host__ __device__ constexpr int num_stages() { return D == 128 ? 4 : 8; }
// Half the output fragments of four warps: the sums are merged in two halves of the columns, which leaves the
// join's first CTAs room beside this kernel's (they are in place when it ends).
template <int D>
__host__ __device__ constexpr int merge_bytes() { return 4 * 16 * (D / 2) * 4; }

struct DecCtl {
  uint64_t full[8];
  uint64_t empty[8];
  int32_t valid[8];             // tokens of the tile to attend (0: its page is outside the cache)
  int32_t warp_sum[10];
  int32_t first_seq, first_start, total;
  int32_t lens[kDecThreads];    // the batch's lengths, where a thread has one at most
  float ml[4][2][16];           // (m, l) rows of the merging warps
};

// A tensor load of data that is read once: its lines leave L2 first.
__device__ __forceinline__ uint64_t evict_first_policy() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ void tma_load_3d_hint(void* dst, const void* map, uint64_t* bar, int c0, int c1, int c2,
                                                 uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], "
      "[%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(dst)),
      "l"(map), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
// (Not volatile: a function of its registers, which the compiler may place among the loads.)
__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_16816_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void compute_bar() {
  asm volatile("bar.sync 1, %0;" ::"n"(32 * kComputeWarps) : "memory");
}
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// A sequence's length as the kernels take it: 0 for one outside its bounds.
__device__ __forceinline__ int seq_len(int L, int max_seqlen) { return (L < 0 || L > max_seqlen) ? 0 : L; }

// First tile of CTA i's run: the tiles in n runs that differ by one at most.
__host__ __device__ __forceinline__ int run_start(int i, int total, int n) {
  const int q = total / n, r = total - q * n;
  return i * q + (i < r ? i : r);
}
__device__ __forceinline__ int run_of(int t, int total, int n) {
  const int q = total / n, r = total - q * n;
  return t < r * (q + 1) ? t / (q + 1) : r + (t - r * (q + 1)) / q;
}

// The lengths of the batch: from shared memory where they fit, else read 32 at a time by a whole warp.
struct SeqLens {
  const int32_t *p, *near;
  int batch, max_seqlen, base, mine;
  __device__ SeqLens(const int32_t* lens, const int32_t* smem, int batch_, int max_, int at)
      : p(lens), near(smem), batch(batch_), max_seqlen(max_), base(0), mine(0) {
    if (batch > kDecThreads) fetch(at);
  }
  __device__ void fetch(int at) {
    const int i = at + (threadIdx.x & 31);
    base = at;
    mine = i < batch ? seq_len(p[i], max_seqlen) : 0;
  }
  __device__ int operator()(int b) {
    if (batch <= kDecThreads) return near[b];
    if (b - base >= 32) fetch(b);
    return __shfl_sync(0xffffffffu, mine, b - base);
  }
};

// What a CTA has summed of a sequence, where something came out infinite or NaN (a
// cache with such a value, or one too large: seldom).  The two terms of a softmax
// weight meet a value v separately, and that breaks an infinite one: a remainder of
// 0 times inf is NaN, a negative one gives inf - inf.  So the warp that has a group's
// sums reads the values of the tiles [first, end) again from their pages, and a column
// that has one that is not finite gets what the formula says for weights above 0:
// that infinity, or NaN for both signs or a NaN: written over what the warp has
// stored, row y of the lane (r, r + 8) where bit y of `rows` says so, to `out` or, of a
// part, to `part`.  Lane (r, c2 / 2) reads the tokens r, r + 8, ... of a tile in its
// own columns.  (Not inlined, and in memory: 32 x 1..8192 tokens, H 64, G 4, d 128, take
// 53.1 us so and 57.6 with it among the main loop's registers.  A context of 1M with
// one infinity takes 1.0 ms in place of 0.31, with infinities everywhere 1.2.)
template <int D>
__device__ __noinline__ void put_infinities(const __nv_bfloat16* __restrict__ v_pages, int G, int g,
                                            const int32_t* __restrict__ table, int64_t num_pages, int L, int first, int end,
                                            __nv_bfloat16* out, float* part, uint32_t rows) {
  const int lane = threadIdx.x & 31, r = lane >> 2, c2 = 2 * (lane & 3);
  const int tok = 64 / G;
  uint32_t pos = 0, neg = 0;                     // a bit per column of the lane: 2 n + parity
  for (int t = first; t < end; ++t) {            // tiles of the sequence
    const int j0 = t * tok, page = table[j0 / kBk];
    if (page < 0 || page >= num_pages) continue;
    for (int x = r; x < min(tok, L - j0); x += 8) {
      const int64_t row = (int64_t)page * kBk + (j0 & (kBk - 1)) + x;
      const uint32_t* src = reinterpret_cast<const uint32_t*>(v_pages + (row * G + g) * D + c2);
#pragma unroll
      for (int n = 0; n < D / 8; ++n) {
        const uint32_t two = src[4 * n];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const uint32_t u = y == 0 ? two & 0xffffu : two >> 16, bit = 1u << (2 * n + y);
          if ((u & 0x7f80u) != 0x7f80u) continue;
          const bool nan = (u & 0x7fu) != 0;
          if (nan || u < 0x8000u) pos |= bit;
          if (nan || u >= 0x8000u) neg |= bit;
        }
      }
    }
  }
#pragma unroll
  for (int x = 4; x <= 16; x <<= 1) {
    pos |= __shfl_xor_sync(0xffffffffu, pos, x);
    neg |= __shfl_xor_sync(0xffffffffu, neg, x);
  }
  for (int y = 0; y < 2; ++y) {
    if ((rows >> y & 1u) == 0) continue;
    for (int i = 0; i < D / 4; ++i) {
      const uint32_t bit = 1u << i;
      if (((pos | neg) & bit) == 0) continue;
      const float v = pos & neg & bit ? __uint_as_float(0x7fffffffu) : pos & bit ? INFINITY : -INFINITY;
      const int at = (r + 8 * y) * D + 8 * (i >> 1) + c2 + (i & 1);
      if (out != nullptr) out[at] = __float2bfloat16_rn(v);
      else part[at] = v;
    }
  }
}

// kFew: at most eight heads a group.  The rows that they leave of the second
// product's operand then hold the remainders: one product does for both terms (in a
// graph, H 32, G 4: 8 x 64K tokens at d 64 83.6 us, 87.8 with two; at d 128 156.5 and
// 157.2).
template <int D, bool kWeights, bool kFew>
__global__ void __launch_bounds__(kDecThreads, 1)
dense_decode_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                    const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ v_pages,
                    __nv_bfloat16* __restrict__ out, float* __restrict__ lse, int batch, int H, int G, float sm_scale,
                    const int32_t* __restrict__ seqlens, const int32_t* __restrict__ block_table, int max_blocks,
                    int max_seqlen, int64_t num_pages,
                    float2* __restrict__ stats, float2* __restrict__ part_ml, float* __restrict__ part_o,
                    float* __restrict__ logits, int logit_tiles, DevError* errors) {
  constexpr int NST = num_stages<D>();
  constexpr int STAGE = stage_bytes<D>();
  constexpr int KV = STAGE / 2;
  constexpr int KK = D / 16;                    // 16-wide steps along d
  constexpr int NY = kFew ? 1 : 2;              // rows of heads a thread has: r, and r + 8
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  float* mbuf = reinterpret_cast<float*>(smem + NST * STAGE);
  DecCtl* ctl = reinterpret_cast<DecCtl*>(smem + NST * STAGE + merge_bytes<D>());

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int Hg = H / G;
  const int tok = 64 / G;                       // tokens per tile
  pdl_launch_dependents();                      // the join waits for this grid's end by itself
  DevError* err = errors + blockIdx.x;          // the join makes one word of them

  // ---- this CTA's run of tiles: one scan over the batch's lengths
  {
    if (threadIdx.x == 0) {
      *err = DevError{0, 0, 0, 0};
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
    const int per = (batch + kDecThreads - 1) / kDecThreads;
    const int b0 = threadIdx.x * per;
    int sum = 0, bad = -1;
    for (int b = b0; b < min(b0 + per, batch); ++b) {
      const int raw_len = seqlens[b];
      const int L = seq_len(raw_len, max_seqlen);
      if (L != raw_len) bad = b;
      if (per == 1) ctl->lens[b] = L;
      sum += (L + tok - 1) / tok;
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) ctl->warp_sum[warp] = incl;
    if (threadIdx.x == 0) {
      for (int i = 0; i < NST; ++i) {
        mbar_init(&ctl->full[i], 1);
        mbar_init(&ctl->empty[i], 4);
      }
      fence_mbar_init();
    }
    __syncthreads();
    if (blockIdx.x == 0 && bad >= 0) report_error(err, MSA_ERR_DEVICE_CHECK, kSiteDenseDecode, bad, seqlens[bad]);
    int before = 0, total = 0;
    for (int w = 0; w <= kComputeWarps; ++w) {
      if (w < warp) before += ctl->warp_sum[w];
      total += ctl->warp_sum[w];
    }
    before += incl - sum;
    const int lo = run_start(blockIdx.x, total, gridDim.x);
    if (lo >= before && lo < before + sum) {    // the run begins in this thread's sequences
      int s = before, b = b0;
      for (;; ++b) {
        const int nt = (seq_len(seqlens[b], max_seqlen) + tok - 1) / tok;
        if (lo < s + nt) break;
        s += nt;
      }
      ctl->first_seq = b;
      ctl->first_start = s;
    }
    if (threadIdx.x == 0) ctl->total = total;
    __syncthreads();
  }
  const int total = ctl->total;
  const int lo = run_start(blockIdx.x, total, gridDim.x);
  const int hi = run_start(blockIdx.x + 1, total, gridDim.x);
  if (lo >= hi) return;
  SeqLens lens(seqlens, ctl->lens, batch, max_seqlen, ctl->first_seq);
  int b = ctl->first_seq, s = ctl->first_start;      // the sequence at hand and its first tile

  if (warp == kComputeWarps) {
    // ------------------------------------------------------------ loads
    const uint64_t once = evict_first_policy();
    bool ok = true;
    int issued = 0;
    for (int t = lo; t < hi;) {
      const int L = lens(b);
      const int nt = (L + tok - 1) / tok;
      if (t >= s + nt) {
        s += nt;
        ++b;
        continue;
      }
      const int e = min(hi, s + nt);
      int page_base = -32, my_page = -1;
      for (; t < e; ++t) {
        const int j0 = (t - s) * tok;                // first token of the tile
        const int blk = j0 / kBk;
        if (blk - page_base >= 32 || page_base < 0) {
          page_base = blk;
          my_page = blk + lane < max_blocks && (int64_t)(blk + lane) * kBk < L
                        ? block_table[(int64_t)b * max_blocks + blk + lane] : -1;
        }
        const int page = __shfl_sync(0xffffffffu, my_page, blk - page_base);
        const int i = t - lo, st = i % NST;
        if (lane == 0 && ok) {
          if (i >= NST) ok = mbar_wait(&ctl->empty[st], ((i / NST) + 1) & 1);
          if (ok) {
            const bool in = page >= 0 && page < num_pages;
            ctl->valid[st] = in ? min(tok, L - j0) : 0;
            if (in) {
              uint8_t* dst = smem + st * STAGE;
              const int row = page * kBk + (j0 & (kBk - 1));
              mbar_arrive_expect_tx(&ctl->full[st], STAGE);
              tma_load_3d_hint(dst, &tm_k, &ctl->full[st], 0, row, 0, once);
              tma_load_3d_hint(dst + KV, &tm_v, &ctl->full[st], 0, row, 0, once);
            } else {
              report_error(err, MSA_ERR_DEVICE_CHECK, kSiteDenseDecode, b, blk);
              mbar_arrive(&ctl->full[st]);
            }
            ++issued;
          }
        }
        __syncwarp();
      }
    }
    if (lane == 0) {
      if (!ok) report_error(err, MSA_ERR_TIMEOUT, kSiteDenseDecode, blockIdx.x, -1);
      // no load may remain in flight when the CTA exits
      for (int i = max(0, issued - NST); i < issued; ++i) mbar_wait(&ctl->full[i % NST], (i / NST) & 1);
    }
    return;
  }

  // -------------------------------------------------------------- compute
  const int set = warp >> 2;                     // takes every other tile of the run
  const int g = (warp & 3) % G, sub = (warp & 3) / G;
  const int nsub = 4 / G;
  const int r = lane >> 2, c2 = 2 * (lane & 3);
  const float c = sm_scale * kLog2e;
  const uint32_t smem0 = smem_u32(smem);
  const uint32_t swz = lane & 7;                 // (row mod 8) of every row this lane addresses
  const uint32_t line = tok * 128;               // bytes of one 64-column block of a tile
  const uint32_t grp = g * (D / 64) * line + sub * kTileTok * 128;
  const uint32_t k_row = ((lane & 7) + ((lane >> 4) & 1) * 8) * 128, k_bit = (lane >> 3) & 1;
  const uint32_t v_row = ((lane & 7) + ((lane >> 3) & 1) * 8) * 128, v_bit = lane >> 4;
  bool dead = false;                             // a wait ran out: no further waits or sums, the barriers still

  for (int t = lo; t < hi;) {
    const int L = lens(b);
    const int nt = (L + tok - 1) / tok;
    if (t >= s + nt) {
      s += nt;
      ++b;
      continue;
    }
    const int t0 = t, e = min(hi, s + nt);
    // the group's query heads as the A operand: rows h = r and r + 8 (zero from Hg on)
    uint32_t qf[KK][4];
    {
      const __nv_bfloat16* qg = q + ((int64_t)b * H + (int64_t)g * Hg) * D;
#pragma unroll
      for (int kk = 0; kk < KK; ++kk)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int h = r + 8 * (x & 1), col = 16 * kk + c2 + 8 * (x >> 1);
          qf[kk][x] = h < Hg ? *reinterpret_cast<const uint32_t*>(qg + (int64_t)h * D + col) : 0u;
        }
    }
    float o[D / 8][4];
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
      for (int x = 0; x < 4; ++x) o[n][x] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

    for (t += ((t - lo) & 1) != set; t < e; t += kSets) {
      const int i = t - lo, st = i % NST;
      if (!dead && !mbar_wait(&ctl->full[st], (i / NST) & 1)) {
        report_error(err, MSA_ERR_TIMEOUT, kSiteDenseDecode, blockIdx.x, warp);
        dead = true;
      }
      if (dead) continue;
      const int valid = ctl->valid[st] - sub * kTileTok;      // tokens of this warp to attend
      auto release = [&] {                                     // the warp's part of the stage is in its registers
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->empty[st]);
      };
      float sc[2][4];                                          // scores: tokens 0-7 and 8-15 of the warp
      const uint32_t base = smem0 + st * STAGE + grp;
      uint32_t f[KK][4];                                       // the keys' fragments, then the values'
      if (valid > 0) {
        // every load ahead of the products, and two chains of products a half: a warp's time on a tile is
        // latency, and it is what holds the stage
#pragma unroll
        for (int kk = 0; kk < KK; ++kk)
          ldsm_x4(base + (kk >> 2) * line + k_row + ((((kk & 3) * 2 + k_bit) ^ swz) << 4), f[kk]);
        float odd[2][4];
        mma_16816_first(sc[0], qf[0], f[0][0], f[0][1]);
        mma_16816_first(sc[1], qf[0], f[0][2], f[0][3]);
        mma_16816_first(odd[0], qf[1], f[1][0], f[1][1]);
        mma_16816_first(odd[1], qf[1], f[1][2], f[1][3]);
#pragma unroll
        for (int kk = 2; kk < KK; kk += 2) {
          mma_16816(sc[0], qf[kk], f[kk][0], f[kk][1]);
          mma_16816(sc[1], qf[kk], f[kk][2], f[kk][3]);
          mma_16816(odd[0], qf[kk + 1], f[kk + 1][0], f[kk + 1][1]);
          mma_16816(odd[1], qf[kk + 1], f[kk + 1][2], f[kk + 1][3]);
        }
#pragma unroll
        for (int n2 = 0; n2 < KK / 2; ++n2)
          ldsm_x4_trans(base + KV + (n2 >> 2) * line + v_row + ((((n2 & 3) * 2 + v_bit) ^ swz) << 4), f[n2]);
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int x = 0; x < 4; ++x) sc[n][x] += odd[n][x];
        if (valid < kTileTok) {
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int x = 0; x < 4; ++x)
              if (8 * n + c2 + (x & 1) >= valid) sc[n][x] = -INFINITY;
        }
      } else {
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int x = 0; x < 4; ++x) sc[n][x] = -INFINITY;
      }
      if constexpr (kWeights) {
        // per 16 tokens and group: row h holds its 16 scores as four lanes' (2 + 2)
        const int64_t tile16 = (int64_t)b * logit_tiles + (int64_t)(t - s) * nsub + sub;
        float4* dst = reinterpret_cast<float4*>(logits + (tile16 * G + g) * (int64_t)(kTileTok * Hg));
        if (r < Hg) dst[lane] = make_float4(sc[0][0], sc[0][1], sc[1][0], sc[1][1]);
        if (r + 8 < Hg) dst[32 + lane] = make_float4(sc[0][2], sc[0][3], sc[1][2], sc[1][3]);
      }
      if (valid > 0) {
        float top[2], sub_m[2];
        bool grew = false;
#pragma unroll
        for (int y = 0; y < NY; ++y) {
          float mx = fmaxf(fmaxf(sc[0][2 * y], sc[0][2 * y + 1]), fmaxf(sc[1][2 * y], sc[1][2 * y + 1]));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          top[y] = mx * c;
          grew |= top[y] > m[y] + kSlack;
        }
        if (__any_sync(0xffffffffu, grew)) {
          float fac[NY];
#pragma unroll
          for (int y = 0; y < NY; ++y) {
            const bool up = top[y] > m[y] + kSlack;
            fac[y] = up ? ex2_approx(m[y] - top[y]) : 1.f;
            if (up) m[y] = top[y];
          }
#pragma unroll
          for (int n = 0; n < D / 8; ++n)
#pragma unroll
            for (int x = 0; x < 4; ++x) o[n][x] *= fac[kFew ? 0 : x >> 1];
#pragma unroll
          for (int y = 0; y < NY; ++y) l[y] *= fac[y];
        }
#pragma unroll
        for (int y = 0; y < NY; ++y) sub_m[y] = m[y] == -INFINITY ? 0.f : m[y];   // no key yet: 2^(-inf - 0) = 0
        uint32_t ph[4], pl[4];                                  // value and remainder of the weights
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int y = 0; y < NY; ++y) {
            const float p0 = ex2_approx(fmaf(sc[n][2 * y], c, -sub_m[y]));
            const float p1 = ex2_approx(fmaf(sc[n][2 * y + 1], c, -sub_m[y]));
            l[y] += p0 + p1;
            const uint32_t hi2 = pack_bf16x2(p0, p1);
            const uint32_t lo2 = pack_bf16x2(p0 - __uint_as_float(hi2 << 16), p1 - __uint_as_float(hi2 & 0xffff0000u));
            ph[2 * n + y] = hi2;
            if constexpr (kFew) ph[2 * n + 1] = lo2;
            else pl[2 * n + y] = lo2;
          }
#pragma unroll
        for (int n2 = KK / 2; n2 < KK; ++n2)     // (all of them ahead of the softmax would not fit in the registers)
          ldsm_x4_trans(base + KV + (n2 >> 2) * line + v_row + ((((n2 & 3) * 2 + v_bit) ^ swz) << 4), f[n2]);
        release();
        // value rows past the last token may hold anything (0 x inf is no 0): cleared in the operand
        uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;
        if (valid < kTileTok) {
          keep0 = (c2 < valid ? 0xffffu : 0u) | (c2 + 1 < valid ? 0xffff0000u : 0u);
          keep1 = (c2 + 8 < valid ? 0xffffu : 0u) | (c2 + 9 < valid ? 0xffff0000u : 0u);
        }
        if (valid < kTileTok) {
#pragma unroll
          for (int n2 = 0; n2 < KK; ++n2) {
            f[n2][0] &= keep0;
            f[n2][1] &= keep1;
            f[n2][2] &= keep0;
            f[n2][3] &= keep1;
          }
        }
#pragma unroll
        for (int n2 = 0; n2 < KK; ++n2) {
          mma_16816(o[2 * n2], ph, f[n2][0], f[n2][1]);
          mma_16816(o[2 * n2 + 1], ph, f[n2][2], f[n2][3]);
        }
        if constexpr (!kFew) {
#pragma unroll
          for (int n2 = 0; n2 < KK; ++n2) {
            mma_16816(o[2 * n2], pl, f[n2][0], f[n2][1]);
            mma_16816(o[2 * n2 + 1], pl, f[n2][2], f[n2][3]);
          }
        }
      } else {
        release();
      }
    }

    t = e;
    // ---- the warps' sums of this part of the sequence become one per group
    if constexpr (kFew) {                        // both terms of the rows r
#pragma unroll
      for (int n = 0; n < D / 8; ++n) {
        o[n][0] += o[n][2];
        o[n][1] += o[n][3];
        o[n][2] = o[n][3] = 0.f;
      }
    }
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      l[y] += __shfl_xor_sync(0xffffffffu, l[y], 1);
      l[y] += __shfl_xor_sync(0xffffffffu, l[y], 2);
    }
    const int part = set * nsub + sub;            // of kSets * nsub parts of group g
    for (int step = kSets * nsub / 2; step >= 1; step >>= 1) {
      const bool gives = part >= step && part < 2 * step, takes = part < step;
      const int slot = (gives ? part - step : part) * G + g;
      float* buf = mbuf + slot * (16 * (D / 2));
      float fa[2] = {0.f, 0.f}, fb[2] = {0.f, 0.f};
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        if (gives) {
#pragma unroll
          for (int n = 0; n < D / 16; ++n)
#pragma unroll
            for (int x = 0; x < 4; ++x) buf[(4 * n + x) * 32 + lane] = o[half * (D / 16) + n][x];
          if (half == 0 && (lane & 3) == 0) {
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              ctl->ml[slot][0][r + 8 * y] = m[y];
              ctl->ml[slot][1][r + 8 * y] = l[y];
            }
          }
        }
        compute_bar();
        if (takes) {
          if (half == 0) {
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const float m2 = ctl->ml[slot][0][r + 8 * y], l2 = ctl->ml[slot][1][r + 8 * y];
              const float mn = fmaxf(m[y], m2);
              const float ms = mn == -INFINITY ? 0.f : mn;
              fa[y] = ex2_approx(m[y] - ms);
              fb[y] = ex2_approx(m2 - ms);
              l[y] = l[y] * fa[y] + l2 * fb[y];
              m[y] = mn;
            }
          }
#pragma unroll
          for (int n = 0; n < D / 16; ++n)
#pragma unroll
            for (int x = 0; x < 4; ++x)
              o[half * (D / 16) + n][x] = o[half * (D / 16) + n][x] * fa[x >> 1] + buf[(4 * n + x) * 32 + lane] * fb[x >> 1];
        }
        compute_bar();
      }
    }
    if (part == 0) {
      float size[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int n = 0; n < D / 8; ++n)
#pragma unroll
        for (int x = 0; x < 2 * NY; ++x) size[x] += fabsf(o[n][x]);
      const bool odd = __any_sync(0xffffffffu, !((size[0] + size[1]) + (size[2] + size[3]) <= 3.402823466e38f));
      const bool whole = t0 == s && e == s + nt;
      const int slot = t0 == s ? 1 : 0;
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int hl = r + 8 * y;
        if (hl >= Hg) continue;
        const int h = g * Hg + hl;
        if (whole) {
          // no weight at all (every score -inf): zeros, whatever the values are
          const bool none = l[y] == 0.f;
          const float inv = none ? 0.f : 1.f / l[y];
          __nv_bfloat16* dst = out + ((int64_t)b * H + h) * D + c2;
#pragma unroll
          for (int n = 0; n < D / 8; ++n)
            *reinterpret_cast<uint32_t*>(dst + 8 * n) =
                none ? 0u : pack_bf16x2(o[n][2 * y] * inv, o[n][2 * y + 1] * inv);
          if ((lane & 3) == 0) {
            if (lse != nullptr)
              lse[(int64_t)b * H + h] = none ? -INFINITY : (m[y] + log2f(l[y])) * kLn2;
            if constexpr (kWeights) stats[(int64_t)b * H + h] = make_float2(m[y], l[y]);
          }
        } else {
          const int64_t at = ((int64_t)blockIdx.x * 2 + slot) * H + h;
          float* dst = part_o + at * D + c2;
#pragma unroll
          for (int n = 0; n < D / 8; ++n)
            *reinterpret_cast<float2*>(dst + 8 * n) = make_float2(o[n][2 * y], o[n][2 * y + 1]);
          if ((lane & 3) == 0) part_ml[at] = make_float2(m[y], l[y]);
        }
      }
      if (odd) {                                  // (a row without any weight keeps its zeros, one with a NaN among them its NaN)
        const uint32_t rows = (r < Hg && (!whole || l[0] > 0.f) ? 1u : 0u) | (r + 8 < Hg && (!whole || l[1] > 0.f) ? 2u : 0u);
        put_infinities<D>(v_pages, G, g, block_table + (int64_t)b * max_blocks, num_pages, L, t0 - s, e - s,
                          whole ? out + ((int64_t)b * H + g * Hg) * D : nullptr,
                          part_o + (((int64_t)blockIdx.x * 2 + slot) * H + g * Hg) * D, rows);
      }
    }
  }
}

// Joins the parts of the sequences that lie in several CTAs' runs, writes the
// rows of sequences without tokens, and makes one error word of the CTAs'.  WPJ
// warps have one (b, h) and VEC columns a lane, so that few sequences in many
// parts and many in few parts both keep the loads in flight: a warp reads the
// parts w, w + WPJ, ... eight at a time.  (What the kernel ahead writes is read through
// pointers without __restrict__: const ones with it may be read before the wait.)
constexpr int kMaxParts = (kDecodeCtas + 31) / 32 * 32;
template <int D, int WPJ, int VEC>
__global__ void __launch_bounds__(256)
dense_join_kernel(__nv_bfloat16* __restrict__ out, float* __restrict__ lse, int batch, int H, int G,
                  const int32_t* __restrict__ seqlens, int max_seqlen, const float2* part_ml, const float* part_o,
                  float2* __restrict__ stats, int ctas, const DevError* errors, DevError* err) {
  constexpr int JPC = 8 / WPJ;                   // (b, h) pairs per CTA
  constexpr int CB = D / (32 * VEC);             // CTAs that share a pair's columns
  constexpr int BATCH = 8;                       // parts in flight per warp
  __shared__ float acc[WPJ > 1 ? 8 : 1][32 * VEC];
  __shared__ float fac[JPC][kMaxParts];
  __shared__ int32_t wsum[2][8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int w = warp % WPJ;
  const int tok = 64 / G;
  pdl_launch_dependents();
  // ---- the first tile of the CTA's first sequence, and all tiles (before the kernel ahead has ended: lengths are
  // no output of it)
  const int64_t pair0 = (int64_t)(blockIdx.x / CB) * JPC;
  const int b0 = (int)(pair0 / H);
  int total, s;
  {
    int sum = 0, mine = 0;
    for (int i = threadIdx.x; i < batch; i += 256) {
      const int n = (seq_len(seqlens[i], max_seqlen) + tok - 1) / tok;
      sum += n;
      if (i < b0) mine += n;
    }
#pragma unroll
    for (int x = 16; x >= 1; x >>= 1) {
      sum += __shfl_xor_sync(0xffffffffu, sum, x);
      mine += __shfl_xor_sync(0xffffffffu, mine, x);
    }
    if (lane == 0) {
      wsum[0][warp] = sum;
      wsum[1][warp] = mine;
    }
    __syncthreads();
    total = 0;
    s = 0;
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      total += wsum[0][x];
      s += wsum[1][x];
    }
  }
  const int64_t pair = pair0 + warp / WPJ;
  const int col = (int)(blockIdx.x % CB) * 32 * VEC + VEC * lane;
  const bool live = pair < (int64_t)batch * H;
  const int b = live ? (int)(pair / H) : b0, h = (int)(pair - (int64_t)b * H);
  for (int i = b0; i < b; ++i) s += (seq_len(seqlens[i], max_seqlen) + tok - 1) / tok;
  const int L = seq_len(seqlens[b], max_seqlen);
  const int nt = (L + tok - 1) / tok;
  const int c0 = L > 0 ? run_of(s, total, ctas) : 0, n = L > 0 ? run_of(s + nt - 1, total, ctas) - c0 + 1 : 0;
  pdl_wait();
  if (blockIdx.x == 0 && warp == 0) {            // the first CTA's that found something
    int first = ctas;
    for (int i = lane; i < ctas; i += 32)
      if (errors[i].code != 0) first = min(first, i);
    first = __reduce_min_sync(0xffffffffu, first);
    if (lane == 0) *err = first < ctas ? errors[first] : DevError{0, 0, 0, 0};
  }
  // with WPJ > 1 every warp of a CTA has the same pair, so the exits are the CTA's
  if (!live || n == 1) return;                   // written by its CTA
  __nv_bfloat16* dst = out + pair * D + col;
  auto store = [&](const float (&y)[VEC]) {
    if constexpr (VEC == 1) {
      dst[0] = __float2bfloat16_rn(y[0]);
    } else {
#pragma unroll
      for (int x = 0; x < VEC; x += 2) reinterpret_cast<uint32_t*>(dst)[x / 2] = pack_bf16x2(y[x], y[x + 1]);
    }
  };
  float o[VEC];
#pragma unroll
  for (int x = 0; x < VEC; ++x) o[x] = 0.f;
  if (n == 0) {
    if (w == 0) {
      store(o);
      if (lane == 0 && blockIdx.x % CB == 0) {
        if (lse != nullptr) lse[pair] = -INFINITY;
        stats[pair] = make_float2(-INFINITY, 0.f);
      }
    }
    return;
  }
  // the part of CTA c0 + i: slot 1 where its run holds the sequence's first tile
  auto at_of = [&](int i) -> int64_t { return ((int64_t)(c0 + i) * 2 + (i == 0 ? 1 : 0)) * H + h; };
  float v[BATCH][VEC];
  auto fetch = [&](int i0) {
#pragma unroll
    for (int u = 0; u < BATCH; ++u) {
      const int i = i0 + u * WPJ;
#pragma unroll
      for (int x = 0; x < VEC; ++x) v[u][x] = 0.f;
      if (i < n) {
        const float* src = part_o + at_of(i) * D + col;
        if constexpr (VEC == 4) {
          const float4 q = *reinterpret_cast<const float4*>(src);
          v[u][0] = q.x; v[u][1] = q.y; v[u][2] = q.z; v[u][3] = q.w;
        } else if constexpr (VEC == 2) {
          const float2 q = *reinterpret_cast<const float2*>(src);
          v[u][0] = q.x; v[u][1] = q.y;
        } else {
          v[u][0] = *src;
        }
      }
    }
  };
  fetch(w);
  // every warp: the maximum, the sum and each part's factor
  float2 ml[kMaxParts / 32];
  float m = -INFINITY, l = 0.f;
#pragma unroll
  for (int x = 0; x < kMaxParts / 32; ++x) {
    const int i = 32 * x + lane;
    ml[x] = i < n ? part_ml[at_of(i)] : make_float2(-INFINITY, 0.f);
    m = fmaxf(m, ml[x].x);
  }
#pragma unroll
  for (int x = 16; x >= 1; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
  const float ms = m == -INFINITY ? 0.f : m;
  float* f = fac[warp / WPJ];
#pragma unroll
  for (int x = 0; x < kMaxParts / 32; ++x) {
    const float e = ex2_approx(ml[x].x - ms);
    l = fmaf(ml[x].y, e, l);
    f[32 * x + lane] = e;                        // the warps of a pair write the same
  }
#pragma unroll
  for (int x = 16; x >= 1; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
  __syncwarp();
  for (int i0 = w;;) {
#pragma unroll
    for (int u = 0; u < BATCH; ++u) {
      const int i = i0 + u * WPJ;
      if (i < n) {
        const float e = f[i];
#pragma unroll
        for (int x = 0; x < VEC; ++x) o[x] = fmaf(v[u][x], e, o[x]);
      }
    }
    i0 += BATCH * WPJ;
    if (i0 >= n) break;
    fetch(i0);
  }
  if constexpr (WPJ > 1) {
#pragma unroll
    for (int x = 0; x < VEC; ++x) acc[warp][VEC * lane + x] = o[x];
    __syncthreads();
    if (w != 0) return;
#pragma unroll
    for (int x = 0; x < VEC; ++x) {
      o[x] = 0.f;
#pragma unroll
      for (int u = 0; u < WPJ; ++u) o[x] += acc[u][VEC * lane + x];
    }
  }
  const float inv = 1.f / l;
#pragma unroll
  for (int x = 0; x < VEC; ++x) o[x] = l == 0.f ? 0.f : o[x] * inv;   // no weight at all: zeros, whatever the values are
  store(o);
  if (lane == 0 && blockIdx.x % CB == 0) {
    if (lse != nullptr) lse[pair] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
    stats[pair] = make_float2(m, l);
  }
}

// weights[b, g, j] = decay weights[b, g, j] + sum_h 2^(c s_hj - m_h) / l_h
// from the kept scores; a warp takes 16 tokens at a time (HBM: 4 Hg + 8 bytes a
// token and group).
constexpr int kWeightTiles = 32;                 // 16-token tiles per CTA
__global__ void __launch_bounds__(256)
dense_weights_kernel(const float* logits, const float2* stats, float* __restrict__ weights,
                     int H, int G, float c, float decay, const int32_t* __restrict__ seqlens, int max_seqlen,
                     int64_t width, int logit_tiles) {
  const int b = blockIdx.z, g = blockIdx.y, Hg = H / G;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2;
  const int first = blockIdx.x * kWeightTiles;
  pdl_wait();
  const int L = seq_len(seqlens[b], max_seqlen);
  if (first * kTileTok >= L) return;
  float mc[2], inv[2];
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    const int h = r + 8 * y;
    float2 st = make_float2(0.f, 0.f);
    if (h < Hg) st = stats[(int64_t)b * H + g * Hg + h];
    mc[y] = st.x == -INFINITY ? 0.f : st.x;
    inv[y] = st.y == 0.f ? 0.f : 1.f / st.y;
  }
  float* wrow = weights + ((int64_t)b * G + g) * width;
#pragma unroll 2
  for (int k = warp; k < kWeightTiles; k += 8) {
    const int tile = first + k;
    if (tile * kTileTok >= L) break;
    const float4* src =
        reinterpret_cast<const float4*>(logits + (((int64_t)b * logit_tiles + tile) * G + g) * (int64_t)(kTileTok * Hg));
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f), p = a;
    if (r < Hg) a = __ldcs(src + lane);
    if (r + 8 < Hg) p = __ldcs(src + 32 + lane);
    // tokens c2, c2 + 1, c2 + 8, c2 + 9 of the tile, c2 = 2 (lane mod 4)
    float v[4];
    v[0] = r < Hg ? ex2_approx(fmaf(a.x, c, -mc[0])) * inv[0] : 0.f;
    v[1] = r < Hg ? ex2_approx(fmaf(a.y, c, -mc[0])) * inv[0] : 0.f;
    v[2] = r < Hg ? ex2_approx(fmaf(a.z, c, -mc[0])) * inv[0] : 0.f;
    v[3] = r < Hg ? ex2_approx(fmaf(a.w, c, -mc[0])) * inv[0] : 0.f;
    if (r + 8 < Hg) {
      v[0] += ex2_approx(fmaf(p.x, c, -mc[1])) * inv[1];
      v[1] += ex2_approx(fmaf(p.y, c, -mc[1])) * inv[1];
      v[2] += ex2_approx(fmaf(p.z, c, -mc[1])) * inv[1];
      v[3] += ex2_approx(fmaf(p.w, c, -mc[1])) * inv[1];
    }
    // sums over the eight row lanes; a lane ends with one token of its four
    const bool up16 = lane & 16, up8 = lane & 8;
    const float s0 = __shfl_xor_sync(0xffffffffu, up16 ? v[0] : v[2], 16);
    const float s1 = __shfl_xor_sync(0xffffffffu, up16 ? v[1] : v[3], 16);
    const float x0 = (up16 ? v[2] : v[0]) + s0, x1 = (up16 ? v[3] : v[1]) + s1;
    const float s2 = __shfl_xor_sync(0xffffffffu, up8 ? x0 : x1, 8);
    float y = (up8 ? x1 : x0) + s2;
    y += __shfl_xor_sync(0xffffffffu, y, 4);
    const int j = tile * kTileTok + 2 * (lane & 3) + (up8 ? 1 : 0) + (up16 ? 8 : 0);
    if ((lane & 4) == 0 && j < L) wrow[j] = decay == 0.f ? y : fmaf(decay, wrow[j], y);
  }
}

template <int D, bool kWeights, bool kFew>
int launch_split(const DenseDecodeArgs& a, int ctas, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                 int logit_tiles, cudaStream_t st) {
  constexpr int smem = 1024 + num_stages<D>() * stage_bytes<D>() + merge_bytes<D>() + (int)sizeof(DecCtl);
  static_assert(smem <= 220 * 1024, "shared memory of one CTA, and 7 KB for the join's beside it");
  static_assert(num_stages<D>() <= 8, "barriers of the stages");
  // a stage belongs to one set: a set that saw every other phase of it could not tell them by parity
  static_assert(num_stages<D>() % kSets == 0, "stages per set");
  static std::atomic<uint64_t> ready{0};
  const int rc = allow_smem(dense_decode_kernel<D, kWeights, kFew>, smem, &ready);
  if (rc != 0) return rc;
  ProfScope p("dense_decode", st);
  dense_decode_kernel<D, kWeights, kFew><<<ctas, kDecThreads, smem, st>>>(
      tm_k, tm_v, static_cast<const __nv_bfloat16*>(a.q), static_cast<const __nv_bfloat16*>(a.v_pages),
      static_cast<__nv_bfloat16*>(a.out), a.lse, a.batch, a.H, a.G, a.sm_scale, a.seqlens, a.block_table, a.max_blocks,
      a.max_seqlen, a.num_pages, a.stats, a.part_ml, a.part_o, a.logits, logit_tiles, a.errors);
  return (int)cudaGetLastError();
}

int logit_tiles_of(int32_t max_seqlen) { return (int)(((int64_t)max_seqlen + 63) / 64 * 4); }   // whole tiles of every G

}  // namespace

DenseDecodeLayout dense_decode_layout(int32_t batch, int32_t H, int32_t d, int32_t max_seqlen, bool with_weights) {
  DenseDecodeLayout L{};
  size_t off = kWsHeader;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = align_up(off + bytes, 256);
    return o;
  };
  L.errors = take(sizeof(DevError) * kDecodeCtas);
  L.stats = take(sizeof(float2) * (size_t)batch * H);
  L.part_ml = take(sizeof(float2) * (size_t)kDecodeCtas * 2 * H);
  L.part_o = take(sizeof(float) * (size_t)kDecodeCtas * 2 * H * d);
  L.logits = take(with_weights ? sizeof(float) * (size_t)batch * logit_tiles_of(max_seqlen) * kTileTok * H : 0);
  L.total = off;
  return L;
}

int launch_dense_decode(const DenseDecodeArgs& a, void* stream) {
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return (int)e;
  const int tok = 64 / a.G;
  const int64_t most = (int64_t)a.batch * (((int64_t)a.max_seqlen + tok - 1) / tok);     // tiles, at most
  int ctas = sms < kDecodeCtas ? sms : kDecodeCtas;
  if (most < ctas) ctas = (int)most;

  alignas(64) CUtensorMap tm_k, tm_v;
  // 64 columns (128 bytes) x rows x (group, half): a tile lies in shared memory as one swizzled
  // [tokens x 128 bytes] block per 64 columns
  const uint64_t dims[3] = {64, (uint64_t)a.num_pages * kBk, (uint64_t)(a.G * a.d / 64)};
  const uint64_t strides[2] = {(uint64_t)a.G * a.d * 2, 128};
  const uint32_t box[3] = {64, (uint32_t)tok, (uint32_t)(a.G * a.d / 64)};
  int rc = make_tmap_bf16(&tm_k, a.k_pages, 3, dims, strides, box, 128);
  if (rc == 0) rc = make_tmap_bf16(&tm_v, a.v_pages, 3, dims, strides, box, 128);
  if (rc != 0) return rc;
  const int lt = logit_tiles_of(a.max_seqlen);
  const bool w = a.weights != nullptr;
  const bool few = a.H / a.G <= 8;
#define MSA_SPLIT(DD, W) \
  (few ? launch_split<DD, W, true>(a, ctas, tm_k, tm_v, lt, st) : launch_split<DD, W, false>(a, ctas, tm_k, tm_v, lt, st))
  if (a.d == 128) rc = w ? MSA_SPLIT(128, true) : MSA_SPLIT(128, false);
  else rc = w ? MSA_SPLIT(64, true) : MSA_SPLIT(64, false);
#undef MSA_SPLIT
  if (rc != 0) return rc;

  const int64_t pairs = (int64_t)a.batch * a.H;
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out);
  {
    ProfScope p("dense_join", stream);
    // few sequences lie in many runs each: eight warps to a (b, h), and up to two sequences its columns over 2 or 4
    // CTAs; many lie in few: one warp.  The three forms, in a graph, H 64, G 4, d 128 (a whole call): 2 x 130K tokens
    // 85.6, 85.7 and 93.5 us, 3 x 87K 87.0, 84.2, 90.6, 16 x 16K 103, 88.2, 86.1, 32 x 8K 123, 94.2, 84.6; d 64, H 32:
    // 16 x 16K 48.2, 45.8, 46.9, 32 x 8K 53.0, 48.4, 46.3
#define MSA_JOIN(DD, W, VEC)                                                                                       \
  rc = launch_after(dense_join_kernel<DD, W, VEC>,                                                                 \
                    dim3((unsigned)((pairs + 8 / W - 1) / (8 / W) * (DD / (32 * VEC)))), 256, st, out, a.lse, a.batch,     \
                    a.H, a.G, a.seqlens, a.max_seqlen, a.part_ml, a.part_o, a.stats, ctas, a.errors, a.err)
    if (a.d == 128) {
      if (a.batch <= 2) MSA_JOIN(128, 8, 1); else if (a.batch <= 16) MSA_JOIN(128, 8, 4); else MSA_JOIN(128, 1, 4);
    } else {
      if (a.batch <= 2) MSA_JOIN(64, 8, 1); else if (a.batch <= 16) MSA_JOIN(64, 8, 2); else MSA_JOIN(64, 1, 2);
    }
#undef MSA_JOIN
  }
  if (rc != 0 || !w) return rc;
  ProfScope p("dense_weights", stream);
  const unsigned gx = (unsigned)(((int64_t)a.max_seqlen + kWeightTiles * kTileTok - 1) / (kWeightTiles * kTileTok));
  for (int b0 = 0; b0 < a.batch; b0 += 65535) {   // grid z is 16 bits
    const int nb = a.batch - b0 < 65535 ? a.batch - b0 : 65535;
    rc = launch_after(dense_weights_kernel, dim3(gx, a.G, nb), 256, st,
                      a.logits + (size_t)b0 * lt * kTileTok * a.H, a.stats + (size_t)b0 * a.H,
                      a.weights + (size_t)b0 * a.G * a.max_blocks * kBk, a.H, a.G, a.sm_scale * kLog2e, a.decay,
                      a.seqlens + b0, a.max_seqlen, (int64_t)a.max_blocks * kBk, lt);
    if (rc != 0) return rc;
  }
  return 0;
}

}  // namespace msa
