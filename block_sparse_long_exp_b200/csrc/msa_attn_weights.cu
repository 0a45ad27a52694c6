// The attention weight that the queries of a prompt give every key
// (include/msa.h: msa_attn_weights):
//   w[b, g, j] = decay w[b, g, j] + sum over the queries t that see key j and the
//                group's heads h of exp(sm_scale <q_th, k_j> - lse_th)
//
// The log-sum-exp is an argument, so there is one product per (query, head,
// key), one exponential and one addition, and no running maximum.  2 d operations
// and an exponential per score, 16 of those a clock and SM: the exponentials take
// longer than the tensor cores' part (d = 128: 1024 clocks against 512 per 128 x
// 128 scores), and both far longer than HBM from some eight queries on.  A
// quarter of them therefore goes by a polynomial on the FMA units.  On a B200: 64
// queries over 4 x 9K..32K keys (H 64, d 128; 246M exponentials, 63 GFLOP) 88 us,
// prompts of 3 x 2.5K..4K (H 32, d 64; 537M) 154 us, the exponentials' unit busy
// 55 % and 63 % of the time; 165 us without the polynomial, 150 to 199 with three
// and four pairs of eight by it.
//   layout: the product is K Q^T, keys as the rows of the accumulator and (query,
//           head) pairs as its columns.  A thread then owns one key (a TMEM lane)
//           and sums its scores' exponentials in registers, with no exchange
//           between lanes; the columns' log-sum-exps come from shared memory.
//   unit  : 256 keys x 128 columns (two products of 128 x 128 that share the
//           query tile: half the queries' traffic from L2 of one), two
//           accumulators of each in TMEM so that one is filled while the other is
//           summed.
//   split : the units of all sequences, groups and key blocks, in order (those
//           that no query of the tile sees are left out), are cut into equal runs,
//           one per CTA.  A key block's 256 keys stay in shared memory while its
//           columns stream by.  A block that lies in one run is written at once;
//           of the others each CTA leaves its 256 sums, and weights_join_kernel
//           adds them in the order of the CTAs: the same from run to run.
#include <cuda_runtime.h>

#include <atomic>

#include "msa_common.cuh"
#include "msa_cache.h"
#include "msa_internal.h"

namespace msa {
namespace {

// A lane of TMEM, that is a key, to a thread.  (Sixteen warps with half the columns each: 148 and 92 us instead of 154
// and 88.)
constexpr int kAwSumWarps = 8;
constexpr int kAwThreads = 32 * (4 + kAwSumWarps);
constexpr int kAwKeys = 256;                      // keys of a unit
constexpr int kAwCols = 128;                      // (query, head) columns of a unit
constexpr uint32_t kAwTmem = 512;                 // 2 units x 2 halves of the keys x 128 columns
constexpr float kLog2e = 1.4426950408889634f;

template <int D>
__host__ __device__ constexpr int k_stage() { return kAwKeys * D * 2; }
template <int D>
__host__ __device__ constexpr int q_stage() { return kAwCols * D * 2; }
template <int D>
__host__ __device__ constexpr int num_q() { return D == 128 ? 3 : 8; }

struct AwCtl {
  uint64_t k_full[2], k_empty[2];
  uint64_t q_full[8], q_empty[8];
  uint64_t s_full[2], s_free[2];
  uint64_t mma_done;
  int64_t warp_sum[kAwThreads / 32];
  int64_t total, first_start;
  int32_t first_seq;
  uint32_t tmem_base;
  int32_t abort_flag;
};

// ---- 2^x for pairs of 32-bit numbers ----

__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float clamp_nan(float x, float lo, float hi) {   // NaN stays NaN
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(lo));
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(r), "f"(hi));
  return r;
}
// acc += 2^x without the exponential's unit, by Cody and Waite's reduction: x =
// i + f with i whole and |f| <= 1/2, 2^f a polynomial of degree 5 (its relative
// error is below 2^-22.5 over [-1/2, 1/2], below 2^-22 with the roundings; the unit's
// own is 2^-22), and 2^i a number whose exponent field is i + 127: what x +
// 3 2^22 + 127 has in its low bits.  Below -127 the result is 0, from 127.5 on infinite.
__device__ __forceinline__ uint64_t add_exp2_poly(uint64_t x, uint64_t acc) {
  float a, b;
  unpair(x, a, b);
  x = pair(clamp_nan(a, -127.f, 128.f), clamp_nan(b, -127.f, 128.f));
  const uint64_t magic = pair(12583039.f, 12583039.f), back = pair(-12583039.f, -12583039.f);
  const uint64_t t = add2(x, magic);
  const uint64_t i = add2(t, back);
  const uint64_t f = fma2(i, pair(-1.f, -1.f), x);
  uint64_t p = pair(0.001327647129073739f, 0.001327647129073739f);
  p = fma2(p, f, pair(0.009675540961325169f, 0.009675540961325169f));
  p = fma2(p, f, pair(0.05550713092088699f, 0.05550713092088699f));
  p = fma2(p, f, pair(0.24022120237350464f, 0.24022120237350464f));
  p = fma2(p, f, pair(0.6931469440460205f, 0.6931469440460205f));
  p = fma2(p, f, pair(1.f, 1.f));
  unpair(t, a, b);
  return fma2(p, pair(__uint_as_float(__float_as_uint(a) << 23), __uint_as_float(__float_as_uint(b) << 23)), acc);
}
// Of eight pairs of columns the ones whose exponentials take that way.
constexpr uint32_t kByPolynomial = 0x12;          // 2 of 8
__device__ __forceinline__ uint64_t add_exp2(uint64_t x, uint64_t acc, int at) {   // `at` a constant once unrolled
  if ((kByPolynomial >> at) & 1u) return add_exp2_poly(x, acc);
  float a, b;
  unpair(x, a, b);
  return add2(acc, pair(ex2_approx(a), ex2_approx(b)));
}

// The units of one sequence: T queries that are the last of S tokens, key blocks
// of 256, column tiles of qt queries.  Block i is seen from column tile
// max(0, R i - Pc) on, R = 256 / qt, Pc = ceil((S - T) / qt).
struct SeqUnits {
  int T, S, nkb, nt, R, Pc;
  int64_t per_group;
  __device__ SeqUnits() : T(0), S(0), nkb(0), nt(0), R(1), Pc(0), per_group(0) {}
  __device__ SeqUnits(int T_, int S_, int qt_log) {
    const bool ok = T_ > 0 && T_ <= S_;
    T = ok ? T_ : 0;
    S = ok ? S_ : 0;
    nkb = (S + kAwKeys - 1) / kAwKeys;
    nt = (T + (1 << qt_log) - 1) >> qt_log;
    R = kAwKeys >> qt_log;
    Pc = (S - T + (1 << qt_log) - 1) >> qt_log;
    per_group = before(nkb);
  }
  __device__ int first_tile(int kb) const {
    const int64_t x = (int64_t)R * kb - Pc;
    return x > 0 ? (int)x : 0;
  }
  // units of key blocks 0 .. kb - 1
  __device__ int64_t before(int kb) const {
    const int i0 = Pc / R + 1;                    // the first block with tiles left out
    int64_t n = (int64_t)nt * kb;
    if (kb > i0) {
      const int64_t c = kb - i0;
      n -= R * (c * (i0 + (int64_t)kb - 1) / 2) - (int64_t)Pc * c;
    }
    return n;
  }
};

// The sequences' offsets on the device, and what bounds them: the rows that the
// host names and the rows of the weights.  A sequence that reaches past them is
// reported and has no units: nothing of it is read or written.
struct Seqs {
  const int32_t *cu_q, *cu_k;
  int32_t total_q, total_k, width;                // (a width beyond 32 bits bounds nothing: a length has 31)
  __device__ bool ok(int b) const {
    const int64_t q0 = cu_q[b], q1 = cu_q[b + 1], k0 = cu_k[b], k1 = cu_k[b + 1];
    if (q1 == q0) return k1 >= k0;                // no queries: left as it is
    return q0 >= 0 && q1 > q0 && q1 <= total_q && k0 >= 0 && k1 <= total_k && q1 - q0 <= k1 - k0 && k1 - k0 <= width;
  }
  __device__ SeqUnits units(int b, int qt_log) const {
    return ok(b) ? SeqUnits(cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b], qt_log) : SeqUnits();
  }
};

__device__ __forceinline__ int64_t run_lo(int i, int64_t total, int n) {
  const int64_t q = total / n;
  const int r = (int)(total - q * n);
  return i * q + (i < r ? i : r);
}
__device__ __forceinline__ int run_of(int64_t t, int64_t total, int n) {
  const int64_t q = total / n;
  const int64_t r = total - q * n;
  return (int)(t < r * (q + 1) ? t / (q + 1) : r + (t - r * (q + 1)) / q);
}

// A walk over a run's units.
struct Walk {
  Seqs seqs;
  int qt_log, G, b, g, kb, ct;
  int q0, k0;                                     // first query and key row of the sequence
  int64_t seq_first, kb_first;                    // unit index of the sequence's and the key block's first unit
  SeqUnits u;
  __device__ void load() {
    q0 = seqs.cu_q[b];
    k0 = seqs.cu_k[b];
    u = seqs.units(b, qt_log);
  }
  __device__ void start(const Seqs& of, int qtl, int groups, int seq, int64_t first, int64_t lo) {
    seqs = of; qt_log = qtl; G = groups; b = seq; seq_first = first;
    load();
    int64_t off = lo - first;
    g = (int)(off / u.per_group);
    off -= g * u.per_group;
    int a = 0, z = u.nkb;                         // the last block with before(kb) <= off
    while (z - a > 1) {
      const int m = (a + z) >> 1;
      if (u.before(m) <= off) a = m; else z = m;
    }
    kb = a;
    kb_first = first + g * u.per_group + u.before(kb);
    ct = u.first_tile(kb) + (int)(off - u.before(kb));
  }
  // the next key block (the run has one)
  __device__ void next_block() {
    kb_first += u.nt - u.first_tile(kb);
    if (++kb == u.nkb) {
      kb = 0;
      if (++g == G) {
        g = 0;
        seq_first = kb_first;
        do {
          ++b;
          load();
        } while (u.per_group == 0);
      }
    }
    ct = u.first_tile(kb);
  }
  __device__ int64_t block_end() const { return kb_first + u.nt - u.first_tile(kb); }
};

__device__ __forceinline__ float decayed(float decay, const float* w, float y) {
  return decay == 0.f ? y : fmaf(decay, *w, y);
}

// Where a run ends inside a key block that began in it: what the join needs.
struct __align__(16) AwOpen {
  int32_t b, g, kb, last;                         // last: the CTA of the block's last unit; b < 0: none
};

template <int D>
__global__ void __launch_bounds__(kAwThreads, 1)
attn_weights_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_q,
                    const float* __restrict__ lse, float* __restrict__ weights, int64_t width, float decay, int batch,
                    int H, int G, int qt_log, float scale_log2, const Seqs seqs, AwOpen* __restrict__ open,
                    float* __restrict__ part, DevError* errors) {
  constexpr int NQ = num_q<D>();
  constexpr int KST = k_stage<D>(), QST = q_stage<D>();
  // the swizzled tiles want 1024-byte boundaries; there is no room to round up (this kernel has no other shared memory)
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* k_s = smem;                            // 2 stages of 256 keys
  uint8_t* q_s = k_s + 2 * KST;                   // NQ stages of 128 columns
  float* l_s = reinterpret_cast<float*>(q_s + NQ * QST);
  AwCtl* ctl = reinterpret_cast<AwCtl*>(l_s + 2 * kAwCols);
  volatile int32_t* abort_flag = &ctl->abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int Hg = H / G, hg_log = 7 - qt_log;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the join waits for this grid's end
  DevError* err = errors + blockIdx.x;            // the join makes one word of them
  const bool placed = (smem_u32(smem) & 1023u) == 0;
  if (tid == 0) {
    *err = placed ? DevError{0, 0, 0, 0} : DevError{MSA_ERR_DEVICE_CHECK, kSiteAttnWeights, -1, -1};
    open[blockIdx.x] = AwOpen{-1, 0, 0, 0};       // until the run is known to leave a block open
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_q);
  }
  if (!placed) return;                            // never seen

  // ---- this CTA's run: one scan over the sequences' numbers of units
  {
    const int per = (batch + kAwThreads - 1) / kAwThreads;
    const int b0 = tid * per, b1 = min(b0 + per, batch);
    int64_t sum = 0;
    int bad = -1;
    for (int b = b0; b < b1; ++b) {
      if (!seqs.ok(b)) bad = b;
      sum += G * seqs.units(b, qt_log).per_group;
    }
    int64_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) ctl->warp_sum[warp] = incl;
    if (tid == 0) {
      for (int i = 0; i < 2; ++i) {
        mbar_init(&ctl->k_full[i], 1);
        mbar_init(&ctl->k_empty[i], 1);
        mbar_init(&ctl->s_full[i], 2);            // the products and the columns' log-sum-exps
        mbar_init(&ctl->s_free[i], kAwSumWarps);
      }
      for (int i = 0; i < NQ; ++i) {
        mbar_init(&ctl->q_full[i], 1);
        mbar_init(&ctl->q_empty[i], 1);
      }
      mbar_init(&ctl->mma_done, 1);
      ctl->abort_flag = 0;
      fence_mbar_init();
    }
    __syncthreads();
    if (blockIdx.x == 0 && bad >= 0)
      report_error(err, MSA_ERR_DEVICE_CHECK, kSiteAttnWeights, bad, seqs.cu_q[bad + 1] - seqs.cu_q[bad]);
    int64_t before = 0, total = 0;
    for (int w = 0; w < kAwThreads / 32; ++w) {
      if (w < warp) before += ctl->warp_sum[w];
      total += ctl->warp_sum[w];
    }
    before += incl - sum;
    const int64_t lo = run_lo(blockIdx.x, total, gridDim.x);
    if (lo >= before && lo < before + sum) {      // the run begins in this thread's sequences
      int64_t s = before;
      int b = b0;
      for (;; ++b) {
        const int64_t n = G * seqs.units(b, qt_log).per_group;
        if (lo < s + n) break;
        s += n;
      }
      ctl->first_seq = b;
      ctl->first_start = s;
    }
    if (tid == 0) ctl->total = total;
    __syncthreads();
  }
  const int64_t total = ctl->total;
  const int64_t lo = run_lo(blockIdx.x, total, gridDim.x), hi = run_lo(blockIdx.x + 1, total, gridDim.x);
  if (lo >= hi) return;                           // the whole CTA
  if (warp == 1) {
    tmem_alloc(&ctl->tmem_base, kAwTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;

  if (warp == 0) {
    // -------------------------------------------------------------- loads
    if (lane == 0) {
      Walk w;
      w.start(seqs, qt_log, G, ctl->first_seq, ctl->first_start, lo);
      bool ok = true;
      int nk = 0, nq = 0;                         // key blocks and column tiles loaded
      for (int64_t t = lo; t < hi && ok;) {
        const int ks = nk & 1;
        ok = !*abort_flag && mbar_wait(&ctl->k_empty[ks], ((nk >> 1) + 1) & 1);
        if (!ok) break;
        mbar_arrive_expect_tx(&ctl->k_full[ks], KST);
        for (int h = 0; h < D / 64; ++h)
          tma_load_3d(k_s + ks * KST + h * kAwKeys * 128, &tm_k, &ctl->k_full[ks], 64 * h, w.g, w.k0 + w.kb * kAwKeys);
        ++nk;
        const int64_t e = min(hi, w.block_end());
        for (; t < e; ++t, ++w.ct) {
          const int st = nq % NQ;
          ok = !*abort_flag && mbar_wait(&ctl->q_empty[st], ((nq / NQ) + 1) & 1);
          if (!ok) break;
          mbar_arrive_expect_tx(&ctl->q_full[st], QST);
          for (int h = 0; h < D / 64; ++h)
            tma_load_3d(q_s + st * QST + h * kAwCols * 128, &tm_q, &ctl->q_full[st], 64 * h, w.g * Hg,
                        w.q0 + (w.ct << qt_log));
          ++nq;
        }
        if (t < hi && ok) w.next_block();
      }
      if (!ok) {
        report_error(err, MSA_ERR_TIMEOUT, kSiteAttnWeights, blockIdx.x, -1);
        *abort_flag = 1;
      }
      // no load may remain in flight when the CTA exits
      for (int i = max(0, nk - 2); i < nk; ++i) mbar_wait(&ctl->k_full[i & 1], (i >> 1) & 1);
      for (int i = max(0, nq - NQ); i < nq; ++i) mbar_wait(&ctl->q_full[i % NQ], (i / NQ) & 1);
    }
  } else if (warp == 1) {
    // ----------------------------------------------------------- products
    if (lane == 0) {
      const uint32_t idesc = idesc_bf16_f32(128, kAwCols, 0, 0);
      const uint64_t kd0 = make_sdesc(smem_u32(k_s), 16, 1024, kSw128);
      const uint64_t qd0 = make_sdesc(smem_u32(q_s), 16, 1024, kSw128);
      Walk w;
      w.start(seqs, qt_log, G, ctl->first_seq, ctl->first_start, lo);
      bool ok = true;
      int nk = 0, n = 0;
      for (int64_t t = lo; t < hi && ok;) {
        const int ks = nk & 1;
        ok = !*abort_flag && mbar_wait(&ctl->k_full[ks], (nk >> 1) & 1);
        const int64_t e = min(hi, w.block_end());
        for (; t < e && ok; ++t, ++n) {
          const int st = n % NQ, slot = n & 1;
          ok = !*abort_flag && mbar_wait(&ctl->q_full[st], (n / NQ) & 1) &&
               mbar_wait(&ctl->s_free[slot], ((n >> 1) + 1) & 1);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int half = 0; half < 2; ++half) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint64_t ko = (uint64_t)((ks * KST + (kk >> 2) * (kAwKeys * 128) + half * (128 * 128) + (kk & 3) * 32) >> 4);
              const uint64_t qo = (uint64_t)((st * QST + (kk >> 2) * (kAwCols * 128) + (kk & 3) * 32) >> 4);
              umma_bf16_ss(tmem + slot * 256 + half * 128, kd0 + ko, qd0 + qo, idesc, kk > 0 ? 1u : 0u);
            }
          }
          umma_commit(&ctl->s_full[slot]);
          umma_commit(&ctl->q_empty[st]);
          if (t + 1 == e) umma_commit(&ctl->k_empty[ks]);
        }
        ++nk;
        if (t < hi && ok) w.next_block();
      }
      if (!ok) {
        report_error(err, MSA_ERR_TIMEOUT, kSiteAttnWeights, blockIdx.x, -2);
        *abort_flag = 1;
      }
      umma_commit(&ctl->mma_done);                // the products read shared memory until here
      mbar_wait(&ctl->mma_done, 0);
    }
  } else if (warp == 2) {
    // ----------------------- the columns' log-sum-exps, in units of log2
    Walk w;
    w.start(seqs, qt_log, G, ctl->first_seq, ctl->first_start, lo);
    const int tq = (4 * lane) >> hg_log, h = (4 * lane) & (Hg - 1);   // a lane's four columns share a query
    auto fetch = [&](float4& v) {
      const int q = (w.ct << qt_log) + tq;
      v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (q < w.u.T) v = *reinterpret_cast<const float4*>(lse + (int64_t)(w.q0 + q) * H + w.g * Hg + h);
    };
    bool ok = true;
    int n = 0;
    float4 v;
    fetch(v);
    for (int64_t t = lo; t < hi; ++t, ++n) {
      float4 next = v;
      if (t + 1 < hi) {                           // the next unit's are on their way meanwhile
        if (t + 1 < w.block_end()) ++w.ct; else w.next_block();
        fetch(next);
      }
      const int st = n & 1;
      if (lane == 0) ok = !*abort_flag && mbar_wait(&ctl->s_free[st], ((n >> 1) + 1) & 1);
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      if (!ok) break;
      // (negated; a log-sum-exp of -inf, nothing seen, as +inf: every 2^(s - inf) is 0)
      auto scaled = [](float l) { return l == -INFINITY ? -INFINITY : l * -kLog2e; };
      reinterpret_cast<float4*>(l_s + st * kAwCols)[lane] =
          make_float4(scaled(v.x), scaled(v.y), scaled(v.z), scaled(v.w));
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->s_full[st]);
      v = next;
    }
    if (!ok && lane == 0) {
      report_error(err, MSA_ERR_TIMEOUT, kSiteAttnWeights, blockIdx.x, -3);
      *abort_flag = 1;
    }
  } else if (warp >= 4) {
    // --------------------------------------------------------------- sums
    const int half = (warp - 4) >> 2;
    const int key = half * 128 + 32 * (warp & 3) + lane;             // in the unit
    const uint32_t col0 = tmem + half * 128 + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
    const uint64_t scale2 = pair(scale_log2, scale_log2);
    Walk w;
    w.start(seqs, qt_log, G, ctl->first_seq, ctl->first_start, lo);
    int n = 0;
    bool ok = true;
    for (int64_t t = lo; t < hi && ok;) {
      const int64_t t0 = t, end = w.block_end();
      const int units = (int)(min(hi, end) - t);
      const int j = w.kb * kAwKeys + key;                             // position of this thread's key
      const int first_q = j - (w.u.S - w.u.T);                        // the first query that sees it
      // tiles from here to there count whole for the warp's 32 keys
      const int whole_from = (max(first_q - lane + 31, 0) + (1 << qt_log) - 1) >> qt_log, whole_to = w.u.T >> qt_log;
      float acc = 0.f, comp = 0.f;                                    // compensated: up to millions of terms
      for (int k = 0; k < units; ++k, ++n, ++w.ct) {
        const int slot = n & 1;
        ok = mbar_wait(&ctl->s_full[slot], (n >> 1) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const float* lv = l_s + slot * kAwCols;
        const uint32_t col = col0 + slot * 256;
        uint64_t s0 = 0, s1 = 0;                                      // pairs of 0.f
        if (w.ct >= whole_from && w.ct < whole_to) {
          uint32_t r[2][32];
          tmem_ld32(col, r[0]);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            tmem_ld_wait();
            if (c < 3) tmem_ld32(col + 32 * (c + 1), r[(c + 1) & 1]);  // on its way meanwhile
#pragma unroll
            for (int x = 0; x < 32; x += 4) {
              const uint32_t* v = r[c & 1] + x;
              const float4 l = *reinterpret_cast<const float4*>(lv + 32 * c + x);
              const uint64_t a = fma2(pair(__uint_as_float(v[0]), __uint_as_float(v[1])), scale2, pair(l.x, l.y));
              const uint64_t b = fma2(pair(__uint_as_float(v[2]), __uint_as_float(v[3])), scale2, pair(l.z, l.w));
              s0 = add_exp2(a, s0, x / 2 % 8);
              s1 = add_exp2(b, s1, x / 2 % 8 + 1);
            }
          }
        } else {
          // columns [xlo, xhi) count for this key; what the others hold does not
          const int q0 = w.ct << qt_log;
          const int xlo = first_q > q0 ? min(first_q - q0, 128) << hg_log : 0;
          const int xhi = min((w.u.T - q0) << hg_log, kAwCols);
          const int none = __shfl_sync(0xffffffffu, xlo, 0);          // the warp's first key sees the most
#pragma unroll 1
          for (int c = none & ~31; c < xhi; c += 32) {
            uint32_t r[32];
            tmem_ld32(col + c, r);
            tmem_ld_wait();
#pragma unroll
            for (int x = 0; x < 32; x += 2) {
              const float p = ex2_approx(fmaf(__uint_as_float(r[x]), scale_log2, lv[c + x]));
              const float q = ex2_approx(fmaf(__uint_as_float(r[x + 1]), scale_log2, lv[c + x + 1]));
              s0 = add2(s0, pair(c + x >= xlo && c + x < xhi ? p : 0.f, c + x + 1 >= xlo && c + x + 1 < xhi ? q : 0.f));
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->s_free[slot]);
        float s[4];
        unpair(s0, s[0], s[1]);
        unpair(s1, s[2], s[3]);
        const float y = ((s[0] + s[1]) + (s[2] + s[3])) - comp, z = acc + y;
        comp = fabsf(z) <= 3.402823466e38f ? (z - acc) - y : 0.f;     // (past the largest number: inf, and no inf - inf)
        acc = z;
      }
      if (!ok) break;
      t += units;
      // whole blocks' sums are written, others left for the join
      if (t0 == w.kb_first && t == end) {
        if (j < w.u.S) {
          float* dst = weights + ((int64_t)w.b * G + w.g) * width + j;
          *dst = decayed(decay, dst, acc);
        }
      } else {
        part[((int64_t)blockIdx.x * 2 + (t0 == w.kb_first ? 1 : 0)) * kAwKeys + key] = acc;
      }
      if (t0 == w.kb_first && t < end && warp == 4 && lane == 0)
        open[blockIdx.x] = AwOpen{w.b, w.g, w.kb, run_of(end - 1, total, gridDim.x)};
      if (t < hi) w.next_block();
    }
    if (!ok && lane == 0) {
      report_error(err, MSA_ERR_TIMEOUT, kSiteAttnWeights, blockIdx.x, warp);
      *abort_flag = 1;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kAwTmem);
  }
}

// Adds the parts of the key block that begins in run i and ends in another, and
// makes one error word of the CTAs'.  (What the kernel ahead writes is read through
// pointers without __restrict__: const ones with it may be read before the wait.)
__global__ void __launch_bounds__(kAwKeys)
weights_join_kernel(const AwOpen* open, const float* part, float* __restrict__ weights, int64_t width, float decay, int G,
                    const int32_t* __restrict__ cu_k, const DevError* errors, DevError* err) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (blockIdx.x == 0 && threadIdx.x < 32) {      // the first CTA's that found something
    int first = gridDim.x;
    for (int i = threadIdx.x; i < gridDim.x; i += 32)
      if (errors[i].code != 0) first = min(first, i);
    first = __reduce_min_sync(0xffffffffu, first);
    if (threadIdx.x == 0) *err = first < gridDim.x ? errors[first] : DevError{0, 0, 0, 0};
  }
  const AwOpen o = open[blockIdx.x];
  if (o.b < 0) return;
  const int j = o.kb * kAwKeys + threadIdx.x;
  if (j >= cu_k[o.b + 1] - cu_k[o.b]) return;
  float acc = part[((int64_t)blockIdx.x * 2 + 1) * kAwKeys + threadIdx.x];
#pragma unroll 4
  for (int i = blockIdx.x + 1; i <= o.last; ++i) acc += part[(int64_t)i * 2 * kAwKeys + threadIdx.x];
  float* dst = weights + ((int64_t)o.b * G + o.g) * width + j;
  *dst = decayed(decay, dst, acc);
}

template <int D>
int launch_units(const AttnWeightsArgs& a, int ctas, cudaStream_t st) {
  CUtensorMap tm_k, tm_q;
  const int hg = a.H / a.G, hg_log = hg == 16 ? 4 : (hg == 8 ? 3 : 2), qt_log = 7 - hg_log;
  {
    const uint64_t dims[3] = {(uint64_t)D, (uint64_t)a.G, (uint64_t)a.total_k};
    const uint64_t strides[2] = {(uint64_t)D * 2, (uint64_t)a.G * D * 2};
    const uint32_t box[3] = {64, 1, kAwKeys};
    const int rc = make_tmap_bf16(&tm_k, a.k, 3, dims, strides, box, 128);
    if (rc != 0) return rc;
  }
  {
    const uint64_t dims[3] = {(uint64_t)D, (uint64_t)a.H, (uint64_t)a.total_q};
    const uint64_t strides[2] = {(uint64_t)D * 2, (uint64_t)a.H * D * 2};
    const uint32_t box[3] = {64, (uint32_t)hg, 1u << qt_log};
    const int rc = make_tmap_bf16(&tm_q, a.q, 3, dims, strides, box, 128);
    if (rc != 0) return rc;
  }
  constexpr int smem = 2 * k_stage<D>() + num_q<D>() * q_stage<D>() + 2 * kAwCols * 4 + (int)sizeof(AwCtl);
  static_assert(smem <= 232448, "shared memory of one CTA");
  static_assert(num_q<D>() <= 8, "barriers of the query stages");
  static std::atomic<uint64_t> ready{0};
  const int rc = allow_smem(attn_weights_kernel<D>, smem, &ready);
  if (rc != 0) return rc;
  const Seqs seqs{a.cu_q, a.cu_k, (int32_t)a.total_q, (int32_t)a.total_k,
                  (int32_t)(a.width < INT32_MAX ? a.width : INT32_MAX)};
  ProfScope p("attn_weights", st);
  attn_weights_kernel<D><<<ctas, kAwThreads, smem, st>>>(
      tm_k, tm_q, a.lse, a.weights, a.width, a.decay, a.batch, a.H, a.G, qt_log, a.sm_scale * kLog2e, seqs,
      static_cast<AwOpen*>(a.open), a.part, a.errors);
  return (int)cudaGetLastError();
}

}  // namespace

AttnWeightsLayout attn_weights_layout() {
  AttnWeightsLayout L{};
  L.errors = kWsHeader;
  L.open = align_up(L.errors + sizeof(DevError) * kDecodeCtas, 256);
  L.part = align_up(L.open + sizeof(AwOpen) * kDecodeCtas, 256);
  L.total = align_up(L.part + sizeof(float) * (size_t)kDecodeCtas * 2 * kAwKeys, 256);
  return L;
}

int launch_attn_weights(const AttnWeightsArgs& a, void* stream) {
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return (int)e;
  const int ctas = sms < kDecodeCtas ? sms : kDecodeCtas;
  const int rc = a.d == 128 ? launch_units<128>(a, ctas, st) : launch_units<64>(a, ctas, st);
  if (rc != 0) return rc;
  ProfScope p("attn_weights_join", st);
  return launch_after(weights_join_kernel, dim3(ctas), kAwKeys, st, static_cast<const AwOpen*>(a.open), a.part,
                      a.weights, a.width, a.decay, a.G, a.cu_k, a.errors, a.err);
}

}  // namespace msa
