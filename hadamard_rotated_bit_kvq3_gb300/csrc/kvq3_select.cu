// Page scores of a decode step and the selection of pages by them.
//
// Scores.  For kv head h of sequence b and page i with key bounds lo, hi,
//   score = max over the G query heads of  sum_j max(q1_j lo_j, q1_j hi_j),
// q1 = U q.  With q1 = q+ + q- (positive and negative part) the sum is
// q- . lo + q+ . hi: a product of the page's 2d fp16 bounds with a vector of
// length 2d, so a tile of 16 pages against the heads is a chain of
// mma.sync m16n8k16 with the bounds as they lie in memory as the A operand
// (each lane loads 16 consecutive bytes of a page's row; the columns of K are
// taken in that order on both sides) and the query parts as B, split into
// hi + lo fp16 halves (two columns per head), so the scores carry about fp32
// accuracy.  Bound by HBM: 4d bytes per (page, kv head) for 4 d G flops.  Each
// row's registers are refilled as they are used, so 8 KB a warp stay in
// flight.  64 sequences of up to 64K tokens, 4 kv heads of 256, 16-token pages
// (549 MB of bounds): 94 us, 5.8 TB/s, 86 % of the measured copy rate (123 us
// with a CTA per tile, loading, then computing; 99 with the bounds through the
// read-only path).  With 8 and 16 heads per kv
// head 97 and 113 us; at d = 128 and 64 with 8 heads 52 and 40 us for half and
// a quarter of the bytes (78 and 52 % of the copy rate).  16 sequences of 32K, 8
// kv heads of 128, 128-token pages (17 MB): 5.9 us, latency.
//
// Selection.  One CTA per (sequence, kv head): the scores as order-preserving
// 32-bit keys (in registers up to 8,192 pages), a histogram search for the
// budget-th largest between the forced first and last pages, and one ordered
// compaction by ballots that breaks ties towards the lower page.  Bound by
// latency, a few block barriers of a row of a few thousand keys; no sort.  256
// rows of up to 4,096 pages, 256 of them chosen: 7.3 us (14.4 with three radix
// passes over keys in shared memory, 11.8 with the keys in registers); 128 rows
// of 256 pages: 3.5 us.  Rows of more than 8,192 pages read their scores again
// in every pass: 25.8 us for 16,384 pages, 112 for 65,536.
//
// Inputs are read with coherent loads (no __restrict__ on them): a kernel
// launched as a programmatic dependent is alive while the one before it still
// writes what it will read.
#include <math.h>

#include "kvq3_internal.h"

using namespace kvq3;

namespace {

constexpr int kScoreWarps = 8;
constexpr int kScoreRounds = 4;

// D: head dimension; NT: n-tiles of 4 heads x (hi, lo) columns.  A CTA takes
// `span` consecutive tiles of 128 pages of one unit, a warp 16 of each.
template <int D, int NT>
__global__ void __launch_bounds__(32 * kScoreWarps, 2)
    page_scores_kernel(const __grid_constant__ RotParams rp, const __grid_constant__ CacheGeom g,
                       const int32_t* page_table, const int32_t* seq_lens,
                       const __half* bounds, const __half* q, int G, int groups, int span,
                       float* __restrict__ scores, int32_t* status, float inv_sqrt_d) {
  constexpr int K = 2 * D;
  constexpr int ROW = K + 32;                // halves per B column in shared memory: 64 bytes of padding, no conflicts
  constexpr int E = D >= 128 ? D / 32 : 4;
  constexpr int L = D / E;
  constexpr int GPW = 32 / L;
  constexpr int CH = D / 32;                 // 16-byte loads per lane and row of one bound
  constexpr int TP = 16 * kScoreWarps;       // pages of a tile
  __shared__ __align__(16) __half qb[NT * 8 * ROW];
  __shared__ float qinv[NT * 4];             // 2^-e of each head, 0 past the last
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int j = lane & 3, r = lane >> 2;
  griddep_wait();
  griddep_launch_dependents();
  const int64_t unit = blockIdx.x / groups;
  const int64_t first = (int64_t)(blockIdx.x - unit * groups) * span * TP;
  const int b = (int)(unit / g.hkv), kvh = (int)(unit - (int64_t)b * g.hkv);
  const int64_t len = seq_lens[b];
  const bool len_ok = len >= 0 && len <= (int64_t)g.max_pages * g.page_size;
  if (!len_ok && threadIdx.x == 0) set_status(status, KVQ3_DEV_BAD_LEN);
  const int64_t n = len_ok ? (len + g.page_size - 1) / g.page_size : 0;
  float* row_out = scores + unit * g.max_pages;
  const int64_t end = min(first + (int64_t)span * TP, (int64_t)g.max_pages);   // the CTA's pages [first, end)
  for (int64_t i = max(first, n) + threadIdx.x; i < end; i += 32 * kScoreWarps) row_out[i] = -INFINITY;
  if (first >= n) return;

  // rows r and r + 8 of this warp's 16 pages of a tile
  const uint4 zero = make_uint4(0, 0, 0, 0);
  auto page_at = [&](int64_t lp) {
    const int64_t p = lp < n ? page_of(g, page_table, b, lp) : -1;
    if (lp < n && p < 0 && j == 0) set_status(status, KVQ3_DEV_BAD_PAGE);
    if (p >= 0 && !KVQ3_CHECK(status, in_range((p * g.hkv + kvh) * K, K, g.num_pages * g.hkv * K))) return (int64_t)-1;
    return p;
  };
  auto row_of = [&](int64_t page) {
    return reinterpret_cast<const uint4*>(bounds + (page < 0 ? 0 : ((page * g.hkv + kvh) * 2) * D)) + j;
  };
  int64_t p0 = first + wid * 16 + r;
  int64_t page[2] = {page_at(p0), page_at(p0 + 8)};
  // the first bound's rows are on their way while the query is rotated; from
  // then on each row's registers are refilled as they are used: the second
  // bound's rows, then the next tile's first
  uint4 a[2][CH];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const uint4* src = row_of(page[e]);
#pragma unroll
    for (int c = 0; c < CH; ++c) a[e][c] = page[e] >= 0 ? src[4 * c] : zero;
  }

  // q1 of the G heads, its negative part against lo and its positive part
  // against hi, scaled by a power of two into [2^7, 2^8) and split hi + lo
  {
    const int rq = lane % L, gq = lane / L;
    const uint32_t sgn = lane_signs<E>(rp, rq);
    for (int g0 = wid * GPW; g0 < NT * 4; g0 += kScoreWarps * GPW) {
      const int gg = g0 + gq;
      float x[E];
      const bool valid = gg < G;
      const __half* qs = q + ((unit * G) + (valid ? gg : 0)) * D + rq * E;
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] = valid ? __half2float(qs[e]) : 0.0f;
      float4 quat[E / 4], quat_r[E / 4];
      lane_quats<E>(rp, rq, quat);
      lane_quats_r<E>(rp, rq, quat_r);
      rotate_forward<E, L>(x, rq, sgn, quat, quat_r, inv_sqrt_d, rot_so4(rp), rot_pair(rp));
      float amax = 0.0f;
#pragma unroll
      for (int e = 0; e < E; ++e) amax = fmaxf(amax, fabsf(x[e]));
#pragma unroll
      for (int o = 1; o < L; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
      int ex = 0;
      if (amax > 0.0f) frexpf(amax, &ex);
      ex = max(-100, min(100, 8 - ex));
      const float sc = ldexpf(1.0f, ex);
      if (gg < NT * 4) {
        __half* hi = qb + (2 * gg) * ROW;
        __half* lo = hi + ROW;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float v = x[e] * sc;
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const float part = s == 0 ? fminf(v, 0.0f) : fmaxf(v, 0.0f);
            const __half h = __float2half_rn(part);
            hi[s * D + rq * E + e] = h;
            lo[s * D + rq * E + e] = __float2half_rn(part - __half2float(h));
          }
        }
        if (rq == 0) qinv[gg] = valid ? ldexpf(1.0f, -ex) : 0.0f;
      }
    }
  }
  __syncthreads();

  for (int it = 0; it < span && first + (int64_t)it * TP < n; ++it) {
    const int64_t p1 = p0 + TP;
    int64_t next[2] = {-1, -1};
    if (it + 1 < span) {
      next[0] = page_at(p1);
      next[1] = page_at(p1 + 8);
    }
    // chains of 8 products at most: a longer one in the tensor core's
    // accumulator rounds every step to its running sum (1.5e-6 of the score at
    // 32 steps), so each chain is added to the total in fp32
    float sum[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t) sum[t][0] = sum[t][1] = sum[t][2] = sum[t][3] = 0.0f;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const uint4* src[2] = {s == 0 ? row_of(page[0]) + D / 8 : row_of(next[0]),
                             s == 0 ? row_of(page[1]) + D / 8 : row_of(next[1])};
      const bool there[2] = {(s == 0 ? page[0] : next[0]) >= 0, (s == 0 ? page[1] : next[1]) >= 0};
#pragma unroll
      for (int c0 = 0; c0 < CH; c0 += 4) {
        float acc[NT][4];
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[t][0] = acc[t][1] = acc[t][2] = acc[t][3] = 0.0f;
#pragma unroll
        for (int c = c0; c < c0 + 4 && c < CH; ++c) {
          const uint4 x = a[0][c], y = a[1][c];
          a[0][c] = there[0] ? src[0][4 * c] : zero;
          a[1][c] = there[1] ? src[1][4 * c] : zero;
          const uint32_t f0[4] = {x.x, y.x, x.y, y.y}, f1[4] = {x.z, y.z, x.w, y.w};
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const uint4 w = *reinterpret_cast<const uint4*>(qb + (8 * t + r) * ROW + s * D + 32 * c + 8 * j);
            mma_16816(acc[t], f0, w.x, w.y);
            mma_16816(acc[t], f1, w.z, w.w);
          }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) sum[t][i] += acc[t][i];
      }
    }
    float best0 = -INFINITY, best1 = -INFINITY;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const float f = qinv[4 * t + j];
      if (4 * t + j < G) {
        // an infinite bound meets a zero query part (0 times infinity): a sum
        // that is no number counts as +infinity, so that its page is attended
        const float s0 = (sum[t][0] + sum[t][1]) * f, s1 = (sum[t][2] + sum[t][3]) * f;
        best0 = fmaxf(best0, s0 == s0 ? s0 : INFINITY);
        best1 = fmaxf(best1, s1 == s1 ? s1 : INFINITY);
      }
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      best0 = fmaxf(best0, __shfl_xor_sync(kFull, best0, o));
      best1 = fmaxf(best1, __shfl_xor_sync(kFull, best1, o));
    }
    if (j < 2) {
      const int64_t i = p0 + 8 * j;
      if (i < n) row_out[i] = (j ? page[1] : page[0]) >= 0 ? (j ? best1 : best0) : -INFINITY;
    }
    p0 = p1;
    page[0] = next[0];
    page[1] = next[1];
  }
}

template <int D, int NT>
cudaError_t launch_scores(const RotParams& rp, const CacheGeom& g, const kvq3_cache* c, const __half* bounds,
                          const __half* q, int G, float* scores, int32_t* st, cudaStream_t stream) {
  // tiles a CTA takes: up to 8 while that leaves kScoreRounds CTAs for each
  // resident one (the query is rotated once a CTA)
  const int64_t tiles = ((int64_t)g.max_pages + 16 * kScoreWarps - 1) / (16 * kScoreWarps);
  const int64_t units = (int64_t)g.batch * g.hkv;
  int span = 1;
  while (span < 8 && units * ((tiles + 2 * span - 1) / (2 * span)) >= (int64_t)kScoreRounds * 2 * sm_count()) span *= 2;
  const int groups = (int)((tiles + span - 1) / span);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * groups));
  cfg.blockDim = dim3(32 * kScoreWarps);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, page_scores_kernel<D, NT>, rp, g, c->page_table, c->seq_lens, bounds, q, G, groups,
                            span, scores, st, inv_sqrt(D));
}

template <int D>
cudaError_t scores_by_heads(const RotParams& rp, const CacheGeom& g, const kvq3_cache* c, const __half* bounds,
                            const __half* q, int G, float* scores, int32_t* st, cudaStream_t stream) {
  if (G <= 4) return launch_scores<D, 1>(rp, g, c, bounds, q, G, scores, st, stream);
  if (G <= 8) return launch_scores<D, 2>(rp, g, c, bounds, q, G, scores, st, stream);
  return launch_scores<D, 4>(rp, g, c, bounds, q, G, scores, st, stream);
}

// ------------------------------------------------------------ selection
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kBinBits = 11;

// The histogram, read four bins at a time.
struct __align__(16) Bins {
  uint32_t n[kBins];
};

// Order-preserving key: larger score, larger key; NaN lowest, -0 as +0.
__device__ __forceinline__ uint32_t score_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.0f);   // -0 + 0 = +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Keys of a row's competing pages, page i = k kSelThreads + thread in round k:
// in registers for rows of up to KPT rounds (the kernel's template), read
// again from memory each time for longer ones (KPT = 0).
template <int KPT>
__global__ void __launch_bounds__(kSelThreads)
    page_select_kernel(const __grid_constant__ CacheGeom g, const int32_t* seq_lens,
                       const float* scores, int budget, int sinks, int recent, int32_t* __restrict__ pages,
                       int32_t* __restrict__ counts, int32_t* status) {
  __shared__ Bins hist;
  __shared__ uint32_t wsum[kSelWarps];
  __shared__ uint2 range_s[kSelWarps];   // smallest and largest key of each warp
  __shared__ uint4 found;                // bin, places left in it, its keys
  __shared__ uint32_t n_cand;
  __shared__ unsigned long long cand[32];
  __shared__ uint2 wcount[(KPT > 0 ? KPT : 1) * kSelWarps];   // larger and equal keys of each warp and round
  const int t = threadIdx.x, lane = t & 31, wid = t >> 5;
  for (int i = t; i < kBins; i += kSelThreads) hist.n[i] = 0;
  griddep_wait();
  griddep_launch_dependents();
  const int64_t unit = blockIdx.x;
  const int b = (int)(unit / g.hkv);
  const float* row = scores + unit * g.max_pages + sinks;
  const int64_t len = seq_lens[b];
  // the scores do not wait for the length: every page of the row can be read
  float raw[KPT > 0 ? KPT : 1];
  if constexpr (KPT > 0) {
#pragma unroll
    for (int k = 0; k < KPT; ++k) {
      const int i = k * kSelThreads + t;
      raw[k] = i < g.max_pages - sinks ? row[i] : 0.0f;
    }
  }
  const bool len_ok = len >= 0 && len <= (int64_t)g.max_pages * g.page_size;
  if (!len_ok && t == 0) set_status(status, KVQ3_DEV_BAD_LEN);
  const int n = len_ok ? (int)((len + g.page_size - 1) / g.page_size) : 0;
  int32_t* out = pages + unit * budget;
  if (t == 0) counts[unit] = min(n, budget);
  if (n <= budget) {
    for (int i = t; i < budget; i += kSelThreads) out[i] = i < n ? i : -1;
    return;
  }
  // pages [sinks, n - recent) compete for `want` places; 0 <= want < m
  const int m = n - sinks - recent, want = budget - sinks - recent;
  for (int i = t; i < sinks; i += kSelThreads) out[i] = i;
  for (int i = t; i < recent; i += kSelThreads) out[budget - recent + i] = n - recent + i;
  if (want == 0) return;
  const int rounds = (m + kSelThreads - 1) / kSelThreads;   // <= KPT where KPT > 0
  uint32_t key[KPT > 0 ? KPT : 1];
  if constexpr (KPT > 0) {
#pragma unroll
    for (int k = 0; k < KPT; ++k) key[k] = score_key(raw[k]);
  }
  // f(key, page, round) for this thread's pages
  auto each = [&](auto f) {
    if constexpr (KPT > 0) {
#pragma unroll
      for (int k = 0; k < KPT; ++k) {
        const int i = k * kSelThreads + t;
        if (i < m) f(key[k], i, k);
      }
    } else {
      for (int i = t; i < m; i += kSelThreads) f(score_key(row[i]), i, 0);
    }
  };

  // The want-th largest key, by a histogram over the range that holds it: the
  // keys of a row differ in few of their top bits, so the first bins divide
  // [smallest, largest] instead of all 32-bit keys (and are not a handful of
  // contended counters).  Each pass narrows the range to one bin of the last;
  // it ends when the bin is taken whole, when 32 keys or fewer are left (one
  // warp ranks them by key, then page), or when they are all equal.
  uint32_t kmin = 0xffffffffu, kmax = 0;
  each([&](uint32_t k, int, int) {
    kmin = min(kmin, k);
    kmax = max(kmax, k);
  });
  kmin = __reduce_min_sync(kFull, kmin);
  kmax = __reduce_max_sync(kFull, kmax);
  if (lane == 0) range_s[wid] = make_uint2(kmin, kmax);
  if (t == 0) n_cand = 0;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kSelWarps; ++w) {
    const uint2 v = range_s[w];
    kmin = min(kmin, v.x);
    kmax = max(kmax, v.y);
  }
  uint32_t base = kmin, span = kmax - kmin;       // the keys [base, base + span] hold the one looked for
  uint32_t left = (uint32_t)want;                 // its rank among them
  uint32_t low = 0, at = 0xffffffffu, equal = 0;  // in: keys above low; at low, pages up to `at` (or the first `equal`)
  bool whole = false;                             // in: keys from low on
#pragma unroll 1
  for (int pass = 0;; ++pass) {
    const int shift = max(0, 32 - __clz((int)span) - kBinBits);   // span >> shift < kBins
    if (pass > 0)
      for (int i = t; i < kBins; i += kSelThreads) hist.n[i] = 0;
    __syncthreads();
    each([&](uint32_t k, int, int) {
      if (k - base <= span) atomicAdd(&hist.n[(k - base) >> shift], 1u);
    });
    __syncthreads();
    // from the top, four bins a thread: the bin that holds the left-th
    constexpr int PER = kBins / kSelThreads;
    static_assert(PER == 4 && alignof(Bins) % alignof(uint4) == 0, "a thread's bins are one 16-byte load");
    const uint4 h4 = *reinterpret_cast<const uint4*>(&hist.n[kBins - PER * (t + 1)]);   // bins ascending
    const uint32_t h[PER] = {h4.w, h4.z, h4.y, h4.x};
    const uint32_t mine = h[0] + h[1] + h[2] + h[3];
    uint32_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) wsum[wid] = incl;
    __syncthreads();
    uint32_t above = incl - mine;
#pragma unroll
    for (int w = 0; w < kSelWarps; ++w) above += w < wid ? wsum[w] : 0u;
    if (above < left && left <= above + mine) {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        if (above < left && left <= above + h[i])
          found = make_uint4((uint32_t)(kBins - 1 - PER * t - i), left - above, h[i], 0);
        above += h[i];
      }
    }
    __syncthreads();
    const uint4 f = found;
    base += f.x << shift;
    span = (shift ? (1u << shift) : 1u) - 1u;   // may reach past the last pass's range, where no key is
    left = f.y;
    low = base;
    if (f.y == f.z) {
      whole = true;
      break;
    }
    if (span == 0) {
      equal = left;
      break;
    }
    if (f.z <= 32) {
      each([&](uint32_t k, int i, int) {
        if (k - base <= span) cand[atomicAdd(&n_cand, 1u)] = ((unsigned long long)k << 32) | (0xffffffffu - (uint32_t)i);
      });
      __syncthreads();
      // every warp ranks the candidates: larger key first, lower page first
      const unsigned long long c = lane < f.z ? cand[lane] : 0ull;
      uint32_t rank = 0;
#pragma unroll
      for (int o = 0; o < 32; ++o) rank += __shfl_sync(kFull, c, o) > c;
      const int src = __ffs(__ballot_sync(kFull, lane < f.z && rank == left - 1u)) - 1;
      const unsigned long long last = __shfl_sync(kFull, c, src);
      low = (uint32_t)(last >> 32);
      at = 0xffffffffu - (uint32_t)last;
      break;
    }
  }

  // in page order: keys above `low`, and at it the pages up to `at` or the
  // first `equal` of them (a bin taken whole: every key from `low` on)
  const bool by_page = !whole && equal == 0;
  auto larger = [&](uint32_t k, int i) {
    return whole ? k >= low : k > low || (by_page && k == low && (uint32_t)i <= at);
  };
  auto same = [&](uint32_t k) { return equal != 0 && k == low; };
  const uint32_t below = (1u << lane) - 1u;
  if constexpr (KPT > 0) {
    uint32_t gt[KPT], eq[KPT];
#pragma unroll
    for (int k = 0; k < KPT; ++k) {
      const bool in = k * kSelThreads + t < m;
      gt[k] = __ballot_sync(kFull, in && larger(key[k], k * kSelThreads + t));
      eq[k] = __ballot_sync(kFull, in && same(key[k]));
      if (lane == 0) wcount[k * kSelWarps + wid] = make_uint2(__popc(gt[k]), __popc(eq[k]));
    }
    __syncthreads();
    if (wid == 0) {   // exclusive sums over (round, warp)
      uint2 base = make_uint2(0, 0);
      for (int i0 = 0; i0 < KPT * kSelWarps; i0 += 32) {
        const uint2 c = i0 + lane < KPT * kSelWarps ? wcount[i0 + lane] : make_uint2(0, 0);
        uint2 s = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t x = __shfl_up_sync(kFull, s.x, o), y = __shfl_up_sync(kFull, s.y, o);
          if (lane >= o) {
            s.x += x;
            s.y += y;
          }
        }
        if (i0 + lane < KPT * kSelWarps) wcount[i0 + lane] = make_uint2(base.x + s.x - c.x, base.y + s.y - c.y);
        base.x += __shfl_sync(kFull, s.x, 31);
        base.y += __shfl_sync(kFull, s.y, 31);
      }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < KPT; ++k) {
      const uint2 c = wcount[k * kSelWarps + wid];
      const uint32_t g0 = c.x + __popc(gt[k] & below), e0 = c.y + __popc(eq[k] & below);
      const bool is_gt = (gt[k] >> lane) & 1u, is_eq = (eq[k] >> lane) & 1u;
      if (is_gt || (is_eq && e0 < equal)) out[sinks + g0 + min(e0, equal)] = sinks + k * kSelThreads + t;
    }
  } else {
    uint32_t g_all = 0, e_all = 0;   // before this round
    for (int k = 0; k < rounds; ++k) {
      const int i = k * kSelThreads + t;
      const uint32_t kk = i < m ? score_key(row[i]) : 0u;
      const uint32_t gt = __ballot_sync(kFull, i < m && larger(kk, i)), eq = __ballot_sync(kFull, i < m && same(kk));
      __syncthreads();
      if (lane == 0) wcount[wid] = make_uint2(__popc(gt), __popc(eq));
      __syncthreads();
      uint32_t g0 = g_all + __popc(gt & below), e0 = e_all + __popc(eq & below);
#pragma unroll
      for (int w = 0; w < kSelWarps; ++w) {
        const uint2 c = wcount[w];
        g0 += w < wid ? c.x : 0u;
        e0 += w < wid ? c.y : 0u;
        g_all += c.x;
        e_all += c.y;
      }
      const bool is_gt = (gt >> lane) & 1u, is_eq = (eq >> lane) & 1u;
      if (is_gt || (is_eq && e0 < equal)) out[sinks + g0 + min(e0, equal)] = sinks + i;
    }
  }
}

}  // namespace

extern "C" {

kvq3_status kvq3_page_scores(kvq3_rotation rot, const kvq3_cache_desc* desc, const kvq3_cache* cache,
                             const void* bounds, const void* q, int32_t num_q_heads, float* scores,
                             int32_t* dev_status, void* stream) {
  CacheGeom g;
  kvq3_status s = make_geom(desc, &g);
  if (s != KVQ3_OK) return s;
  if (!rot || rot->d != g.d || !q || !bounds || !scores) return KVQ3_ERR_INVALID_ARG;
  if ((s = check_cache(g, cache, true)) != KVQ3_OK) return s;
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(bounds)) % 16 != 0 ||
      reinterpret_cast<uintptr_t>(scores) % 4 != 0)
    return KVQ3_ERR_INVALID_ARG;
  if (num_q_heads < 1 || num_q_heads % g.hkv != 0) return KVQ3_ERR_INVALID_ARG;
  const int G = num_q_heads / g.hkv;
  if (G > 16) return KVQ3_ERR_UNSUPPORTED;
  const int64_t tiles = ((int64_t)g.max_pages + 16 * kScoreWarps - 1) / (16 * kScoreWarps);
  if ((int64_t)g.batch * g.hkv >= ((int64_t)1 << 31) / tiles) return KVQ3_ERR_UNSUPPORTED;   // one CTA per tile
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const __half* bh = static_cast<const __half*>(bounds);
  const __half* qh = static_cast<const __half*>(q);
  cudaError_t e;
  switch (g.d) {
    case 64: e = scores_by_heads<64>(rot->params, g, cache, bh, qh, G, scores, dev_status, st); break;
    case 128: e = scores_by_heads<128>(rot->params, g, cache, bh, qh, G, scores, dev_status, st); break;
    case 256: e = scores_by_heads<256>(rot->params, g, cache, bh, qh, G, scores, dev_status, st); break;
    default: return KVQ3_ERR_UNSUPPORTED;
  }
  return cuda_status(e);
}

kvq3_status kvq3_page_select(const kvq3_cache_desc* desc, const kvq3_cache* cache, const float* scores,
                             int32_t budget, int32_t sinks, int32_t recent, int32_t* pages, int32_t* counts,
                             int32_t* dev_status, void* stream) {
  CacheGeom g;
  kvq3_status s = make_geom(desc, &g);
  if (s != KVQ3_OK) return s;
  if (!cache || !cache->seq_lens || !scores || !pages || !counts) return KVQ3_ERR_INVALID_ARG;
  if (budget < 1 || sinks < 0 || recent < 1 || (int64_t)sinks + recent > budget) return KVQ3_ERR_INVALID_ARG;
  if ((int64_t)g.batch * g.hkv >= ((int64_t)1 << 31)) return KVQ3_ERR_UNSUPPORTED;   // one CTA per row
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((int64_t)g.batch * g.hkv));
  cfg.blockDim = dim3(kSelThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // the rounds that the longest row can take
  auto run = [&](auto kernel) {
    return cuda_status(cudaLaunchKernelEx(&cfg, kernel, g, cache->seq_lens, scores, budget, sinks, recent, pages, counts,
                                          dev_status));
  };
  // Measured for 128 rows (us): a kernel with more rounds than the row needs
  // pays 0.1 to 0.2 a round (512 pages: 1, 2, 3, 4, 8 rounds 3.5, 3.7, 3.9,
  // 4.0, 4.8), so that 2 or 4 rounds of their own would gain 0.1 and 0.7 at
  // most (2,048 pages: 4, 6, 8 rounds 4.4, 4.7, 5.0), 12 another 0.9 (6,144
  // pages: 6.4, and 7.2 with 16); reading again costs 6.7 for 2,048 pages, 9.5
  // for 4,096, 15.0 for 8,192 (7.6 with 16 rounds).
  const int64_t most = (int64_t)g.max_pages - sinks - recent;
  if (most <= kSelThreads) return run(page_select_kernel<1>);
  if (most <= 3 * kSelThreads) return run(page_select_kernel<3>);
  if (most <= 8 * kSelThreads) return run(page_select_kernel<8>);
  if (most <= 16 * kSelThreads) return run(page_select_kernel<16>);
  return run(page_select_kernel<0>);
}

}  // extern "C"
