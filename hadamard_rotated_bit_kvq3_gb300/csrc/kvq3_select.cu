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
// accuracy.  Bound by HBM: 4d bytes per (page, kv head) for 4 d G flops.
//
// Selection.  One CTA per (sequence, kv head): the scores as order-preserving
// 32-bit keys, a radix select of the budget-th largest between the forced
// first and last pages, and one ordered compaction that breaks ties towards
// the lower page.  A few microseconds of latency, no sort.
#include <math.h>

#include "kvq3_internal.h"

using namespace kvq3;

namespace {

constexpr int kScoreWarps = 8;

// D: head dimension; NT: n-tiles of 4 heads x (hi, lo) columns.
template <int D, int NT>
__global__ void __launch_bounds__(32 * kScoreWarps)
    page_scores_kernel(const __grid_constant__ RotParams rp, const __grid_constant__ CacheGeom g,
                       const int32_t* __restrict__ page_table, const int32_t* __restrict__ seq_lens,
                       const __half* __restrict__ bounds, const __half* __restrict__ q, int G, int tiles,
                       float* __restrict__ scores, int32_t* status, float inv_sqrt_d) {
  constexpr int K = 2 * D;
  constexpr int ROW = K + 32;                // halves per B column in shared memory: 64 bytes of padding, no conflicts
  constexpr int E = D >= 128 ? D / 32 : 4;
  constexpr int L = D / E;
  constexpr int GPW = 32 / L;
  constexpr int CH = D / 32;                 // 16-byte loads per lane and row of one bound
  __shared__ __align__(16) __half qb[NT * 8 * ROW];
  __shared__ float qinv[NT * 4];             // 2^-e of each head, 0 past the last
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int j = lane & 3, r = lane >> 2;
  griddep_wait();
  griddep_launch_dependents();
  const int64_t unit = blockIdx.x / tiles;
  const int tile = (int)(blockIdx.x - unit * tiles);
  const int b = (int)(unit / g.hkv), kvh = (int)(unit - (int64_t)b * g.hkv);
  const int64_t len = seq_lens[b];
  const bool len_ok = len >= 0 && len <= (int64_t)g.max_pages * g.page_size;
  if (!len_ok && threadIdx.x == 0) set_status(status, KVQ3_DEV_BAD_LEN);
  const int64_t n = len_ok ? (len + g.page_size - 1) / g.page_size : 0;
  float* row_out = scores + unit * g.max_pages;
  const int64_t p0 = (int64_t)tile * (16 * kScoreWarps) + wid * 16;   // this warp's pages
  if ((int64_t)tile * (16 * kScoreWarps) >= n) {                      // nothing there for the whole CTA
    const int64_t i = (int64_t)tile * (16 * kScoreWarps) + threadIdx.x;
    if (threadIdx.x < 16 * kScoreWarps && i < g.max_pages) row_out[i] = -INFINITY;
    return;
  }
  // rows r and r + 8 of the tile: pages p0 + r, p0 + r + 8
  int64_t page[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int64_t lp = p0 + r + 8 * e;
    page[e] = lp < n ? page_of(g, page_table, b, lp) : -1;
    if (lp < n && page[e] < 0 && j == 0) set_status(status, KVQ3_DEV_BAD_PAGE);
  }
  const uint4* src[2];
#pragma unroll
  for (int e = 0; e < 2; ++e)
    src[e] = reinterpret_cast<const uint4*>(bounds + (page[e] < 0 ? 0 : ((page[e] * g.hkv + kvh) * 2) * D)) + j;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  // the first bound's rows are on their way while the query is rotated
  uint4 a[2][CH];
#pragma unroll
  for (int e = 0; e < 2; ++e)
#pragma unroll
    for (int c = 0; c < CH; ++c) a[e][c] = page[e] >= 0 ? __ldg(src[e] + 4 * c) : zero;

  // q1 of the G heads, its negative part against lo and its positive part
  // against hi, scaled by a power of two into (2^7, 2^8] and split hi + lo
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

  float acc[NT][4];
#pragma unroll
  for (int t = 0; t < NT; ++t) acc[t][0] = acc[t][1] = acc[t][2] = acc[t][3] = 0.0f;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const uint4 x = a[0][c], y = a[1][c];
      if (s == 0) {   // the second bound's row in the first one's registers
        a[0][c] = page[0] >= 0 ? __ldg(src[0] + D / 8 + 4 * c) : zero;
        a[1][c] = page[1] >= 0 ? __ldg(src[1] + D / 8 + 4 * c) : zero;
      }
      const uint32_t f0[4] = {x.x, y.x, x.y, y.y}, f1[4] = {x.z, y.z, x.w, y.w};
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const uint4 w = *reinterpret_cast<const uint4*>(qb + (8 * t + r) * ROW + s * D + 32 * c + 8 * j);
        mma_16816(acc[t], f0, w.x, w.y);
        mma_16816(acc[t], f1, w.z, w.w);
      }
    }
  }
  float best0 = -INFINITY, best1 = -INFINITY;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const float f = qinv[4 * t + j];
    if (4 * t + j < G) {
      best0 = fmaxf(best0, (acc[t][0] + acc[t][1]) * f);
      best1 = fmaxf(best1, (acc[t][2] + acc[t][3]) * f);
    }
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    best0 = fmaxf(best0, __shfl_xor_sync(kFull, best0, o));
    best1 = fmaxf(best1, __shfl_xor_sync(kFull, best1, o));
  }
  if (j < 2) {
    const int64_t i = p0 + r + 8 * j;
    if (i < g.max_pages) row_out[i] = (j ? page[1] : page[0]) >= 0 ? (j ? best1 : best0) : -INFINITY;
  }
}

template <int D, int NT>
cudaError_t launch_scores(const RotParams& rp, const CacheGeom& g, const kvq3_cache* c, const __half* bounds,
                          const __half* q, int G, float* scores, int32_t* st, cudaStream_t stream) {
  const int tiles = (int)(((int64_t)g.max_pages + 16 * kScoreWarps - 1) / (16 * kScoreWarps));
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((int64_t)g.batch * g.hkv * tiles));
  cfg.blockDim = dim3(32 * kScoreWarps);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, page_scores_kernel<D, NT>, rp, g, c->page_table, c->seq_lens, bounds, q, G, tiles,
                            scores, st, inv_sqrt(D));
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
constexpr int kBins = 2048;          // 11 bits a pass: 11 + 11 + 10
constexpr int kSelCache = 8192;      // keys held in shared memory (longer rows are read again)

// Order-preserving key: larger score, larger key; NaN lowest, -0 as +0.
__device__ __forceinline__ uint32_t score_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.0f);   // -0 + 0 = +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive block sum of v over the threads; *total receives the sum.
__device__ __forceinline__ uint32_t block_excl(uint32_t v, uint32_t* wsum, uint32_t* total) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  uint32_t incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t t = __shfl_up_sync(kFull, incl, o);
    if (lane >= o) incl += t;
  }
  __syncthreads();
  if (lane == 31) wsum[wid] = incl;
  __syncthreads();
  uint32_t base = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kSelThreads / 32; ++w) {
    const uint32_t t = wsum[w];
    base += w < wid ? t : 0u;
    all += t;
  }
  *total = all;
  return base + incl - v;
}

__global__ void __launch_bounds__(kSelThreads)
    page_select_kernel(const __grid_constant__ CacheGeom g, const int32_t* __restrict__ seq_lens,
                       const float* __restrict__ scores, int budget, int sinks, int recent, int32_t* __restrict__ pages,
                       int32_t* __restrict__ counts, int32_t* status) {
  __shared__ uint32_t keys[kSelCache];
  __shared__ uint32_t hist[kBins];
  __shared__ uint32_t wsum[kSelThreads / 32];
  __shared__ uint32_t found[2];
  griddep_wait();
  griddep_launch_dependents();
  const int t = threadIdx.x;
  const int64_t unit = blockIdx.x;
  const int b = (int)(unit / g.hkv);
  const int64_t len = seq_lens[b];
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
  const float* row = scores + unit * g.max_pages + sinks;
  for (int i = t; i < sinks; i += kSelThreads) out[i] = i;
  for (int i = t; i < recent; i += kSelThreads) out[budget - recent + i] = n - recent + i;
  if (want == 0) return;
  const bool cached = m <= kSelCache;
  if (cached)
    for (int i = t; i < m; i += kSelThreads) keys[i] = score_key(row[i]);
  auto key_at = [&](int i) { return cached ? keys[i] : score_key(row[i]); };

  // radix select of the want-th largest key: bits [31..21], [20..10], [9..0]
  uint32_t prefix = 0, left = (uint32_t)want;   // places left within the prefix
  uint32_t equal = 0;                           // keys equal to the one found, at the end
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const int bins = pass == 2 ? 1024 : kBins;
    for (int i = t; i < bins; i += kSelThreads) hist[i] = 0;
    __syncthreads();
    for (int i = t; i < m; i += kSelThreads) {
      const uint32_t k = key_at(i);
      if (pass == 0 || (k >> (pass == 1 ? 21 : 10)) == prefix) atomicAdd(&hist[(k >> shift) & (bins - 1)], 1u);
    }
    __syncthreads();
    // from the top: the bin that holds the left-th
    const int per = bins / kSelThreads, top = bins - 1 - t * per;
    uint32_t mine = 0;
    for (int i = 0; i < per; ++i) mine += hist[top - i];
    uint32_t total;
    uint32_t above = block_excl(mine, wsum, &total);
    if (above < left && left <= above + mine) {
      for (int i = 0; i < per; ++i) {
        const uint32_t h = hist[top - i];
        if (left <= above + h) {
          found[0] = (uint32_t)(top - i);
          found[1] = left - above;
          break;
        }
        above += h;
      }
    }
    __syncthreads();
    prefix = pass == 0 ? found[0] : (prefix << (pass == 1 ? 11 : 10)) | found[0];
    left = found[1];
    __syncthreads();
  }
  equal = left;   // of the keys equal to `prefix`, the first `equal` by page

  // each thread a run of consecutive pages: larger keys and, in order, the
  // first of the equal ones
  const int per = (m + kSelThreads - 1) / kSelThreads;
  const int i0 = min(m, t * per), i1 = min(m, i0 + per);
  uint32_t gt = 0, eq = 0;
  for (int i = i0; i < i1; ++i) {
    const uint32_t k = key_at(i);
    gt += k > prefix;
    eq += k == prefix;
  }
  uint32_t total;
  const uint32_t gt0 = block_excl(gt, wsum, &total);
  uint32_t eq0 = block_excl(eq, wsum, &total);
  uint32_t at = (uint32_t)sinks + gt0 + min(eq0, equal);
  for (int i = i0; i < i1; ++i) {
    const uint32_t k = key_at(i);
    const bool take = k > prefix || (k == prefix && eq0++ < equal);
    if (take) out[at++] = sinks + i;
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
  return cuda_status(cudaLaunchKernelEx(&cfg, page_select_kernel, g, cache->seq_lens, scores, budget, sinks, recent,
                                        pages, counts, dev_status));
}

}  // extern "C"
