// Key bounds of the cache's pages: the cheap summary that page scores read in
// place of the keys.
//
// For page p, kv head h and rotated coordinate j, over the page's tokens t of
// the sequence,
//   lo[p][h][j] = min_t k_hat[t][j],   hi[p][h][j] = max_t k_hat[t][j],
// k_hat = s_q c (or s_q u + z_q) as the attention reads it.  For any query q1
// = U q and any token of the page, q1 . k_hat <= sum_j max(q1_j lo_j, q1_j
// hi_j), which is what the scores compute.  The bounds are held in fp16, each
// the rounding to nearest of the exact minimum or maximum: rounding is
// monotone, so taking the minimum of rounded products gives the same value,
// and the product of an fp16 (or E4M3) scale and a small integer rounds once
// in half2 arithmetic.  That inequality then holds up to 2^-11 relative, far
// below what a page ranking resolves, at half the bytes of fp32.
//
// One lane owns 32 coordinates of a (page, kv head) and walks the page's
// tokens, two batches of four in flight in turn, so the minima and maxima stay
// in registers; 2 to 16 lanes share a page's tokens and meet by shuffles where
// that fills the GPU (the append of a decode step, the last round over a long
// prompt).  What bounds it is the unpacking: per 32 coordinates of a token 32
// packed minima and maxima, 16 masks and about 12 shifts on the half-rate
// integer pipe (70 % busy) and 32 half2 products on another half-rate one.
// 16 sequences of 32K tokens (8 kv heads of 128, 3-bit codes, 128-token pages):
// 87 us, 2.7 TB/s of 235 MB.  Runs of consecutive tokens per lane (constant
// address steps) took 95 us (one 48-byte piece per memory wavefront), window
// tables with 5 kinds of field position instead of 8 84 to 88.  The other
// formats on the same tokens: 83 us at 2 bits, 91 at 4, 87 with E4M3 scales, 95
// with zero points, 146 with fp32 scales (products in fp32, rounded at the
// end); 50 us at d = 64 and 169 at d = 256.
//
// Inputs are read with coherent loads (no __restrict__ on them): a kernel
// launched as a programmatic dependent is alive while the one before it still
// writes what it will read.
#include <algorithm>
#include <atomic>

#include "kvq3_decode.cuh"

using namespace kvq3;

namespace {

constexpr int kThreads = 128;
constexpr int kLaneTokens = 32;
constexpr int kSeg = 1024;   // sequences whose page counts are held in shared memory at a time

// Page count of every sequence of a segment as an inclusive running sum in
// shared memory; `first` (nullable) gives the position from which pages count.
__device__ __forceinline__ int64_t segment_pages(const CacheGeom& g, const int32_t* seq_lens, const int32_t* first,
                                                 int b0, int64_t* psum, int32_t* pfirst, int32_t* status, bool flag) {
  __shared__ int64_t wsum[kThreads / 32];
  constexpr int PER = kSeg / kThreads;
  const int t = threadIdx.x, lane = t & 31, wid = t >> 5;
  const int64_t cap = (int64_t)g.max_pages * g.page_size;
  int64_t n[PER], sum = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int b = b0 + t * PER + i;
    int64_t pages = 0;
    int32_t lp0 = 0;
    if (b < g.batch) {
      const int64_t len = seq_lens[b];
      const int64_t f = first ? first[b] : 0;
      if (len < 0 || len > cap || f < 0) {
        if (flag) set_status(status, KVQ3_DEV_BAD_LEN);
      } else if (f < len) {
        lp0 = (int32_t)(f / g.page_size);
        pages = (len + g.page_size - 1) / g.page_size - lp0;
      }
    }
    n[i] = pages;
    sum += pages;
    pfirst[t * PER + i] = lp0;
  }
  int64_t incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(kFull, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) wsum[wid] = incl;
  __syncthreads();
  int64_t base = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < wid) base += wsum[w];
    total += wsum[w];
  }
  base += incl - sum;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    base += n[i];
    psum[t * PER + i] = base;
  }
  __syncthreads();
  return total;
}

__device__ __forceinline__ uint32_t hmul2_bits(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t hfma2_bits(uint32_t a, uint32_t b, uint32_t c) {
  const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b),
                            *reinterpret_cast<const __half2*>(&c));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t hmin2_bits(uint32_t a, uint32_t b) {
  const __half2 r = __hmin2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t hmax2_bits(uint32_t a, uint32_t b) {
  const __half2 r = __hmax2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// fp16 bits of a power of two 2^-k (0 <= k <= 7) and of the offset -(2^(10-k) + ofs)
__host__ __device__ constexpr uint32_t half_pow2(int k) { return (uint32_t)(15 - k) << 10; }
__host__ __device__ constexpr uint32_t half_int(int v) {   // 0 < v <= 2048, exact in fp16
  int e = 0;
  while ((v >> (e + 1)) != 0) ++e;
  return ((uint32_t)(15 + e) << 10) | (((uint32_t)v << 10 >> e) & 0x3ffu);
}

// Pair P of a 16-field window (lo:hi) as the exact half2 of its codes (UNS:
// unsigned fields).  The window's sign bits are flipped beforehand, so a field
// reads u = c + 2^(b-1); or-ed into a half of exponent 2^10 at mantissa bit k
// it is 1024 + u 2^k, and one half2 fma gives (1024 + u 2^k) 2^-k -
// (2^(10-k) + 2^(b-1)) = c exactly.
template <int NBIT, bool UNS, int P>
__device__ __forceinline__ uint32_t code_pair(uint32_t lo, uint32_t hi, uint32_t magic) {
  constexpr int kl = kp_kl(NBIT, 16, P), kh = kp_kh(NBIT, 16, P);
  constexpr uint32_t F = (1u << NBIT) - 1u;
  constexpr uint32_t M = (F << kl) | (F << (16 + kh));
  uint32_t w;
  if constexpr (NBIT == 3) {
    constexpr int o = kp3_o(16, P);
    if constexpr (o < 0) w = lo << (-o);
    else if constexpr (o == 0) w = lo;
    else w = __funnelshift_r(lo, hi, o);
  } else if constexpr (NBIT == 4) {
    w = (P < 4 ? lo : hi) >> ((P % 4) >= 2 ? 8 : 0);
  } else {
    w = __byte_perm(lo, 0u, (P / 4) == 0 ? 0x1100u : 0x3322u);
  }
  uint32_t v;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(v) : "r"(w), "n"(M), "r"(magic));   // (w & M) | magic
  constexpr int OFS = UNS ? 0 : 1 << (NBIT - 1);
  constexpr uint32_t mul = half_pow2(kl) | (half_pow2(kh) << 16);
  constexpr uint32_t add = 0x80008000u | half_int((1024 >> kl) + OFS) | (half_int((1024 >> kh) + OFS) << 16);
  return hfma2_bits(v, mul, add);
}

// 32 codes of one token: NBIT words.
template <int NBIT>
struct Codes {
  uint32_t w[NBIT];
};

template <int NBIT>
__device__ __forceinline__ Codes<NBIT> load_codes(const uint8_t* p) {
  Codes<NBIT> c;
  if constexpr (NBIT == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    c.w[0] = v.x; c.w[1] = v.y;
  } else if constexpr (NBIT == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    c.w[0] = v.x; c.w[1] = v.y; c.w[2] = v.z; c.w[3] = v.w;
  } else {
    const uint32_t* q = reinterpret_cast<const uint32_t*>(p);
    c.w[0] = q[0]; c.w[1] = q[1]; c.w[2] = q[2];
  }
  return c;
}

// Raw scale bits of a block (scale byte | zero-point byte << 8 in the
// asymmetric variant).
template <int SCALE>
__device__ __forceinline__ uint32_t load_scale(const uint8_t* p) {
  if constexpr (SCALE == KVQ3_SCALE_F32) return *reinterpret_cast<const uint32_t*>(p);
  else if constexpr (SCALE == KVQ3_SCALE_E4M3) return *p;
  else return *reinterpret_cast<const uint16_t*>(p);
}

template <int NBIT, int SCALE>
struct Accum {
  static constexpr bool WIDE = SCALE == KVQ3_SCALE_F32;   // fp32 products, rounded at the end
  static constexpr bool ASYM = SCALE == KVQ3_SCALE_E4M3_ZP;
  static constexpr int N = WIDE ? 32 : 16;
  uint32_t lo[N], hi[N];   // half2 pairs (window i, pair P at 8 i + P), or fp32 bits (twice as many)

  __device__ __forceinline__ void init() {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      lo[i] = WIDE ? 0x7f800000u : 0x7c007c00u;
      hi[i] = WIDE ? 0xff800000u : 0xfc00fc00u;
    }
  }

  __device__ __forceinline__ void add(const Codes<NBIT>& c, uint32_t sbits) {
    uint32_t s2 = 0, z2 = 0;
    float sf = 0.0f;
    if constexpr (WIDE) {
      sf = __uint_as_float(sbits);
    } else if constexpr (SCALE == KVQ3_SCALE_F16) {
      s2 = sbits | (sbits << 16);
    } else {
      const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)sbits, __NV_E4M3);
      s2 = (uint32_t)hr.x | ((uint32_t)hr.x << 16);
      z2 = (uint32_t)hr.y | ((uint32_t)hr.y << 16);
    }
    // sign bits of the fields flipped (bits 3i + 2 of the 96-bit string; the
    // top bit of every nibble or bit pair)
    uint32_t w[NBIT];
#pragma unroll
    for (int i = 0; i < NBIT; ++i) {
      const uint32_t sgn = NBIT == 4 ? kSign4 : NBIT == 2 ? kSign2 : i == 0 ? kSignRes2 : i == 1 ? kSignRes0 : 0x92492492u;
      w[i] = ASYM ? c.w[i] : c.w[i] ^ sgn;
    }
    const uint32_t magic = 0x64006400u;
    static_for<2>([&](auto ic) {
      constexpr int i = decltype(ic)::value;
      uint32_t l, h;
      if constexpr (NBIT == 2) {
        l = w[i]; h = 0;
      } else if constexpr (NBIT == 4) {
        l = w[(2 * i) % NBIT]; h = w[(2 * i + 1) % NBIT];
      } else if constexpr (i == 0) {
        l = w[0]; h = w[1];
      } else {
        l = __funnelshift_r(w[1], w[2 % NBIT], 16); h = w[2 % NBIT] >> 16;
      }
      static_for<8>([&](auto pc) {
        constexpr int P = decltype(pc)::value;
        const uint32_t v = code_pair<NBIT, ASYM, P>(l, h, magic);
        if constexpr (WIDE) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v));
          const float x = f.x * sf, y = f.y * sf;
          constexpr int k = (2 * (8 * i + P)) % N;
          lo[k] = __float_as_uint(fminf(__uint_as_float(lo[k]), x));
          hi[k] = __float_as_uint(fmaxf(__uint_as_float(hi[k]), x));
          lo[k + 1] = __float_as_uint(fminf(__uint_as_float(lo[k + 1]), y));
          hi[k + 1] = __float_as_uint(fmaxf(__uint_as_float(hi[k + 1]), y));
        } else {
          const uint32_t x = ASYM ? hfma2_bits(v, s2, z2) : hmul2_bits(v, s2);
          constexpr int k = (8 * i + P) % N;
          lo[k] = hmin2_bits(lo[k], x);
          hi[k] = hmax2_bits(hi[k], x);
        }
      });
    });
  }

  // minima and maxima over the lanes that differ from this one in bit m
  __device__ __forceinline__ void meet(int m) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t a = __shfl_xor_sync(kFull, lo[i], m), b = __shfl_xor_sync(kFull, hi[i], m);
      if constexpr (WIDE) {
        lo[i] = __float_as_uint(fminf(__uint_as_float(lo[i]), __uint_as_float(a)));
        hi[i] = __float_as_uint(fmaxf(__uint_as_float(hi[i]), __uint_as_float(b)));
      } else {
        lo[i] = hmin2_bits(lo[i], a);
        hi[i] = hmax2_bits(hi[i], b);
      }
    }
  }

  // the 32 coordinates in order, 16 words of half2, 64 bytes at dst
  __device__ __forceinline__ static void store(const uint32_t (&v)[N], __half* dst) {
    uint16_t h[32];
    static_for<16>([&](auto pc) {
      constexpr int i = decltype(pc)::value / 8, P = decltype(pc)::value % 8;
      constexpr int fl = 16 * i + kp_fl(NBIT, 16, P), fh = 16 * i + kp_fh(NBIT, 16, P);
      if constexpr (WIDE) {
        constexpr int k = (2 * (8 * i + P)) % N;
        h[fl] = __half_as_ushort(__float2half_rn(__uint_as_float(v[k])));
        h[fh] = __half_as_ushort(__float2half_rn(__uint_as_float(v[k + 1])));
      } else {
        h[fl] = (uint16_t)(v[(8 * i + P) % N] & 0xffffu);
        h[fh] = (uint16_t)(v[(8 * i + P) % N] >> 16);
      }
    });
    uint4* d = reinterpret_cast<uint4*>(dst);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = (uint32_t)h[8 * k + 2 * e] | ((uint32_t)h[8 * k + 2 * e + 1] << 16);
      d[k] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
};

template <int NBIT, int SCALE>
__global__ void __launch_bounds__(kThreads)
    key_bounds_kernel(const __grid_constant__ CacheGeom g, const uint8_t* pool,
                      const int32_t* page_table, const int32_t* seq_lens,
                      const int32_t* first, __half* __restrict__ bounds, int32_t* status) {
  __shared__ int64_t psum[kSeg];
  __shared__ int32_t pfirst[kSeg];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t nthreads = (int64_t)gridDim.x * kThreads;
  const int64_t thread = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int ng = g.d / 32;   // lanes of a token
  for (int b0 = 0; b0 < g.batch; b0 += kSeg) {
    __syncthreads();
    const int64_t pages = segment_pages(g, seq_lens, first, b0, psum, pfirst, status, blockIdx.x == 0);
    const int64_t units = pages * g.hkv;
    // lanes that share a page's tokens: two more while the GPU is not full, or
    // while its last round would idle and each keeps kLaneTokens tokens
    int sub = 1;
    while (sub * ng < 32 && (units * ng * sub < nthreads / 2 ||
                             (units * ng * sub < 8 * nthreads && g.page_size >= 2 * sub * kLaneTokens)))
      sub <<= 1;
    const int per = ng * sub;                 // lanes of a unit
    const int64_t lanes = (units * per + 31) / 32 * 32;   // whole warps: shuffles below
    for (int64_t i = thread; i < lanes; i += nthreads) {
      const int64_t unit = i / per;
      const bool on = unit < units;
      const int grp = lane % ng, s = (lane % per) / ng;
      const int64_t item = on ? unit / g.hkv : 0;
      const int kvh = on ? (int)(unit - item * g.hkv) : 0;
      int l = 0, h = kSeg - 1;                // the sequence: first running sum above item
      while (l < h) {
        const int m = (l + h) >> 1;
        if (psum[m] > item) h = m;
        else l = m + 1;
      }
      const int b = min(b0 + l, g.batch - 1);
      const int64_t lp = on ? pfirst[l] + item - (l ? psum[l - 1] : 0) : 0;
      const int64_t page = on ? page_of(g, page_table, b, lp) : -1;
      const bool ok = page >= 0 && KVQ3_CHECK(status, in_range(record_offset(g, page, kvh, 0), g.record_bytes,
                                                              g.num_pages * g.page_bytes) &&
                                                         in_range((page * g.hkv + kvh) * 2 * g.d, 2 * g.d,
                                                                  g.num_pages * g.hkv * 2 * g.d));
      if (on && page < 0 && grp == 0 && s == 0) set_status(status, KVQ3_DEV_BAD_PAGE);
      Accum<NBIT, SCALE> acc;
      acc.init();
      if (ok) {
        const int n = (int)min((int64_t)g.page_size, seq_lens[b] - lp * g.page_size);   // >= 1
        const uint8_t* rec = pool + record_offset(g, page, kvh, 0);
        const uint8_t* codes = rec + g.scale_hdr_bytes + grp * (4 * NBIT);
        const uint8_t* scales = rec + (grp * 32 / g.block) * g.sb;
        const int tb = g.nb * g.sb;
        // U tokens at a time, the next U on their way meanwhile; a token index
        // past the last is clamped to it (minima and maxima do not mind a
        // token twice)
        constexpr int U = 4;
        Codes<NBIT> c[U], cn[U];
        uint32_t sc[U], scn[U];
        auto load = [&](int t0, Codes<NBIT>(&cc)[U], uint32_t(&ss)[U]) {
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int t = min(t0 + u * sub, n - 1);
            cc[u] = load_codes<NBIT>(codes + (uint32_t)(t * g.cb));
            ss[u] = load_scale<SCALE>(scales + (uint32_t)(t * tb));
          }
        };
        const int step = U * sub;
        load(s, c, sc);
        for (int t0 = s; t0 < n; t0 += 2 * step) {
          if (t0 + step < n) load(t0 + step, cn, scn);
#pragma unroll
          for (int u = 0; u < U; ++u) acc.add(c[u], sc[u]);
          if (t0 + step < n) {
            if (t0 + 2 * step < n) load(t0 + 2 * step, c, sc);
#pragma unroll
            for (int u = 0; u < U; ++u) acc.add(cn[u], scn[u]);
          }
        }
      }
      for (int m = ng; m < per; m <<= 1) acc.meet(m);
      if (ok && s == 0) {
        __half* dst = bounds + ((page * g.hkv + kvh) * 2) * g.d + grp * 32;
        Accum<NBIT, SCALE>::store(acc.lo, dst);
        Accum<NBIT, SCALE>::store(acc.hi, dst + g.d);
      }
    }
  }
}

template <int NBIT, int SCALE>
cudaError_t launch_bounds(const CacheGeom& g, const kvq3_cache* c, const int32_t* first, __half* bounds, int32_t* st,
                          cudaStream_t stream) {
  static std::atomic<int> resident{0};   // CTAs per SM (the same on every sm_103a device)
  int per_sm = resident.load(std::memory_order_relaxed);
  if (per_sm == 0) {
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, key_bounds_kernel<NBIT, SCALE>, kThreads, 0) != cudaSuccess)
      return cudaErrorUnknown;
    resident.store(per_sm, std::memory_order_relaxed);
  }
  // no more CTAs than a lane for each coordinate of each page that the cache's tables can name
  const double most = (double)g.batch * g.max_pages * g.hkv * g.d / kThreads + 1.0;
  int64_t blocks = (int64_t)sm_count() * std::max(1, per_sm);
  if ((double)blocks > most) blocks = (int64_t)most;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(blocks > 0 ? blocks : 1));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, key_bounds_kernel<NBIT, SCALE>, g, static_cast<const uint8_t*>(c->pool), c->page_table,
                            c->seq_lens, first, bounds, st);
}

template <int SCALE>
cudaError_t bounds_by_bits(const CacheGeom& g, const kvq3_cache* c, const int32_t* first, __half* bounds, int32_t* st,
                           cudaStream_t stream) {
  if (g.bits == 2) return launch_bounds<2, SCALE>(g, c, first, bounds, st, stream);
  if (g.bits == 4) return launch_bounds<4, SCALE>(g, c, first, bounds, st, stream);
  return launch_bounds<3, SCALE>(g, c, first, bounds, st, stream);
}

}  // namespace

extern "C" kvq3_status kvq3_key_bounds(const kvq3_cache_desc* desc, const kvq3_cache* cache, const int32_t* first_pos,
                                       void* bounds, int32_t* dev_status, void* stream) {
  CacheGeom g;
  kvq3_status s = make_geom(desc, &g);
  if (s != KVQ3_OK) return s;
  if ((s = check_cache(g, cache, true)) != KVQ3_OK) return s;
  if (!bounds || reinterpret_cast<uintptr_t>(bounds) % 16 != 0) return KVQ3_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  __half* out = static_cast<__half*>(bounds);
  cudaError_t e;
  switch (g.scale_type) {
    case KVQ3_SCALE_F32: e = bounds_by_bits<KVQ3_SCALE_F32>(g, cache, first_pos, out, dev_status, st); break;
    case KVQ3_SCALE_F16: e = bounds_by_bits<KVQ3_SCALE_F16>(g, cache, first_pos, out, dev_status, st); break;
    case KVQ3_SCALE_E4M3: e = bounds_by_bits<KVQ3_SCALE_E4M3>(g, cache, first_pos, out, dev_status, st); break;
    default: e = launch_bounds<3, KVQ3_SCALE_E4M3_ZP>(g, cache, first_pos, out, dev_status, st); break;
  }
  return cuda_status(e);
}
