// Page management of a paged cache: remapping sequences onto pages (fork,
// reorder, grow, truncate, free) and compacting kept tokens into fresh pages.
//
// Remap.  The new table is a function of the old one: whole pages of a row's
// source are shared, a part-filled page has one owner (the lowest row, unless
// some row shares it whole) and is copied for the others, and the rest of the
// entries take the lowest pages that no row of the new table holds.  Nothing
// is kept between calls: which pages are free follows from the table itself,
// so there are no reference counts to drift and the outcome does not depend
// on the order of any atomic (the marks are bit-ors, the owner a minimum, the
// free pages a rank over a bitmap).
//
// The bookkeeping is a chain of dependent passes over the table and the page
// bitmap (a few hundred KB at most), bound by the latency of its loads and
// barriers.  For a small table (up to 512 rows and 64K entries) every CTA of
// one launch does all of it for itself, with the rows' state and the bitmap in
// shared memory and block barriers between the passes; the first CTA writes
// the result, and each then copies its share of the part-filled pages without
// waiting for another.  A larger table is a thread-block cluster's work, its
// state in the workspace and the hardware cluster barrier between, and the
// copies, the only bulk traffic, are a second kernel's, its programmatic
// dependent.  Only the slots in use are copied.  16 sequences that grow by a
// token: 5.0 us; 64 sequences in beams of 8, a third of them with a page to
// copy (2.3 MB): 8.4 us (13.4 and 18.1 as a cluster with a copy kernel).  Where
// the two meet: 16 rows of up to 4,095 pages 38.2 us in the one launch, 512 rows
// of up to 64 pages 27.5; 600 rows of up to 64 pages 23.8 as a cluster.  64 rows
// of up to 4,096 pages: 67 us, six cluster barriers and eight SMs that walk 2 MB
// of table.
//
// Compaction is a gather of packed vectors (codes and scales as stored); one
// CTA takes a run of kept tokens of a (sequence, kv head), resolves each
// token's record addresses once into shared memory, and moves the code strings
// and scale headers with the widest accesses their sizes allow, every load
// under way before the first store.  Bound by HBM sectors: a kept token at
// random reads 48 + 4 bytes per vector but touches about 104 (whole 32-byte
// sectors).  16 x 8 heads, 4,096 of 16,384 tokens kept: 31.4 us, 3.5 TB/s of
// the bytes moved, 5.2 TB/s of sectors (35.6 us with one access at a time).
//
// Inputs are read with coherent loads (no __restrict__ on them): a kernel
// launched as a programmatic dependent is alive while the one before it still
// writes what it will read.
#include <cooperative_groups.h>

#include <algorithm>

#include "kvq3_internal.h"

namespace cg = cooperative_groups;
using namespace kvq3;

namespace {

constexpr int kMapThreads = 1024;
constexpr int kMapCluster = 8;      // CTAs of the remap cluster (the portable maximum)
// The tables that remap_small_kernel takes, whose every CTA does the whole
// bookkeeping for itself: a cluster barrier costs over a microsecond with the
// workspace's writes in flight, a block barrier almost nothing, but one SM
// moves only about 100 GB/s of table.
constexpr int kSmallRows = 512;
constexpr int kSmallEntries = 65536;
constexpr int kSmallPages = 65536;
constexpr int kCopyPieces = 5;      // pieces of a record's copy: its codes in quarters, its scales

// What the remap keeps in its workspace.
struct RemapWs {
  uint32_t* bits;       // [ceil(num_pages / 32)] pages held by the new table
  int32_t* owner;       // [num_pages] lowest row whose part-filled page it is (only such pages are written)
  int32_t* freed;       // [num_pages] the lowest free pages in order
  int32_t* need;        // [batch] entries a row takes from the free pages
  int64_t* first;       // [batch] rank of the first of them
  int4* rows;           // [batch] source row (-1: none), whole pages, tokens of the part-filled page, entries
  int32_t* tail;        // [batch] the part-filled page's id, -1 where there is none
  int4* copies;         // [batch] copy of a part-filled page: from, to, tokens (0: no copy)
  size_t bytes;
};

RemapWs remap_layout(const CacheGeom& g, void* base) {
  RemapWs w;
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t o = at;
    at += (n + 255) / 256 * 256;
    return static_cast<char*>(base) + o;
  };
  const size_t n = (size_t)g.num_pages, b = (size_t)g.batch;
  w.bits = reinterpret_cast<uint32_t*>(take((n + 31) / 32 * 4));
  w.owner = reinterpret_cast<int32_t*>(take(n * 4));
  w.freed = reinterpret_cast<int32_t*>(take(n * 4));
  w.need = reinterpret_cast<int32_t*>(take(b * 4));
  w.first = reinterpret_cast<int64_t*>(take(b * 8));
  w.rows = reinterpret_cast<int4*>(take(b * 16));
  w.tail = reinterpret_cast<int32_t*>(take(b * 4));
  w.copies = reinterpret_cast<int4*>(take(b * 16));
  w.bytes = at;
  return w;
}

// Exclusive sum of v over the CTA's threads; *total receives the sum.
__device__ __forceinline__ int64_t cta_excl(int64_t v, int64_t* wsum, int64_t* total) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  int64_t incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t t = __shfl_up_sync(kFull, incl, o);
    if (lane >= o) incl += t;
  }
  __syncthreads();
  if (lane == 31) wsum[wid] = incl;
  __syncthreads();
  int64_t base = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kMapThreads / 32; ++w) {
    const int64_t t = wsum[w];
    base += w < wid ? t : 0;
    all += t;
  }
  *total = all;
  return base + incl - v;
}

__global__ void __launch_bounds__(kMapThreads)
    remap_kernel(const __grid_constant__ CacheGeom g, const int32_t* table, const int32_t* seq_lens, const int32_t* src,
                 const int32_t* new_lens, int32_t* table_out, int32_t* lens_out, const __grid_constant__ RemapWs ws,
                 int32_t* status) {
  __shared__ int64_t wsum[kMapThreads / 32];
  __shared__ int64_t part[2];   // this CTA's free pages and wanted entries
  griddep_wait();
  griddep_launch_dependents();
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ncta = (int)cluster.num_blocks();
  const int t = threadIdx.x, lane = t & 31;
  const int64_t th = (int64_t)rank * kMapThreads + t, nth = (int64_t)ncta * kMapThreads;
  const int64_t wp = th >> 5, nwp = nth >> 5;
  const int64_t words = (g.num_pages + 31) / 32;
  const int P = g.page_size;
  const int64_t cap = (int64_t)g.max_pages * P;

  // the rows, and an empty bitmap
  for (int64_t i = th; i < words; i += nth) ws.bits[i] = 0;
  for (int64_t b = th; b < g.batch; b += nth) {
    const int s = src[b];
    const int64_t want = new_lens[b];
    int64_t held = 0, entries = 0;
    int from = -1;
    if (s < -1 || s >= g.batch) {
      set_status(status, KVQ3_DEV_BAD_SEQ);
    } else if (want < 0 || want > cap || (s >= 0 && (seq_lens[s] < 0 || seq_lens[s] > cap))) {
      set_status(status, KVQ3_DEV_BAD_LEN);
    } else {
      from = s;
      held = s >= 0 ? min((int64_t)seq_lens[s], want) : 0;
      entries = (want + P - 1) / P;
    }
    const int full = (int)(held / P), rest = (int)(held % P);
    int tail = -1;
    if (rest) {
      tail = table[(int64_t)from * g.max_pages + full];
      if (tail < 0 || tail >= g.num_pages) {
        set_status(status, KVQ3_DEV_BAD_PAGE);
        tail = -1;
      } else {
        ws.owner[tail] = 0x7fffffff;
      }
    }
    ws.rows[b] = make_int4(from, full, rest, (int)entries);
    ws.tail[b] = tail;
    ws.copies[b] = make_int4(0, 0, 0, 0);
    lens_out[b] = (int32_t)held;
  }
  cluster.sync();
  // whole pages are shared as they are
  for (int64_t b = wp; b < g.batch; b += nwp) {
    const int4 r = ws.rows[b];
    for (int i = lane; i < g.max_pages; i += 32) {
      int32_t page = -1;
      if (i < r.y) {
        page = table[(int64_t)r.x * g.max_pages + i];
        if (page < 0 || page >= g.num_pages) {
          set_status(status, KVQ3_DEV_BAD_PAGE);
          page = -1;
        } else {
          atomicOr(&ws.bits[page >> 5], 1u << (page & 31));
        }
      }
      table_out[b * g.max_pages + i] = page;
    }
  }
  cluster.sync();
  // owners of part-filled pages
  for (int64_t b = th; b < g.batch; b += nth) {
    const int tail = ws.tail[b];
    if (tail >= 0) atomicMin(&ws.owner[tail], (int32_t)b);
  }
  cluster.sync();
  for (int64_t b = th; b < g.batch; b += nth) {
    const int4 r = ws.rows[b];
    const int tail = ws.tail[b];
    int keeps = 0;
    if (tail >= 0 && __ldcg(&ws.owner[tail]) == b) {
      // only the owner may set this bit here, so it is clear unless some row shares the page whole
      const uint32_t bit = 1u << (tail & 31);
      if ((atomicOr(&ws.bits[tail >> 5], bit) & bit) == 0) {
        keeps = 1;
        table_out[b * g.max_pages + r.y] = tail;
        ws.tail[b] = -1;   // nothing to copy
      }
    }
    // an unreadable part-filled page keeps its entry at -1
    const int lost = r.z && tail < 0;
    ws.need[b] = r.w - r.y - (keeps | lost);
  }
  cluster.sync();
  // ranks: every CTA counts the free pages and the wanted entries of its slice
  const int64_t w0 = words * rank / ncta, w1 = words * (rank + 1) / ncta;
  const int64_t b0 = (int64_t)g.batch * rank / ncta, b1 = (int64_t)g.batch * (rank + 1) / ncta;
  auto free_of = [&](int64_t w) {
    uint32_t f = ~__ldcg(&ws.bits[w]);
    if (w == words - 1 && (g.num_pages & 31)) f &= (1u << (g.num_pages & 31)) - 1u;
    return f;
  };
  {
    int64_t f = 0, n = 0, total;
    for (int64_t w = w0 + t; w < w1; w += kMapThreads) f += __popc(free_of(w));
    for (int64_t b = b0 + t; b < b1; b += kMapThreads) n += ws.need[b];
    cta_excl(f, wsum, &total);
    if (t == 0) part[0] = total;
    cta_excl(n, wsum, &total);
    if (t == 0) part[1] = total;
  }
  cluster.sync();
  int64_t free_before = 0, want_before = 0, free_all = 0, want_all = 0;
  for (int c = 0; c < ncta; ++c) {
    const int64_t* other = cluster.map_shared_rank(part, c);
    const int64_t f = other[0], n = other[1];
    if (c < rank) {
      free_before += f;
      want_before += n;
    }
    free_all += f;
    want_all += n;
  }
  const bool enough = want_all <= free_all;
  if (!enough && th == 0) set_status(status, KVQ3_DEV_NO_PAGE);
  // the slice's free pages below the number wanted, in order
  for (int64_t base = w0; base < w1 && free_before < want_all; base += kMapThreads) {
    const int64_t w = base + t;
    uint32_t f = w < w1 ? free_of(w) : 0u;
    int64_t total;
    int64_t at = free_before + cta_excl(__popc(f), wsum, &total);
    while (f && at < want_all) {
      ws.freed[at++] = (int32_t)(w * 32 + __ffs(f) - 1);
      f &= f - 1;
    }
    free_before += total;
  }
  for (int64_t base = b0; base < b1; base += kMapThreads) {
    const int64_t b = base + t;
    int64_t total;
    const int64_t at = want_before + cta_excl(b < b1 ? ws.need[b] : 0, wsum, &total);
    if (b < b1) ws.first[b] = at;
    want_before += total;
  }
  cluster.sync();   // also: no CTA leaves while another reads its shared memory
  if (!enough) return;
  for (int64_t b = wp; b < g.batch; b += nwp) {
    const int4 r = ws.rows[b];
    const int n = ws.need[b];
    const int64_t at = ws.first[b];
    const int tail = ws.tail[b];
    for (int i = lane; i < n; i += 32) {
      const int32_t page = ws.freed[at + i];
      table_out[b * g.max_pages + r.w - n + i] = page;
      if (i == 0 && tail >= 0) ws.copies[b] = make_int4(tail, page, r.z, 0);
    }
  }
}

// Copies `bytes` bytes from src to dst, both 16-byte aligned: thread t of n.
__device__ __forceinline__ void copy_bytes(uint8_t* dst, const uint8_t* src, int64_t bytes, int t, int n) {
  const int64_t n16 = bytes / 16;
#pragma unroll 4
  for (int64_t i = t; i < n16; i += n)
    reinterpret_cast<uint4*>(dst)[i] = __ldcs(reinterpret_cast<const uint4*>(src) + i);
  for (int64_t i = n16 * 16 + t; i < bytes; i += n) dst[i] = src[i];
}

__global__ void __launch_bounds__(256)
    remap_copy_kernel(const __grid_constant__ CacheGeom g, uint8_t* pool, const int4* copies, int32_t* status) {
  griddep_wait();
  griddep_launch_dependents();
  const int recs = 2 * g.hkv;
  const int64_t items = (int64_t)g.batch * recs;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int64_t b = it / recs;
    const int4 c = copies[b];
    if (c.z == 0) continue;
    const int64_t rec = (it - b * recs) * g.record_bytes;
    const int64_t from = c.x * g.page_bytes + rec, to = c.y * g.page_bytes + rec;
    if (!KVQ3_CHECK(status, in_range(from, g.record_bytes, g.num_pages * g.page_bytes) &&
                                in_range(to, g.record_bytes, g.num_pages * g.page_bytes)))
      continue;
    copy_bytes(pool + to, pool + from, (int64_t)c.z * g.nb * g.sb, threadIdx.x, blockDim.x);
    copy_bytes(pool + to + g.scale_hdr_bytes, pool + from + g.scale_hdr_bytes, (int64_t)c.z * g.cb, threadIdx.x, blockDim.x);
  }
}

// The whole remap of a small table, by every CTA for itself: the first CTA
// writes the new table and lengths, all copy.
__global__ void __launch_bounds__(kMapThreads)
    remap_small_kernel(const __grid_constant__ CacheGeom g, uint8_t* pool, const int32_t* table,
                       const int32_t* seq_lens, const int32_t* src,
                       const int32_t* new_lens, int32_t* __restrict__ table_out,
                       int32_t* __restrict__ lens_out, int32_t* status) {
  __shared__ uint32_t bits[kSmallPages / 32];        // pages held by the new table
  __shared__ uint32_t free_before[kSmallPages / 32]; // free pages before each word
  __shared__ int4 rows[kSmallRows];                  // source row, then: keeps its part-filled page; whole pages; tokens
                                                     // of the part-filled one; entries
  __shared__ int32_t tail[kSmallRows];               // the part-filled page, -1 where there is none
  __shared__ uint32_t first[kSmallRows];             // entries from the free pages, then the rank of the first
  __shared__ int32_t copy_from[kSmallRows], copy_to[kSmallRows];
  __shared__ uint32_t copy_tokens[kSmallRows];
  __shared__ unsigned long long wsum[kMapThreads / 32];
  const int t = threadIdx.x, lane = t & 31, wid = t >> 5;
  const int words = (int)((g.num_pages + 31) / 32), batch = g.batch;
  for (int i = t; i < words; i += kMapThreads) bits[i] = 0;
  griddep_wait();
  griddep_launch_dependents();
  const bool lead = blockIdx.x == 0;
  int32_t* st = lead ? status : nullptr;
  const int P = g.page_size;
  const int64_t cap = (int64_t)g.max_pages * P;
  if (t < batch) {
    const int s = src[t];
    const int64_t want = new_lens[t];
    const int64_t len = s >= 0 && s < batch ? seq_lens[s] : 0;
    int64_t held = 0, entries = 0;
    int from = -1;
    if (s < -1 || s >= batch) {
      set_status(st, KVQ3_DEV_BAD_SEQ);
    } else if (want < 0 || want > cap || len < 0 || len > cap) {
      set_status(st, KVQ3_DEV_BAD_LEN);
    } else {
      from = s;
      held = min(len, want);
      entries = (want + P - 1) / P;
    }
    const int full = (int)(held / P), rest = (int)(held % P);
    int page = -1;
    if (rest) {
      page = table[(int64_t)from * g.max_pages + full];
      if (page < 0 || page >= g.num_pages) {
        set_status(st, KVQ3_DEV_BAD_PAGE);
        page = -1;
      }
    }
    rows[t] = make_int4(from, full, rest, (int)entries);
    tail[t] = page;
    if (lead) lens_out[t] = (int32_t)held;
  }
  __syncthreads();
  // whole pages are shared as they are
  for (int b = wid; b < batch; b += kMapThreads / 32) {
    const int4 r = rows[b];
    const int end = lead ? g.max_pages : r.y;
    for (int i = lane; i < end; i += 32) {
      int32_t page = -1;
      if (i < r.y) {
        page = table[(int64_t)r.x * g.max_pages + i];
        if (page < 0 || page >= g.num_pages) {
          set_status(st, KVQ3_DEV_BAD_PAGE);
          page = -1;
        } else {
          atomicOr(&bits[page >> 5], 1u << (page & 31));
        }
      }
      if (lead) table_out[(int64_t)b * g.max_pages + i] = page;
    }
  }
  __syncthreads();
  // a part-filled page stays with the lowest row that has it, unless some row shares it whole
  for (int b = wid; b < batch; b += kMapThreads / 32) {
    const int page = tail[b];
    bool lower = false;
    if (page >= 0)
      for (int c = lane; c < b; c += 32) lower |= tail[c] == page;
    lower = __any_sync(kFull, lower);
    if (lane == 0) {
      const bool keeps = page >= 0 && !lower && !((bits[page >> 5] >> (page & 31)) & 1u);
      const int4 r = rows[b];
      rows[b].x = keeps;
      first[b] = (uint32_t)(r.w - r.y - (keeps || (r.z && page < 0) ? 1 : 0));   // an unreadable one keeps its -1
    }
  }
  __syncthreads();
  const bool keeps = t < batch && rows[t].x, copies = t < batch && tail[t] >= 0 && !keeps;
  const uint32_t need = t < batch ? first[t] : 0;
  if (keeps) {
    atomicOr(&bits[tail[t] >> 5], 1u << (tail[t] & 31));
    if (lead) table_out[(int64_t)t * g.max_pages + rows[t].y] = tail[t];
  }
  __syncthreads();
  // ranks of the free pages, the wanted entries and the copies (the same in
  // every CTA: each takes its share of the copies by rank), in one sum of
  // three fields: at most 2^16 free pages, 2^16 entries, 2^9 copies
  constexpr int WPT = kSmallPages / 32 / kMapThreads;
  uint32_t mine[WPT], free_here = 0;
#pragma unroll
  for (int i = 0; i < WPT; ++i) {
    const int w = t * WPT + i;
    uint32_t f = w < words ? ~bits[w] : 0u;
    if (w == words - 1 && (g.num_pages & 31)) f &= (1u << (g.num_pages & 31)) - 1u;
    mine[i] = __popc(f);
    free_here += mine[i];
  }
  const unsigned long long v = ((unsigned long long)free_here << 40) | ((unsigned long long)need << 16) | (copies ? 1 : 0);
  unsigned long long incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long x = __shfl_up_sync(kFull, incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 31) wsum[wid] = incl;
  __syncthreads();
  unsigned long long before = incl - v, total = 0;
#pragma unroll
  for (int w = 0; w < kMapThreads / 32; ++w) {
    before += w < wid ? wsum[w] : 0;
    total += wsum[w];
  }
  static_assert(kSmallEntries < (1 << 24) && kSmallRows < (1 << 16) && kSmallPages < (1 << 24), "fields of the sum");
  const uint32_t want_all = (uint32_t)(total >> 16) & 0xffffffu, n_copies = (uint32_t)total & 0xffffu;
  uint32_t at = (uint32_t)(before >> 40);
#pragma unroll
  for (int i = 0; i < WPT; ++i) {
    if (t * WPT + i < words) free_before[t * WPT + i] = at;
    at += mine[i];
  }
  if (t < batch) first[t] = (uint32_t)(before >> 16) & 0xffffffu;
  if (want_all > (uint32_t)(total >> 40)) {   // fewer free pages than wanted: nothing is copied
    if (t == 0) set_status(st, KVQ3_DEV_NO_PAGE);
    return;
  }
  __syncthreads();
  // the free page of a rank
  auto free_page = [&](uint32_t rank) {
    int lo = 0, hi = words - 1;
    while (lo < hi) {   // the last word with at most `rank` free pages before it
      const int m = (lo + hi + 1) >> 1;
      if (free_before[m] <= rank) lo = m;
      else hi = m - 1;
    }
    uint32_t f = ~bits[lo];
    for (uint32_t k = rank - free_before[lo]; k > 0; --k) f &= f - 1;
    return lo * 32 + __ffs(f) - 1;
  };
  if (copies) {
    const uint32_t k = (uint32_t)before & 0xffffu;
    copy_from[k] = tail[t];
    copy_to[k] = free_page(first[t]);
    copy_tokens[k] = rows[t].z;
  }
  if (lead) {
    for (int b = wid; b < batch; b += kMapThreads / 32) {
      const int4 r = rows[b];
      const uint32_t at0 = first[b];
      const int start = r.y + (r.x || (r.z && tail[b] < 0) ? 1 : 0);
      for (int i = start + lane; i < r.w; i += 32)
        table_out[(int64_t)b * g.max_pages + i] = free_page(at0 + (uint32_t)(i - start));
    }
  }
  __syncthreads();
  // a warp copies the scales of a record's slots in use, or a quarter of their
  // codes: a few accesses a lane, all under way together
  const int recs = 2 * g.hkv;
  const int64_t items = (int64_t)n_copies * recs * kCopyPieces;
  for (int64_t it = (int64_t)wid * gridDim.x + blockIdx.x; it < items; it += (int64_t)gridDim.x * (kMapThreads / 32)) {
    const int64_t whole = it / kCopyPieces;
    const int piece = (int)(it - whole * kCopyPieces), c = (int)(whole / recs);
    const int64_t rec = (whole - (int64_t)c * recs) * g.record_bytes;
    const int64_t from = copy_from[c] * g.page_bytes + rec, to = copy_to[c] * g.page_bytes + rec;
    if (!KVQ3_CHECK(status, in_range(from, g.record_bytes, g.num_pages * g.page_bytes) &&
                                in_range(to, g.record_bytes, g.num_pages * g.page_bytes)))
      continue;
    if (piece == kCopyPieces - 1) {
      copy_bytes(pool + to, pool + from, (int64_t)copy_tokens[c] * g.nb * g.sb, lane, 32);
    } else {
      const int64_t bytes = (int64_t)copy_tokens[c] * g.cb;
      const int64_t part = (bytes / 16 + kCopyPieces - 2) / (kCopyPieces - 1) * 16;
      const int64_t b0 = min(bytes, piece * part), b1 = piece == kCopyPieces - 2 ? bytes : min(bytes, b0 + part);
      copy_bytes(pool + to + g.scale_hdr_bytes + b0, pool + from + g.scale_hdr_bytes + b0, b1 - b0, lane, 32);
    }
  }
}

// ------------------------------------------------------------ compaction
constexpr int kKeepTile = 128;   // kept tokens per CTA, one per thread

// CV: a code access (16 or 8 bytes), CN of them in a code string; HV: a header
// access, dividing a token's scales.
template <typename CV, int CN, typename HV, int HN>
__global__ void __launch_bounds__(kKeepTile)
    compact_kernel(const __grid_constant__ CacheGeom g, uint8_t* pool, const int32_t* page_table,
                   const int32_t* seq_lens, const int32_t* src_seq,
                   const int32_t* dst_seq, const int32_t* keep,
                   const int32_t* n_keep, int keep_stride, int tiles, int32_t* status) {
  __shared__ int64_t from_s[kKeepTile], to_s[kKeepTile];   // K records, -1: skip
  __shared__ int32_t slots_s[kKeepTile];                   // source slot, destination slot << 16
  griddep_wait();
  griddep_launch_dependents();
  const int t = threadIdx.x;
  const int64_t unit = blockIdx.x / tiles;
  const int tile = (int)(blockIdx.x - unit * tiles);
  const int i = (int)(unit / g.hkv), kvh = (int)(unit - (int64_t)i * g.hkv);
  const int64_t cap = (int64_t)g.max_pages * g.page_size;
  const int64_t at = (int64_t)tile * kKeepTile + t;
  const int64_t pos = at < keep_stride ? keep[unit * keep_stride + at] : -1;   // with the pair's ids and count
  const int s = src_seq[i], d = dst_seq[i], n = n_keep[i];
  int bad = 0;
  int64_t len = 0;
  if (s < 0 || s >= g.batch || d < 0 || d >= g.batch || s == d) bad = KVQ3_DEV_BAD_SEQ;
  else {
    len = seq_lens[s];
    if (len < 0 || len > cap || n < 0 || n > keep_stride || n > cap) bad = KVQ3_DEV_BAD_LEN;
  }
  if (bad) {
    if (t == 0) set_status(status, bad);
    return;
  }
  const int m = (int)min((int64_t)kKeepTile, n - (int64_t)tile * kKeepTile);
  if (m <= 0) return;
  int64_t a = -1, z = -1;
  if (t < m) {
    if (pos < 0 || pos >= len) {
      set_status(status, KVQ3_DEV_BAD_POS);
    } else {   // 32-bit positions: below 2^31
      const uint32_t P = (uint32_t)g.page_size;
      const uint32_t lp = (uint32_t)pos / P, ld = (uint32_t)at / P;
      const int64_t ps = page_of(g, page_table, s, lp), pd = page_of(g, page_table, d, ld);
      if (ps < 0 || pd < 0) set_status(status, KVQ3_DEV_BAD_PAGE);
      else {
        a = record_offset(g, ps, kvh, 0);
        z = record_offset(g, pd, kvh, 0);
        slots_s[t] = (int32_t)((uint32_t)pos - lp * P) | ((int32_t)((uint32_t)at - ld * P) << 16);
        if (!KVQ3_CHECK(status, in_range(a, 2 * g.record_bytes, g.num_pages * g.page_bytes) &&
                                    in_range(z, 2 * g.record_bytes, g.num_pages * g.page_bytes)))
          a = -1;
      }
    }
  }
  from_s[t] = a;
  to_s[t] = z;
  __syncthreads();
  // consecutive threads move consecutive pieces of a code string; every load
  // of the thread is under way before its first store
  CV c[2][CN];
  HV h[2][HN];
#pragma unroll
  for (int k = 0; k < CN; ++k) {
    const int x = k * kKeepTile + t, tok = x / CN, e = x - tok * CN;
    const int64_t f = from_s[tok];
    if (f < 0) continue;
    const uint8_t* p = pool + f + g.scale_hdr_bytes + (slots_s[tok] & 0xffff) * g.cb;
    c[0][k] = reinterpret_cast<const CV*>(p)[e];
    c[1][k] = reinterpret_cast<const CV*>(p + g.record_bytes)[e];
  }
#pragma unroll
  for (int k = 0; k < HN; ++k) {
    const int x = k * kKeepTile + t, tok = x / HN, e = x - tok * HN;
    const int64_t f = from_s[tok];
    if (f < 0) continue;
    const uint8_t* p = pool + f + (slots_s[tok] & 0xffff) * (HN * (int)sizeof(HV));
    h[0][k] = reinterpret_cast<const HV*>(p)[e];
    h[1][k] = reinterpret_cast<const HV*>(p + g.record_bytes)[e];
  }
#pragma unroll
  for (int k = 0; k < CN; ++k) {
    const int x = k * kKeepTile + t, tok = x / CN, e = x - tok * CN;
    if (from_s[tok] < 0) continue;
    uint8_t* p = pool + to_s[tok] + g.scale_hdr_bytes + (slots_s[tok] >> 16) * g.cb;
    reinterpret_cast<CV*>(p)[e] = c[0][k];
    reinterpret_cast<CV*>(p + g.record_bytes)[e] = c[1][k];
  }
#pragma unroll
  for (int k = 0; k < HN; ++k) {
    const int x = k * kKeepTile + t, tok = x / HN, e = x - tok * HN;
    if (from_s[tok] < 0) continue;
    uint8_t* p = pool + to_s[tok] + (slots_s[tok] >> 16) * (HN * (int)sizeof(HV));
    reinterpret_cast<HV*>(p)[e] = h[0][k];
    reinterpret_cast<HV*>(p + g.record_bytes)[e] = h[1][k];
  }
}

struct CompactArgs {
  const kvq3_cache* cache;
  const int32_t *src_seq, *dst_seq, *keep, *n_keep;
  int64_t units;
  int keep_stride;
  int32_t* status;
  cudaStream_t stream;
};

template <typename CV, int CN, typename HV, int HN>
cudaError_t launch_compact(const CacheGeom& g, const CompactArgs& a) {
  const int tiles = (int)(((int64_t)a.keep_stride + kKeepTile - 1) / kKeepTile);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.units * tiles));
  cfg.blockDim = dim3(kKeepTile);
  cfg.stream = a.stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, compact_kernel<CV, CN, HV, HN>, g, static_cast<uint8_t*>(a.cache->pool),
                            a.cache->page_table, a.cache->seq_lens, a.src_seq, a.dst_seq, a.keep, a.n_keep,
                            a.keep_stride, tiles, a.status);
}

// A token's scales take d/64 (one-byte scales, blocks of 64) to d/8 bytes
// (fp32, blocks of 32), a power of two.
template <int D, typename CV, int CN>
cudaError_t compact_by_header(const CacheGeom& g, const CompactArgs& a) {
  switch (g.nb * g.sb) {
    case 1: if constexpr (D <= 64) return launch_compact<CV, CN, uint8_t, 1>(g, a); break;
    case 2: if constexpr (D <= 128) return launch_compact<CV, CN, uint16_t, 1>(g, a); break;
    case 4: return launch_compact<CV, CN, uint32_t, 1>(g, a);
    case 8: return launch_compact<CV, CN, uint2, 1>(g, a);
    case 16: if constexpr (D >= 128) return launch_compact<CV, CN, uint4, 1>(g, a); break;
    case 32: if constexpr (D >= 256) return launch_compact<CV, CN, uint4, 2>(g, a); break;
  }
  return cudaErrorInvalidValue;
}

// A code string takes b d / 8 bytes: a multiple of 16 but for 3-bit codes at d = 64.
template <int D>
cudaError_t compact_by_codes(const CacheGeom& g, const CompactArgs& a) {
  if (g.bits == 2) return compact_by_header<D, uint4, D / 64>(g, a);
  if (g.bits == 4) return compact_by_header<D, uint4, D / 32>(g, a);
  if constexpr (D == 64) return compact_by_header<D, uint2, 3>(g, a);
  else return compact_by_header<D, uint4, 3 * D / 128>(g, a);
}

}  // namespace

extern "C" {

kvq3_status kvq3_remap_workspace_size(const kvq3_cache_desc* desc, size_t* bytes) {
  CacheGeom g;
  const kvq3_status s = make_geom(desc, &g);
  if (s != KVQ3_OK) return s;
  if (!bytes) return KVQ3_ERR_INVALID_ARG;
  if (g.num_pages >= ((int64_t)1 << 31)) return KVQ3_ERR_UNSUPPORTED;   // int32 page ids
  *bytes = remap_layout(g, nullptr).bytes;
  return KVQ3_OK;
}

kvq3_status kvq3_remap(const kvq3_cache_desc* desc, const kvq3_cache* cache, const int32_t* src, const int32_t* new_lens,
                       int32_t* table_out, int32_t* lens_out, void* workspace, size_t ws_bytes, int32_t* dev_status,
                       void* stream) {
  CacheGeom g;
  kvq3_status s = make_geom(desc, &g);
  if (s != KVQ3_OK) return s;
  if ((s = check_cache(g, cache, true)) != KVQ3_OK) return s;
  if (!cache->page_table || !src || !new_lens || !table_out || !lens_out) return KVQ3_ERR_INVALID_ARG;
  // the inputs are read while the outputs are written
  auto apart = [](const int32_t* a, int64_t na, const int32_t* b, int64_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x + na * 4 <= y || y + nb * 4 <= x;
  };
  const int64_t n = g.batch, cells = (int64_t)g.batch * g.max_pages;
  for (const int32_t* in : {cache->seq_lens, src, new_lens})
    if (!apart(lens_out, n, in, n) || !apart(table_out, cells, in, n)) return KVQ3_ERR_INVALID_ARG;
  if (!apart(lens_out, n, cache->page_table, cells) || !apart(table_out, cells, cache->page_table, cells) ||
      !apart(table_out, cells, lens_out, n))
    return KVQ3_ERR_INVALID_ARG;
  if (g.num_pages >= ((int64_t)1 << 31)) return KVQ3_ERR_UNSUPPORTED;
  const RemapWs ws = remap_layout(g, workspace);
  if (!workspace || ws_bytes < ws.bytes || reinterpret_cast<uintptr_t>(workspace) % 256) return KVQ3_ERR_WORKSPACE;
  const int64_t copies = (int64_t)g.batch * 2 * g.hkv;   // records that may be copied
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kMapCluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kMapThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  if (g.batch <= kSmallRows && (int64_t)g.batch * g.max_pages <= kSmallEntries && g.num_pages <= kSmallPages) {
    cfg.gridDim = dim3((unsigned)std::min<int64_t>(std::max(1, sm_count()), (copies * kCopyPieces + 31) / 32));
    cfg.numAttrs = 1;
    return cuda_status(cudaLaunchKernelEx(&cfg, remap_small_kernel, g, static_cast<uint8_t*>(cache->pool),
                                          cache->page_table, cache->seq_lens, src, new_lens, table_out, lens_out,
                                          dev_status));
  }
  cfg.gridDim = dim3(kMapCluster);
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, remap_kernel, g, cache->page_table, cache->seq_lens, src, new_lens, table_out, lens_out, ws,
                         dev_status) != cudaSuccess)
    return KVQ3_ERR_CUDA;
  cfg.gridDim = dim3((unsigned)std::min<int64_t>(copies, (int64_t)std::max(1, sm_count()) * 8));
  cfg.blockDim = dim3(256);
  cfg.numAttrs = 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, remap_copy_kernel, g, static_cast<uint8_t*>(cache->pool),
                                        static_cast<const int4*>(ws.copies), dev_status));
}

kvq3_status kvq3_compact(const kvq3_cache_desc* desc, const kvq3_cache* cache, const int32_t* src_seq,
                         const int32_t* dst_seq, int32_t n_seq, const int32_t* keep, const int32_t* n_keep,
                         int32_t keep_stride, int32_t* dev_status, void* stream) {
  CacheGeom g;
  kvq3_status s = make_geom(desc, &g);
  if (s != KVQ3_OK) return s;
  if ((s = check_cache(g, cache, true)) != KVQ3_OK) return s;
  if (n_seq < 0 || keep_stride < 0) return KVQ3_ERR_INVALID_ARG;
  if (n_seq == 0 || keep_stride == 0) return KVQ3_OK;
  if (!src_seq || !dst_seq || !keep || !n_keep) return KVQ3_ERR_INVALID_ARG;
  const int64_t units = (int64_t)n_seq * g.hkv, tiles = ((int64_t)keep_stride + kKeepTile - 1) / kKeepTile;
  if (units >= ((int64_t)1 << 31) / tiles) return KVQ3_ERR_UNSUPPORTED;   // one CTA per tile
  const CompactArgs a{cache, src_seq, dst_seq, keep, n_keep, units, keep_stride, dev_status,
                      static_cast<cudaStream_t>(stream)};
  switch (g.d) {
    case 64: return cuda_status(compact_by_codes<64>(g, a));
    case 128: return cuda_status(compact_by_codes<128>(g, a));
    case 256: return cuda_status(compact_by_codes<256>(g, a));
  }
  return KVQ3_ERR_UNSUPPORTED;
}

}  // extern "C"
