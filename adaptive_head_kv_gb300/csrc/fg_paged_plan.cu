// Paged 8-bit caches: layout of the prompt's caches, the decode work list and
// the coding of the kept prompt rows (Model Tells You What to Discard, Method:
// K_C, V_C = f(K, V, C), with rows of 8 bits in pages).
#include "fg_paged.cuh"

namespace fg {
namespace {

// Layout and list are single-CTA scans, made once a prompt.  Measured (a call of
// fastgen_paged_plan and of fastgen_paged_schedule, which wait for the result):
// 1024 caches 50 and 29 us, 8192 caches 128 and 51 us, 40960 caches 386 and 153
// us.
constexpr int kPlanThreads = 1024;

// One CTA: exclusive scans over the caches of their prompt pages and table
// entries.  A cache's entries hold room for `reserve` more rows; the first
// page of a cache is left in its first entry for the fill kernel.
__global__ void __launch_bounds__(kPlanThreads) paged_plan_kernel(
    const int2* __restrict__ cinfo, int G, int w, int reserve, fg_paged_desc* __restrict__ caches,
    int32_t* __restrict__ rows, int32_t* __restrict__ table, int32_t* __restrict__ next_page,
    long long* __restrict__ totals) {
  __shared__ long long scr[33];
  long long page_base = 0, entry_base = 0;
  for (int base = 0; base < G; base += blockDim.x) {
    const int c = base + threadIdx.x;
    long long pages = 0, entries = 0;
    int policy = 0, n_static = 0, wg = 0, seg = 0, ring = 0;
    if (c < G) {
      policy = cinfo[c].x;
      n_static = cinfo[c].y;
      wg = policy == FG_POLICY_SPFL ? w : 0;
      seg = max(1, cdiv(n_static + reserve, kPageRows));
      ring = cdiv(wg, kPageRows);
      pages = cdiv(n_static, kPageRows) + ring;
      entries = seg + ring;
    }
    long long ptot, etot;
    const long long p0 = page_base + block_exclusive_scan(pages, scr, &ptot);
    const long long e0 = entry_base + block_exclusive_scan(entries, scr, &etot);
    if (c < G) {
      fg_paged_desc d;
      d.policy = policy;
      d.w = wg;
      d.first_page = (int)e0;
      d.max_pages = seg;
      d.ring_page = (int)e0 + seg;
      d.ring_pages = ring;
      caches[c] = d;
      rows[c] = n_static;
      table[e0] = (int)p0;
    }
    page_base += ptot;
    entry_base += etot;
  }
  if (threadIdx.x == 0) {
    *next_page = (int)page_base;
    totals[0] = page_base;
    totals[1] = entry_base;  // every entry filled
    totals[2] = entry_base;
  }
}

// One warp per cache: its prompt pages in order, -1 where it may grow.
__global__ void __launch_bounds__(256) paged_fill_kernel(const fg_paged_desc* __restrict__ caches,
                                                         const int32_t* __restrict__ rows, int G,
                                                         int32_t* __restrict__ table) {
  const int c = blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (c >= G) return;
  const fg_paged_desc d = caches[c];
  const int now = cdiv(rows[c], kPageRows);
  const int page = table[d.first_page];
  __syncwarp();  // every lane has read the first entry before it is overwritten
  for (int i = lane; i < d.max_pages; i += 32) table[d.first_page + i] = i < now ? page + i : -1;
  for (int i = lane; i < d.ring_pages; i += 32) table[d.ring_page + i] = page + now + i;
}

// Pages of a cache that a decode step reads: its never-evicted segment's (at
// least one) and its ring's.  Descriptors the plan did not write may say
// anything: what lies past the table is not counted, nor a ring of more than max_w slots.
__device__ __forceinline__ int2 cache_pages(const fg_paged_desc& d, int rows, int max_w,
                                            int table_len) {
  const int seg = min(max(d.max_pages, 0), table_len), ring = min(max(d.ring_pages, 0), table_len);
  return make_int2(max(1, min(cdiv(max(rows, 0), kPageRows), seg)),
                   min(cdiv(ring_slots(d, max_w), kPageRows), ring));
}

// One CTA: how the decode step is cut into items.
//
// Small steps: every cache on its own, in equal items of at most kItemPages
// pages with a thread block each, for the shortest chain.  Larger ones: the
// caches' pages end to end, each cache led by item_cost pages' worth for what
// an item costs beside its pages, cut into equal lengths for a whole number
// of waves of resident thread blocks, so that no wave is part empty; a block
// takes the one or more items that fall in its length.
// ranges[c] = (first item, items, start of the cache end to end, length or 0).
// What an item costs grows with the queries of a group, whose sums the warps
// merge: fitted to thread blocks' times, 3.1 pages' worth for one query, 4.2
// for 4, 6 to 7 for 8 (d = 128).
int item_cost(int R) { return 3 + R / 2; }
constexpr int kLengthTarget = 128; // pages a thread block takes in a wave, about

__global__ void __launch_bounds__(kPlanThreads) paged_schedule_kernel(
    const fg_paged_desc* __restrict__ caches, const int32_t* __restrict__ rows, int G, int max_w,
    int table_len, int slots, int item_cost, int4* __restrict__ ranges,
    long long* __restrict__ totals) {
  __shared__ long long scr[33];
  long long small = 0, cost = 0;
  for (int base = 0; base < G; base += blockDim.x) {
    const int c = base + threadIdx.x;
    long long items = 0, pages = 0, tot;
    if (c < G) {
      const int2 p = cache_pages(caches[c], rows[c], max_w, table_len);
      pages = (long long)p.x + p.y + item_cost;
      items = ((long long)p.x + p.y + kItemPages - 1) / kItemPages;
    }
    block_exclusive_scan(items, scr, &tot);
    small += tot;
    block_exclusive_scan(pages, scr, &tot);
    cost += tot;
  }
  long long len = 0;
  if (small > 2LL * slots) {
    const long long wave = (long long)slots * kLengthTarget;
    const long long waves = max(1LL, (cost + wave / 2) / wave);
    len = (cost + slots * waves - 1) / (slots * waves);
  }
  long long item_base = 0, cost_base = 0;
  for (int base = 0; base < G; base += blockDim.x) {
    const int c = base + threadIdx.x;
    long long items = 0, pages = 0, tot;
    if (c < G) {
      const int2 p = cache_pages(caches[c], rows[c], max_w, table_len);
      pages = (long long)p.x + p.y;
    }
    const long long span = c < G ? pages + item_cost : 0;
    const long long at = cost_base + block_exclusive_scan(span, scr, &tot);
    cost_base += tot;
    if (c < G)
      items = len > 0 ? (at + span - 1) / len - at / len + 1
                      : (pages + kItemPages - 1) / kItemPages;
    const long long first = item_base + block_exclusive_scan(items, scr, &tot);
    item_base += tot;
    if (c < G)
      ranges[c] = make_int4((int)min(first, 0x7fffffffLL), (int)items,
                            (int)min(at, 0x7fffffffLL), (int)len);
  }
  if (threadIdx.x == 0) {
    totals[3] = cost > 0x7fffffffLL ? -1 : item_base;
    totals[4] = len > 0 ? (cost + len - 1) / len : item_base;
  }
}

// One warp per cache: its items, and where they begin a thread block.
__global__ void __launch_bounds__(256) paged_items_kernel(
    const fg_paged_desc* __restrict__ caches, const int32_t* __restrict__ rows, int G, int max_w,
    int table_len, int item_cost, const int4* __restrict__ ranges, int max_work,
    PagedItem* __restrict__ items, int32_t* __restrict__ cta_first,
    const long long* __restrict__ totals) {
  const int c = blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (c >= G || totals[3] < 0 || totals[3] > max_work || totals[4] > max_work) return;
  const int4 r = ranges[c];
  const int2 p = cache_pages(caches[c], rows[c], max_w, table_len);
  const int pages = p.x + p.y;
  for (int i = lane; i < r.y; i += 32) {
    long long p0, p1;
    if (r.w > 0) {
      const long long k = r.z / r.w + i, start = (long long)r.z + item_cost;
      p0 = max(0LL, k * r.w - start);
      p1 = min((long long)pages, (k + 1) * r.w - start);
      if (p1 < p0) p1 = p0 = 0;  // the length ends within the cache's lead
      if (i > 0 || r.z % r.w == 0) cta_first[k] = r.x + i;
    } else {
      p0 = (long long)i * pages / r.y;
      p1 = (long long)(i + 1) * pages / r.y;
      cta_first[r.x + i] = r.x + i;
    }
    PagedItem it;
    it.cache = c;
    it.last = p0 <= p.x - 1 && p.x - 1 < p1;
    it.seg0 = (int)min(p0, (long long)p.x);
    it.seg1 = (int)min(p1, (long long)p.x);
    it.ring0 = (int)max(p0 - p.x, 0LL);
    it.ring1 = (int)max(p1 - p.x, 0LL);
    items[r.x + i] = it;
  }
  if (c == G - 1 && lane == 0) cta_first[totals[4]] = (int)totals[3];
}

// ---------------------------------------------------------------------------
// Coding the kept rows.  One CTA per (cache, a chunk of the rows of
// its never-evicted segment or of its ring).  A segment's CTA first finds the
// positions of its rows: every thread turns kScanPer keep codes into bits, and
// a scan of their counts ranks them.  Then each warp takes the K or the V of a
// block of 16 rows: the rows in registers (one pass over the data), the
// block's largest magnitude, the exponent, the codes.  Bound by HBM: 2 * eb + 2
// bytes a value.  Measured (device time; bf16, d = 128, 2048 positions): 256
// caches (192 MB) 37 us, 5.2 TB/s; 4096 caches (3.1 GB) 478 us, 6.4 TB/s.
//
// A CTA has as many threads as its chunk has rows: 128, so that one CTA's
// search hides behind its neighbours' rows, or 512 where a long prompt or a
// large group makes the search (every CTA reads the codes before its chunk)
// outweigh 128 rows.  Measured with 128 / 512, groups of 1 and 8: 2048
// positions 36.7 / 39.8 us, 16384 38.2 / 37.3, 32768 25.5 / 22.1; 8 x 4096
// 24.9 / 23.6, 8 x 8192 29.2 / 24.3, 8 x 16384 39.1 / 25.0.
constexpr int kLongSearch = 12288;  // codes of a group
constexpr int kScanPer = 32;  // positions per thread and scan step

// Bit i: byte i of the 16 bytes at p is FG_KEEP_STATIC.  p is 16-byte aligned
// and may reach over the ends of the buffer [lo, hi), of which nothing else is
// read.
__device__ __forceinline__ uint32_t static_bits16(const uint8_t* p, const uint8_t* lo,
                                                  const uint8_t* hi) {
  uint32_t bits = 0;
  if (p >= lo && p + 16 <= hi) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t s = __vcmpeq4(w[k], 0x01010101u * FG_KEEP_STATIC) & 0x01010101u;
      bits |= ((s * 0x01020408u) >> 24) << (4 * k);  // byte i's flag to bit i
    }
  } else {
    for (int k = 0; k < 16; ++k)
      if (p + k >= lo && p + k < hi && p[k] == FG_KEEP_STATIC) bits |= 1u << k;
  }
  return bits;
}

// Bit i: code at p + i is FG_KEEP_STATIC, for 32 codes at any address.
__device__ __forceinline__ uint32_t static_bits32(const uint8_t* p, const uint8_t* lo,
                                                  const uint8_t* hi) {
  const int s = (int)(reinterpret_cast<uintptr_t>(p) & 15);
  const uint8_t* q = p - s;
  const uint32_t w = static_bits16(q, lo, hi) | static_bits16(q + 16, lo, hi) << 16;
  return s ? __funnelshift_r(w, static_bits16(q + 32, lo, hi), s) : w;
}

// Codes a block of 16 rows: src[i] is the prompt position of row i, or -1.
template <typename T, int D>
__device__ __forceinline__ void code_block(const T* __restrict__ X, const int* src, uint8_t* dst,
                                           int8_t* exp_dst) {
  constexpr int E = Vec16<T>::kElems;
  constexpr int LPR = D / E;              // lanes per row
  constexpr int RPI = 32 / LPR;           // rows per load
  constexpr int NI = kBlockRows / RPI;
  const int lane = threadIdx.x & 31;
  const int sub = lane / LPR, gl = lane % LPR;
  uint4 x[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int j = src[i * RPI + sub];
    x[i] = j >= 0 ? ldg_stream(X + (size_t)j * D + gl * E) : make_uint4(0, 0, 0, 0);
  }
  const int e = block_exponent(__reduce_max_sync(0xffffffffu, lane_top(x, (const T*)nullptr)));
  const float inv = pow2f(-e);
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int r = i * RPI + sub;
    if (src[r] >= 0) code16(x[i], inv, dst + (size_t)r * D + gl * E, (const T*)nullptr);
  }
  if (lane == 0) *exp_dst = (int8_t)e;
}

// CTAs of `chunk` threads that an SM is to hold, by the bytes of a row: a warp's
// 16 rows take as many registers a lane as a row has 8 bytes.  With / without
// the bound: 128 bytes (bf16, d = 64; 128 threads) 41.4 / 45.6 us, 256 bytes
// 478 / 489 us (4096 caches; 512 threads, 32768 positions 22.1 / 23.0); rows of
// 512 bytes would spill (65 / 55 us).
constexpr int compact_blocks(int row_bytes, int chunk) {
  return row_bytes > 256 ? 1 : chunk > 128 ? 2 : row_bytes > 128 ? 8 : 12;
}

template <typename T, int D, int kChunkRows>
__global__ void __launch_bounds__(kChunkRows, compact_blocks(D * sizeof(T), kChunkRows))
    compact_q8_kernel(
    const T* __restrict__ K, const T* __restrict__ V, const uint8_t* __restrict__ keep, int n,
    int G, int H, int R, int seg_chunks, int chunks, const PagedArgs a) {
  constexpr int kCodeThreads = kChunkRows;
  __shared__ int src[kChunkRows];
  __shared__ int scr[33];
  const int c = blockIdx.x / chunks;
  int chunk = blockIdx.x % chunks;
  griddep_wait();
  griddep_launch_dependents();
  const fg_paged_desc d = a.caches[c];
  const int rows = a.rows[c];
  const bool ring = chunk >= seg_chunks;
  if (ring) chunk -= seg_chunks;
  const int lo = chunk * kChunkRows;
  const int w = ring_slots(d, a.max_w), total = ring ? w : live_rows(d, rows);
  const bool first = !ring && chunk == 0;
  if (first && threadIdx.x == 0 && (rows != total || rows > n || d.w != w))
    atomicOr(a.dev_err, kErrInvalid);
  if (lo >= total && !first) return;
  const int hi = min(lo + kChunkRows, total);
  const int Hkv = H / R;
  const size_t g0 = (size_t)(c / Hkv) * H + (size_t)(c % Hkv) * R;  // first query head
  src[threadIdx.x] = -1;
  __syncthreads();
  if (!ring) {
    const uint8_t* end = keep + (size_t)G * n;
    int seen = 0;  // never-evicted rows before the step
    // (the CTA of the last rows looks at the whole prompt: every kept position has a row)
    for (int base = 0; base < n && (seen < hi || hi == total); base += kCodeThreads * kScanPer) {
      const int j0 = base + threadIdx.x * kScanPer;
      uint32_t bits = 0;  // any member keeps the position so
      if (j0 < n) {
        for (int m = 0; m < R; ++m)
          bits |= static_bits32(keep + (g0 + m) * (size_t)n + j0, keep, end);
        if (n - j0 < kScanPer) bits &= (1u << (n - j0)) - 1;
      }
      int tot;
      int rank = seen + block_exclusive_scan(__popc(bits), scr, &tot);
      if (rank < hi && rank + __popc(bits) > lo)
        while (bits) {
          const int k = __ffs(bits) - 1;
          bits &= bits - 1;
          if (rank >= lo && rank < hi) src[rank - lo] = j0 + k;
          ++rank;
        }
      seen += tot;
    }
    if (hi == total && seen != total && threadIdx.x == 0) atomicOr(a.dev_err, kErrInvalid);
  } else {
    // slot s holds the one position of [n - w, n) that is s modulo w
    for (int s = lo + threadIdx.x; s < hi; s += kCodeThreads) {
      const int back = (n - 1 - s) % w;
      const int j = n - 1 - (back < 0 ? back + w : back);
      int st = 0, win = 0;
      for (int m = 0; m < R && j >= 0; ++m) {
        const int code = keep[(g0 + m) * (size_t)n + j];
        st |= code == FG_KEEP_STATIC;
        win |= code == FG_KEEP_WINDOW;
      }
      src[s - lo] = win && !st ? j : -1;
    }
  }
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int blocks = cdiv(hi - lo, kBlockRows);
  for (int task = warp; task < 2 * blocks; task += kCodeThreads / 32) {
    const int b = task >> 1, which = task & 1;
    const int row = lo + b * kBlockRows;
    const int page = ring ? page_at(a, d.ring_page, d.ring_pages, row / kPageRows)
                          : page_at(a, d.first_page, d.max_pages, row / kPageRows);
    if (page < 0) {
      if (lane == 0) atomicOr(a.dev_err, kErrInvalid);
      continue;
    }
    const int r = row % kPageRows;
    const int* bs = src + b * kBlockRows;
    if (which == 0 && lane < kBlockRows && row + lane < hi && (ring || bs[lane] >= 0))
      a.pos[(size_t)page * kPageRows + r + lane] = bs[lane];
    code_block<T, D>((which ? V : K) + (size_t)c * n * D, bs,
                     (which ? a.vp : a.kp) + ((size_t)page * kPageRows + r) * D,
                     a.exps + ((size_t)page * kPageBlocks + r / kBlockRows) * 2 + which);
  }
}

template <typename T, int D, int kChunkRows>
cudaError_t run_compact_chunk(const ProfileDims& pd, const void* K, const void* V,
                           const uint8_t* keep, const PagedArgs& a, cudaStream_t s) {
  const int seg = cdiv(pd.n, kChunkRows), chunks = seg + cdiv(pd.w, kChunkRows);
  const long long grid = (long long)pd.Gkv * chunks;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  return launch_pdl(compact_q8_kernel<T, D, kChunkRows>, (unsigned)grid, kChunkRows, 0, s,
                    (const T*)K, (const T*)V, keep, pd.n, pd.G, pd.H, pd.R, seg, chunks, a);
}

template <typename T, int D>
cudaError_t run_compact_q8(const ProfileDims& pd, const void* K, const void* V,
                           const uint8_t* keep, const PagedArgs& a, cudaStream_t s) {
  return (long long)pd.n * pd.R > kLongSearch ? run_compact_chunk<T, D, 512>(pd, K, V, keep, a, s)
                            : run_compact_chunk<T, D, 128>(pd, K, V, keep, a, s);
}

}  // namespace

cudaError_t launch_paged_plan(int Gkv, int w, int reserve, const int2* cinfo, fg_paged_desc* caches,
                              int32_t* rows, int32_t* table, int32_t* next_page,
                              long long* totals, cudaStream_t s) {
  paged_plan_kernel<<<1, kPlanThreads, 0, s>>>(cinfo, Gkv, w, reserve, caches, rows, table,
                                               next_page, totals);
  paged_fill_kernel<<<cdiv(Gkv, 8), 256, 0, s>>>(caches, rows, Gkv, table);
  return cudaGetLastError();
}

cudaError_t launch_paged_schedule(int Gkv, int R, const fg_paged_desc* caches, const int32_t* rows,
                                  int max_w, int table_len, int max_work, int slots, int4* ranges,
                                  PagedItem* items, int32_t* cta_first, long long* totals,
                                  cudaStream_t s) {
  paged_schedule_kernel<<<1, kPlanThreads, 0, s>>>(caches, rows, Gkv, max_w, table_len, slots,
                                                   item_cost(R), ranges, totals);
  paged_items_kernel<<<cdiv(Gkv, 8), 256, 0, s>>>(caches, rows, Gkv, max_w, table_len,
                                                  item_cost(R), ranges, max_work, items, cta_first,
                                                  totals);
  return cudaGetLastError();
}

cudaError_t launch_compact_q8(const ProfileDims& pd, const void* K, const void* V,
                              const uint8_t* keep, const PagedArgs& a, cudaStream_t s) {
  if (pd.dtype == FG_FP32)
    return pd.d == 64 ? run_compact_q8<float, 64>(pd, K, V, keep, a, s)
                      : run_compact_q8<float, 128>(pd, K, V, keep, a, s);
  return pd.d == 64 ? run_compact_q8<__nv_bfloat16, 64>(pd, K, V, keep, a, s)
                    : run_compact_q8<__nv_bfloat16, 128>(pd, K, V, keep, a, s);
}

}  // namespace fg
