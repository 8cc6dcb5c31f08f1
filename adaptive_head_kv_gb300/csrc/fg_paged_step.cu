// fastgen_decode_attn_q8_ex: the split kernel of fg_paged_decode.cuh over every
// sequence's own caches, the join of its partial results with those of the
// shared caches (fg_prefix.cu), and the rows' weights.
//
// A softmax over several sets of rows: each set gives a query its maximum m,
// its sum l = sum_j 2^(s_j - m) and its mean y of the values, and
//   M = max m,  L = sum l 2^(m - M),  out = sum y l 2^(m - M) / L.
// With M and L final a row's weight is 2^(s - M) / L: the split kernel leaves the
// scores of the segment rows behind, and weigh_kernel adds the group's weights.
#include "fg_paged_decode.cuh"

namespace fg {
namespace {

// The parts that a query's result is made of, kAhead at a time: maximum, sum and kPer values of the
// mean of each.
template <int kAhead, int kPer>
struct Joined {
  float M = kNoScore, L = 0.f, acc[kPer] = {};
  __device__ __forceinline__ void add(const float (&m)[kAhead], const float (&l)[kAhead],
                                      const float (&x)[kAhead][kPer]) {
    float Mn = M;
#pragma unroll
    for (int j = 0; j < kAhead; ++j) Mn = fmaxf(Mn, m[j]);
    // 2^(m - Mn) as the square of h: a weight below what a float holds may still meet values
    // that make it count
    const float fh = exp2f(0.5f * (M - Mn));
    float h[kAhead], Ln = L * fh * fh;
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      h[j] = exp2f(0.5f * (m[j] - Mn));
      Ln = fmaf(l[j] * h[j], h[j], Ln);
    }
    // means of means: nothing passes the largest value
    const float r = Ln == 0.f ? 0.f : 1.f / Ln;
#pragma unroll
    for (int k = 0; k < kPer; ++k) acc[k] = acc[k] * (L * r) * fh * fh;
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
#pragma unroll
      for (int k = 0; k < kPer; ++k) acc[k] = fmaf(x[j][k] * (l[j] * r) * h[j], h[j], acc[k]);
    L = Ln;
    M = Mn;
  }
};

// The count of a cache's rows after the step (all lanes of a warp call, with the same cache).
__device__ __forceinline__ int rows_after(const PagedArgs& a, const StepArgs& n,
                                          const fg_paged_desc& hd, int had, bool special,
                                          bool punct) {
  const bool stored = n.k_new && joins_static(hd.policy, special, special || punct) && had >= 0 &&
                      page_at(a, hd.first_page, hd.max_pages, had / kPageRows) >= 0;
  return had + (stored ? 1 : 0);
}

// Without shared caches: one warp per query head.
constexpr int kCombineWarps = 4;

template <typename T, int D>
__global__ void __launch_bounds__(kCombineWarps * 32)
    step_combine_kernel(const PagedArgs a, const StepArgs n, int G, int H, int R, int HLkv) {
  constexpr int PER = D / 32, kAhead = 4;
  const int gq = blockIdx.x * kCombineWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const bool in = gq < G;
  const int c = in ? kv_head(gq, H, R) : 0, qi = (gq % H) % R, b = c / HLkv;
  int4 range = a.ranges[c];
  range.x = max(0, min(range.x, a.n_work));
  range.y = min(range.y, a.n_work - range.x);
  const bool listed = same_list(a);
  griddep_wait();
  griddep_launch_dependents();
  const LaneSet special(n.special, n.ns), punct(n.punct, n.np);
  if (!in || !listed) return;
  const fg_paged_desc hd = a.caches[c];
  const int t = n.pos[b], had = a.rows[c], tau = n.k_new ? n.ids[b] : 0;
  if (t < 0) {
    if (qi == 0 && lane == 0) a.rows_out[c] = had;
    return;
  }
  Joined<kAhead, PER> o;
  for (int i0 = 0; i0 < range.y; i0 += kAhead) {
    float m[kAhead], l[kAhead], x[kAhead][PER];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const bool ok = i0 + j < range.y;
      const size_t slot = ((size_t)range.x + i0 + j) * R + qi;
      const float2 ml = ok ? *reinterpret_cast<const float2*>(n.part_ml + 2 * slot)
                           : make_float2(kNoScore, 0.f);
      m[j] = ml.x;
      l[j] = ml.y;
      if (ok) load_row<PER>(n.part_acc + slot * D, x[j]);
      else
#pragma unroll
        for (int k = 0; k < PER; ++k) x[j][k] = 0.f;
    }
    o.add(m, l, x);
  }
#pragma unroll
  for (int k = 0; k < PER; ++k) store_out((T*)n.out + (size_t)gq * D + lane * PER + k, o.acc[k]);
  if (n.head_ml && lane == 0)
    *reinterpret_cast<float2*>(n.head_ml + 2 * (size_t)gq) = make_float2(o.M, o.L);
  if (qi == 0) {
    const int now = rows_after(a, n, hd, had, special.has(tau), punct.has(tau));
    if (lane == 0) a.rows_out[c] = now;
  }
}

// With shared caches: their parts hold the queries of a tile side by side, so a lane takes a query
// and a warp 4 kFours dimensions of 32 of them.  kSplit warps share the parts of these (where few
// caches leave many parts to each), eight warps a block.  What a warp asks for before the values (the
// sequence, its list's items, the parts) is a chain of loads, which bounds it (16384 queries of 4
// parts, 37 MB, 18 us): it takes more dimensions where there are warps enough (20 us with four).
constexpr int kJoinWarps = 8;

template <typename T, int D, int kSplit, int kFours>
__global__ void __launch_bounds__(kJoinWarps * 32)
    step_join_kernel(const PagedArgs a, const StepArgs n, const PrefixParts px, int H, int R,
                     int HL) {
  constexpr int kAhead = 4, kQuads = kJoinWarps / kSplit, kPer = 4 * kFours;
  constexpr int kSlices = D / kPer / kQuads;
  __shared__ float sm[kSplit > 1 ? kSplit - 1 : 1][kQuads][kPer + 2][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int split = warp / kQuads, dq = warp % kQuads;
  const int d4 = (blockIdx.x % kSlices * kQuads + dq) * kFours;
  const int quads = cdiv(px.rows, 32);  // of 32 queries, of a tile
  const int rest = blockIdx.x / kSlices, quad = rest % quads, unit = rest / quads;
  const int pc = unit / px.tiles, tile = unit % px.tiles;
  const int row = quad * 32 + lane, j = tile * kPrefixTile + row, b = j / R, qi = j % R;
  const bool in = row < px.rows && j < px.nq;
  const int c = in ? b * px.caches + pc : 0;  // the query's own cache
  const size_t g =
      in ? (size_t)b * HL + (size_t)(pc / (H / R)) * H + (size_t)(pc % (H / R)) * R + qi : 0;
  int4 range = a.ranges[c];
  range.x = max(0, min(range.x, a.n_work));
  range.y = min(range.y, a.n_work - range.x);
  const bool listed = same_list(a);
  griddep_wait();
  griddep_launch_dependents();
  if (!listed) return;
  const int t = in ? n.pos[b] : -1;
  // of every thread block that had pages of the unit one part, or two where the block's two streams
  // took its pages in turns
  int parts = 0;
  const int streams = px.pair ? 1 : 2, grp = px.pair ? tile / 2 : tile;
  const long long c0 = px.cum[pc], pages = px.cum[pc + 1] - c0;
  size_t part = 0;  // the first one
  if (pages > 0) {
    const long long all = px.cum[px.caches] * px.groups;
    const int ctas = prefix_ctas(all, px.ctas);
    const long long x = c0 * px.groups + grp * pages;
    const int i0 = prefix_cta(all, ctas, x), i1 = prefix_cta(all, ctas, x + pages - 1);
    parts = (i1 - i0 + 1) * streams;
    part = ((size_t)i0 + (size_t)pc * px.groups + grp) * 2 + (px.pair ? tile & 1 : 0);
  }
  Joined<kAhead, kPer> o;
  const int most = parts + __reduce_max_sync(0xffffffffu, t >= 0 ? range.y : 0);
  for (int i0 = split; i0 < most; i0 += kAhead * kSplit) {
    float m[kAhead], l[kAhead], x[kAhead][kPer];
    float2 ml[kAhead];
    float4 v[kAhead][kFours];
#pragma unroll
    for (int z = 0; z < kAhead; ++z) {
      const int i = i0 + z * kSplit;
      const bool shared = i < parts, ok = t >= 0 && i < parts + range.y;
      const size_t p = part + (size_t)i * (2 / streams);
      const size_t slot = shared ? p * px.rows + row : ((size_t)range.x + i - parts) * R + qi;
      ml[z] = ok ? *reinterpret_cast<const float2*>((shared ? px.ml : n.part_ml) + 2 * slot)
                 : make_float2(kNoScore, 0.f);
#pragma unroll
      for (int f = 0; f < kFours; ++f)
        v[z][f] = ok ? *reinterpret_cast<const float4*>(
                           shared ? px.acc + ((p * (D / 4) + d4 + f) * px.rows + row) * 4
                                  : n.part_acc + slot * D + (d4 + f) * 4)
                     : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int z = 0; z < kAhead; ++z) {
      m[z] = ml[z].x;
      l[z] = ml[z].y;
      const bool some = l[z] != 0.f;  // (a part without a row has no values)
#pragma unroll
      for (int f = 0; f < kFours; ++f) {
        x[z][4 * f] = some ? v[z][f].x : 0.f;
        x[z][4 * f + 1] = some ? v[z][f].y : 0.f;
        x[z][4 * f + 2] = some ? v[z][f].z : 0.f;
        x[z][4 * f + 3] = some ? v[z][f].w : 0.f;
      }
    }
    o.add(m, l, x);
  }
  if constexpr (kSplit > 1) {
    if (split > 0) {
      float(&s)[kPer + 2][32] = sm[split - 1][dq];
#pragma unroll
      for (int k = 0; k < kPer; ++k) s[k][lane] = o.acc[k];
      s[kPer][lane] = o.M;
      s[kPer + 1][lane] = o.L;
    }
    __syncthreads();
    Joined<kSplit - 1, kPer> all;
    all.M = o.M;
    all.L = o.L;
    float m[kSplit - 1], l[kSplit - 1], x[kSplit - 1][kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) all.acc[k] = o.acc[k];
#pragma unroll
    for (int z = 0; z < kSplit - 1; ++z) {
      float(&s)[kPer + 2][32] = sm[z][dq];
#pragma unroll
      for (int k = 0; k < kPer; ++k) x[z][k] = s[k][lane];
      m[z] = s[kPer][lane];
      l[z] = s[kPer + 1][lane];
    }
    all.add(m, l, x);
#pragma unroll
    for (int k = 0; k < kPer; ++k) o.acc[k] = all.acc[k];
    o.M = all.M;
    o.L = all.L;
  }
  // a query's dimensions of this block side by side in memory: the lanes of a warp take fours of
  // the block's dimensions of the same queries
  constexpr int kOut = kQuads * kFours;
  __shared__ float4 sm_out[32][kOut + 1];
  __shared__ long long sm_at[32];
  if (split == 0) {
#pragma unroll
    for (int f = 0; f < kFours; ++f)
      sm_out[lane][dq * kFours + f] =
          make_float4(o.acc[4 * f], o.acc[4 * f + 1], o.acc[4 * f + 2], o.acc[4 * f + 3]);
    if (dq == 0) sm_at[lane] = t >= 0 ? (long long)g : -1;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 32 * kOut; i += kJoinWarps * 32) {
    const float4 v = sm_out[i / kOut][i % kOut];
    const long long at = sm_at[i / kOut];
    T* out = (T*)n.out + at * D + (blockIdx.x % kSlices * kOut + i % kOut) * 4;
    if (at < 0) continue;
    if constexpr (sizeof(T) == 4)
      *reinterpret_cast<float4*>(out) = v;
    else
      *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
  }
  if (d4 != 0 || split != 0) return;
  if (t >= 0 && n.head_ml) *reinterpret_cast<float2*>(n.head_ml + 2 * g) = make_float2(o.M, o.L);
  const LaneSet special(n.special, n.ns), punct(n.punct, n.np);
  const int tau = n.k_new && t >= 0 ? n.ids[b] : 0;
  const bool s = special.has_mine(tau), p = punct.has_mine(tau);
  if (in && qi == 0) {
    const int had = a.rows[c];
    a.rows_out[c] = t < 0 ? had : rows_after(a, n, a.caches[c], had, s, p);
  }
}

template <typename T, int D, int kSplit, int kFours>
cudaError_t run_join(const ProfileDims& pd, const PagedArgs& a, const StepArgs& n,
                     const PrefixParts& px, cudaStream_t s) {
  const long long grid =
      (long long)px.caches * px.tiles * cdiv(px.rows, 32) * (D / 4 / kFours / (kJoinWarps / kSplit));
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  return launch_pdl(step_join_kernel<T, D, kSplit, kFours>, (unsigned)grid, kJoinWarps * 32, 0, s, a,
                    n, px, pd.H, pd.R, pd.HL);
}

// Adds the step's weights to the rows of a work item's part of the segment: a warp takes pages in
// turns, a lane two rows of each.  It reads R scores of a row and reads and writes its weight so far,
// 4 R + 8 bytes beside the 2 d of its codes: 11 of 68 us (192 caches of 8192 positions, groups of
// 8), which the chain item, table, row bounds more than their bytes (26 MB, 4 us at HBM's rate).
constexpr int kWeighWarps = 8;

template <int R>
__global__ void __launch_bounds__(kWeighWarps * 32)
    weigh_kernel(const PagedArgs a, const StepArgs n, int Gkv, int H, int HLkv) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const PagedItem it = a.items[blockIdx.x];
  const bool listed = same_list(a);
  griddep_wait();
  griddep_launch_dependents();
  const int c = it.cache;
  if (!listed || (unsigned)c >= (unsigned)Gkv) return;
  const size_t g0 = (size_t)(c / (H / R)) * H + (size_t)(c % (H / R)) * R;
  const int t = n.pos[c / HLkv], now = a.rows_out[c];
  const fg_paged_desc hd = a.caches[c];
  float M[R], r[R];
#pragma unroll
  for (int q = 0; q < R; ++q) {
    const float2 ml = *reinterpret_cast<const float2*>(n.head_ml + 2 * (g0 + q));
    M[q] = ml.x;
    r[q] = ml.y == 0.f ? 0.f : 1.f / ml.y;
  }
  if (t < 0) return;
  const int rows = live_rows(hd, now);
  const int end = it.last ? rows : (int)min((long long)rows, (long long)it.seg1 * kPageRows);
  constexpr int kAhead = R > 2 ? 1 : 2;
  for (int j = it.seg0 + warp; j * kPageRows < end; j += kAhead * kWeighWarps) {
    float s[kAhead][2][R];
    float2 w[kAhead];
    long long at[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int p = j + u * kWeighWarps, row = p * kPageRows + 2 * lane;
      const int page = row < end ? page_at(a, hd.first_page, hd.max_pages, p) : -1;
      at[u] = page < 0 ? -1 : (long long)page * kPageRows + 2 * lane;  // (flagged by the split kernel)
      if (at[u] < 0) continue;
      w[u] = *reinterpret_cast<const float2*>(n.row_w + at[u]);
      // two rows' scores lie side by side
      const float* x = n.row_sc + at[u] * R;
      if constexpr (R == 1) {
        const float2 y = *reinterpret_cast<const float2*>(x);
        s[u][0][0] = y.x;
        s[u][1][0] = y.y;
      } else {
#pragma unroll
        for (int k = 0; k < 2 * R; k += 4) {
          const float4 y = *reinterpret_cast<const float4*>(x + k);
          s[u][k / R][k % R] = y.x;
          s[u][(k + 1) / R][(k + 1) % R] = y.y;
          s[u][(k + 2) / R][(k + 2) % R] = y.z;
          s[u][(k + 3) / R][(k + 3) % R] = y.w;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (at[u] < 0) continue;
      float y[2] = {0.f, 0.f};
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int q = 0; q < R; ++q) y[h] = fmaf(ex2(s[u][h][q] - M[q]), r[q], y[h]);
      const int row = (j + u * kWeighWarps) * kPageRows + 2 * lane;
      // a pinned row stays pinned, also where a weight is NaN
      const float w0 = w[u].x == -FG_NEG_INF ? w[u].x : w[u].x + y[0];
      const float w1 = w[u].y == -FG_NEG_INF ? w[u].y : w[u].y + y[1];
      if (row + 1 < end)
        *reinterpret_cast<float2*>(n.row_w + at[u]) = make_float2(w0, w1);
      else
        n.row_w[at[u]] = w0;
    }
  }
}

__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

// Many small caches: a warp an item.  The split kernel's streaming warp opens one item after the
// other, a chain of dependent loads each, which its pages hide only where there are enough of them:
// 16384 caches of some 30 rows took 4.5 us an item of a block.  Here an SM's warps open a dozen
// items at a time and read each lane's operands where they lie; the arithmetic is the split kernel's,
// with keys and values in their own order.  Pages of a ring without a row that counts (rings behind
// a shared prompt begin empty) are passed over.  Those caches take 80 us: 1600 instructions an item, at
// a third of the schedulers' rate with the four warps each that registers leave room for.  (Warps that
// take over blocks not yet started: 85 us.)
constexpr int kSmallWarps = 1;  // (a block of four waits for its longest: 194 us, with one 181)

template <typename T, int D, bool kFold, int kMode>
__global__ void __launch_bounds__(kSmallWarps * 32, 16)
    q8_small_kernel(const PagedArgs a, const StepArgs n, int Gkv, int H, int R, int HLkv,
                    float sl2) {
  constexpr bool kWide = wide<T>(kFold, kMode), kTwo = kFold || kWide;
  constexpr int NQ = kFold ? 1 : 2;  // queries of a lane
  constexpr int PER = D / 32, KI = D / 64, PW = D / 32, MT = D / 16;
  constexpr int kQNext = (kFold ? 2 : 1) * D, kQTerm = (kFold ? 1 : kMaxR) * D;  // in f16
  constexpr int kQueries = kFold ? kMaxR / 2 : kMaxR;
  __shared__ __align__(16) uint16_t sm_q[kSmallWarps][kMaxR * D + (kWide ? kQTerm : 0)];
  __shared__ float sm_e[kSmallWarps][kMaxR];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  const int q0 = NQ * t4;  // the lane's first query
  const int wi = blockIdx.x * kSmallWarps + warp;
  const bool have = wi < a.n_work;
  const PagedItem it = a.items[have ? wi : 0];
  const bool listed = same_list(a);
  if (n.beside) {
    if (!start_beside()) return;
  } else {
    griddep_wait();
    griddep_launch_dependents();
  }
  if (!listed) {
    if (threadIdx.x == 0) atomicOr(a.dev_err, kErrInvalid);
    return;
  }
  if (!have) return;
  const int c = it.cache, b = c / HLkv;
  if ((unsigned)c >= (unsigned)Gkv) {
    if (lane == 0) atomicOr(a.dev_err, kErrInvalid);
    return;
  }
  // what opens an item is asked for together: the sequence, the cache, the queries, the new row
  const int t = n.pos[b], had = a.rows[c], tau = n.k_new ? n.ids[b] : 0;
  const fg_paged_desc hd = a.caches[c];
  const size_t g0 = (size_t)(c / (H / R)) * H + (size_t)(c % (H / R)) * R;
  float x[kQueries][PER], xk[PER], xv[PER];
#pragma unroll
  for (int qi = 0; qi < kQueries; ++qi)
    if (qi < R) load_row<PER>((const T*)n.q + (g0 + qi) * D, x[qi]);
#pragma unroll
  for (int k = 0; k < PER; ++k) xk[k] = xv[k] = 0.f;
  if (n.k_new) {
    load_row<PER>((const T*)n.k_new + (size_t)c * D, xk);
    load_row<PER>((const T*)n.v_new + (size_t)c * D, xv);
  }
  const LaneSet special(n.special, n.ns), punct(n.punct, n.np);
  if (t < 0) return;  // the sequence takes no part
  const int w = ring_slots(hd, a.max_w), old = live_rows(hd, had);
  if ((old != had || w != hd.w) && it.last && lane == 0) atomicOr(a.dev_err, kErrInvalid);
  const Put put = item_put(n, it, hd, special, punct, w, old, t, tau);
  int seg_end = it.last ? old : (int)min((long long)old, (long long)it.seg1 * kPageRows);
  const int ring_end = (int)min((long long)w, (long long)it.ring1 * kPageRows);
  // a page's number, exponents and which of its rows count, asked for a page ahead
  int page_next = -1;
  uint2 ex_next = make_uint2(0, 0);
  int2 p_next = make_int2(-1, -1);
  int n_seg = max(0, cdiv(seg_end - it.seg0 * kPageRows, kPageRows));
  const int n_ring =
      it.ring1 > it.ring0 ? max(0, cdiv(ring_end - it.ring0 * kPageRows, kPageRows)) : 0;
  auto ask = [&](int j) {
    page_next = -1;
    p_next = make_int2(-1, -1);
    if (j >= n_seg + n_ring) return;
    page_next = j < n_seg ? page_at(a, hd.first_page, hd.max_pages, it.seg0 + j)
                          : page_at(a, hd.ring_page, hd.ring_pages, it.ring0 + j - n_seg);
    if (page_next < 0) {
      if (lane == 0) atomicOr(a.dev_err, kErrInvalid);
      return;
    }
    ex_next = __ldcg(reinterpret_cast<const uint2*>(a.exps + (size_t)page_next * kPageBlocks * 2));
    if (j < n_seg) {  // its rows, on their way while what opens the item is looked up
      const int bytes = min(kPageRows, seg_end - (it.seg0 + j) * kPageRows) * D;
      for (int i = lane * 128; i < bytes; i += 32 * 128) {
        prefetch_l2(a.kp + (size_t)page_next * kPageRows * D + i);
        prefetch_l2(a.vp + (size_t)page_next * kPageRows * D + i);
      }
    } else {
      const int32_t* p = a.pos + (size_t)page_next * kPageRows + lane;
      p_next = make_int2(__ldcg(p), __ldcg(p + 32));
    }
  };
  int new_page = -1, new_k = 0, new_v = 0;
  if (put.at >= 0) {
    new_page = put_page(a, hd, put);
    __syncwarp();  // its entry is there
    if (new_page >= 0) {
      const int8_t* ex =
          a.exps + ((size_t)new_page * kPageBlocks + put.at % kPageRows / kBlockRows) * 2;
      new_k = ex[0];
      new_v = ex[1];
      if (!put.ring) {
        seg_end = put.at + 1;
        n_seg = max(0, cdiv(seg_end - it.seg0 * kPageRows, kPageRows));
      }
    }
  }
  ask(0);
  // the queries: rotated, divided by the power of two that brings the largest value to
  // [2^13, 2^14), as f16 (two terms: and what f16 loses, times 2^11)
  {
    float2 cs[PER];
    if (n.rope.rot > 0) {
      row_angles<PER>(cs, n.rope.rot, n.rope.style, [&](int p) {
        float2 y;
        rope_cos_sin((unsigned)t, n.rope.turns[p], y.x, y.y);
        return y;
      });
      if (put.at >= 0) rotate_row<PER>(xk, cs, n.rope.rot, n.rope.style);
    }
#pragma unroll
    for (int qi = 0; qi < kQueries; ++qi) {
      if (qi >= R) break;
      if (n.rope.rot > 0) rotate_row<PER>(x[qi], cs, n.rope.rot, n.rope.style);
      uint32_t top = 0;
#pragma unroll
      for (int k = 0; k < PER; ++k) top = max(top, finite_bits(x[qi][k]));
      top = __reduce_max_sync(0xffffffffu, top);
      const int eq = max(-110, (int)(top >> 23) - 127 - 13);
      const float inv = pow2f(-eq);
#pragma unroll
      for (int k = 0; k < PER; k += 2) {
        const float u = x[qi][k] * inv, v = x[qi][k + 1] * inv;
        const uint32_t hi = pack_f16x2(u, v);
        uint16_t* q = sm_q[warp] + qi * kQNext + lane * PER + k;
        *reinterpret_cast<uint32_t*>(q) = hi;
        if constexpr (kTwo) {
          const float2 f = unpack_f16x2(hi);
          *reinterpret_cast<uint32_t*>(q + kQTerm) =
              pack_f16x2((u - f.x) * 2048.f, (v - f.y) * 2048.f);
        }
      }
      if (lane == 0) sm_e[warp][qi] = pow2f(eq) * sl2;
    }
  }
  if (new_page >= 0) {
    const float2 f = put_row<D, kMode>(a, n, put, new_page, t, kMode == kScores && special.has(tau),
                                       put_opens(put) ? -128 : new_k, put_opens(put) ? -128 : new_v,
                                       xk, xv);
    new_k = 127 - (int)(__float_as_uint(f.x) >> 23);  // the exponents now
    new_v = 127 - (int)(__float_as_uint(f.y) >> 23);
  }
  __syncwarp();  // the queries and the new row are there
  uint32_t qa[4 * KI][kWide ? 4 : 2];  // (kWide: the second terms behind the first)
  float fq[NQ];
#pragma unroll
  for (int i = 0; i < KI; ++i)
#pragma unroll
    for (int z = 0; z < 4; ++z) {
      uint2 x = make_uint2(0, 0), y = make_uint2(0, 0);
      if (g < (kFold ? 2 * R : R)) {
        const uint16_t* q = sm_q[warp] + g * D + 64 * i + 16 * t4 + 4 * z;
        x = *reinterpret_cast<const uint2*>(q);
        if constexpr (kWide) y = *reinterpret_cast<const uint2*>(q + kQTerm);
      }
      qa[4 * i + z][0] = x.x;
      qa[4 * i + z][1] = x.y;
      if constexpr (kWide) {
        qa[4 * i + z][2] = y.x;
        qa[4 * i + z][3] = y.y;
      }
    }
  float m[NQ], ms[NQ], l[NQ];
#pragma unroll
  for (int q = 0; q < NQ; ++q) {
    fq[q] = q0 + q < R ? sm_e[warp][q0 + q] : 0.f;
    m[q] = ms[q] = q0 + q < R ? kNoScore : 1e30f;
    l[q] = 0.f;
  }
  float o[MT][4];
#pragma unroll
  for (int j = 0; j < MT; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;

#pragma unroll 1
  for (int j = 0; j < n_seg + n_ring; ++j) {
    const int page = page_next;
    uint2 ex = ex_next;
    const int2 p = p_next;
    const bool ring = j >= n_seg;
    // (what this step put may have been asked for before)
    const bool fresh_page = page >= 0 && page == new_page;
    if (fresh_page) {
      const int blk = put.at % kPageRows / kBlockRows, shift = 16 * (blk & 1);
      const uint32_t e = (uint32_t)(new_k & 0xff) | (uint32_t)(new_v & 0xff) << 8;
      uint32_t& word = blk < 2 ? ex.x : ex.y;
      word = (word & ~(0xffffu << shift)) | e << shift;
    }
    uint32_t live0, live1;  // rows 0-31 and 32-63 that count
    if (ring) {
      const int left = ring_end - (it.ring0 + j - n_seg) * kPageRows;
      auto counts = [&](int row, int pos) {
        return row < left && pos >= 0 && (unsigned)t - (unsigned)pos < (unsigned)w;
      };
      live0 = __ballot_sync(0xffffffffu, counts(lane, p.x));
      live1 = __ballot_sync(0xffffffffu, counts(lane + 32, p.y));
    } else {
      const int left = seg_end - (it.seg0 + j) * kPageRows;
      live0 = left >= 32 ? 0xffffffffu : (1u << max(left, 0)) - 1;
      live1 = left >= 64 ? 0xffffffffu : left > 32 ? (1u << (left - 32)) - 1 : 0u;
    }
    if (ring && fresh_page) {
      const int slot = put.at % kPageRows;
      (slot < 32 ? live0 : live1) |= 1u << (slot & 31);
    }
    ask(j + 1);
    if (page < 0) continue;
#pragma unroll 1
    for (int blk = 0; blk < kPageBlocks; ++blk) {
      const uint32_t live = (blk < 2 ? live0 : live1) >> (16 * (blk & 1)) & 0xffffu;
      if (live == 0) continue;
      const size_t row = (size_t)page * kPageRows + blk * kBlockRows;
      const uint8_t *kb = a.kp + row * D, *vb = a.vp + row * D;
      uint4 k0[KI], k1[KI];
#pragma unroll
      for (int i = 0; i < KI; ++i) {
        k0[i] = __ldcg(reinterpret_cast<const uint4*>(kb + g * D + (t4 + 4 * i) * 16));
        k1[i] = __ldcg(reinterpret_cast<const uint4*>(kb + (g + 8) * D + (t4 + 4 * i) * 16));
      }
      uint32_t v[4][PW];  // keys 2 t4, 2 t4 + 1 and those + 8
#pragma unroll
      for (int z = 0; z < 4; ++z) {
        const uint8_t* p = vb + (2 * t4 + (z & 1) + (z >> 1) * 8) * D + g * (D / 8);
        if constexpr (D == 128) {
          const uint4 y = __ldcg(reinterpret_cast<const uint4*>(p));
          v[z][0] = y.x, v[z][1] = y.y, v[z][2] = y.z, v[z][3] = y.w;
        } else {
          const uint2 y = __ldcg(reinterpret_cast<const uint2*>(p));
          v[z][0] = y.x, v[z][1] = y.y;
        }
      }
      const uint32_t e2 = (blk < 2 ? ex.x : ex.y) >> (16 * (blk & 1));
      const int ek = (int)(signed char)(e2 & 0xff), ev = (int)(signed char)(e2 >> 8 & 0xff);
      // columns 2 t4 and 2 t4 + 1 of key g ([0], [1]) and of key g + 8 ([2], [3])
      float x[4] = {0.f, 0.f, 0.f, 0.f}, xl[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < KI; ++i)
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          const uint32_t y0 = word4(k0[i], z), y1 = word4(k1[i], z);
          const uint32_t(&q)[kWide ? 4 : 2] = qa[4 * i + z];
          const uint32_t f0 = decode2(y0), f1 = decode2(y1), f2 = decode2(y0 >> 16),
                         f3 = decode2(y1 >> 16);
          mma_f16_16816(x, f0, f1, f2, f3, q[0], q[1]);
          if constexpr (kWide) mma_f16_16816(xl, f0, f1, f2, f3, q[2], q[3]);
        }
      const float fv = (float)ev, fk = pow2f(ek);
      float sc[NQ][2];
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        const float kf = fminf(fk * fq[q], 1.7e38f);  // (a score of 0 stays 0)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float y = kFold   ? fmaf(x[2 * h + 1], 1.f / 2048.f, x[2 * h])
                          : kWide ? fmaf(xl[2 * h + q], 1.f / 2048.f, x[2 * h + q])
                                  : x[2 * h + q];
          sc[q][h] = live >> (g + 8 * h) & 1 ? y * kf : FG_NEG_INF;
        }
      }
      if (live != 0xffffu) {  // such a row may hold anything, also NaN
#pragma unroll
        for (int z = 0; z < 4; ++z)
          if (!(live >> (2 * t4 + (z & 1) + (z >> 1) * 8) & 1))
#pragma unroll
            for (int k = 0; k < PW; ++k) v[z][k] = 0;
      }
      if constexpr (kMode == kScores) {
        if (!ring && q0 < R) {
          float* p = n.row_sc + row * R + q0;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if constexpr (NQ == 2)  // R = 8
              *reinterpret_cast<float2*>(p + (g + 8 * h) * R) = make_float2(sc[0][h], sc[1][h]);
            else
              p[(g + 8 * h) * R] = sc[0][h];
          }
        }
      }
      float top[NQ];
      bool rises = false;
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        top[q] = fmaxf(sc[q][0], sc[q][1]);
        rises |= top[q] > ms[q] || top[q] + fv > m[q];
      }
      if (__any_sync(0xffffffffu, rises)) {
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
#pragma unroll
          for (int d = 4; d < 32; d <<= 1)
            top[q] = fmaxf(top[q], __shfl_xor_sync(0xffffffffu, top[q], d));
          const float mn = fmaxf(m[q], top[q] + fv), sn = fmaxf(ms[q], top[q]);
          const float corr = ex2(m[q] - mn);
          l[q] *= ex2(ms[q] - sn);
          m[q] = mn;
          ms[q] = sn;
#pragma unroll
          for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (kFold || (k & 1) == q) o[i][k] *= corr;
        }
      }
      float p[NQ][2];
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        const float up = fv - m[q] + kPBits;
        p[q][0] = ex2(sc[q][0] + up);
        p[q][1] = ex2(sc[q][1] + up);
        l[q] += ex2(sc[q][0] - ms[q]) + ex2(sc[q][1] - ms[q]);
      }
      uint32_t p01, p23, r01 = 0, r23 = 0;  // of keys g and g + 8; r: second terms
      if constexpr (kFold) {
        const float2 f = unpack_f16x2(pack_f16x2(p[0][0], p[0][1]));
        p01 = transpose8x8(pack_f16x2(f.x, p[0][0] - f.x));
        p23 = transpose8x8(pack_f16x2(f.y, p[0][1] - f.y));
      } else {
        const uint32_t lo = pack_f16x2(p[0][0], p[NQ - 1][0]), hi = pack_f16x2(p[0][1], p[NQ - 1][1]);
        p01 = transpose8x8(lo);
        p23 = transpose8x8(hi);
        if constexpr (kWide) {
          const float2 f01 = unpack_f16x2(lo), f23 = unpack_f16x2(hi);
          r01 = transpose8x8(pack_f16x2(p[0][0] - f01.x, p[NQ - 1][0] - f01.y));
          r23 = transpose8x8(pack_f16x2(p[0][1] - f23.x, p[NQ - 1][1] - f23.y));
        }
      }
#pragma unroll
      for (int z = 0; z < PW; ++z) {
        // byte pairs (key, next key) of dimensions 4 z, 4 z + 1 and 4 z + 2, 4 z + 3
        const uint32_t lo01 = __byte_perm(v[0][z], v[1][z], 0x5140),
                       hi01 = __byte_perm(v[0][z], v[1][z], 0x7362),
                       lo23 = __byte_perm(v[2][z], v[3][z], 0x5140),
                       hi23 = __byte_perm(v[2][z], v[3][z], 0x7362);
        const uint32_t f0 = decode2(lo01), f1 = decode2(lo01 >> 16), f2 = decode2(lo23),
                       f3 = decode2(lo23 >> 16);
        const uint32_t h0 = decode2(hi01), h1 = decode2(hi01 >> 16), h2 = decode2(hi23),
                       h3 = decode2(hi23 >> 16);
        mma_f16_16816(o[2 * z], f0, f1, f2, f3, p01, p23);
        mma_f16_16816(o[2 * z + 1], h0, h1, h2, h3, p01, p23);
        if constexpr (kWide) {
          mma_f16_16816(o[2 * z], f0, f1, f2, f3, r01, r23);
          mma_f16_16816(o[2 * z + 1], h0, h1, h2, h3, r01, r23);
        }
      }
    }
  }
  // O^T: rows 16 j + g, + 8 are dimensions (D / 8) g + 2 j, + 1; the columns as the queries'
#pragma unroll
  for (int q = 0; q < NQ; ++q) {
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) l[q] += __shfl_xor_sync(0xffffffffu, l[q], d);
    const int qi = q0 + q;
    if (qi >= R) continue;
    // the sums are in units of 2^(m - kPBits), l in 2^ms
    const float f = l[q] == 0.f ? 0.f : exp2f(m[q] - ms[q] - kPBits) / l[q];
    float* out = n.part_acc + ((size_t)wi * R + qi) * D + (D / 8) * g;
#pragma unroll
    for (int j = 0; j < MT; j += 2) {
      float4 y;
      if constexpr (kFold)
        y = make_float4((o[j][0] + o[j][1]) * f, (o[j][2] + o[j][3]) * f,
                        (o[j + 1][0] + o[j + 1][1]) * f, (o[j + 1][2] + o[j + 1][3]) * f);
      else
        y = make_float4(o[j][q] * f, o[j][q + 2] * f, o[j + 1][q] * f, o[j + 1][q + 2] * f);
      *reinterpret_cast<float4*>(out + 2 * j) = y;
    }
    if (g == 0)
      *reinterpret_cast<float2*>(n.part_ml + 2 * ((size_t)wi * R + qi)) = make_float2(ms[q], l[q]);
  }
}

// A list whose thread blocks have this many items each has small ones: a block's length is at most
// 192 pages' worth, of which an item takes 3 to 7 beside its pages.
constexpr int kSmallItems = 4;

template <typename T, int D, bool kFold, int kMode>
cudaError_t run_items(const ProfileDims& pd, const PagedArgs& a, const StepArgs& n,
                      cudaStream_t s) {
  if (a.n_work < kSmallItems * a.n_ctas) return launch_split<T, D, kFold, kMode>(pd, a, n, s);
  return launch_pdl(q8_small_kernel<T, D, kFold, kMode>, cdiv(a.n_work, kSmallWarps) + n.beside,
                    kSmallWarps * 32, 0, s, a, n, pd.Gkv, pd.H, pd.R, pd.HLkv, pd.sl2);
}

template <typename T, int D, bool kFold>
cudaError_t run_split(const ProfileDims& pd, const PagedArgs& a, const StepArgs& n,
                      cudaStream_t s) {
  return n.row_w ? run_items<T, D, kFold, kScores>(pd, a, n, s)
                 : run_items<T, D, kFold, kParts>(pd, a, n, s);
}

template <typename T, int D>
cudaError_t run_step(const ProfileDims& pd, const PagedArgs& a, const StepArgs& n,
                     const PrefixParts& px, cudaStream_t s) {
  cudaError_t e = pd.R <= kFoldR ? run_split<T, D, true>(pd, a, n, s)
                                 : run_split<T, D, false>(pd, a, n, s);
  if (e == cudaSuccess && px.caches == 0)
    e = launch_pdl(step_combine_kernel<T, D>, cdiv(pd.G, kCombineWarps), kCombineWarps * 32, 0, s,
                   a, n, pd.G, pd.H, pd.R, pd.HLkv);
  if (e == cudaSuccess && px.caches > 0) {
    // few queries: warps share a query's parts (8 caches of 8192 positions, 64 queries each: 71 us
    // by a warp a query, 33 with a lane a query, 9 shared); many: each part has work enough for all
    // SMs (32 caches, 512 queries each: 25, shared 58)
    const long long blocks =
        (long long)px.caches * px.tiles * cdiv(px.rows, 32) * (D / 4 / kJoinWarps);
    e = blocks <= 2 * px.sms ? run_join<T, D, 4, 1>(pd, a, n, px, s)
                             : run_join<T, D, 1, 2>(pd, a, n, px, s);
  }
  if (e != cudaSuccess || !n.row_w) return e;
  const auto weigh = pd.R == 1   ? weigh_kernel<1>
                     : pd.R == 2 ? weigh_kernel<2>
                     : pd.R == 4 ? weigh_kernel<4>
                                 : weigh_kernel<8>;
  return launch_pdl(weigh, a.n_work, kWeighWarps * 32, 0, s, a, n, pd.Gkv, pd.H, pd.HLkv);
}

}  // namespace

constexpr int kFewPages = 8;  // an SM's, of the shared caches

cudaError_t launch_step_q8(const ProfileDims& pd, const PagedArgs& a, const StepArgs& n,
                           const PagedArgs& pre, const PrefixParts& px0, cudaStream_t s) {
  PrefixParts px = px0;
  if (px.caches > 0) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    // Few pages: half of the SMs take them as fast, and the others have the sequences' own caches
    // meanwhile (8 caches of 8192 positions, 64 queries each: 31 -> 25 us, with 40 of 152 SMs
    // 29).  8 caches, 64 queries each, all SMs and half: 2.3 pages an SM 28.3 and 23.2 us, 4.7 31.3
    // and 28.7, 7.0 32.8 and 32.2, 9.3 35.2 and 40.0, 28 57 and 76; 256 queries each 7.0 53.5 and
    // 53.8, 9.3 55.7 and 63.1; 4 queries a cache 2.3 24.2 and 24.8, 6.4 27.4 and 31.1.  Pages are
    // counted by the room of the prompt's table, which the host knows: with eight times the room
    // the first case takes all SMs.
    px.sms = sms;
    const long long pages = (long long)(pre.table_len < pre.n_pages ? pre.table_len : pre.n_pages);
    if (pages * px.groups < (long long)kFewPages * sms) sms = (sms + 1) / 2;
    px.ctas = sms < kPrefixMaxCtas ? sms : kPrefixMaxCtas;
    if (e == cudaSuccess) e = launch_prefix(pd, n, pre, px, s);
    if (e != cudaSuccess) return e;
  }
  if (pd.dtype == FG_FP32)
    return pd.d == 64 ? run_step<float, 64>(pd, a, n, px, s) : run_step<float, 128>(pd, a, n, px, s);
  return pd.d == 64 ? run_step<__nv_bfloat16, 64>(pd, a, n, px, s)
                    : run_step<__nv_bfloat16, 128>(pd, a, n, px, s);
}

}  // namespace fg
