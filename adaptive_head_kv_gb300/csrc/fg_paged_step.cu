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
__device__ __forceinline__ int rows_after(const PagedArgs& a, const PagedDecodeArgs& n,
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
    step_combine_kernel(const PagedArgs a, const PagedDecodeArgs n, int G, int H, int R, int HLkv) {
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
// and a warp four dimensions of 32 of them.  kSplit warps share the parts of these (where few caches
// leave many parts to each), eight warps a block.
constexpr int kJoinWarps = 8;

template <typename T, int D, int kSplit>
__global__ void __launch_bounds__(kJoinWarps * 32)
    step_join_kernel(const PagedArgs a, const PagedDecodeArgs n, const PrefixParts px, int H, int R,
                     int HL) {
  constexpr int kAhead = 4, kQuads = kJoinWarps / kSplit, kSlices = D / 4 / kQuads;
  __shared__ float sm[kSplit > 1 ? kSplit - 1 : 1][kQuads][6][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int split = warp / kQuads, dq = warp % kQuads;
  const int d4 = blockIdx.x % kSlices * kQuads + dq;
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
  Joined<kAhead, 4> o;
  const int most = parts + __reduce_max_sync(0xffffffffu, t >= 0 ? range.y : 0);
  for (int i0 = split; i0 < most; i0 += kAhead * kSplit) {
    float m[kAhead], l[kAhead], x[kAhead][4];
    float2 ml[kAhead];
    float4 v[kAhead];
#pragma unroll
    for (int z = 0; z < kAhead; ++z) {
      const int i = i0 + z * kSplit;
      const bool shared = i < parts, ok = t >= 0 && i < parts + range.y;
      const size_t p = part + (size_t)i * (2 / streams);
      const size_t slot = shared ? p * px.rows + row : ((size_t)range.x + i - parts) * R + qi;
      ml[z] = ok ? *reinterpret_cast<const float2*>((shared ? px.ml : n.part_ml) + 2 * slot)
                 : make_float2(kNoScore, 0.f);
      v[z] = ok ? *reinterpret_cast<const float4*>(
                      shared ? px.acc + (p * (D / 4) + d4) * px.rows * 4 + (size_t)row * 4
                             : n.part_acc + slot * D + d4 * 4)
                : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int z = 0; z < kAhead; ++z) {
      m[z] = ml[z].x;
      l[z] = ml[z].y;
      const bool some = l[z] != 0.f;  // (a part without a row has no values)
      x[z][0] = some ? v[z].x : 0.f;
      x[z][1] = some ? v[z].y : 0.f;
      x[z][2] = some ? v[z].z : 0.f;
      x[z][3] = some ? v[z].w : 0.f;
    }
    o.add(m, l, x);
  }
  if constexpr (kSplit > 1) {
    if (split > 0) {
      float(&s)[6][32] = sm[split - 1][dq];
#pragma unroll
      for (int k = 0; k < 4; ++k) s[k][lane] = o.acc[k];
      s[4][lane] = o.M;
      s[5][lane] = o.L;
    }
    __syncthreads();
    Joined<kSplit - 1, 4> all;
    all.M = o.M;
    all.L = o.L;
    float m[kSplit - 1], l[kSplit - 1], x[kSplit - 1][4];
#pragma unroll
    for (int k = 0; k < 4; ++k) all.acc[k] = o.acc[k];
#pragma unroll
    for (int z = 0; z < kSplit - 1; ++z) {
      float(&s)[6][32] = sm[z][dq];
#pragma unroll
      for (int k = 0; k < 4; ++k) x[z][k] = s[k][lane];
      m[z] = s[4][lane];
      l[z] = s[5][lane];
    }
    all.add(m, l, x);
#pragma unroll
    for (int k = 0; k < 4; ++k) o.acc[k] = all.acc[k];
    o.M = all.M;
    o.L = all.L;
  }
  // a query's dimensions of this block side by side in memory: the lanes of a warp take kQuads of
  // the block's fours of each of 32 / kQuads queries
  __shared__ float4 sm_out[32][kQuads + 1];
  __shared__ long long sm_at[32];
  if (split == 0) {
    sm_out[lane][dq] = make_float4(o.acc[0], o.acc[1], o.acc[2], o.acc[3]);
    if (dq == 0) sm_at[lane] = t >= 0 ? (long long)g : -1;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 32 * kQuads; i += kJoinWarps * 32) {
    const float4 v = sm_out[i / kQuads][i % kQuads];
    const long long at = sm_at[i / kQuads];
    T* out = (T*)n.out + at * D + (blockIdx.x % kSlices * kQuads + i % kQuads) * 4;
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

template <typename T, int D, int kSplit>
cudaError_t run_join(const ProfileDims& pd, const PagedArgs& a, const PagedDecodeArgs& n,
                     const PrefixParts& px, cudaStream_t s) {
  const long long grid =
      (long long)px.caches * px.tiles * cdiv(px.rows, 32) * (D / 4 / (kJoinWarps / kSplit));
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  return launch_pdl(step_join_kernel<T, D, kSplit>, (unsigned)grid, kJoinWarps * 32, 0, s, a, n, px,
                    pd.H, pd.R, pd.HL);
}

// Adds the step's weights to the rows of a work item's part of the segment, a thread a row.
constexpr int kWeighThreads = 256;

template <int R>
__global__ void __launch_bounds__(kWeighThreads)
    weigh_kernel(const PagedArgs a, const PagedDecodeArgs n, int Gkv, int H, int HLkv) {
  const PagedItem it = a.items[blockIdx.x];
  const bool listed = same_list(a);
  griddep_wait();
  griddep_launch_dependents();
  const int c = it.cache;
  if (!listed || (unsigned)c >= (unsigned)Gkv) return;
  if (n.pos[c / HLkv] < 0) return;
  const fg_paged_desc hd = a.caches[c];
  const int rows = live_rows(hd, a.rows_out[c]);
  const int end = it.last ? rows : (int)min((long long)rows, (long long)it.seg1 * kPageRows);
  const size_t g0 = (size_t)(c / (H / R)) * H + (size_t)(c % (H / R)) * R;
  float M[R], r[R];
#pragma unroll
  for (int q = 0; q < R; ++q) {
    const float2 ml = *reinterpret_cast<const float2*>(n.head_ml + 2 * (g0 + q));
    M[q] = ml.x;
    r[q] = ml.y == 0.f ? 0.f : 1.f / ml.y;
  }
  for (int row = it.seg0 * kPageRows + threadIdx.x; row < end; row += kWeighThreads) {
    const int page = page_at(a, hd.first_page, hd.max_pages, row / kPageRows);
    if (page < 0) continue;  // flagged by the split kernel
    const size_t at = (size_t)page * kPageRows + row % kPageRows;
    float w = 0.f;
#pragma unroll
    for (int q = 0; q < R; ++q) w = fmaf(ex2(n.row_sc[at * R + q] - M[q]), r[q], w);
    n.row_w[at] += w;
  }
}

template <typename T, int D, bool kFold>
cudaError_t run_split(const ProfileDims& pd, const PagedArgs& a, const PagedDecodeArgs& n,
                      cudaStream_t s) {
  return n.row_w ? launch_split<T, D, kFold, kScores>(pd, a, n, s)
                 : launch_split<T, D, kFold, kParts>(pd, a, n, s);
}

template <typename T, int D>
cudaError_t run_step(const ProfileDims& pd, const PagedArgs& a, const PagedDecodeArgs& n,
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
    const long long blocks = (long long)px.caches * px.tiles * cdiv(px.rows, 32) * (D / 4 / kJoinWarps);
    e = blocks <= 2 * px.ctas ? run_join<T, D, 4>(pd, a, n, px, s) : run_join<T, D, 1>(pd, a, n, px, s);
  }
  if (e != cudaSuccess || !n.row_w) return e;
  const auto weigh = pd.R == 1   ? weigh_kernel<1>
                     : pd.R == 2 ? weigh_kernel<2>
                     : pd.R == 4 ? weigh_kernel<4>
                                 : weigh_kernel<8>;
  return launch_pdl(weigh, a.n_work, kWeighThreads, 0, s, a, n, pd.Gkv, pd.H, pd.HLkv);
}

}  // namespace

cudaError_t launch_step_q8(const ProfileDims& pd, const PagedArgs& a, const PagedDecodeArgs& n,
                           const PagedArgs& pre, const PrefixParts& px0, cudaStream_t s) {
  PrefixParts px = px0;
  if (px.caches > 0) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
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
