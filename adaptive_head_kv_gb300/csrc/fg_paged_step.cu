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

constexpr int kCombineWarps = 4;

// One warp per query head.
template <typename T, int D>
__global__ void __launch_bounds__(kCombineWarps * 32)
    step_combine_kernel(const PagedArgs a, const PagedDecodeArgs n, const PrefixParts px, int G,
                        int H, int R, int HLkv) {
  constexpr int PER = D / 32;
  constexpr int kAhead = 4;  // parts with loads in flight
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
  // the shared cache's parts of this query: of every thread block that had pages of its unit, one,
  // or two where the block's two streams shared the unit's pages
  int parts = 0, streams = 1, row = 0;
  size_t pre0 = 0;  // the first part
  if (px.caches > 0) {
    const int pc = c % HLkv, j = b * R + qi, tile = j / kPrefixTile;
    const int grp = px.pair ? tile / 2 : tile;
    const long long c0 = px.cum[pc], pages = px.cum[pc + 1] - c0;
    const long long all = px.cum[px.caches] * px.groups;
    if (pages > 0) {
      const int ctas = prefix_ctas(all, px.ctas);
      const long long x = c0 * px.groups + grp * pages;
      const int i0 = prefix_cta(all, ctas, x), i1 = prefix_cta(all, ctas, x + pages - 1);
      streams = px.pair ? 1 : 2;
      parts = (i1 - i0 + 1) * streams;
      pre0 = ((size_t)i0 + (size_t)pc * px.groups + grp) * 2 + (px.pair ? tile & 1 : 0);
      row = j % kPrefixTile;
    }
  }
  const int total = range.y + parts;
  float M = kNoScore, L = 0.f, acc[PER];  // of the parts so far: maximum, sum, output
#pragma unroll
  for (int k = 0; k < PER; ++k) acc[k] = 0.f;
  for (int i0 = 0; i0 < total; i0 += kAhead) {
    float m[kAhead], l[kAhead], x[kAhead][PER];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int i = i0 + j;
      const bool own = i < range.y;
      const size_t part = pre0 + (size_t)(i - range.y) * (2 / streams);
      const size_t slot = own ? ((size_t)range.x + i) * R + qi : part * px.rows + row;
      const float2 ml = i < total
                            ? *reinterpret_cast<const float2*>((own ? n.part_ml : px.ml) + 2 * slot)
                            : make_float2(kNoScore, 0.f);
      m[j] = ml.x;
      l[j] = ml.y;
      if (l[j] == 0.f) {  // no row: nothing was written
#pragma unroll
        for (int k = 0; k < PER; ++k) x[j][k] = 0.f;
      } else if (own) {
        load_row<PER>(n.part_acc + slot * D, x[j]);
      } else {
        const float* p = px.acc + part * px.rows * D + ((size_t)(lane * PER / 4) * px.rows + row) * 4;
#pragma unroll
        for (int k = 0; k < PER; k += 2) {
          const float2 y = *reinterpret_cast<const float2*>(p + lane * PER % 4 + k);
          x[j][k] = y.x;
          x[j][k + 1] = y.y;
        }
      }
    }
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
    for (int k = 0; k < PER; ++k) acc[k] = acc[k] * (L * r) * fh * fh;
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
#pragma unroll
      for (int k = 0; k < PER; ++k) acc[k] = fmaf(x[j][k] * (l[j] * r) * h[j], h[j], acc[k]);
    L = Ln;
    M = Mn;
  }
#pragma unroll
  for (int k = 0; k < PER; ++k) store_out((T*)n.out + (size_t)gq * D + lane * PER + k, acc[k]);
  if (n.head_ml && lane == 0)
    *reinterpret_cast<float2*>(n.head_ml + 2 * (size_t)gq) = make_float2(M, L);
  if (qi == 0) {
    bool stored = false;  // the new token joined the never-evicted segment and found a page
    if (n.k_new) {
      const bool s = special.has(tau), sp = s || punct.has(tau);
      stored = joins_static(hd.policy, s, sp) && had >= 0 &&
               page_at(a, hd.first_page, hd.max_pages, had / kPageRows) >= 0;
    }
    if (lane == 0) a.rows_out[c] = had + (stored ? 1 : 0);
  }
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
  if (e == cudaSuccess)
    e = launch_pdl(step_combine_kernel<T, D>, cdiv(pd.G, kCombineWarps), kCombineWarps * 32, 0, s,
                   a, n, px, pd.G, pd.H, pd.R, pd.HLkv);
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
