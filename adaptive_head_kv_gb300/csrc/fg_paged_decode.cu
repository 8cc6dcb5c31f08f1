// fastgen_decode_attn_q8: the split kernel of fg_paged_decode.cuh, the combine
// of caches with several items, and their launches.
#include "fg_paged_decode.cuh"

namespace fg {
namespace {

// One warp per query head of a cache with several items: merges them and
// writes the output; one member of a group also writes the cache's new row
// count.
constexpr int kCombineWarps = 4;

template <typename T, int D>
__global__ void __launch_bounds__(kCombineWarps * 32)
    q8_combine_kernel(const PagedArgs a, const PagedDecodeArgs n, int G, int H, int R, int HLkv) {
  constexpr int PER = D / 32;
  constexpr int kAhead = 4;  // items with loads in flight
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
  // (a cache's only item has written the result and the count)
  if (!in || range.y == 1 || !listed) return;
  const fg_paged_desc hd = a.caches[c];
  const int t = n.pos[b], had = a.rows[c], tau = n.k_new ? n.ids[b] : 0;
  if (t < 0) {
    if (qi == 0 && lane == 0) a.rows_out[c] = had;
    return;
  }
  float M = kNoScore, L = 0.f, acc[PER];  // of the items so far: maximum, sum, output
#pragma unroll
  for (int k = 0; k < PER; ++k) acc[k] = 0.f;
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
  for (int k = 0; k < PER; ++k)
    store_out((T*)n.out + (size_t)gq * D + lane * PER + k, acc[k]);
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

template <typename T, int D, bool kFold>
cudaError_t run_decode_q8(const ProfileDims& pd, const PagedArgs& a, const PagedDecodeArgs& n,
                          cudaStream_t s) {
  cudaError_t e = launch_split<T, D, kFold, kDecode>(pd, a, n, s);
  if (D == 64 && e == cudaSuccess)  // as the split kernel
    e = cudaFuncSetAttribute(q8_combine_kernel<T, D>, cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared);
  if (e == cudaSuccess && a.n_work > pd.Gkv)  // else every cache has one item
    e = launch_pdl(q8_combine_kernel<T, D>, cdiv(pd.G, kCombineWarps), kCombineWarps * 32, 0, s, a,
                   n, pd.G, pd.H, pd.R, pd.HLkv);
  return e;
}

template <typename T, int D>
cudaError_t run_decode_q8(const ProfileDims& pd, const PagedArgs& a, const PagedDecodeArgs& n,
                          cudaStream_t s) {
  return pd.R <= kFoldR ? run_decode_q8<T, D, true>(pd, a, n, s)
                        : run_decode_q8<T, D, false>(pd, a, n, s);
}

// As many as the SMs hold less one or two: right behind the previous step's
// combine the last block at times found no room, and started only when another
// ended (grouped 4k shape: 456 blocks on 152 SMs 63 us, 452 blocks 54.5 us).
// Shared memory (228 KB an SM, of which a block also takes 1 KB and its static
// part) is the limit for fp32 groups of 8 at d = 128: two blocks (counting on three
// left a part-filled second wave: 128 caches of 8192 positions 51.6 us, now 37).
template <typename T, int D>
int slots(int R, int sms) {
  const int smem =
      R <= kFoldR ? split_smem<T, D, true, kDecode>(R) : split_smem<T, D, false, kDecode>(R);
  const int room = 228 * 1024 / (smem + 1024 + 1024);
  return (room < kBlocks(D) ? room : kBlocks(D)) * sms - sms / 64;
}

}  // namespace

int q8_slots(const ProfileDims& pd, int sms) {
  if (pd.dtype == FG_FP32)
    return pd.d == 64 ? slots<float, 64>(pd.R, sms) : slots<float, 128>(pd.R, sms);
  return pd.d == 64 ? slots<__nv_bfloat16, 64>(pd.R, sms) : slots<__nv_bfloat16, 128>(pd.R, sms);
}

cudaError_t launch_decode_q8(const ProfileDims& pd, const PagedArgs& a, const PagedDecodeArgs& n,
                             cudaStream_t s) {
  if (pd.dtype == FG_FP32)
    return pd.d == 64 ? run_decode_q8<float, 64>(pd, a, n, s)
                      : run_decode_q8<float, 128>(pd, a, n, s);
  return pd.d == 64 ? run_decode_q8<__nv_bfloat16, 64>(pd, a, n, s)
                    : run_decode_q8<__nv_bfloat16, 128>(pd, a, n, s);
}

}  // namespace fg
