// Caches that stay within a budget: the weights their rows start with, the cut
// to the budget, and empty caches behind a shared prompt.
#include "fg_paged.cuh"

namespace fg {
namespace {

// ------------------------------------------------------------- empty caches
__global__ void __launch_bounds__(256) fork_kernel(const fg_paged_desc* __restrict__ prefix,
                                                   int one, int Gkv, int2* __restrict__ cinfo) {
  const int c = blockIdx.x * blockDim.x + threadIdx.x;
  if (c >= Gkv) return;
  const int policy = prefix[c % one].policy;
  cinfo[c] = make_int2(policy >= FG_POLICY_S && policy <= FG_POLICY_FULL ? policy : FG_POLICY_FULL,
                       0);
}

// One warp per cache: no rows, no ring slot in use, the ring's blocks at the least exponent.
__global__ void __launch_bounds__(256) clear_kernel(const PagedArgs a, int32_t* rows, int Gkv) {
  const int c = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (c >= Gkv) return;
  const fg_paged_desc hd = a.caches[c];
  const int w = ring_slots(hd, a.max_w);
  if (lane == 0) {
    if (w != hd.w) atomicOr(a.dev_err, kErrInvalid);
    rows[c] = 0;
    a.rows_out[c] = 0;
  }
  for (int i = 0; i < cdiv(w, kPageRows); ++i) {
    const int page = page_at(a, hd.ring_page, hd.ring_pages, i);
    if (page < 0) {
      if (lane == 0) atomicOr(a.dev_err, kErrInvalid);
      continue;
    }
    for (int r = lane; r < kPageRows; r += 32) a.pos[(size_t)page * kPageRows + r] = -1;
    if (lane < kPageBlocks * 2) a.exps[(size_t)page * kPageBlocks * 2 + lane] = (int8_t)kExpMin;
  }
}

// ------------------------------------------------------- weights to start with
__global__ void __launch_bounds__(256) scores_kernel(const PagedArgs a, const ScoreArgs n, int H,
                                                     int R, int HLkv) {
  griddep_wait();
  griddep_launch_dependents();
  const int c = blockIdx.x, b = c / HLkv;
  const int first = n.pos ? n.pos[b] : 0;
  const int count = n.n_new ? min(n.n_new[b], n.m) : n.m;
  if (first < 0) return;
  const fg_paged_desc hd = a.caches[c];
  const int rows = live_rows(hd, a.rows[c]);
  const size_t g0 = (size_t)(c / (H / R)) * H + (size_t)(c % (H / R)) * R;
  for (int r = threadIdx.x; r < rows; r += 256) {
    const int page = page_at(a, hd.first_page, hd.max_pages, r / kPageRows);
    if (page < 0) {
      atomicOr(a.dev_err, kErrInvalid);
      continue;
    }
    const size_t at = (size_t)page * kPageRows + r % kPageRows;
    const long long i = (long long)a.pos[at] - first;
    if (i < 0 || i >= count) continue;
    float y = 0.f;
    if (n.colsum)
      for (int q = 0; q < R; ++q) y += n.colsum[(g0 + q) * n.m + i];
    n.scores[at] = id_in(n.ids[(size_t)b * n.m + i], n.special, n.ns) ? -FG_NEG_INF : y;
  }
}

// ------------------------------------------------------------------- the cut
// Order of the rows that stay: recent ones, then by weight; ties to the lower row.
__device__ __forceinline__ uint32_t row_key(float score, int p, int t, int recent) {
  if (p <= t && (long long)p > (long long)t - recent) return 0xffffffffu;
  return score > 0.f ? __float_as_uint(score) : 0u;
}

constexpr int kSelectThreads = 1024;

// One CTA per cache: which rows stay, and which of those behind the budget come to which place
// below it.
__global__ void __launch_bounds__(kSelectThreads) evict_select_kernel(const PagedArgs a,
                                                                      const EvictArgs n, int HLkv) {
  __shared__ int hist[256];
  __shared__ int scr[33];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  griddep_wait();
  griddep_launch_dependents();
  const int c = blockIdx.x, tid = threadIdx.x;
  const fg_paged_desc hd = a.caches[c];
  const int t = n.pos[c / HLkv], had = a.rows[c], rows = live_rows(hd, had);
  __syncthreads();  // every thread has read the count
  if (tid == 0) {
    if (rows != had) atomicOr(a.dev_err, kErrInvalid);
    a.rows_out[c] = t >= 0 && rows > n.budget ? n.budget : had;
    n.moves[c] = 0;
  }
  if (t < 0 || rows <= n.budget) return;
  auto key_of = [&](int r) {
    const int page = page_at(a, hd.first_page, hd.max_pages, r / kPageRows);
    if (page < 0) {  // a row that is not there
      atomicOr(a.dev_err, kErrInvalid);
      return 0u;
    }
    const size_t at = (size_t)page * kPageRows + r % kPageRows;
    return row_key(n.scores[at], a.pos[at], t, n.recent);
  };
  // the budget-th largest key, eight bits at a time
  uint32_t prefix = 0;
  int need = n.budget;
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
    for (int r = tid; r < rows; r += kSelectThreads) {
      const uint32_t k = key_of(r);
      if (shift == 24 || k >> (shift + 8) == prefix >> (shift + 8))
        atomicAdd(&hist[k >> shift & 255], 1);
    }
    __syncthreads();
    if (tid == 0) {
      int bin = 255;
      for (; bin > 0 && hist[bin] < need; --bin) need -= hist[bin];
      s_prefix = prefix | (uint32_t)bin << shift;
      s_need = need;
    }
    __syncthreads();
    prefix = s_prefix;
    need = s_need;
  }
  // rows a thread, in order: how many tie, then who stays
  const int per = cdiv(rows, kSelectThreads), r0 = min(tid * per, rows), r1 = min(r0 + per, rows);
  int ties = 0, total;
  for (int r = r0; r < r1; ++r) ties += key_of(r) == prefix;
  const int before = block_exclusive_scan(ties, scr, &total);
  auto each = [&](auto hole, auto mover) {
    int tie = before;
    for (int r = r0; r < r1; ++r) {
      const uint32_t k = key_of(r);
      const bool stays = k > prefix || (k == prefix && tie++ < need);
      if (r < n.budget ? !stays : stays) {
        if (r < n.budget) hole(r);
        else mover(r);
      }
    }
  };
  int holes = 0, movers = 0;
  each([&](int) { ++holes; }, [&](int) { ++movers; });
  int h0 = block_exclusive_scan(holes, scr, &total);
  int m0 = block_exclusive_scan(movers, scr, &total);
  // src[i] first lists the movers in order, then is read by who fills hole i
  int32_t* list = n.src + (size_t)gridDim.x * n.budget + (size_t)c * n.budget;
  int32_t* src = n.src + (size_t)c * n.budget;
  for (int r = tid; r < n.budget; r += kSelectThreads) src[r] = -1;
  each([](int) {}, [&](int r) { list[m0++] = r; });
  __syncthreads();
  each([&](int r) { src[r] = list[h0++]; }, [](int) {});
  if (tid == 0) n.moves[c] = total;
}

// One warp per block of 16 places below the budget.
template <int D>
__global__ void __launch_bounds__(128) evict_move_kernel(const PagedArgs a, const EvictArgs n,
                                                         int blocks) {
  constexpr int PER = D / 32;
  const int quads = cdiv(blocks, 4);
  const int c = blockIdx.x / quads, lane = threadIdx.x & 31;
  const int blk = blockIdx.x % quads * 4 + (threadIdx.x >> 5);
  griddep_wait();
  griddep_launch_dependents();
  if (blk >= blocks || n.moves[c] == 0) return;
  const int src = lane < kBlockRows ? n.src[(size_t)c * n.budget + blk * kBlockRows + lane] : -1;
  const uint32_t mask = __ballot_sync(0xffffffffu, src >= 0);
  if (mask == 0) return;
  const fg_paged_desc hd = a.caches[c];
  const int row0 = blk * kBlockRows;
  const int page = page_at(a, hd.first_page, hd.max_pages, row0 / kPageRows);
  const int from = src >= 0 ? page_at(a, hd.first_page, hd.max_pages, src / kPageRows) : -1;
  const bool ok = page >= 0 && from >= 0;
  if (src >= 0 && !ok) atomicOr(a.dev_err, kErrInvalid);
  const uint32_t todo = __ballot_sync(0xffffffffu, ok);
  if (todo == 0) return;
  const size_t to = (size_t)page * kPageRows + row0 % kPageRows;
  const int b0 = row0 % kPageRows / kBlockRows;
  const long long at = ok ? (long long)from * kPageRows + src % kPageRows : 0;
  if (ok) {
    a.pos[to + lane] = a.pos[at];
    n.scores[to + lane] = n.scores[at];
  }
  for (int side = 0; side < 2; ++side) {
    uint8_t* codes = (side ? a.vp : a.kp);
    int8_t* ex = a.exps + ((size_t)page * kPageBlocks + b0) * 2 + side;
    float x[kBlockRows][PER];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kBlockRows; ++i) {
      const long long z = __shfl_sync(0xffffffffu, at, i);
#pragma unroll
      for (int k = 0; k < PER; ++k) x[i][k] = 0.f;
      if (!(todo >> i & 1)) continue;
      const float f = pow2f(a.exps[z / kBlockRows * 2 + side]);
#pragma unroll
      for (int k = 0; k < PER; k += 2) {
        const uint16_t w = *reinterpret_cast<const uint16_t*>(codes + z * D + lane * PER + k);
        const uint32_t h = decode2(w);
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
            : "=f"(x[i][k]), "=f"(x[i][k + 1])
            : "r"(h));
        x[i][k] *= f;
        x[i][k + 1] *= f;
      }
      top = max(top, top_bits<PER>(x[i]));
    }
    const float inv = open_block<D>(top, ex[0], codes + to * D, ex);
#pragma unroll
    for (int i = 0; i < kBlockRows; ++i)
      if (todo >> i & 1) code_row<PER>(x[i], inv, codes + (to + i) * D);
  }
}

}  // namespace

cudaError_t launch_fork(const ProfileDims& pd, const fg_paged_desc* prefix, int2* cinfo,
                        cudaStream_t s) {
  fork_kernel<<<cdiv(pd.Gkv, 256), 256, 0, s>>>(prefix, pd.HLkv, pd.Gkv, cinfo);
  return cudaGetLastError();
}

cudaError_t launch_paged_clear(const ProfileDims& pd, const PagedArgs& a, int32_t* rows,
                               cudaStream_t s) {
  clear_kernel<<<cdiv(pd.Gkv, 8), 256, 0, s>>>(a, rows, pd.Gkv);
  return cudaGetLastError();
}

cudaError_t launch_scores_q8(const ProfileDims& pd, const PagedArgs& a, const ScoreArgs& n,
                             cudaStream_t s) {
  return launch_pdl(scores_kernel, pd.Gkv, 256, 0, s, a, n, pd.H, pd.R, pd.HLkv);
}

cudaError_t launch_evict_q8(const ProfileDims& pd, const PagedArgs& a, const EvictArgs& n,
                            cudaStream_t s) {
  cudaError_t e = launch_pdl(evict_select_kernel, pd.Gkv, kSelectThreads, 0, s, a, n, pd.HLkv);
  if (e != cudaSuccess) return e;
  const int blocks = n.budget / kBlockRows;
  const long long grid = (long long)cdiv(blocks, 4) * pd.Gkv;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  return launch_pdl(pd.d == 64 ? evict_move_kernel<64> : evict_move_kernel<128>, (unsigned)grid,
                    128, 0, s, a, n, blocks);
}

}  // namespace fg
