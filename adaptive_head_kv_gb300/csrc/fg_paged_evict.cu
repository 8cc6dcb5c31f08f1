// Caches that stay within a budget: the weights their rows start with, the cut
// to the budget, and empty caches behind a shared prompt.
#include <type_traits>

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
  const int had = a.rows[c], rows = live_rows(hd, had);
  if (threadIdx.x == 0 && (rows != had || ring_slots(hd, a.max_w) != hd.w))
    atomicOr(a.dev_err, kErrInvalid);
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
__device__ __forceinline__ float2 half2_values(uint32_t w) {
  float2 f;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(w));
  return f;
}

// Order of the rows that stay: recent ones, then by weight; ties to the lower row.
__device__ __forceinline__ uint32_t row_key(float score, int p, int t, int recent) {
  if (p <= t && (long long)p > (long long)t - recent) return 0xffffffffu;
  return score > 0.f ? __float_as_uint(score) : 0u;
}

// One CTA per cache: which rows stay, and which of those behind the budget come to which place
// below it.  The keys are read once, into shared memory (of a cache with more than kKeys rows they
// are read seven times); the budget-th largest is found eleven bits at a time.  A chain of loads, scans and barriers bounds it: 1024 caches
// of 1280 rows about 10 us, 16 of 32768 rows 25 us (with clusters of eight blocks a cache, whose
// barriers cost as much as the shorter runs save, 30 us).
template <int kThreads, int kKeys>
__global__ void __launch_bounds__(kThreads)
    evict_select_kernel(const PagedArgs a, const EvictArgs n, int HLkv) {
  constexpr int kBins = 2048, kPerThread = kBins / kThreads, kPasses = 3;
  extern __shared__ uint32_t keys[];  // [kKeys]
  __shared__ int hist[kBins];
  __shared__ int scr[33];
  __shared__ int s_bin, s_need;
  griddep_wait();
  griddep_launch_dependents();
  const int c = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const fg_paged_desc hd = a.caches[c];
  const int t = n.pos[c / HLkv], had = a.rows[c], rows = live_rows(hd, had);
  __syncthreads();  // every thread has read the count
  if (tid == 0) {
    if (rows != had || ring_slots(hd, a.max_w) != hd.w) atomicOr(a.dev_err, kErrInvalid);
    a.rows_out[c] = t >= 0 && rows > n.budget ? n.budget : had;
    n.moves[c] = 0;
  }
  if (t < 0 || rows <= n.budget) return;
  auto key_of = [&](int r, int page) {
    if (page < 0) {  // a row that is not there
      atomicOr(a.dev_err, kErrInvalid);
      return 0u;
    }
    const size_t at = (size_t)page * kPageRows + r % kPageRows;
    return row_key(n.scores[at], a.pos[at], t, n.recent);
  };
  const bool kept_here = rows <= kKeys;
  auto key = [&](int r) {
    return kept_here ? keys[r] : key_of(r, page_at(a, hd.first_page, hd.max_pages, r / kPageRows));
  };
  for (int i = tid; i < kBins; i += kThreads) hist[i] = 0;
  if (kept_here) {
    // a warp takes pages in turns, each lane two rows; four pages under way
    constexpr int kAhead = 4, kWarps = kThreads / 32;
    for (int p0 = warp; p0 * kPageRows < rows; p0 += kAhead * kWarps) {
      int page[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        page[u] = page_at(a, hd.first_page, hd.max_pages, p0 + u * kWarps);
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = (p0 + u * kWarps) * kPageRows + h * 32 + lane;
          if (r < rows) keys[r] = key_of(r, page[u]);
        }
    }
  }
  __syncthreads();
  uint32_t prefix = 0;
  int need = n.budget;
#pragma unroll 1
  for (int pass = 0; pass < kPasses; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t bins = pass == 2 ? 1024 : 2048;
    for (int r = tid; r < rows; r += kThreads) {
      const uint32_t k = key(r);
      if (pass == 0 || k >> (pass == 1 ? 21 : 10) == prefix >> (pass == 1 ? 21 : 10))
        atomicAdd(&hist[k >> shift & (bins - 1)], 1);
    }
    __syncthreads();
    // thread i counts the bins below 2048 - kPerThread i; the scan gives how many keys lie above
    int own[kPerThread], sum = 0, total;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) sum += own[i] = hist[kBins - 1 - tid * kPerThread - i];
    const int above = block_exclusive_scan(sum, scr, &total);
    if (above < need && need <= above + sum) {
      int left = need - above, i = 0;
      while (i < kPerThread - 1 && own[i] < left) left -= own[i++];
      s_bin = kBins - 1 - tid * kPerThread - i;
      s_need = left;
    }
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) hist[kBins - 1 - tid * kPerThread - i] = 0;
    __syncthreads();
    prefix |= (uint32_t)s_bin << shift;
    need = s_need;
  }
  // rows a thread, in order: how many tie, then who stays (an odd number, for the banks)
  const int per = cdiv(rows, kThreads) | 1, r0 = min(tid * per, rows), r1 = min(r0 + per, rows);
  int ties = 0, total;
  for (int r = r0; r < r1; ++r) ties += key(r) == prefix;
  const int before = block_exclusive_scan(ties, scr, &total);
  auto each = [&](auto hole, auto mover) {
    int tie = before;
    for (int r = r0; r < r1; ++r) {
      const uint32_t k = key(r);
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
  // the movers in order, then who fills which hole
  int32_t* list = n.src + (size_t)n.caches * n.budget + (size_t)c * n.budget;
  int32_t* src = n.src + (size_t)c * n.budget;
  for (int r = tid; r < n.budget; r += kThreads) src[r] = -1;
  each([](int) {}, [&](int r) { list[m0++] = r; });
  __syncthreads();
  each([&](int r) { src[r] = list[h0++]; }, [](int) {});
  if (tid == 0) n.moves[c] = total;
}

// A warp takes kMoveBlocks blocks of 16 places below the budget in turn.  The codes of K and of V of
// all rows that come to a block are asked for before any is used; they lie far apart, and the chain
// list, page, row, exponent bounds it (1024 caches of 1280 rows cut to 1024: 10 us, 20 MB).
constexpr int kMoveWarps = 4, kMoveBlocks = 4;

template <int D>
__global__ void __launch_bounds__(kMoveWarps * 32)
    evict_move_kernel(const PagedArgs a, const EvictArgs n, int blocks) {
  constexpr int PER = D / 32;
  using Word = typename std::conditional<PER == 4, uint32_t, uint16_t>::type;  // a lane's codes of a row
  const int warps = cdiv(blocks, kMoveBlocks), lane = threadIdx.x & 31;
  const long long wi = (long long)blockIdx.x * kMoveWarps + (threadIdx.x >> 5);
  griddep_wait();
  griddep_launch_dependents();
  const int c = (int)(wi / warps), blk0 = (int)(wi % warps) * kMoveBlocks;
  if (c >= n.caches || n.moves[c] == 0) return;
  const fg_paged_desc hd = a.caches[c];
  int src_l[kMoveBlocks / 2];  // of two blocks
#pragma unroll
  for (int i = 0; i < kMoveBlocks / 2; ++i) {
    const int place = (blk0 + 2 * i) * kBlockRows + lane;
    src_l[i] = place < n.budget ? n.src[(size_t)c * n.budget + place] : -1;
  }
#pragma unroll 1
  for (int i = 0; i < kMoveBlocks; ++i) {
    int src = i < 2 ? src_l[0] : src_l[kMoveBlocks / 2 - 1];
    src = __shfl_sync(0xffffffffu, src, (lane & 15) + 16 * (i & 1));
    if (lane >= kBlockRows) src = -1;
    if (__ballot_sync(0xffffffffu, src >= 0) == 0) continue;
    const int row0 = (blk0 + i) * kBlockRows, b0 = row0 % kPageRows / kBlockRows;
    const int page = page_at(a, hd.first_page, hd.max_pages, row0 / kPageRows);
    const int from = src >= 0 ? page_at(a, hd.first_page, hd.max_pages, src / kPageRows) : -1;
    const bool ok = page >= 0 && from >= 0;
    if (src >= 0 && !ok) atomicOr(a.dev_err, kErrInvalid);
    const uint32_t todo = __ballot_sync(0xffffffffu, ok);
    if (todo == 0) continue;
    const size_t to = (size_t)page * kPageRows + row0 % kPageRows;
    const long long at = ok ? (long long)from * kPageRows + src % kPageRows : 0;
    Word x[2][kBlockRows];
#pragma unroll
    for (int r = 0; r < kBlockRows; ++r) {
      const long long z = __shfl_sync(0xffffffffu, at, r);
      x[0][r] = x[1][r] = 0;
      if (todo >> r & 1) {
        x[0][r] = __ldcg(reinterpret_cast<const Word*>(a.kp + z * D) + lane);
        x[1][r] = __ldcg(reinterpret_cast<const Word*>(a.vp + z * D) + lane);
      }
    }
    int e_k = 0, e_v = 0;
    if (ok) {
      const int8_t* e = a.exps + at / kBlockRows * 2;
      e_k = e[0];
      e_v = e[1];
      a.pos[to + lane] = a.pos[at];
      n.scores[to + lane] = n.scores[at];
    }
    int8_t* ex = a.exps + ((size_t)page * kPageBlocks + b0) * 2;
    const int had_k = ex[0], had_v = ex[1];
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      uint8_t* codes = side ? a.vp : a.kp;
      auto values = [&](int r, float (&y)[PER]) {
        const float f = pow2f(__shfl_sync(0xffffffffu, side ? e_v : e_k, r));
#pragma unroll
        for (int k = 0; k < PER; k += 2) {
          const float2 z = half2_values(decode2((uint32_t)x[side][r] >> (8 * k)));
          y[k] = z.x * f;
          y[k + 1] = z.y * f;
        }
      };
      uint32_t top = 0;
#pragma unroll
      for (int r = 0; r < kBlockRows; ++r) {
        if (!(todo >> r & 1)) continue;
        float y[PER];
        values(r, y);
        top = max(top, top_bits<PER>(y));
      }
      const float inv = open_block<D>(top, side ? had_v : had_k, codes + to * D, ex + side);
#pragma unroll
      for (int r = 0; r < kBlockRows; ++r) {
        if (!(todo >> r & 1)) continue;
        float y[PER];
        values(r, y);
        code_row<PER>(y, inv, codes + (to + r) * D);
      }
    }
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

template <int kThreads, int kKeys>
static cudaError_t run_select(const ProfileDims& pd, const PagedArgs& a, const EvictArgs& n,
                              cudaStream_t s) {
  const auto k = evict_select_kernel<kThreads, kKeys>;
  const int smem = kKeys * (int)sizeof(uint32_t);
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  return e == cudaSuccess ? launch_pdl(k, pd.Gkv, kThreads, smem, s, a, n, pd.HLkv) : e;
}

cudaError_t launch_evict_q8(const ProfileDims& pd, const PagedArgs& a, const EvictArgs& n,
                            cudaStream_t s) {
  // Rows that do not fit cost the small form dear: 77 of 256 caches cut from 7801 rows 167 us, the
  // large form 19; 307 of 1024 from 7001 (d = 64) 331 and 70.  Where all fit it has more caches on
  // an SM: 4096 cut from 2001 rows 190 us and 285 (32 of them 23 and 16).  What is known here is the
  // room that the table gives a cache on average, and the prompt's length: of a prompt longer than
  // what fits some head may keep every row, unless the caches are those of sequences behind it, with
  // room for their own tokens alone (a mix of all policies has room for 0.4 of the prompt).
  constexpr int kFits = 4096;
  const long long room = (long long)a.table_len * kPageRows / pd.Gkv;
  const bool longer = room > kFits || (pd.n > kFits && room > pd.n / 8);
  const cudaError_t e =
      longer ? run_select<1024, 49152>(pd, a, n, s) : run_select<256, kFits>(pd, a, n, s);
  if (e != cudaSuccess) return e;
  const int blocks = n.budget / kBlockRows;
  const long long warps = (long long)cdiv(blocks, kMoveBlocks) * pd.Gkv;
  const long long grid = (warps + kMoveWarps - 1) / kMoveWarps;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  return launch_pdl(pd.d == 64 ? evict_move_kernel<64> : evict_move_kernel<128>, (unsigned)grid,
                    kMoveWarps * 32, 0, s, a, n, blocks);
}

}  // namespace fg
