// Appending new tokens' rows to paged 8-bit caches (Model Tells You What to
// Discard, Method: keys and values appended at each step by the prompt-time
// policy), with the position rotation of the keys on the way.
//
// Up to kFew tokens, one launch: a CTA per cache, in which every warp
// classifies the tokens, one a lane, and takes the K or the V rows of a
// destination block of 16 rows at a time.
//
// More, two launches.  The first (per sequence and 256 caches) classifies the
// tokens once, lists the special and the special-or-punctuation ones (every
// cache of the sequence takes its never-evicted rows from one of these lists
// or from all tokens), takes the pages that the segments grow into, writes
// the new row counts and forms the (cos, sin) of every position once for all
// caches.  The second gives each warp the K or the V rows of one destination
// block of 16 rows.  In both a block's exponent is settled once and its codes
// are rounded again at most once.
//
// Short chains of dependent loads, not bytes, set the time of all but long
// calls: what does not depend on each other is asked for together.
#include "fg_paged.cuh"

namespace fg {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ int new_tokens(const AppendArgs& n, int b) {
  if (n.pos[b] < 0) return 0;
  return n.n_new ? max(0, min(n.n_new[b], n.m)) : n.m;
}

__global__ void __launch_bounds__(kThreads) append_plan_kernel(const PagedArgs a,
                                                               const AppendArgs n, int HLkv) {
  __shared__ int scr[33];
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.y;
  const int cnt = new_tokens(n, b);
  const int local = blockIdx.x * kThreads + threadIdx.x;  // cache of the sequence
  int n_s = 0, n_sp = 0;  // special, special or punctuation tokens
  if (blockIdx.x * kThreads < HLkv) {  // uniform over the CTA
    int32_t* ls = n.lists + (size_t)b * 2 * n.m;
    int32_t* lsp = ls + n.m;
    for (int base = 0; base < cnt; base += kThreads) {
      const int i = base + threadIdx.x;
      bool s = false, sp = false;
      if (i < cnt) {
        const int tau = n.ids[(size_t)b * n.m + i];
        s = id_in(tau, n.special, n.ns);
        sp = s || id_in(tau, n.punct, n.np);
      }
      int tot;
      const int before = block_exclusive_scan((int)s + ((int)sp << 16), scr, &tot);
      if (blockIdx.x == 0) {
        if (s) ls[n_s + (before & 0xffff)] = i;
        if (sp) lsp[n_sp + (before >> 16)] = i;
      }
      n_s += tot & 0xffff;
      n_sp += tot >> 16;
    }
  }
  if (local < HLkv) {
    const int c = b * HLkv + local;
    const fg_paged_desc d = a.caches[c];
    const int had = a.rows[c];
    const long long cap = (long long)d.max_pages * kPageRows;
    const int old = (int)max(0LL, min((long long)had, cap));
    if (old != had) atomicOr(a.dev_err, kErrInvalid);
    const int want = d.policy == FG_POLICY_FULL ? cnt : d.policy == FG_POLICY_S ? n_s : n_sp;
    int now = (int)min((long long)old + want, min(cap, 0x7fffffffLL));
    if (now - old < want) atomicOr(a.dev_err, kErrCapacity);
    if (now > old) {
      for (int i = old / kPageRows; i <= (now - 1) / kPageRows; ++i) {
        if (d.first_page < 0 || d.first_page > a.table_len - 1 - i) {
          atomicOr(a.dev_err, kErrInvalid);
          now = max(old, i * kPageRows);
          break;
        }
        int32_t* entry = a.table + d.first_page + i;
        int page = *entry;
        if (page < 0) {
          page = atomicAdd(a.next_page, 1);
          if (page < 0 || page >= a.n_pages) {
            atomicOr(a.dev_err, kErrCapacity);
            now = max(old, i * kPageRows);
            break;
          }
          *entry = page;
        } else if (page >= a.n_pages) {
          atomicOr(a.dev_err, kErrInvalid);
          now = max(old, i * kPageRows);
          break;
        }
      }
    }
    n.old[2 * c] = old;
    n.old[2 * c + 1] = now - old;
    a.rows_out[c] = cnt > 0 ? now : had;
  }
  const int pairs = n.rope.rot / 2;
  if (pairs > 0 && cnt > 0) {
    const unsigned first = (unsigned)n.pos[b];
    float2* out = n.angles + (size_t)b * n.m * pairs;
    for (int x = local; x < cnt * pairs; x += gridDim.x * kThreads) {
      float2 cs;
      rope_cos_sin(first + x / pairs, n.rope.turns[x % pairs], cs.x, cs.y);
      out[x] = cs;
    }
  }
}

// Puts the rows of one destination block (all lanes of a warp call): lane i's
// tok goes to row i, or none (-1).  angle(tok, pair) gives (cos, sin).  Up to
// kHold rows stay in registers between the search for the largest value and
// the coding; more are read twice.
template <typename T, int D, int kHold, typename Angle>
__device__ __forceinline__ void append_block(const PagedArgs& a, const AppendArgs& n, int c,
                                             int tok, unsigned p0, int page, int r, int which,
                                             bool fresh, Angle angle) {
  constexpr int PER = D / 32;
  const int lane = threadIdx.x & 31;
  const uint32_t mask = __ballot_sync(0xffffffffu, tok >= 0);
  if (mask == 0) return;
  if (page < 0) {
    if (lane == 0) atomicOr(a.dev_err, kErrInvalid);
    return;
  }
  if (which == 0 && tok >= 0) a.pos[(size_t)page * kPageRows + r + lane] = (int)(p0 + tok);
  const T* src = (const T*)(which ? n.v_new : n.k_new) + (size_t)c * n.m * D;
  uint8_t* codes = (which ? a.vp : a.kp) + ((size_t)page * kPageRows + r) * D;
  const bool turn = which == 0 && n.rope.rot > 0;
  float x[kHold][PER];
  auto read = [&](uint32_t m) {  // the rows of m's first kHold bits, rotated
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
      if (m == 0) break;
      load_row<PER>(src + (size_t)__shfl_sync(0xffffffffu, tok, __ffs(m) - 1) * D, x[i]);
      m &= m - 1;
    }
  };
  auto rotate = [&](uint32_t m) {
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
      if (m == 0) break;
      const int t = __shfl_sync(0xffffffffu, tok, __ffs(m) - 1);
      m &= m - 1;
      float2 cs[PER];
      row_angles<PER>(cs, n.rope.rot, n.rope.style, [&](int p) { return angle(t, p); });
      rotate_row<PER>(x[i], cs, n.rope.rot, n.rope.style);
    }
    return m;
  };
  auto skip = [](uint32_t m) {
#pragma unroll
    for (int i = 0; i < kHold; ++i) m &= m - 1;  // 0 stays 0
    return m;
  };
  uint32_t top = 0;
  for (uint32_t m = mask; m; m = skip(m)) {
    read(m);
    if (turn) rotate(m);
    uint32_t left = m;
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
      if (left == 0) break;
      left &= left - 1;
      top = max(top, row_top<PER>(x[i]));
    }
  }
  const float inv = open_block<D>(
      top, fresh, codes, a.exps + ((size_t)page * kPageBlocks + r / kBlockRows) * 2 + which);
  const bool held = skip(mask) == 0;
  for (uint32_t m = mask; m; m = skip(m)) {
    if (!held) {
      read(m);
      if (turn) rotate(m);
    }
    uint32_t left = m;
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
      if (left == 0) break;
      code_row<PER>(x[i], inv, codes + (__ffs(left) - 1) * D);
      left &= left - 1;
    }
  }
}

// Where the last `in` of cnt tokens go in a ring of w slots: the j-th block
// they touch, and the token (the one of that slot among them) of row `lane`.
struct RingBlock {
  int block, tok;
};
__device__ __forceinline__ RingBlock ring_block(unsigned p0, int cnt, int in, int w, int j) {
  const int lane = threadIdx.x & 31;
  const unsigned last = p0 + (unsigned)cnt - 1, uw = (unsigned)w;
  RingBlock o;
  o.block = (int)(((last + 1 - (unsigned)in) % uw / kBlockRows + (unsigned)j) %
                  (unsigned)cdiv(w, kBlockRows));
  o.tok = -1;
  const unsigned slot = (unsigned)(o.block * kBlockRows + lane);
  if (lane < kBlockRows && slot < uw) {
    const unsigned back = (last % uw + uw - slot) % uw;  // the slot's position is last - back
    if (back < (unsigned)in) o.tok = cnt - 1 - (int)back;
  }
  return o;
}

// Blocks of 16 rows that m consecutive rows may touch (wrap: a ring's last
// block may be short, which costs one more).
__host__ __device__ inline int touched(int m, bool wrap) {
  return m <= 1 ? m : (m + kBlockRows - 2) / kBlockRows + 1 + (wrap ? 1 : 0);
}

constexpr int kFew = 32;
constexpr int kFewWarps = 4;

// One CTA per cache, at most kFew tokens (lane i: token i).
template <typename T, int D>
__global__ void __launch_bounds__(kFewWarps * 32)
    append_few_kernel(const PagedArgs a, const AppendArgs n, int HLkv) {
  __shared__ int sm_page[2], sm_stored;
  __shared__ float2 sm_angle[kFew][D / 2];
  const int c = blockIdx.x, b = c / HLkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const fg_paged_desc d = a.caches[c];
  const LaneSet special(n.special, n.ns), punct(n.punct, n.np);
  griddep_wait();
  griddep_launch_dependents();
  const int pos = n.pos[b], had = a.rows[c];
  const int tau = lane < n.m ? n.ids[(size_t)b * n.m + lane] : 0;
  int cnt = n.n_new ? max(0, min(n.n_new[b], n.m)) : n.m;
  if (pos < 0) cnt = 0;
  const unsigned p0 = (unsigned)pos;
  const int old = live_rows(d, had);
  // the pages that the new rows may fall in (at most two), as they are
  const int page0 = old / kPageRows;
  int page = lane < 2 ? page_at(a, d.first_page, d.max_pages, page0 + lane) : -1;
  const bool s = special.has_mine(tau), sp = punct.has_mine(tau) || s;
  const bool to_static = lane < cnt && (d.policy == FG_POLICY_FULL ? true
                                        : d.policy == FG_POLICY_S  ? s
                                                                   : sp);
  const uint32_t st = __ballot_sync(0xffffffffu, to_static);
  if (warp == 0) {
    const int want = __popc(st);
    int stored = (int)min((long long)want,
                          min((long long)d.max_pages * kPageRows, 0x7fffffffLL) - old);
    stored = max(stored, 0);
    if (lane == 0) {
      if (old != had && cnt > 0) atomicOr(a.dev_err, kErrInvalid);
      if (stored < want) atomicOr(a.dev_err, kErrCapacity);
    }
    const int need = stored > 0 ? (old + stored - 1) / kPageRows - page0 + 1 : 0;
    for (int i = 0; i < need; ++i) {
      int p = __shfl_sync(0xffffffffu, page, i);
      if (p < 0) {  // uniform over the warp
        if (lane == 0) {
          int err = kErrInvalid;
          const int e = page0 + i;
          if (d.first_page >= 0 && d.first_page <= a.table_len - 1 - e &&
              a.table[d.first_page + e] < 0) {
            p = atomicAdd(a.next_page, 1);
            if (p >= 0 && p < a.n_pages) {
              a.table[d.first_page + e] = p;
            } else {
              p = -1;
              err = kErrCapacity;
            }
          }
          if (p < 0) atomicOr(a.dev_err, err);
        }
        p = __shfl_sync(0xffffffffu, p, 0);
        if (p < 0) {  // what fits before this page is stored
          stored = max(0, (page0 + i) * kPageRows - old);
          break;
        }
        if (lane == i) page = p;
      }
    }
    if (lane < 2) sm_page[lane] = page;
    if (lane == 0) sm_stored = stored;
  }
  const int pairs = n.rope.rot / 2;
  for (int x = threadIdx.x; x < cnt * pairs; x += kFewWarps * 32) {
    float2 cs;
    rope_cos_sin(p0 + (unsigned)(x / pairs), n.rope.turns[x % pairs], cs.x, cs.y);
    sm_angle[x / pairs][x % pairs] = cs;
  }
  __syncthreads();
  const int stored = sm_stored;
  if (threadIdx.x == 0) a.rows_out[c] = cnt > 0 ? old + stored : had;  // every warp has read it
  const int seg = stored > 0 ? (old + stored - 1) / kBlockRows - old / kBlockRows + 1 : 0;
  const int in = d.policy == FG_POLICY_SPFL && d.w > 0 ? min(cnt, d.w) : 0;
  const int ring = in > 0 ? min(cdiv(d.w, kBlockRows), touched(in, true)) : 0;
  auto angle = [&](int tok, int p) { return sm_angle[tok][p]; };
  for (int task = warp; task < 2 * (seg + ring); task += kFewWarps) {
    const int which = task & 1, j = task >> 1;
    if (j < seg) {
      const int block = old / kBlockRows + j, row = block * kBlockRows;
      const int k = row + lane - old;
      const int tok = lane < kBlockRows && k >= 0 && k < stored ? (int)__fns(st, 0, k + 1) : -1;
      append_block<T, D, 4>(a, n, c, tok, p0, sm_page[row / kPageRows - page0], row % kPageRows,
                         which, row >= old, angle);
    } else {
      RingBlock o = ring_block(p0, cnt, in, d.w, j - seg);
      if (o.tok >= 0 && (st >> o.tok & 1)) o.tok = -1;
      const int row = o.block * kBlockRows;
      append_block<T, D, 4>(a, n, c, o.tok, p0,
                         page_at(a, d.ring_page, d.ring_pages, row / kPageRows), row % kPageRows,
                         which, false, angle);
    }
  }
}

// One warp per (cache, destination block, K or V).  seg_blocks: blocks that
// the call's rows of a never-evicted segment may touch; ring_blocks likewise.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) append_q8_kernel(const PagedArgs a, const AppendArgs n,
                                                             int HLkv, int seg_blocks,
                                                             int ring_blocks, int max_w,
                                                             long long tasks) {
  const long long task = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int which = (int)(task & 1), per = seg_blocks + ring_blocks;
  const int j = (int)((task >> 1) % per);
  const bool in_grid = task < tasks;
  const int c = in_grid ? (int)((task >> 1) / per) : 0, b = c / HLkv;
  const fg_paged_desc d = a.caches[c];
  const LaneSet special(n.special, n.ns), punct(n.punct, n.np);
  griddep_wait();
  griddep_launch_dependents();
  if (!in_grid) return;
  const int2 rows = *reinterpret_cast<const int2*>(n.old + 2 * c);  // before the call, stored
  const int cnt = new_tokens(n, b);
  if (cnt == 0) return;
  const unsigned p0 = (unsigned)n.pos[b];
  int tok = -1, row, page;  // tok: token that goes to row `lane` of the block
  bool fresh = false;
  if (j < seg_blocks) {
    row = (rows.x / kBlockRows + j) * kBlockRows;
    if (row >= rows.x + rows.y) return;
    page = page_at(a, d.first_page, d.max_pages, row / kPageRows);
    fresh = row >= rows.x;
    const int k = row + lane - rows.x;
    if (lane < kBlockRows && k >= 0 && k < rows.y) {
      const int32_t* list = n.lists + ((size_t)b * 2 + (d.policy != FG_POLICY_S)) * n.m;
      tok = d.policy == FG_POLICY_FULL ? k : list[k];
    }
  } else {
    if (d.policy != FG_POLICY_SPFL || d.w <= 0) return;
    if (d.w > max_w) {  // a descriptor of another shape: ring_blocks would not reach all of it
      if (lane == 0) atomicOr(a.dev_err, kErrInvalid);
      return;
    }
    const int in = min(cnt, d.w);  // only the last w tokens can be in the window
    if (j - seg_blocks >= cdiv(d.w, kBlockRows)) return;
    const RingBlock o = ring_block(p0, cnt, in, d.w, j - seg_blocks);
    row = o.block * kBlockRows;
    page = page_at(a, d.ring_page, d.ring_pages, row / kPageRows);
    tok = o.tok;
    const int tau = tok >= 0 ? n.ids[(size_t)b * n.m + tok] : 0;
    const bool s = special.has_mine(tau), sp = punct.has_mine(tau) || s;
    if (sp) tok = -1;  // the never-evicted segment takes it
  }
  const float2* angles = n.angles + (size_t)b * n.m * (n.rope.rot / 2);
  append_block<T, D, kBlockRows>(a, n, c, tok, p0, page, row % kPageRows, which, fresh,
                     [&](int t, int p) { return angles[(size_t)t * (n.rope.rot / 2) + p]; });
}

template <typename T, int D>
cudaError_t run_append(const ProfileDims& pd, const PagedArgs& a, const AppendArgs& n,
                       cudaStream_t s) {
  if (n.m <= kFew)
    return launch_pdl(append_few_kernel<T, D>, pd.Gkv, kFewWarps * 32, 0, s, a, n, pd.HLkv);
  // enough CTAs per sequence for its caches and, in long calls, its angles
  const int for_angles = (int)min((long long)64, ((long long)n.m * (n.rope.rot / 2) + 1023) / 1024);
  const int per_seq = max(cdiv(pd.HLkv, kThreads), for_angles);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(per_seq, pd.B);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, append_plan_kernel, a, n, pd.HLkv);
  if (e != cudaSuccess) return e;
  const int seg = touched(n.m, false);
  const int ring = min(cdiv(pd.w, kBlockRows), touched(min(n.m, pd.w), true));
  const long long tasks = 2LL * pd.Gkv * (seg + ring);
  const long long grid = (tasks + kThreads / 32 - 1) / (kThreads / 32);
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  return launch_pdl(append_q8_kernel<T, D>, (unsigned)grid, kThreads, 0, s, a, n, pd.HLkv, seg,
                    ring, pd.w, tasks);
}

}  // namespace

cudaError_t launch_append_q8(const ProfileDims& pd, const PagedArgs& a, const AppendArgs& n,
                             cudaStream_t s) {
  if (pd.dtype == FG_FP32)
    return pd.d == 64 ? run_append<float, 64>(pd, a, n, s) : run_append<float, 128>(pd, a, n, s);
  return pd.d == 64 ? run_append<__nv_bfloat16, 64>(pd, a, n, s)
                    : run_append<__nv_bfloat16, 128>(pd, a, n, s);
}

}  // namespace fg
