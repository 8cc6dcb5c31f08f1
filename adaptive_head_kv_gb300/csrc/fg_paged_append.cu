// Appending new tokens' rows to paged 8-bit caches (Model Tells You What to
// Discard, Method: keys and values appended at each step by the prompt-time
// policy), with the position rotation of the keys on the way.
//
// Two launches.  The first (per sequence and 256 caches) classifies the
// tokens once, lists the special and the special-or-punctuation ones (every
// cache of the sequence takes its never-evicted rows from one of these lists
// or from all tokens), takes the pages that the segments grow into, writes
// the new row counts and forms the (cos, sin) of every position once for all
// caches.  The second gives each warp the K or the V rows of one destination
// block of 16 rows, so the block's exponent is settled once and its codes are
// rounded again at most once.
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

// One warp per (cache, destination block, K or V).  seg_blocks: blocks that
// the call's rows of a never-evicted segment may touch; ring_blocks likewise.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) append_q8_kernel(const PagedArgs a, const AppendArgs n,
                                                             int HLkv, int seg_blocks,
                                                             int ring_blocks, int max_w,
                                                             long long tasks) {
  constexpr int PER = D / 32;
  const long long task = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  griddep_wait();
  griddep_launch_dependents();
  if (task >= tasks) return;
  const int which = (int)(task & 1), per = seg_blocks + ring_blocks;
  const int j = (int)((task >> 1) % per), c = (int)((task >> 1) / per);
  const int b = c / HLkv;
  const int cnt = new_tokens(n, b);
  if (cnt == 0) return;
  const unsigned p0 = (unsigned)n.pos[b];
  const fg_paged_desc d = a.caches[c];
  int tok = -1;  // token that goes to row `lane` of the block
  int block, first, entries;
  bool fresh = false;
  if (j < seg_blocks) {
    const int old = n.old[2 * c], stored = n.old[2 * c + 1];
    block = old / kBlockRows + j;
    first = d.first_page;
    entries = d.max_pages;
    fresh = block * kBlockRows >= old;
    const int k = block * kBlockRows + lane - old;
    if (lane < kBlockRows && k >= 0 && k < stored) {
      const int32_t* list = n.lists + ((size_t)b * 2 + (d.policy != FG_POLICY_S)) * n.m;
      tok = d.policy == FG_POLICY_FULL ? k : list[k];
    }
  } else {
    if (d.policy != FG_POLICY_SPFL || d.w <= 0) return;
    const unsigned w = (unsigned)d.w;
    if (d.w > max_w) {  // a descriptor of another shape: ring_blocks would not reach all of it
      if (lane == 0) atomicOr(a.dev_err, kErrInvalid);
      return;
    }
    const int in = min(cnt, d.w);  // only the last w tokens can be in the window
    const int blocks = cdiv(d.w, kBlockRows);
    const unsigned last = p0 + (unsigned)cnt - 1;
    if (j - seg_blocks >= blocks) return;
    block = (int)(((last + 1 - (unsigned)in) % w / kBlockRows + (unsigned)(j - seg_blocks)) %
                  (unsigned)blocks);
    first = d.ring_page;
    entries = d.ring_pages;
    const unsigned slot = (unsigned)(block * kBlockRows + lane);
    if (lane < kBlockRows && slot < w) {
      const unsigned back = (last % w + w - slot) % w;  // the slot's position is last - back
      if (back < (unsigned)in) {
        const int i = cnt - 1 - (int)back;
        const int tau = n.ids[(size_t)b * n.m + i];
        if (!id_in(tau, n.special, n.ns) && !id_in(tau, n.punct, n.np)) tok = i;
      }
    }
  }
  const uint32_t mask = __ballot_sync(0xffffffffu, tok >= 0);
  if (mask == 0) return;
  const int row = block * kBlockRows;
  const int page = page_at(a, first, entries, row / kPageRows);
  if (page < 0) {
    if (lane == 0) atomicOr(a.dev_err, kErrInvalid);
    return;
  }
  const int r = row % kPageRows;
  if (which == 0 && tok >= 0) a.pos[(size_t)page * kPageRows + r + lane] = (int)(p0 + tok);
  const T* src = (const T*)(which ? n.v_new : n.k_new) + (size_t)c * n.m * D;
  float x[kBlockRows][PER];
#pragma unroll
  for (int i = 0; i < kBlockRows; ++i) {
    const int t = __shfl_sync(0xffffffffu, tok, i);
    if (t >= 0) {
      load_row<PER>(src + (size_t)t * D, x[i]);
    } else {
#pragma unroll
      for (int k = 0; k < PER; ++k) x[i][k] = 0.f;
    }
  }
  if (which == 0 && n.rope.rot > 0) {
    const int pairs = n.rope.rot / 2;
#pragma unroll
    for (int i = 0; i < kBlockRows; ++i) {
      const int t = __shfl_sync(0xffffffffu, tok, i);
      if (t < 0) continue;
      const float2* at = n.angles + ((size_t)b * n.m + t) * pairs;
      float2 cs[PER];
      row_angles<PER>(cs, n.rope.rot, n.rope.style, [&](int p) { return at[p]; });
      rotate_row<PER>(x[i], cs, n.rope.rot, n.rope.style);
    }
  }
  put_rows<D, kBlockRows>(x, mask, 0, fresh, (which ? a.vp : a.kp) + ((size_t)page * kPageRows + r) * D,
                          a.exps + ((size_t)page * kPageBlocks + r / kBlockRows) * 2 + which);
}

// Blocks of 16 rows that m consecutive rows may touch (wrap: a ring's last
// block may be short, which costs one more).
int touched(int m, bool wrap) {
  return m <= 1 ? m : (m + kBlockRows - 2) / kBlockRows + 1 + (wrap ? 1 : 0);
}

template <typename T, int D>
cudaError_t run_append(const ProfileDims& pd, const PagedArgs& a, const AppendArgs& n,
                       cudaStream_t s) {
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
