// Appending new tokens' rows to paged 8-bit caches (Model Tells You What to
// Discard, Method: keys and values appended at each step by the prompt-time
// policy), with the position rotation of the keys on the way.
//
// Up to kFew tokens, one launch: a CTA per cache, in which every warp
// classifies the tokens, one a lane, and takes the K or the V rows of a
// destination block of 16 rows at a time.
//
// More, two launches.  In the first, every CTA counts its sequence's special
// and special-or-punctuation tokens (one also lists them: a cache takes its
// never-evicted rows from one of these lists or from all tokens), its warps
// take the pages that kPlanCaches caches grow into, 32 at a time, and write
// the new row counts; its threads form the (cos, sin) of every position once
// for all caches.  The second gives each warp the K or the V rows of one destination
// block of 16 rows.  In both a block's exponent is settled once and its codes
// are rounded again at most once.
//
// Short chains of dependent loads, not bytes, set the time of all but long
// calls: what does not depend on each other is asked for together.  Measured
// (device time): one token in 1024 caches 4.0 us, five in 2048 caches 10.6 us
// (two warps a cache take its blocks one after the other, and rows past the
// fourth of a block are read and rotated twice), 701 (fp32, d = 64) in 128
// caches 17 us, 512 in 1024 caches (229 MB) 93 us.
#include "fg_paged.cuh"

namespace fg {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ int new_tokens(const AppendArgs& n, int b) {
  const int pos = n.pos[b], cnt = n.n_new ? n.n_new[b] : n.m;  // asked for together
  return pos < 0 ? 0 : max(0, min(cnt, n.m));
}

constexpr int kPlanCaches = 8;   // caches of a CTA of the first launch

__global__ void __launch_bounds__(kThreads) append_plan_kernel(const PagedArgs a,
                                                               const AppendArgs n, int HLkv) {
  __shared__ int scr[33];
  __shared__ int sm_count[2][kThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  griddep_wait();
  griddep_launch_dependents();
  const LaneSet special(n.special, n.ns), punct(n.punct, n.np);
  const int b = blockIdx.y;
  const int cnt = new_tokens(n, b);
  int n_s = 0, n_sp = 0;  // special, special or punctuation tokens
  if (blockIdx.x == 0) {
    int32_t* ls = n.lists + (size_t)b * 2 * n.m;
    int32_t* lsp = ls + n.m;
    for (int base = 0; base < cnt; base += kThreads) {
      const int i = base + threadIdx.x;
      const int tau = i < cnt ? n.ids[(size_t)b * n.m + i] : 0;
      const bool is_s = special.has_mine(tau), is_p = punct.has_mine(tau);  // every lane asks
      const bool s = is_s && i < cnt, sp = (is_s || is_p) && i < cnt;
      int tot;
      const int before = block_exclusive_scan((int)s + ((int)sp << 16), scr, &tot);
      if (s) ls[n_s + (before & 0xffff)] = i;
      if (sp) lsp[n_sp + (before >> 16)] = i;
      n_s += tot & 0xffff;
      n_sp += tot >> 16;
    }
  } else if (blockIdx.x * kPlanCaches < HLkv) {  // the counts alone
    for (int base = 0; base < cnt; base += 4 * kThreads) {
      int tau[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = base + u * kThreads + threadIdx.x;
        tau[u] = i < cnt ? n.ids[(size_t)b * n.m + i] : 0;
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const bool in = base + u * kThreads + threadIdx.x < cnt;
        const bool s = special.has_mine(tau[u]), p = punct.has_mine(tau[u]);
        n_s += __popc(__ballot_sync(0xffffffffu, s && in));
        n_sp += __popc(__ballot_sync(0xffffffffu, (s || p) && in));
      }
    }
    if (lane == 0) {
      sm_count[0][warp] = n_s;
      sm_count[1][warp] = n_sp;
    }
    __syncthreads();
    n_s = n_sp = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      n_s += sm_count[0][w];
      n_sp += sm_count[1][w];
    }
  }
  for (int k = warp; k < kPlanCaches; k += kThreads / 32) {
    const int local = blockIdx.x * kPlanCaches + k;  // cache of the sequence
    if (local >= HLkv) break;
    const int c = b * HLkv + local;
    const fg_paged_desc d = a.caches[c];
    const int had = a.rows[c], old = live_rows(d, had);
    const int want = d.policy == FG_POLICY_FULL ? cnt : d.policy == FG_POLICY_S ? n_s : n_sp;
    const long long cap = min((long long)d.max_pages * kPageRows, 0x7fffffffLL);
    int now = (int)min((long long)old + want, max(cap, (long long)old));
    int err = (old != had || d.w != ring_slots(d, a.max_w)) && cnt > 0 ? kErrInvalid : 0;
    if (now - old < want) err |= kErrCapacity;
    const int end = now > old ? (now - 1) / kPageRows + 1 : 0;
    for (int base = old / kPageRows; base < end; base += 32) {
      const int i = base + lane;
      const bool need = i < end;
      const bool in_table = d.first_page >= 0 && d.first_page <= a.table_len - 1 - i;
      int page = need && in_table ? a.table[d.first_page + i] : a.n_pages;
      const uint32_t missing = __ballot_sync(0xffffffffu, need && page < 0);
      if (missing) {
        int first = 0;
        if (lane == 0) first = take_pages(a, __popc(missing));
        first = __shfl_sync(0xffffffffu, first, 0);
        if (missing >> lane & 1) {
          const long long p = (long long)first + __popc(missing & ((1u << lane) - 1));
          if (first >= 0 && p < a.n_pages) {
            page = (int)p;
            a.table[d.first_page + i] = page;
          } else {
            err |= kErrCapacity;
          }
        } else if (need && page >= a.n_pages) {
          err |= kErrInvalid;
        }
      } else if (need && page >= a.n_pages) {
        err |= kErrInvalid;
      }
      // what fits before the first page that is not there is stored
      const uint32_t bad = __ballot_sync(0xffffffffu, need && (page < 0 || page >= a.n_pages));
      if (bad) {
        now = max(old, (base + __ffs(bad) - 1) * kPageRows);
        break;
      }
    }
    if (err) atomicOr(a.dev_err, err);
    if (lane == 0) {
      n.old[2 * c] = old;
      n.old[2 * c + 1] = now - old;
      a.rows_out[c] = cnt > 0 ? now : had;
    }
  }
  const int pairs = n.rope.rot / 2;
  if (pairs > 0 && cnt > 0) {
    const unsigned first = (unsigned)n.pos[b];
    float2* out = n.angles + (size_t)b * n.m * pairs;
    for (long long x = (long long)blockIdx.x * kThreads + threadIdx.x; x < (long long)cnt * pairs;
         x += gridDim.x * kThreads) {
      float2 cs;
      rope_cos_sin(first + (unsigned)(x / pairs), n.rope.turns[x % pairs], cs.x, cs.y);
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
  int8_t* exp_at = a.exps + ((size_t)page * kPageBlocks + r / kBlockRows) * 2 + which;
  const int had = fresh ? -128 : *exp_at;  // asked for before the rows
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
      top = max(top, top_bits<PER>(x[i]));
    }
  }
  const float inv = open_block<D>(top, had, codes, exp_at);
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

// The same for many rows: 16-byte pieces, a row over D / E lanes, all of the
// block's rows in registers (a lane of a warp that held whole rows would have
// two or four values of each and spend most of its instructions on addresses).
template <typename T, int D>
__device__ __forceinline__ void append_full_block(const PagedArgs& a, const AppendArgs& n, int c,
                                                  int tok, unsigned p0, int page, int r,
                                                  int which, bool fresh,
                                                  const float2* __restrict__ angles) {
  constexpr int E = Vec16<T>::kElems, LPR = D / E, RPI = 32 / LPR, NI = kBlockRows / RPI;
  const int lane = threadIdx.x & 31, sub = lane / LPR, gl = lane % LPR, e0 = gl * E;
  if (!__any_sync(0xffffffffu, tok >= 0)) return;
  if (page < 0) {
    if (lane == 0) atomicOr(a.dev_err, kErrInvalid);
    return;
  }
  int8_t* exp_at = a.exps + ((size_t)page * kPageBlocks + r / kBlockRows) * 2 + which;
  const int had = fresh ? -128 : *exp_at;
  if (which == 0 && tok >= 0) a.pos[(size_t)page * kPageRows + r + lane] = (int)(p0 + tok);
  const T* src = (const T*)(which ? n.v_new : n.k_new) + (size_t)c * n.m * D + e0;
  uint8_t* codes = (which ? a.vp : a.kp) + ((size_t)page * kPageRows + r) * D;
  uint8_t* dst = codes + sub * D + e0;
  int t[NI];
  uint4 x[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    t[i] = __shfl_sync(0xffffffffu, tok, i * RPI + sub);
    x[i] = t[i] >= 0 ? ldg_stream(src + (size_t)t[i] * D) : make_uint4(0, 0, 0, 0);
  }
  const int rot = n.rope.rot, h = rot / 2;
  if (which == 0 && rot > 0) {
    const bool inter = n.rope.style == FG_ROPE_INTERLEAVED, first = e0 < h;
    // the lane that holds the other half of this lane's pairs
    const int other = inter || e0 >= rot ? lane : first ? lane + h / E : lane - h / E;
    float f[NI][E];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      unpack16(x[i], f[i], (const T*)nullptr);
      float y[E];
      if (!inter) {
        uint4 z;
        z.x = __shfl_sync(0xffffffffu, x[i].x, other);
        z.y = __shfl_sync(0xffffffffu, x[i].y, other);
        z.z = __shfl_sync(0xffffffffu, x[i].z, other);
        z.w = __shfl_sync(0xffffffffu, x[i].w, other);
        unpack16(z, y, (const T*)nullptr);
      }
      if (t[i] >= 0 && e0 < rot) {
        // two pairs' (cos, sin) a load
        const float4* cs = reinterpret_cast<const float4*>(
            angles + (size_t)t[i] * h + (inter ? e0 / 2 : e0 - (first ? 0 : h)));
        if (inter) {
#pragma unroll
          for (int k = 0; k < E; k += 4) {
            const float4 w = __ldg(cs + k / 4);
            const float u = f[i][k], v = f[i][k + 2];
            f[i][k] = u * w.x - f[i][k + 1] * w.y;
            f[i][k + 1] = f[i][k + 1] * w.x + u * w.y;
            f[i][k + 2] = v * w.z - f[i][k + 3] * w.w;
            f[i][k + 3] = f[i][k + 3] * w.z + v * w.w;
          }
        } else {
          const float sign = first ? -1.f : 1.f;
#pragma unroll
          for (int k = 0; k < E; k += 2) {
            const float4 w = __ldg(cs + k / 2);
            f[i][k] = f[i][k] * w.x + sign * y[k] * w.y;
            f[i][k + 1] = f[i][k + 1] * w.z + sign * y[k + 1] * w.w;
          }
        }
      }
      top = max(top, top_bits<E>(f[i]));
    }
    const float inv = open_block<D>(top, had, codes, exp_at);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      if (t[i] < 0) continue;
      uint32_t w[E / 4];
#pragma unroll
      for (int k = 0; k < E / 4; ++k)
        w[k] = code4(f[i][4 * k] * inv, f[i][4 * k + 1] * inv, f[i][4 * k + 2] * inv,
                     f[i][4 * k + 3] * inv);
      uint8_t* p = dst + i * RPI * D;
      if constexpr (E == 8) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
      else *reinterpret_cast<uint32_t*>(p) = w[0];
    }
  } else {
    const float inv = open_block<D>(lane_top<NI>(x, (const T*)nullptr), had, codes, exp_at);
#pragma unroll
    for (int i = 0; i < NI; ++i)
      if (t[i] >= 0) code16(x[i], inv, dst + i * RPI * D, (const T*)nullptr);
  }
}

// Where the last `in` of cnt tokens go in a ring of w slots: the j-th block
// they touch, and the token (the one of that slot among them) of row `lane`.
struct RingBlock {
  int block, tok;
};
__device__ __forceinline__ RingBlock ring_block(unsigned p0, int cnt, int in, int w, int j) {
  const int lane = threadIdx.x & 31, blocks = cdiv(w, kBlockRows);
  const int last = (int)((p0 + (unsigned)cnt - 1) % (unsigned)w);  // the last token's slot
  const int first = last + 1 - in;                                 // the first's, in (-w, w)
  RingBlock o;
  o.block = (first < 0 ? first + w : first) / kBlockRows + j;  // j <= blocks
  if (o.block >= blocks) o.block -= blocks;
  o.tok = -1;
  const int slot = o.block * kBlockRows + lane;
  if (lane < kBlockRows && slot < w) {
    // the slot's position is the last token's less `back`
    const int back = last - slot + (slot > last ? w : 0);
    if (back < in) o.tok = cnt - 1 - back;
  }
  return o;
}

// Blocks of 16 rows that m consecutive rows may touch (wrap: a ring's last
// block may be short, which costs one more).
__host__ __device__ inline int touched(int m, bool wrap) {
  return m <= 1 ? m : (m + kBlockRows - 2) / kBlockRows + 1 + (wrap ? 1 : 0);
}

// Calls of up to kFew tokens take one launch: its time grows by a microsecond a
// token, the other's first 16 tokens cost nothing.  32 caches: 12 tokens 11.6
// against 8.9 us, 32 tokens 27 against 9.6; 2048 caches: 9 tokens 16 against 19
// us, 16 tokens 26 against 23.6.  (At most 32: a token a lane.)
constexpr int kFew = 8;
constexpr int kFewWarps = 2;

// One CTA per cache, at most kFew tokens (lane i: token i).
template <typename T, int D>
__global__ void __launch_bounds__(kFewWarps * 32)
    append_few_kernel(const PagedArgs a, const AppendArgs n, int HLkv) {
  __shared__ int sm_page[2], sm_stored;
  extern __shared__ float2 sm_angle[];  // [m][rot / 2]
  const int c = blockIdx.x, b = c / HLkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  griddep_wait();
  griddep_launch_dependents();
  const fg_paged_desc d = a.caches[c];
  const LaneSet special(n.special, n.ns), punct(n.punct, n.np);
  const int pos = n.pos[b], had = a.rows[c];
  const int tau = lane < n.m ? n.ids[(size_t)b * n.m + lane] : 0;
  int cnt = n.n_new ? max(0, min(n.n_new[b], n.m)) : n.m;
  if (pos < 0) cnt = 0;
  const unsigned p0 = (unsigned)pos;
  const int old = live_rows(d, had), w = ring_slots(d, a.max_w);
  // the pages that the new rows may fall in (at most two), as they are
  const int page0 = old / kPageRows;
  int page = lane < 2 ? page_at(a, d.first_page, d.max_pages, page0 + lane) : -1;
  const bool s = special.has_mine(tau), p = punct.has_mine(tau), sp = s || p;
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
      if ((old != had || d.w != w) && cnt > 0) atomicOr(a.dev_err, kErrInvalid);
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
            p = take_pages(a, 1);
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
    sm_angle[x] = cs;
  }
  __syncthreads();
  const int stored = sm_stored;
  if (threadIdx.x == 0) a.rows_out[c] = cnt > 0 ? old + stored : had;  // every warp has read it
  const int seg = stored > 0 ? (old + stored - 1) / kBlockRows - old / kBlockRows + 1 : 0;
  const int in = d.policy == FG_POLICY_SPFL ? min(cnt, w) : 0;
  const int ring = in > 0 ? min(cdiv(w, kBlockRows), touched(in, true)) : 0;
  auto angle = [&](int tok, int p) { return sm_angle[tok * pairs + p]; };
  for (int task = warp; task < 2 * (seg + ring); task += kFewWarps) {
    const int which = task & 1, j = task >> 1;
    if (j < seg) {
      const int block = old / kBlockRows + j, row = block * kBlockRows;
      const int k = row + lane - old;
      const int tok = lane < kBlockRows && k >= 0 && k < stored ? (int)__fns(st, 0, k + 1) : -1;
      append_block<T, D, 4>(a, n, c, tok, p0, sm_page[row / kPageRows - page0], row % kPageRows,
                         which, row >= old, angle);
    } else {
      RingBlock o = ring_block(p0, cnt, in, w, j - seg);
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
// Four blocks an SM, although a block of rotated rows then leaves some of them
// in local memory: the chain of loads that opens a block needs the warps
// (7B shape, 512 tokens: three blocks without spills 135 us, four 92, five
// 105).  Without the blocks' work the same grid takes 29 us.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 4)
    append_q8_kernel(const PagedArgs a, const AppendArgs n, int HLkv, int seg_blocks,
                     int ring_blocks, uint32_t tasks) {
  const uint32_t task = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const uint32_t per = seg_blocks + ring_blocks;
  const int which = (int)(task & 1), j = (int)((task >> 1) % per);
  const bool in_grid = task < tasks;
  const int c = in_grid ? (int)((task >> 1) / per) : 0, b = c / HLkv;
  griddep_wait();
  griddep_launch_dependents();
  if (!in_grid) return;
  const fg_paged_desc d = a.caches[c];
  const LaneSet special(n.special, n.ns), punct(n.punct, n.np);
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
    const int w = ring_slots(d, a.max_w);
    if (d.policy != FG_POLICY_SPFL || w == 0) return;
    const int in = min(cnt, w);  // only the last w tokens can be in the window
    if (j - seg_blocks >= cdiv(w, kBlockRows)) return;
    const RingBlock o = ring_block(p0, cnt, in, w, j - seg_blocks);
    row = o.block * kBlockRows;
    page = page_at(a, d.ring_page, d.ring_pages, row / kPageRows);
    tok = o.tok;
    const int tau = tok >= 0 ? n.ids[(size_t)b * n.m + tok] : 0;
    const bool s = special.has_mine(tau), p = punct.has_mine(tau);
    if (s || p) tok = -1;  // the never-evicted segment takes it
  }
  const float2* angles = n.angles + (size_t)b * n.m * (n.rope.rot / 2);
  append_full_block<T, D>(a, n, c, tok, p0, page, row % kPageRows, which, fresh, angles);
}

template <typename T, int D>
cudaError_t run_append(const ProfileDims& pd, const PagedArgs& a, const AppendArgs& n,
                       cudaStream_t s) {
  if (n.m <= kFew)
    return launch_pdl(append_few_kernel<T, D>, pd.Gkv, kFewWarps * 32,
                      (size_t)n.m * (n.rope.rot / 2) * sizeof(float2), s, a, n, pd.HLkv);
  // enough CTAs per sequence for its caches and, in long calls, its angles
  const int for_angles = (int)min((long long)64, ((long long)n.m * (n.rope.rot / 2) + 1023) / 1024);
  const int per_seq = max(cdiv(pd.HLkv, kPlanCaches), for_angles);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(per_seq, pd.B);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const int seg = touched(n.m, false);
  const int ring = min(cdiv(pd.w, kBlockRows), touched(min(n.m, pd.w), true));
  const long long tasks = 2LL * pd.Gkv * (seg + ring);
  const long long grid = (tasks + kThreads / 32 - 1) / (kThreads / 32);
  if (tasks > 0xffffffffLL - kThreads / 32) return cudaErrorInvalidValue;
  cudaError_t e = cudaLaunchKernelEx(&cfg, append_plan_kernel, a, n, pd.HLkv);
  if (e != cudaSuccess) return e;
  return launch_pdl(append_q8_kernel<T, D>, (unsigned)grid, kThreads, 0, s, a, n, pd.HLkv, seg,
                    ring, (uint32_t)tasks);
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
