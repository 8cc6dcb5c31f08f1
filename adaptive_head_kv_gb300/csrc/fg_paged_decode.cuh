// One generation step over paged 8-bit caches (Model Tells You What to
// Discard, Method: head-specific caches, the prompt-time policy reused).
//
// Split-K over the work list: an item is a run of pages of one cache (its
// never-evicted segment, the last item's run growing with the rows appended
// later, then its ring).  A CTA takes one or more items in turn.  Its last
// warp streams their pages into a ring of kStages pages in shared memory by
// cp.async, across the items' borders: while the four other warps work on one
// item, the next one's descriptors, page numbers and queries are read, so the
// chain of dependent loads that opens an item (about 2 us) hides behind the
// pages in the ring.  Each of the four warps takes 16 rows of every page.
// New tokens' rows are coded by those four warps before they start; the page
// that holds one is streamed last of its item, once that is done.
//
// Both products run as warp MMAs in f16, which holds every e4m3 code exactly:
//   S^T[16 keys x 8] = K[16 keys x d] . Q^T
//   O^T[d x 8]      += V^T[d x 16 keys] . P^T
// Queries and weights take two f16 terms each (22 bits): a group of up to four
// has them side by side, column 2 i the first term of query i and 2 i + 1 the
// second, so that a lane holds both and they cost no MMA.  A group of eight takes
// a second MMA for the second terms in fp32, and one term (11 bits) in bf16:
// second MMAs cost it 19 % (192 caches of 16384 positions 75 -> 89 us; the
// queries' alone 84, the weights' alone 84), where its outputs' distance from
// the definition, 0.00156, is 0.00150 by their own rounding to bf16.
// The dimension order inside a product is free as long as both operands agree,
// so a lane's operand fragments are 16 consecutive bytes of a row; S^T's
// accumulators become P^T's operand with one 8x8 transpose per 8 keys.  The
// order of the keys is free as well: with 16-byte pieces swizzled by the row, slot_key
// puts the rows that a load phase touches on different banks.  The exponents
// of a block are two numbers for the whole MMA: K's scales the scores, V's is
// added to them in base 2, so that a weight of the product carries it.  The
// softmax's own sum is kept apart, against the maximum of the scores alone: a
// row counts in it however small its values are beside others (a block of zeros
// has the least exponent).  A weight enters the product in f16, times 2^15:
// nothing below 2^-40 of the largest weight times 2^exponent.
//
// Bound by HBM: 2 d bytes a row.  Unpacking costs one conversion per two
// codes; scoring on the SIMT lanes would cost four instructions per two
// codes and query, past the row stream's pace at two queries already.  The
// MMA that takes e4m3 operands (k = 32, queries as sums of three e4m3 terms)
// was slower (7B shape 52 -> 64 us): with operands that change it runs at
// 0.30 a nanosecond and SM, the f16 one (k = 16) at 0.66.
//
// Measured (device time; bf16, d = 128, of the 6.78 TB/s that a copy reaches):
// 1024 caches of the 7B shape (278 MB) 51.5 us, 0.80; 8192 caches 349 us, 0.94;
// 512 caches of 32768 positions 287 us, 0.99; 128 caches of 16384 positions,
// groups of 8, 303 us, 0.94, groups of 4 292 us, 0.97; 8192 caches, fp32 351 us,
// 0.94, d = 64 204 us, 0.80 (a block of 16 rows costs a warp about 1500 cycles,
// less than half of them for its bytes); 32 caches of 128 positions 6.1 us.
// A list made before the caches grew costs more: the last item of a segment
// takes every later row (32 caches, 8192 rows since: 77 us, with a new list 14).
#pragma once

#include <type_traits>

#include "fg_paged.cuh"
#include "fg_sm100.cuh"

namespace fg {
namespace {

constexpr int kWarps = 4;  // that compute
constexpr int kThreads = (kWarps + 1) * 32;
constexpr int kMaxR = 8;
// Maximum before the first score, finite so that differences are: what has none weighs 0, and a
// NaN in its sum stays.
constexpr float kNoScore = -3.402823466e38f;
constexpr float kPBits = 15.f;  // weights are formed times 2^15, near the top of f16's range

__device__ __forceinline__ void mma_f16_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// (lo, hi) -> f16x2, nearest even; values past f16's range become infinite.
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 unpack_f16x2(uint32_t w) {
  float2 f;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(w));
  return f;
}

using sm100::ex2;

__device__ __forceinline__ uint4 lds16(uint32_t p) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(p)
               : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t p) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(p) : "memory");
  return v;
}
template <int D>
struct Piece;  // a lane's D / 8 codes of a V row
template <>
struct Piece<128> {
  uint4 v;
  __device__ void load(uint32_t p) { v = lds16(p); }
  __device__ void zero() { v = make_uint4(0, 0, 0, 0); }
  __device__ uint32_t word(int i) const { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
};
template <>
struct Piece<64> {
  uint2 v;
  __device__ void load(uint32_t p) { v = lds8(p); }
  __device__ void zero() { v = make_uint2(0, 0); }
  __device__ uint32_t word(int i) const { return i == 0 ? v.x : v.y; }
};

// What a stage of the ring holds beside the codes: its page's rows and
// exponents, and the item it belongs to.
struct StageInfo {
  int row, end;      // first row (or slot) of the page, end of the item's rows
  int flags;         // kSeg, kRing or kNone (no page); kLast: the item's last page
  int t;             // the sequence's position
  uint32_t exps[2];  // of the page's four blocks: (K, V) bytes
  int w;             // ring slots
  int alone;         // the cache's only item: its sums are the result
  int item, cache;   // item -1: of a sequence that takes no part
  int page;          // (kScores)
};
enum { kSeg, kRing, kNone, kKind = 3, kLast = 4 };

// What becomes of an item's sums.  kDecode: of a cache's only item they are the
// result, else partial results for the combine.  kParts: partial results always (the
// combine joins them with what lies outside the cache).  kScores: also every
// segment row's scores are written, for the rows' weights.
enum Mode { kDecode, kParts, kScores };
template <int kMode>
using ModeArgs = typename std::conditional<kMode == kDecode, PagedDecodeArgs, StepArgs>::type;

// Second MMAs for the queries' and weights' second terms?  Weights that add up over a
// generation are formed from 22-bit queries in bf16 groups of eight too.
template <typename T>
__host__ __device__ constexpr bool wide(bool fold, int mode) {
  return !fold && (sizeof(T) == 4 || mode == kScores);
}

// The merge of an item's warps takes the queries of a group of eight in two halves where the
// scores' second terms fill the stages, so that three blocks still fit an SM (192 caches of 8192
// positions: two blocks 99 us, three 70 us).
template <bool kFold, int kMode>
__host__ __device__ constexpr int kHalves() {
  return kMode == kScores && !kFold ? 2 : 1;
}

// A stage: a page's K and V codes, its rows' positions, StageInfo, and, in an
// item's first stage, the group's queries: f16 terms and the power of
// two each query was divided by.  Row r's 16-byte piece c sits at piece c ^ swizzle(r).
// A load phase (8 lanes of 16 bytes, 16 of 8) of the K fragments touches all
// pieces of one half (d = 128) or all pieces (d = 64) of two rows, one of the
// V fragments two adjacent pieces of four rows; slot_key orders the 8 keys of
// a tile so that these fall on different banks.
template <int D, bool kFold, bool kWide>
struct Ring {
  static constexpr int kStages = D == 128 ? 3 : 4;
  static constexpr int kV = kPageRows * D, kPos = 2 * kV, kInfo = kPos + kPageRows * 4;
  static constexpr int kQExp = kInfo + 64, kQ = kQExp + 64;
  // term t of query i: column 2 i + t, or of two sets of columns
  static constexpr int kQNext = (kFold ? 2 : 1) * D * 2;
  static constexpr int kQTerm = (kFold ? 1 : kMaxR) * D * 2;
  static constexpr int kStride = (kQ + kMaxR * D * 2 + (kWide ? kQTerm : 0) + 127) / 128 * 128;
  static constexpr int kBytes = kStages * kStride;
  __device__ static int swizzle(int r) { return D == 128 ? r & 7 : r & 2; }
  __device__ static int slot_key(int n) {
    const int k = n >> 1;
    return D == 128 ? (n & 1 ? (n + 4) & 7 : n) : (n & 1 ? 4 + (k ^ 1) : k);
  }
};
static_assert(sizeof(StageInfo) <= 64 && kMaxR * 4 <= 64, "room in a stage");

// Barrier waits end after a second at most: the CTA then runs on without
// waiting (every address it forms stays in bounds) and reports FG_EDEVICE.
struct Bars {
  uint64_t full[5], empty[5], puts, sync;
  int stop;
};
// False once a wait has run out.
__device__ __forceinline__ bool wait_bar(Bars* s, uint64_t* bar, uint32_t parity, int32_t* err) {
  if (sm100::mbar_try_wait(bar, parity)) return true;
  if (*(volatile int*)&s->stop) return false;
  if (sm100::mbar_wait(bar, parity)) return true;
  *(volatile int*)&s->stop = 1;
  atomicOr(err, kErrDevice);
  return false;
}
__device__ __forceinline__ void arrive_after_copies(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(sm100::smem_addr(bar))
               : "memory");
}

// Where the step's token goes in a cache, if it falls in an item's pages.
struct Put {
  int at;     // row of the segment or slot of the ring, -1: not in this item
  bool ring;
};
// All lanes call; w: slots of the ring, `old`: rows of the segment before the step.
__device__ __forceinline__ Put item_put(const PagedDecodeArgs& n, const PagedItem& it,
                                        const fg_paged_desc& hd, const LaneSet& special,
                                        const LaneSet& punct, int w, int old, int t, int tau) {
  Put p{-1, false};
  if (!n.k_new) return p;
  const int page = old / kPageRows;
  const bool seg_mine = page >= it.seg0 && (it.last || page < it.seg1);
  const int slot = hd.policy == FG_POLICY_SPFL && w > 0 ? t % w : -1;
  const bool ring_mine = slot >= 0 && slot / kPageRows >= it.ring0 && slot / kPageRows < it.ring1;
  if (!seg_mine && !ring_mine) return p;
  const bool s = special.has(tau), sp = s || punct.has(tau);
  p.ring = !joins_static(hd.policy, s, sp);
  if (p.ring ? ring_mine : seg_mine) p.at = p.ring ? slot : old;
  return p;
}
__device__ __forceinline__ uint32_t word4(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// The page of an item's new row, taken if it is the segment's first there (all lanes call); -1 and a
// flag if there is none.
__device__ __forceinline__ int put_page(const PagedArgs& a, const fg_paged_desc& hd,
                                        const Put& put) {
  const int first = put.ring ? hd.ring_page : hd.first_page;
  const int entries = put.ring ? hd.ring_pages : hd.max_pages;
  const int i = put.at / kPageRows;
  int page = page_at(a, first, entries, i);
  if (page < 0) {
    if ((threadIdx.x & 31) == 0) {
      int err = kErrInvalid;
      if (!put.ring && i >= entries) {
        err = kErrCapacity;
      } else if (!put.ring && first >= 0 && first <= a.table_len - 1 - i &&
                 a.table[first + i] < 0) {
        page = take_pages(a, 1);
        if (page >= 0 && page < a.n_pages) {
          a.table[first + i] = page;
        } else {
          page = -1;
          err = kErrCapacity;
        }
      }
      if (page < 0) atomicOr(a.dev_err, err);
    }
    page = __shfl_sync(0xffffffffu, page, 0);
  }
  return page;
}

// Is the new row the first of a block, which then starts afresh?
__device__ __forceinline__ bool put_opens(const Put& put) {
  return !put.ring && put.at % kBlockRows == 0;
}

// Codes the new row, K rotated, into that page; had_k, had_v: its block's exponents, -128 if it
// opens the block.  Returns the powers of two that K and V were multiplied by.
template <int D, int kMode>
__device__ __forceinline__ float2 put_row(const PagedArgs& a, const ModeArgs<kMode>& n,
                                          const Put& put, int page, int t, bool pinned, int had_k,
                                          int had_v,
                                          const float (&xk)[D / 32], const float (&xv)[D / 32]) {
  constexpr int PER = D / 32;
  const int r = put.at % kPageRows, blk = r / kBlockRows;
  const size_t row = (size_t)page * kPageRows + blk * kBlockRows;
  int8_t* ex = a.exps + ((size_t)page * kPageBlocks + blk) * 2;
  uint8_t *kb = a.kp + row * D, *vb = a.vp + row * D;
  float2 f;
  f.x = open_block<D>(top_bits<PER>(xk), had_k, kb, ex);
  code_row<PER>(xk, f.x, kb + r % kBlockRows * D);
  f.y = open_block<D>(top_bits<PER>(xv), had_v, vb, ex + 1);
  code_row<PER>(xv, f.y, vb + r % kBlockRows * D);
  if ((threadIdx.x & 31) == 0) {
    a.pos[(size_t)page * kPageRows + r] = t;
    if constexpr (kMode == kScores)  // nothing received yet; a special token's row is pinned
      if (!put.ring) n.row_w[(size_t)page * kPageRows + r] = pinned ? -FG_NEG_INF : 0.f;
  }
  return f;
}

// Codes the new token's row of an item into its page (all lanes call).
template <typename T, int D, int kMode>
__device__ __forceinline__ void put_token(const PagedArgs& a, const ModeArgs<kMode>& n, int c,
                                          const fg_paged_desc& hd, const Put& put, int t,
                                          bool pinned) {
  constexpr int PER = D / 32;
  float xk[PER], xv[PER];
  load_row<PER>((const T*)n.k_new + (size_t)c * D, xk);
  load_row<PER>((const T*)n.v_new + (size_t)c * D, xv);
  const int page = put_page(a, hd, put);
  if (page < 0) return;
  if (n.rope.rot > 0) {
    float2 cs[PER];
    row_angles<PER>(cs, n.rope.rot, n.rope.style, [&](int p) {
      float2 y;
      rope_cos_sin((unsigned)t, n.rope.turns[p], y.x, y.y);
      return y;
    });
    rotate_row<PER>(xk, cs, n.rope.rot, n.rope.style);
  }
  const int8_t* ex =
      a.exps + ((size_t)page * kPageBlocks + put.at % kPageRows / kBlockRows) * 2;
  const bool opens = put_opens(put);
  put_row<D, kMode>(a, n, put, page, t, pinned, opens ? -128 : ex[0], opens ? -128 : ex[1], xk, xv);
}

// The streaming warp.
template <typename T, int D, bool kFold, int kMode>
__device__ __forceinline__ void stream_items(const PagedArgs& a, const ModeArgs<kMode>& n, int Gkv,
                                             int H, int R, int HLkv, uint8_t* ring_smem, Bars* bars,
                                             int wi, int wi_end, PagedItem it, fg_paged_desc hd,
                                             int items, const LaneSet& special,
                                             const LaneSet& punct) {
  constexpr bool kWide = wide<T>(kFold, kMode), kTwo = kFold || kWide;
  using RG = Ring<D, kFold, kWide>;
  constexpr int PER = D / 32, CPR = D / 16;  // values per lane of a row; 16-byte pieces per row
  constexpr int kQueries = kFold ? kMaxR / 2 : kMaxR;
  const int lane = threadIdx.x & 31;
  const uint32_t base = sm100::smem_addr(ring_smem);
  bool puts_done = false;
  auto wait_puts = [&]() {
    if (!puts_done) wait_bar(bars, &bars->puts, 0, a.dev_err);
    puts_done = true;
  };
  int stage = 0;
  bool opened = true;  // hd and items are the first item's
  for (; wi < wi_end; ++wi) {
    const bool known = (unsigned)it.cache < (unsigned)Gkv;
    if (!known && lane == 0) atomicOr(a.dev_err, kErrInvalid);
    const int c = known ? it.cache : 0, b = c / HLkv;
    if (!opened) {
      hd = a.caches[c];
      items = a.ranges[c].y;
    }
    opened = false;
    const bool alone = kMode == kDecode && items == 1 && known;
    const int t = known ? n.pos[b] : -1, had = a.rows[c], tau = n.k_new ? n.ids[b] : 0;
    const PagedItem cur = it;
    if (wi + 1 < wi_end) it = a.items[wi + 1];  // known by the time this item is through
    // the group's queries and the angles' turns, on their way while the pages are looked up
    const size_t g0 = (size_t)(c / (H / R)) * H + (size_t)(c % (H / R)) * R;
    float x[kQueries][PER];
#pragma unroll
    for (int qi = 0; qi < kQueries; ++qi)
      if (qi < R) load_row<PER>((const T*)n.q + (g0 + qi) * D, x[qi]);
    if (t < 0) {  // the sequence takes no part: one empty stage says so
      const int slot = stage % RG::kStages;
      wait_bar(bars, &bars->empty[slot], (stage / RG::kStages & 1) ^ 1, a.dev_err);
      if (lane == 0) {
        StageInfo* info = reinterpret_cast<StageInfo*>(ring_smem + slot * RG::kStride + RG::kInfo);
        info->flags = kNone | kLast;
        info->item = -1;
        if (alone) a.rows_out[c] = had;
      }
      arrive_after_copies(&bars->full[slot]);
      sm100::mbar_arrive(&bars->full[slot]);
      ++stage;
      continue;
    }
    if (hd.w != ring_slots(hd, a.max_w)) hd.w = -1;  // flagged below
    const int old = live_rows(hd, had);
    if ((old != had || hd.w < 0) && cur.last && lane == 0) atomicOr(a.dev_err, kErrInvalid);
    const Put put = item_put(n, cur, hd, special, punct, hd.w, old, t, tau);
    int seg_end = cur.last ? old : (int)min((long long)old, (long long)cur.seg1 * kPageRows);
    const int ring_end = (int)min((long long)hd.w, (long long)cur.ring1 * kPageRows);
    auto pages_of = [](int page0, int end) {
      const int rows = end - page0 * kPageRows;
      return rows > 0 ? cdiv(rows, kPageRows) : 0;
    };
    int n_seg = pages_of(cur.seg0, seg_end);
    const int n_ring = cur.ring1 > cur.ring0 ? pages_of(cur.ring0, ring_end) : 0;
    bool grown = false;  // the new row opens a page of its own
    if (put.at >= 0 && !put.ring) {
      grown = old % kPageRows == 0;
      if (grown) ++n_seg;
    }
    const int pages = n_seg + n_ring;
    // the page of the new row goes last
    const int put_j = put.at < 0 ? -1
                      : put.ring ? n_seg + put.at / kPageRows - cur.ring0
                                 : put.at / kPageRows - cur.seg0;
    auto page_j = [&](int j) {
      return j < n_seg ? page_at(a, hd.first_page, hd.max_pages, cur.seg0 + j)
                       : page_at(a, hd.ring_page, hd.ring_pages, cur.ring0 + j - n_seg);
    };
    // pages 32 at a time, in streaming order: lane l holds one and its exponents
    int page_l = -1;
    uint2 exp_l = make_uint2(0, 0);
    auto fetch = [&](int group) {
      int k = group * 32 + lane;
      page_l = -1;
      if (k >= pages - (put_j >= 0 ? 1 : 0)) return;  // the new row's page is looked up later
      if (k == put_j) k = pages - 1;
      page_l = page_j(k);
      if (page_l < 0)
        atomicOr(a.dev_err, kErrInvalid);
      else
        exp_l = *reinterpret_cast<const uint2*>(a.exps + (size_t)page_l * kPageBlocks * 2);
    };
    fetch(0);
    // the group's queries into an item's first stage: rotated, divided by the power of two that
    // brings the largest value to [2^13, 2^14), as f16 (two terms: and what f16 loses, times 2^11)
    auto put_queries = [&](uint8_t* st) {
      float2 cs[PER];
      if (n.rope.rot > 0)
        row_angles<PER>(cs, n.rope.rot, n.rope.style, [&](int p) {
          float2 y;
          rope_cos_sin<kTwo>((unsigned)t, n.rope.turns[p], y.x, y.y);
          return y;
        });
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
          uint8_t* q = st + RG::kQ + qi * RG::kQNext + (lane * PER + k) * 2;
          *reinterpret_cast<uint32_t*>(q) = hi;
          if constexpr (kTwo) {
            const float2 f = unpack_f16x2(hi);
            *reinterpret_cast<uint32_t*>(q + RG::kQTerm) =
                pack_f16x2((u - f.x) * 2048.f, (v - f.y) * 2048.f);
          }
        }
        if (lane == 0) reinterpret_cast<float*>(st + RG::kQExp)[qi] = pow2f(eq);
      }
    };
    const bool late = stage == 0 && pages > RG::kStages;
    // an item without a page has one empty stage
    for (int k = 0; k == 0 || k < pages; ++k, ++stage) {
      const int slot = stage % RG::kStages;
      if (k > 0 && (k & 31) == 0) fetch(k >> 5);
      wait_bar(bars, &bars->empty[slot], (stage / RG::kStages & 1) ^ 1, a.dev_err);
      int page = __shfl_sync(0xffffffffu, page_l, k & 31);
      uint2 ex = make_uint2(0, 0);
      const bool with_put = put_j >= 0 && k == pages - 1;
      int j = k == put_j ? pages - 1 : k;
      if (with_put) {
        j = put_j;
        wait_puts();
        page = page_j(j);
        if (page >= 0)
          ex = __ldcg(reinterpret_cast<const uint2*>(a.exps + (size_t)page * kPageBlocks * 2));
        if (page < 0 && !grown && lane == 0) atomicOr(a.dev_err, kErrInvalid);
        if (page >= 0 && !put.ring) seg_end = put.at + 1;
      }
      const bool ring = j >= n_seg;
      const int row = (ring ? cur.ring0 + j - n_seg : cur.seg0 + j) * kPageRows;
      const int end = ring ? ring_end : seg_end;
      if (page >= 0 && pages > 0) {
        const uint32_t st = base + (uint32_t)(slot * RG::kStride);
        const uint8_t* kb = a.kp + (size_t)page * kPageRows * D + lane * 16;
        const uint8_t* vb = a.vp + (size_t)page * kPageRows * D + lane * 16;
        const int blocks = min(kPageBlocks, cdiv(end - row, kBlockRows));  // with rows
        constexpr int kPer = kBlockRows * CPR / 32;  // pieces per lane of a block
#pragma unroll
        for (int i = 0; i < kPageBlocks * kPer; ++i) {
          if (i / kPer < blocks) {
            const int r = i * (32 / CPR) + lane / CPR;
            const uint32_t dst = st + (uint32_t)(r * D + (((lane % CPR) ^ RG::swizzle(r)) << 4));
            cp_async16(dst, kb + i * 512);
            cp_async16(dst + RG::kV, vb + i * 512);
          }
        }
        if (ring && lane < kPageRows / 4)
          cp_async16(st + RG::kPos + lane * 16, a.pos + (size_t)page * kPageRows + lane * 4);
      }
      // while the ring is empty, its other stages' copies go out before the queries are formed
      const bool queries = late ? k + 1 == min(max(pages, 1), RG::kStages) : k == 0;
      if (queries) put_queries(ring_smem + (late ? 0 : slot) * RG::kStride);
      if (!with_put) {
        ex.x = __shfl_sync(0xffffffffu, exp_l.x, k & 31);
        ex.y = __shfl_sync(0xffffffffu, exp_l.y, k & 31);
      }
      if (lane == 0) {
        StageInfo* info = reinterpret_cast<StageInfo*>(ring_smem + slot * RG::kStride + RG::kInfo);
        info->row = row;
        info->end = end;
        info->flags = (page < 0 || pages == 0 ? kNone : ring ? kRing : kSeg) |
                      (k + 1 >= pages ? kLast : 0);
        info->exps[0] = ex.x;
        info->exps[1] = ex.y;
        info->item = wi;
        info->cache = c;
        info->alone = alone;
        info->t = t;
        info->w = hd.w;
        if constexpr (kMode == kScores) info->page = page;
      }
      arrive_after_copies(&bars->full[slot]);
      if (k > 0 || !late) sm100::mbar_arrive(&bars->full[slot]);
      if (queries && late) sm100::mbar_arrive(&bars->full[0]);  // the first stage is complete now
    }
    if (alone) {  // no other reader of the count is left once the rows are put
      wait_puts();
      const bool stored = put.at >= 0 && !put.ring && had >= 0 &&
                          page_at(a, hd.first_page, hd.max_pages, had / kPageRows) >= 0;
      if (lane == 0) a.rows_out[c] = had + (stored ? 1 : 0);
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// Thread blocks that an SM's registers hold.
constexpr int kBlocks(int d) { return d == 64 ? 4 : 3; }

// Is the list the one that the call was made (or captured) with?
__device__ __forceinline__ bool same_list(const PagedArgs& a) {
  return a.totals[3] == a.n_work && a.totals[4] == a.n_ctas;
}

// kFold: groups of up to four queries.  A lane then has one query (t4) and, in
// its two columns, that query's two terms; else two queries (2 t4, 2 t4 + 1).
template <typename T, int D, bool kFold, int kMode>
__global__ void __launch_bounds__(kThreads, kBlocks(D))
    q8_split_kernel(const PagedArgs a, const ModeArgs<kMode> n, int G, int H, int R, int HLkv,
                    float sl2) {
  constexpr bool kWide = wide<T>(kFold, kMode);
  using RG = Ring<D, kFold, kWide>;
  constexpr int NQ = kFold ? 1 : 2;  // queries of a lane
  constexpr int KI = D / 64;   // 16-byte pieces of a K row per lane
  constexpr int PW = D / 32;   // words of a lane's V piece
  constexpr int MT = D / 16;   // 16-row tiles of O^T
  extern __shared__ __align__(128) uint8_t ring_smem[];
  __shared__ float sm_ml[2][3][kWarps][kMaxR];
  __shared__ Bars bars;
  float* sums = reinterpret_cast<float*>(ring_smem + RG::kBytes);  // [kWarps][R / kHalves][D]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t4 = lane & 3;
  const int q0 = NQ * t4;  // the lane's first query
  bool beside = false;
  if constexpr (kMode != kDecode) {
    beside = n.beside;
    if (beside && !start_beside()) return;
  }
  // a list of another cache may say anything: its items are bounded here, its
  // caches where they are used
  const int wi0 = max(0, min(a.cta_first[blockIdx.x], a.n_work - 1));
  const int wi_end = max(wi0 + 1, min(a.cta_first[blockIdx.x + 1], a.n_work));
  const int Gkv = G / R;
  if (threadIdx.x == 0) {
    for (int i = 0; i < RG::kStages; ++i) {
      sm100::mbar_init(&bars.full[i], 64);  // every streaming lane: its copies, and its stores
      sm100::mbar_init(&bars.empty[i], kWarps);
    }
    sm100::mbar_init(&bars.puts, kWarps);
    sm100::mbar_init(&bars.sync, kWarps);
    bars.stop = 0;
    sm100::fence_barrier_init();
  }
  // the work list is read before the wait (fastgen_paged_schedule waits until it is there); the
  // caller's own buffers, descriptors too, behind it
  const int own = min(wi0 + (warp == kWarps ? 0 : warp), wi_end - 1);
  const PagedItem own_item = a.items[own];
  const int own_c = (unsigned)own_item.cache < (unsigned)Gkv ? own_item.cache : 0;
  const int own_items = a.ranges[own_c].y;
  const bool listed = same_list(a);
  __syncthreads();
  if (!beside) {
    griddep_wait();
    griddep_launch_dependents();
  }
  const fg_paged_desc own_cache = a.caches[own_c];
  if (!listed) {
    if (threadIdx.x == 0) atomicOr(a.dev_err, kErrInvalid);
    return;
  }
  const LaneSet special(n.special, n.ns), punct(n.punct, n.np);
  if (warp == kWarps) {
    stream_items<T, D, kFold, kMode>(a, n, Gkv, H, R, HLkv, ring_smem, &bars, wi0, wi_end, own_item,
                              own_cache, own_items, special, punct);
    return;
  }

  // the new tokens' rows of this CTA's items
  if (n.k_new) {
    for (int wi = wi0 + warp; wi < wi_end; wi += kWarps) {
      const PagedItem it = wi == own ? own_item : a.items[wi];
      const int c = it.cache, b = c / HLkv;
      if ((unsigned)c >= (unsigned)Gkv) continue;
      const fg_paged_desc hd = wi == own ? own_cache : a.caches[c];
      const int t = n.pos[b], tau = n.ids[b], had = a.rows[c];
      if (t < 0) continue;
      const Put put = item_put(n, it, hd, special, punct, ring_slots(hd, a.max_w),
                               live_rows(hd, had), t, tau);
      if (put.at >= 0)
        put_token<T, D, kMode>(a, n, c, hd, put, t, kMode == kScores && special.has(tau));
    }
    __syncwarp();
    if (lane == 0) sm100::mbar_arrive(&bars.puts);
  } else if (lane == 0) {
    sm100::mbar_arrive(&bars.puts);
  }

  // this lane's rows of a block and their places in a stage: key kr (and + 8) for the scores,
  // keys va, vb (and + 8) for the values and the weights
  const uint32_t base = sm100::smem_addr(ring_smem) + (uint32_t)(warp * kBlockRows * D);
  const int kr = RG::slot_key(g), va = RG::slot_key(2 * t4), vb = RG::slot_key(2 * t4 + 1);
  uint32_t k_off[KI];
#pragma unroll
  for (int i = 0; i < KI; ++i)
    k_off[i] = (uint32_t)(kr * D + (((t4 + 4 * i) ^ RG::swizzle(kr)) << 4));
  const int vp = D == 128 ? g : g >> 1, vo = D == 128 ? 0 : (g & 1) * 8;
  const uint32_t va_off = (uint32_t)(RG::kV + va * D + ((vp ^ RG::swizzle(va)) << 4) + vo);
  const uint32_t vb_off = (uint32_t)(RG::kV + vb * D + ((vp ^ RG::swizzle(vb)) << 4) + vo);
  uint32_t syncs = 0;
  auto sync_warps = [&]() {  // the four computing warps
    __syncwarp();
    if (lane == 0) sm100::mbar_arrive(&bars.sync);
    wait_bar(&bars, &bars.sync, syncs++ & 1, a.dev_err);
  };

  int stage = 0, half = 0;
#pragma unroll 1
  for (int wi = wi0; wi < wi_end; ++wi) {
    // of the lane's queries over its keys; lanes without a query keep a maximum that no score
    // passes: weight 0
    float m[NQ], ms[NQ], l[NQ];  // maximum of score + V's exponent; of the scores, and their sum
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      m[q] = ms[q] = q0 + q < R ? kNoScore : 1e30f;
      l[q] = 0.f;
    }
    float o[MT][4];
#pragma unroll
    for (int j = 0; j < MT; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
    uint32_t qa[4 * KI][kWide ? 4 : 2];  // (kWide: the second terms behind the first)
    float fq[NQ] = {};  // what the queries were divided by, times the softmax scale
    int last = 0, item = 0, cache = 0, alone = 0;
#pragma unroll 1
    for (bool opening = true; !last; opening = false, ++stage) {
      const int slot = stage % RG::kStages;
      if (!wait_bar(&bars, &bars.full[slot], stage / RG::kStages & 1, a.dev_err))
        return;  // the copies in flight are the streaming warp's
      // everything that the block needs first is asked for together
      const uint8_t* sp = ring_smem + slot * RG::kStride;
      const StageInfo* info = reinterpret_cast<const StageInfo*>(sp + RG::kInfo);
      const uint32_t st = base + (uint32_t)(slot * RG::kStride);
      const uint4 head = *reinterpret_cast<const uint4*>(info);
      const uint32_t exps = info->exps[warp >> 1];
      uint4 k0[KI], k1[KI];
#pragma unroll
      for (int i = 0; i < KI; ++i) {
        k0[i] = lds16(st + k_off[i]);
        k1[i] = lds16(st + k_off[i] + 8 * D);
      }
      const int row = (int)head.x + warp * kBlockRows, end = (int)head.y;
      const int kind = head.z & kKind;
      last = head.z & kLast;
      if (last) {
        item = info->item;
        cache = info->cache;
        alone = info->alone;
      }
      if (opening) {
        // operand fragments: k-step 4 i + w takes dimensions 64 i + 16 t4 + 4 w + 0..3
#pragma unroll
        for (int i = 0; i < KI; ++i)
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            uint2 x = make_uint2(0, 0), y = make_uint2(0, 0);
            if (g < (kFold ? 2 * R : R)) {
              const uint8_t* q = sp + RG::kQ + (g * D + 64 * i + 16 * t4 + 4 * w) * 2;
              x = *reinterpret_cast<const uint2*>(q);
              if constexpr (kWide) y = *reinterpret_cast<const uint2*>(q + RG::kQTerm);
            }
            qa[4 * i + w][0] = x.x;
            qa[4 * i + w][1] = x.y;
            if constexpr (kWide) {
              qa[4 * i + w][2] = y.x;
              qa[4 * i + w][3] = y.y;
            }
          }
#pragma unroll
        for (int q = 0; q < NQ; ++q)
          fq[q] = q0 + q < R ? reinterpret_cast<const float*>(sp + RG::kQExp)[q0 + q] * sl2 : 0.f;
      }
      if (kind == kNone || row >= end) {  // uniform over the warp: no rows here
        __syncwarp();
        if (lane == 0) sm100::mbar_arrive(&bars.empty[slot]);
        continue;
      }
      const uint32_t ex = exps >> (16 * (warp & 1));
      const int ek = (int)(signed char)(ex & 0xff), ev = (int)(signed char)((ex >> 8) & 0xff);
      // columns 2 t4 and 2 t4 + 1 of key kr ([0], [1]) and of key kr + 8 ([2], [3])
      float x[4] = {0.f, 0.f, 0.f, 0.f}, xl[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < KI; ++i) {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const uint32_t y0 = word4(k0[i], w), y1 = word4(k1[i], w);
          const uint32_t(&q)[kWide ? 4 : 2] = qa[4 * i + w];
          const uint32_t f0 = decode2(y0), f1 = decode2(y1), f2 = decode2(y0 >> 16),
                         f3 = decode2(y1 >> 16);
          mma_f16_16816(x, f0, f1, f2, f3, q[0], q[1]);
          if constexpr (kWide) mma_f16_16816(xl, f0, f1, f2, f3, q[2], q[3]);
        }
      }
      Piece<D> v[4];  // keys va, vb, va + 8, vb + 8
      v[0].load(st + va_off);
      v[1].load(st + vb_off);
      v[2].load(st + va_off + 8 * D);
      v[3].load(st + vb_off + 8 * D);
      // scores of the lane's queries with keys kr and kr + 8 in base 2
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
          sc[q][h] = y * kf;
        }
      }
      if (kind == kRing || row + kBlockRows > end) {  // uniform: rows may be missing
        const int t = (int)head.w, w = info->w;
        auto there = [&](int key) {
          bool ok = row + key < end;
          if (kind == kRing) {  // in the window: position in (t - w, t]
            const int p = reinterpret_cast<const int*>(sp + RG::kPos)[warp * kBlockRows + key];
            ok = ok && p >= 0 && (unsigned)t - (unsigned)p < (unsigned)w;
          }
          return ok;
        };
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (!there(kr + 8 * h))
#pragma unroll
            for (int q = 0; q < NQ; ++q) sc[q][h] = FG_NEG_INF;
#pragma unroll
        for (int i = 0; i < 4; ++i)  // such a row may hold anything, also NaN
          if (!there((i & 1 ? vb : va) + (i & 2 ? 8 : 0))) v[i].zero();
      }
      if constexpr (kMode == kScores) {
        if (kind == kSeg && q0 < R) {
          // (rows past the end too: their slots belong to the page)
          float* p = n.row_sc + ((size_t)info->page * kPageRows + warp * kBlockRows) * R + q0;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if constexpr (NQ == 2)  // R = 8
              *reinterpret_cast<float2*>(p + (kr + 8 * h) * R) = make_float2(sc[0][h], sc[1][h]);
            else
              p[(kr + 8 * h) * R] = sc[0][h];
          }
        }
      }
      __syncwarp();  // every lane has read the stage
      if (lane == 0) sm100::mbar_arrive(&bars.empty[slot]);
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
      uint32_t p01, p23, r01 = 0, r23 = 0;  // of keys kr and kr + 8; r: second terms
      if constexpr (kFold) {
        const float2 f = unpack_f16x2(pack_f16x2(p[0][0], p[0][1]));
        p01 = transpose8x8(pack_f16x2(f.x, p[0][0] - f.x));
        p23 = transpose8x8(pack_f16x2(f.y, p[0][1] - f.y));
      } else {
        const uint32_t lo = pack_f16x2(p[0][0], p[NQ - 1][0]),
                       hi = pack_f16x2(p[0][1], p[NQ - 1][1]);
        p01 = transpose8x8(lo);
        p23 = transpose8x8(hi);
        if constexpr (kWide) {
          const float2 f01 = unpack_f16x2(lo), f23 = unpack_f16x2(hi);
          r01 = transpose8x8(pack_f16x2(p[0][0] - f01.x, p[NQ - 1][0] - f01.y));
          r23 = transpose8x8(pack_f16x2(p[0][1] - f23.x, p[NQ - 1][1] - f23.y));
        }
      }
#pragma unroll
      for (int w = 0; w < PW; ++w) {
        const uint32_t a0 = v[0].word(w), a1 = v[1].word(w), a2 = v[2].word(w), a3 = v[3].word(w);
        // byte pairs (key, next key) of dimensions 4 w, 4 w + 1 and 4 w + 2, 4 w + 3
        const uint32_t lo01 = __byte_perm(a0, a1, 0x5140), hi01 = __byte_perm(a0, a1, 0x7362);
        const uint32_t lo23 = __byte_perm(a2, a3, 0x5140), hi23 = __byte_perm(a2, a3, 0x7362);
        const uint32_t f0 = decode2(lo01), f1 = decode2(lo01 >> 16), f2 = decode2(lo23),
                       f3 = decode2(lo23 >> 16);
        const uint32_t h0 = decode2(hi01), h1 = decode2(hi01 >> 16), h2 = decode2(hi23),
                       h3 = decode2(hi23 >> 16);
        mma_f16_16816(o[2 * w], f0, f1, f2, f3, p01, p23);
        mma_f16_16816(o[2 * w + 1], h0, h1, h2, h3, p01, p23);
        if constexpr (kWide) {
          mma_f16_16816(o[2 * w], f0, f1, f2, f3, r01, r23);
          mma_f16_16816(o[2 * w + 1], h0, h1, h2, h3, r01, r23);
        }
      }
    }
    if (item < 0) continue;
    // the item is through: merge the four warps
    float(&sm_m)[kWarps][kMaxR] = sm_ml[half][0], (&sm_s)[kWarps][kMaxR] = sm_ml[half][1],
        (&sm_l)[kWarps][kMaxR] = sm_ml[half][2];
    half ^= 1;  // the other half may still be read
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) l[q] += __shfl_xor_sync(0xffffffffu, l[q], d);
      if (g == 0 && q0 + q < R) {
        sm_m[warp][q0 + q] = m[q];
        sm_s[warp][q0 + q] = ms[q];
        sm_l[warp][q0 + q] = l[q];
      }
    }
    sync_warps();
    // O^T: rows 16 j + g, + 8 are dimensions (D / 8) g + 2 j, + 1; the columns as the queries'
    constexpr int kMerges = kHalves<kFold, kMode>();
    const int RH = R / kMerges;
#pragma unroll
    for (int z = 0; z < kMerges; ++z) {
      const int r0 = z * RH;    // its first query
      if (z > 0) sync_warps();  // the half before has been read
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        const int qi = q0 + q;
        if (kMerges == 1 ? qi < R : qi >= r0 && qi < r0 + RH) {
          float M = kNoScore;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm_m[w][qi]);
          const float f = exp2f(m[q] - M);
#pragma unroll
          for (int j = 0; j < MT; ++j)
            *reinterpret_cast<float2*>(
                &sums[(warp * RH + qi - r0) * D + (D / 8) * g + 2 * j]) =
                kFold ? make_float2((o[j][0] + o[j][1]) * f, (o[j][2] + o[j][3]) * f)
                      : make_float2(o[j][q] * f, o[j][q + 2] * f);
        }
      }
      sync_warps();
      const size_t g0 = (size_t)(cache / (H / R)) * H + (size_t)(cache % (H / R)) * R + r0;
      for (int x = warp * 32 + lane; x < RH * D; x += kWarps * 32) {
        const int qi = r0 + x / D;
        float A = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) A += sums[w * RH * D + x];
        float M = kNoScore, S = kNoScore, L = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          M = fmaxf(M, sm_m[w][qi]);
          S = fmaxf(S, sm_s[w][qi]);
        }
#pragma unroll
        for (int w = 0; w < kWarps; ++w) L += sm_l[w][qi] * exp2f(sm_s[w][qi] - S);
        // the item's own output: the sums are in units of 2^(M - kPBits), L in 2^S
        const float y = L == 0.f ? 0.f : A / L * exp2f(M - S - kPBits);
        if (alone) {
          store_out((T*)n.out + g0 * D + x, y);
        } else {
          n.part_acc[((size_t)item * R + r0) * D + x] = y;
          if (x % D == 0) {
            n.part_ml[2 * ((size_t)item * R + qi)] = S;
            n.part_ml[2 * ((size_t)item * R + qi) + 1] = L;
          }
        }
      }
    }
  }
}

constexpr int kFoldR = 4;  // queries whose two terms fill the MMA's eight columns

template <typename T, int D, bool kFold, int kMode>
int split_smem(int R) {
  return Ring<D, kFold, wide<T>(kFold, kMode)>::kBytes +
         kWarps * (R / kHalves<kFold, kMode>()) * D * (int)sizeof(float);
}

template <typename T, int D, bool kFold, int kMode>
cudaError_t launch_split(const ProfileDims& pd, const PagedArgs& a, const ModeArgs<kMode>& n,
                         cudaStream_t s) {
  const auto split = q8_split_kernel<T, D, kFold, kMode>;
  const int smem = split_smem<T, D, kFold, kMode>(pd.R);
  cudaError_t e = cudaFuncSetAttribute(split, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  // d = 64: with the split of an SM's memory that its own size asks for, SMs at
  // times took in fewer than four blocks beside the previous combine's (64 -> 59
  // us, 2048 caches of 2048 positions); d = 128 runs slower with less L1 (51.3 ->
  // 52.0 us, 7B shape)
  if (D == 64 && e == cudaSuccess)
    e = cudaFuncSetAttribute(split, cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared);
  int grid = a.n_ctas;
  if constexpr (kMode != kDecode) grid += n.beside;
  if (e == cudaSuccess)
    e = launch_pdl(split, grid, kThreads, smem, s, a, n, pd.G, pd.H, pd.R, pd.HLkv, pd.sl2);
  return e;
}

}  // namespace
}  // namespace fg
