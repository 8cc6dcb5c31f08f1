// Attention of a batch over the caches of a prompt that its sequences share:
// every query of sequence b and head h over cache h / R of the prompt, which is
// read once for all sequences.
//
// With B sequences and groups of R a cache meets B R queries, so both products
// are matrix products of the tensor cores, a page of 64 keys at a time:
//   S [128 queries x 64 keys] = Q K^T,  O [128 x d] += P V,
// accumulators and P in tensor memory, operands in shared memory.  The codes of
// a page are widened to f16, which holds them exactly, on their way; the
// exponents of a block of 16 keys are two numbers for 16 columns of S: K's
// scales the scores, V's goes into the weights that enter the product.
// Queries are f16 after the division by a power of two (11 bits; fp32 inputs two
// terms, 22 bits: Q = Qh + Ql along the product's depth, P = Ph + Pl likewise).
// One term in bf16 also where the split kernel takes two (groups of up to four): the
// outputs' distance from the definition is then 0.00149 to 0.00172 of their size, with
// two terms 0.00144 to 0.00164, nearly all of it their own rounding, and two terms
// cost a step 10 to 55 % (4 queries a cache 23.0 -> 25.5 us, 64 in groups of 4 25.0 ->
// 29.5, 64 in groups of 1 161 -> 189, 512 127 -> 197: a block then has room for one
// tile of queries).
//
// A thread block per SM: a warp that loads the pages' codes (bulk copies of 4 or
// 8 KB), one that describes the pages, four that widen codes into the swizzled
// layout the tensor cores read, two threads that issue products, and two
// warpgroups of softmax, a thread a query.  The two work on separate streams
// with S and O of their own: two tiles of queries over the same pages (each
// widened once for both), or, where there is one tile of queries, the even and
// the odd pages.  A stream has two places of S, so that the next page's scores
// are there before the softmax asks; P takes S's place in tensor memory.
//
// The softmax is one pass over the rows: sums and products are kept relative
// to reference maxima that follow the true ones when those get 2^kSlack ahead
// (then O is rescaled in tensor memory).  The sum's maximum is that of the
// scores, the product's that of score + V's exponent, as in the split kernel.
//
// What bounds it: 32 caches of 16384 positions (about 4800 pages), 512 queries each, take 81 us, 63
// pages of two tiles an SM, 2350 cycles each, in which the threads that issue products wait for the
// tensor cores and these for shared memory: it moves 192 KB a page, 1540 cycles (for each tile
// S reads 32 KB of queries and 16 of keys, the product with V 16; codes come in, are read and
// written widened, 64).  S of 64 keys alone takes 405 cycles where 260 would be the tensor cores'.
// Exponentials have 510 cycles, the warps' instructions 1130 of each scheduler's.  Without the softmax
// it takes 20 us less, without the products 10, without both 32, with pages from L2 alone 1.
// With one tile of 64 queries (256 caches of 4096, 133 MB) 60 us, 3 times HBM's: widening a page
// takes its warps 1300 cycles, and rows of a tile that no query fills are computed all the same.
//   The kernel's code has to fit the instruction cache: with the roles' loops unrolled it was 78 KB,
// and the same case took 342 us.  Taken and dropped: key tiles of 128 with one place of S (197), S
// in registers with a register split of the warps (198), eight warps that widen (180 -> 179).
#include "fg_paged_decode.cuh"

namespace fg {
namespace {

using namespace sm100;

constexpr int kTile = kPrefixTile;  // queries of a tile (rows of tensor memory)
// warps 0-7 softmax (warp w reads tensor memory lanes 32 (w % 4) ..), 8-11 widen
constexpr int kSoftWarps = 8, kUnpackWarps = 4;
constexpr int kLoadWarp = kSoftWarps + kUnpackWarps, kMetaWarp = kLoadWarp + 1;
constexpr int kMmaWarp = kMetaWarp + 1;  // and the next
constexpr int kPrefixThreads = (kMmaWarp + 2) * 32;
constexpr int kMetas = 8;  // pages whose description is there
constexpr float kSlack = 8.f;
constexpr float kProdBits = 7.f;  // weights enter the product times 2^7, at most 2^15
constexpr int kSmem = 227 * 1024;

// A page of a segment or of a ring.
struct PageMeta {
  uint32_t exps[2];     // of the page's blocks: (K, V) bytes
  int cnt;              // rows (0: no page)
  int w;                // ring slots, 0: a segment's page
  int pos[kPageRows];   // of a ring's rows
};

template <int D, int kTerms, bool kPair>
struct Plan {
  static constexpr int kQHalf = kTile * 128;  // bytes of 64 dimensions of a tile of queries
  static constexpr int kQTerm = kTile * D * 2;                        // one term of a tile of queries
  static constexpr int kQBytes = (kPair ? 2 : 1) * kTerms * kQTerm;   // the queries in shared memory
  static constexpr int kPiece = kPageRows * D;                        // codes of K or of V of a page
  static constexpr int kHalf = kPageRows * 128;  // bytes of 64 dimensions of an operand
  static constexpr int kOpBytes = kPageRows * D * 2;
  // Widened K or V pages in shared memory.  Where the streams take pages in turns, a multiple of
  // four, so that a place always has the same stream's pages.
  static constexpr int kOperands = kPair ? 6 : kTerms == 2 && D == 128 ? 4 : 8;
  static constexpr int kRoom = (kSmem - 1024 - 3584 - kQBytes - kOperands * kOpBytes) / (2 * kPiece);
  static constexpr int kRaw = kRoom > 8 ? 8 : kRoom;  // pages of codes in shared memory
  static_assert(kRaw >= 2 && (kPair || kOperands % 4 == 0), "rings of a block");
};

template <int D, int kTerms, bool kPair>
struct alignas(1024) Smem {
  using P = Plan<D, kTerms, kPair>;
  uint8_t q[P::kQBytes];
  uint8_t op[P::kOperands][P::kOpBytes];
  alignas(128) uint8_t raw[P::kRaw][2 * P::kPiece];  // K, V
  alignas(16) PageMeta meta[kMetas];
  uint64_t raw_full[P::kRaw], raw_empty[P::kRaw];
  uint64_t meta_full[kMetas], meta_empty[kMetas];
  uint64_t op_full[P::kOperands], op_empty[P::kOperands];
  uint64_t s_full[2][2], p_full[2][2], pv_done[2][2];  // of a stream's two places of S
  uint64_t q_full, q_free, drain[2];
  int abort;
  uint32_t tmem;
  int first_cache;  // of this block's range
};

// tensor memory: two places of S (and P) of each stream, then O
constexpr uint32_t kTmemCols = 512;
__device__ __forceinline__ uint32_t s_col(int st, int b) { return st * 128 + b * kPageRows; }
__device__ __forceinline__ uint32_t o_col(int st) { return 256 + st * 128; }

// Waits for at most about a second (2^31 cycles), or until another wait has run out.
__device__ __forceinline__ bool wait_or_stop(uint64_t* bar, uint32_t parity, volatile int* abort) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
#pragma unroll 1
  while (!mbar_try_wait(bar, parity)) {
    if (clock64() - t0 > (1ll << 31)) *abort = 1;
    if (*abort) return false;
  }
  return true;
}
__device__ __forceinline__ bool test_bar(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
// The same by a whole warp.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  return __all_sync(0xffffffffu, wait_or_stop(bar, parity, abort));
}
__device__ __forceinline__ void fence_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// f16 operands, f32 accumulator, M x N, A K-major; B K-major or (mn) MN-major.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool mn) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24) | (mn ? 1u << 16 : 0u);
}
// An MN-major operand of rows of 64 elements in the 128-byte swizzled layout: 8-row groups (along
// K) 1024 bytes apart, 64-element column blocks mn_stride apart.
__device__ __forceinline__ uint64_t desc_mn_sw128(uint32_t saddr, uint32_t mn_stride) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | (uint64_t)((mn_stride >> 4) & 0x3FFFu) << 16 |
         (uint64_t)(1024u >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}
// 16 columns, and the wait for them.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld16(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                 "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]),
                 "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Pages of a cache: of its segment, of its ring.
__device__ __forceinline__ int2 key_pages(const PagedArgs& a, const fg_paged_desc& hd, int rows) {
  return make_int2(cdiv(live_rows(hd, rows), kPageRows), cdiv(ring_slots(hd, a.max_w), kPageRows));
}

// ------------------------------------------------------------- before the products
// A warp a query: rotated, divided by the power of two that brings its largest value to
// [2^13, 2^14), as f16 in the tensor cores' layout.  (Rows of a tile without a query stay as they
// are: no other row's result depends on them.)  The last CTA counts the caches' pages.
constexpr int kPrepThreads = 256;

template <typename T, int D, int kTerms>
__global__ void __launch_bounds__(kPrepThreads)
    prefix_prep_kernel(const PagedArgs a, const PagedDecodeArgs n, const PrefixParts px, int G,
                       int H, int R, int HL, float sl2) {
  constexpr int PER = D / 32;
  __shared__ long long scr[33];
  const int lane = threadIdx.x & 31;
  griddep_wait();
  griddep_launch_dependents();
  if (blockIdx.x == gridDim.x - 1) {
    long long sum = 0, tot;
    for (int base = 0; base < px.caches; base += kPrepThreads) {
      const int c = base + threadIdx.x;
      long long x = 0;
      if (c < px.caches) {
        const fg_paged_desc hd = a.caches[c];
        const int rows = a.rows[c];
        if (live_rows(hd, rows) != rows || ring_slots(hd, a.max_w) != hd.w)
          atomicOr(a.dev_err, kErrInvalid);
        const int2 k = key_pages(a, hd, rows);
        x = (long long)k.x + k.y;
      }
      const long long at = sum + block_exclusive_scan(x, scr, &tot);
      if (c < px.caches) px.cum[c] = at;
      sum += tot;
    }
    if (threadIdx.x == 0) px.cum[px.caches] = sum;
    return;
  }
  const int g = blockIdx.x * (kPrepThreads / 32) + (threadIdx.x >> 5);
  if (g >= G) return;
  const int b = g / HL, c = kv_head(g % HL, H, R), j = b * R + g % H % R;
  const int t = n.pos[b];
  if (t < 0) return;
  float x[PER];
  load_row<PER>((const T*)n.q + (size_t)g * D, x);
  if (n.rope.rot > 0) {
    float2 cs[PER];
    row_angles<PER>(cs, n.rope.rot, n.rope.style, [&](int p) {
      float2 y;
      rope_cos_sin((unsigned)t, n.rope.turns[p], y.x, y.y);
      return y;
    });
    rotate_row<PER>(x, cs, n.rope.rot, n.rope.style);
  }
  uint32_t top = 0;
#pragma unroll
  for (int k = 0; k < PER; ++k) top = max(top, finite_bits(x[k]));
  top = __reduce_max_sync(0xffffffffu, top);
  const int eq = max(-110, (int)(top >> 23) - 127 - 13);
  const float inv = pow2f(-eq);
  const size_t tile = (size_t)c * px.tiles + j / kTile;
  const int r = j % kTile, e = lane * PER;
  uint8_t* p = px.q + tile * kTerms * kTile * D * 2 + e / 64 * (kTile * 128) + r * 128 +
               ((((e % 64) / 8) ^ (r & 7)) << 4) + e % 8 * 2;
#pragma unroll
  for (int k = 0; k < PER; k += 2) {
    const float u = x[k] * inv, v = x[k + 1] * inv;
    const uint32_t hi = pack_f16x2(u, v);
    *reinterpret_cast<uint32_t*>(p + 2 * k) = hi;
    if constexpr (kTerms == 2) {  // what f16 loses, down to 2^-38 of the largest value
      const float2 z = unpack_f16x2(hi);
      *reinterpret_cast<uint32_t*>(p + 2 * k + kTile * D * 2) = pack_f16x2(u - z.x, v - z.y);
    }
  }
  if (lane == 0) px.qf[tile * kTile + r] = pow2f(eq) * sl2;
}

// ------------------------------------------------------------------- the products
// The parts of units' pages that a thread block takes.
struct Walk {
  const PrefixParts& px;
  long long x, end;  // of the block's range
  int c, grp;
  long long c0, pages;  // of the cache
  __device__ Walk(const PrefixParts& p, int first_cache, long long x0, long long x1)
      : px(p), x(x0), end(x1), c(first_cache) {
    c0 = px.cum[c];
    pages = px.cum[c + 1] - c0;
    grp = pages > 0 ? (int)((x - c0 * px.groups) / pages) : 0;
  }
  __device__ bool more() const { return x < end; }
  __device__ int first() const { return (int)(x - c0 * px.groups - grp * pages); }  // page
  __device__ int count() const { return (int)min(pages - first(), end - x); }
  __device__ bool both() const { return px.pair && 2 * grp + 1 < px.tiles; }
  __device__ int tile() const { return px.pair ? 2 * grp : grp; }  // of the queries
  __device__ size_t unit() const { return (size_t)c * px.groups + grp; }
  __device__ void next() {
    x += count();
    if (x >= end) return;
    if (++grp < px.groups) return;
    grp = 0;
    do {
      c0 = px.cum[++c];
      pages = px.cum[c + 1] - c0;
    } while (pages == 0);
  }
};

// Calls page(k, page number or -1, exponents, first row, rows, is it a ring's, ring slots) for every
// page of the block in order, until that returns false (all lanes; one warp).
template <typename F>
__device__ __forceinline__ void each_page(const PagedArgs& a, Walk wk, F&& page) {
  const int lane = threadIdx.x & 31;
  int k = 0;
  for (; wk.more(); wk.next()) {
    const fg_paged_desc hd = a.caches[wk.c];
    const int rows = live_rows(hd, a.rows[wk.c]), w = ring_slots(hd, a.max_w);
    const int seg = cdiv(rows, kPageRows), t0 = wk.first(), nt = wk.count();
    int page_l = -1;
    uint2 exp_l = make_uint2(0, 0);
#pragma unroll 1
    for (int i = 0; i < nt; ++i, ++k) {
      const int t = t0 + i;
      if ((i & 31) == 0) {  // the next 32 pages: lane l holds one and its exponents
        page_l = -1;
        if (i + lane < nt) {
          const int e = t + lane;
          page_l = e < seg ? page_at(a, hd.first_page, hd.max_pages, e)
                           : page_at(a, hd.ring_page, hd.ring_pages, e - seg);
          if (page_l < 0)
            atomicOr(a.dev_err, kErrInvalid);
          else
            exp_l = *reinterpret_cast<const uint2*>(a.exps + (size_t)page_l * kPageBlocks * 2);
        }
      }
      const bool ring = t >= seg;
      uint2 ex;
      ex.x = __shfl_sync(0xffffffffu, exp_l.x, i & 31);
      ex.y = __shfl_sync(0xffffffffu, exp_l.y, i & 31);
      if (!page(k, __shfl_sync(0xffffffffu, page_l, i & 31), ex,
                (ring ? w : rows) - (ring ? t - seg : t) * kPageRows, ring ? w : 0))
        return;
    }
  }
}

// The warp that loads the pages' codes.
template <int D, int kTerms, bool kPair>
__device__ __forceinline__ void load_pages(Smem<D, kTerms, kPair>& s, const PagedArgs& a, Walk wk) {
  using P = Plan<D, kTerms, kPair>;
  volatile int* abort = &s.abort;
  int pages = 0;  // asked for so far
  each_page(a, wk, [&](int k, int page, uint2, int, int) {
    bool go = true;
    if ((threadIdx.x & 31) == 0) {
      const int slot = k % P::kRaw;
      go = k < P::kRaw || wait_or_stop(&s.raw_empty[slot], (k / P::kRaw - 1) & 1, abort);
      if (go) {
        ++pages;
        if (page < 0) {
          mbar_arrive(&s.raw_full[slot]);
        } else {
          mbar_expect_tx(&s.raw_full[slot], 2 * P::kPiece);
          bulk_load(s.raw[slot], a.kp + (size_t)page * P::kPiece, P::kPiece, &s.raw_full[slot]);
          bulk_load(s.raw[slot] + P::kPiece, a.vp + (size_t)page * P::kPiece, P::kPiece,
                    &s.raw_full[slot]);
        }
      }
    }
    return (bool)__shfl_sync(0xffffffffu, go, 0);
  });
  if (*abort && (threadIdx.x & 31) == 0)  // what is in flight lands before the block ends
    for (int i = max(0, pages - P::kRaw); i < pages; ++i)
      mbar_wait(&s.raw_full[i % P::kRaw], i / P::kRaw & 1);
}

// The warp that describes them.
template <int D, int kTerms, bool kPair>
__device__ __forceinline__ void load_metas(Smem<D, kTerms, kPair>& s, const PagedArgs& a, Walk wk) {
  volatile int* abort = &s.abort;
  int metas = 0;
  each_page(a, wk, [&](int k, int page, uint2 ex, int left, int w) {
    bool go = true;
    if ((threadIdx.x & 31) == 0) {
      const int slot = k % kMetas;
      go = k < kMetas || wait_or_stop(&s.meta_empty[slot], (k / kMetas - 1) & 1, abort);
      if (go) {
        PageMeta& m = s.meta[slot];
        *reinterpret_cast<uint4*>(&m) = make_uint4(ex.x, ex.y, page < 0 ? 0 : min(kPageRows, left), w);
        const bool copy = w > 0 && page >= 0;
        mbar_expect_tx(&s.meta_full[slot], copy ? kPageRows * 4 : 0);
        ++metas;
        if (copy)
          bulk_load(m.pos, a.pos + (size_t)page * kPageRows, kPageRows * 4, &s.meta_full[slot]);
      }
    }
    return (bool)__shfl_sync(0xffffffffu, go, 0);
  });
  if (*abort && (threadIdx.x & 31) == 0)
    for (int i = max(0, metas - kMetas); i < metas; ++i)
      mbar_wait(&s.meta_full[i % kMetas], i / kMetas & 1);
}

// One of the four warps that widen codes: rows 16 w .. of every page (a warp that skipped pages could
// take a barrier's phase for the one two before it), where an operand row that is
// not there is zero.  A lane's 16 bytes and the 32 it makes of them are chosen so that the eight
// lanes of a phase meet eight different banks, in the codes and in the swizzled operand.
template <int D, int kTerms, bool kPair>
__device__ __forceinline__ void widen(Smem<D, kTerms, kPair>& s, int uw, int total) {
  using P = Plan<D, kTerms, kPair>;
  constexpr int kIter = kBlockRows * (D / 16) / 32;  // 16-byte pieces of a lane
  const int lane = threadIdx.x & 31, lr = lane & 7;
  volatile int* abort = &s.abort;
  auto row_of = [&](int i) { return lr + (i & 1) * 8; };
  auto piece_of = [&](int i) {
    return D == 128 ? ((lane >> 3) + 4 * (i >> 1) + lr) & 7
                    : (((((lr >> 2) ^ (lr >> 1)) & 1) << 1 | (lr >> 2)) ^ (lane >> 3)) & 3;
  };
#pragma unroll 1
  for (int k = 0; k < total; ++k) {
    const int ms = k % kMetas, raw = k % P::kRaw;
    const int seq[2] = {2 * k, 2 * k + 1}, slot[2] = {seq[0] % P::kOperands, seq[1] % P::kOperands};
    auto has_room = [&](int side) {
      return seq[side] < P::kOperands ||
             test_bar(&s.op_empty[slot[side]], (seq[side] / P::kOperands - 1) & 1);
    };
    auto wait_room = [&](int side) {
      return seq[side] < P::kOperands ||
             warp_wait(&s.op_empty[slot[side]], (seq[side] / P::kOperands - 1) & 1, abort);
    };
    // What the page needs is asked for at once: one after the other the answers took 1000 of a page's
    // 1650 cycles.
    const bool ready = test_bar(&s.meta_full[ms], k / kMetas & 1) &
                       test_bar(&s.raw_full[raw], k / P::kRaw & 1) & has_room(0);
    const bool room = __all_sync(0xffffffffu, has_room(1));
    if (!__all_sync(0xffffffffu, ready)) {
      if (!warp_wait(&s.meta_full[ms], k / kMetas & 1, abort)) return;
      if (!warp_wait(&s.raw_full[raw], k / P::kRaw & 1, abort)) return;
      if (!wait_room(0)) return;
    }
    const uint8_t* codes = s.raw[raw] + uw * kBlockRows * D;
    // K and V are read before either is written: one wait for both
    uint4 x[2][kIter];
#pragma unroll
    for (int side = 0; side < 2; ++side)
#pragma unroll
      for (int i = 0; i < kIter; ++i)
        x[side][i] = *reinterpret_cast<const uint4*>(codes + side * P::kPiece + row_of(i) * D +
                                                     piece_of(i) * 16);
    const PageMeta& m = s.meta[ms];
    const int cnt = m.cnt, w = m.w;
    uint32_t here = 0xffffu, poison = 0;
    if (w > 0 || cnt < kPageRows) {
      const int row = uw * kBlockRows + lane;
      bool ok = lane < kBlockRows && row < cnt;
      if (ok && w > 0) ok = m.pos[row] >= 0;
      here = __ballot_sync(0xffffffffu, ok);
    }
    if (w > 0) {
      // A ring's row may be seen by some queries and not by others, and 0 times a NaN value is
      // NaN: its NaN values become zeros, and its key NaN, which only who sees it takes.
      const uint8_t* v = codes + P::kPiece;
#pragma unroll 1
      for (int r = 0; r < kBlockRows; r += 8) {
        bool nan = false;
#pragma unroll
        for (int z = 0; z < D / 64; ++z) {
          const uint4 x = *reinterpret_cast<const uint4*>(v + (r + lane / 4) * D +
                                                          (lane % 4 * (D / 64) + z) * 16);
          const uint32_t w4[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {  // a code's NaN is 0x7f: the only one that 1 carries into bit 7
            const uint32_t y = (w4[i] & 0x7f7f7f7fu) + 0x01010101u;
            nan |= (y & 0x80808080u) != 0;
          }
        }
        const uint32_t hit = __ballot_sync(0xffffffffu, nan);
        for (int i = 0; i < 8; ++i)
          if (hit >> (4 * i) & 15u) poison |= 1u << (r + i);
      }
      poison &= here;
    }
    const bool plain = here == 0xffffu && poison == 0;
    auto put = [&](uint8_t* dst, int r, int c, const uint32_t (&y)[8]) {
      uint8_t* p = dst + c / 4 * P::kHalf + r * 128;
      const int z = c % 4 * 2;
      *reinterpret_cast<uint4*>(p + ((z ^ lr) << 4)) = make_uint4(y[0], y[1], y[2], y[3]);
      *reinterpret_cast<uint4*>(p + (((z + 1) ^ lr) << 4)) = make_uint4(y[4], y[5], y[6], y[7]);
    };
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      if (side == 1 && !room && !wait_room(1)) return;
      uint8_t* dst = s.op[slot[side]] + uw * kBlockRows * 128;
      if (plain) {
#pragma unroll
        for (int i = 0; i < kIter; ++i) {
          const uint4 z = x[side][i];
          const uint32_t y[8] = {decode2(z.x), decode2(z.x >> 16), decode2(z.y), decode2(z.y >> 16),
                                 decode2(z.z), decode2(z.z >> 16), decode2(z.w), decode2(z.w >> 16)};
          put(dst, row_of(i), piece_of(i), y);
        }
      } else {
#pragma unroll 1
        for (int i = 0; i < kIter; ++i) {
          const int r = row_of(i), c = piece_of(i);
          const bool ok = here >> r & 1, bad = poison >> r & 1;
          const uint4 z4 = *reinterpret_cast<const uint4*>(codes + side * P::kPiece + r * D + c * 16);
          uint32_t y[8] = {decode2(z4.x), decode2(z4.x >> 16), decode2(z4.y), decode2(z4.y >> 16),
                           decode2(z4.z), decode2(z4.z >> 16), decode2(z4.w), decode2(z4.w >> 16)};
#pragma unroll
          for (int z = 0; z < 8; ++z) {
            if (bad)  // the codes' NaN is f16's 0x7fff
              y[z] = side == 0 ? 0x7fff7fffu
                               : ((y[z] & 0x7fffu) == 0x7fffu ? 0u : y[z] & 0xffffu) |
                                     ((y[z] & 0x7fff0000u) == 0x7fff0000u ? 0u : y[z] & 0xffff0000u);
            if (!ok) y[z] = 0;
          }
          put(dst, r, c, y);
        }
      }
      fence_async_shared();  // the tensor cores read what the lanes have written
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&s.op_full[slot[side]]);
        mbar_arrive(side == 0 ? &s.meta_empty[ms] : &s.raw_empty[raw]);
      }
    }
  }
}

// The thread that issues stream st's products.  A page's scores go to one of two places, when P of
// the page two before, which lay there, has been used: so the softmax has the next page's scores
// before it while the tensor cores take its weights.
template <int D, int kTerms, bool kPair>
__device__ __forceinline__ void issue(Smem<D, kTerms, kPair>& s, const PrefixParts& px, int st,
                                      Walk wk) {
  using P = Plan<D, kTerms, kPair>;
  constexpr uint32_t kScores = idesc_f16(kTile, kPageRows, false);
  constexpr uint32_t kValues = idesc_f16(kTile, D, true);
  constexpr int kStep = kPair ? 1 : 2;
  volatile int* abort = &s.abort;
  const uint32_t oc = s.tmem + o_col(st);
  int base = 0, units = 0;  // pages, units
  int ns = 0, np = 0;       // this stream's pages whose scores, whose weighted values were asked for
  bool asked = false, go = true;
  for (; wk.more() && go; wk.next(), ++units) {
    const int nt = wk.count();
    const bool both = wk.both();
    if (st == 0) {
      const uint32_t bytes = (both ? 2 : 1) * kTerms * P::kQTerm;
      if (units > 0 && !wait_or_stop(&s.q_free, (units - 1) & 1, abort)) break;
      mbar_expect_tx(&s.q_full, bytes);
      bulk_load(s.q, px.q + ((size_t)wk.c * px.tiles + wk.tile()) * kTerms * P::kQTerm, bytes,
                &s.q_full);
      asked = true;
    }
    if (!wait_or_stop(&s.q_full, units & 1, abort)) break;
    asked = false;
    if (kPair && st == 1 && !both) {  // no second tile of queries: the pages pass by
#pragma unroll 1
      for (int seq = 2 * base; seq < 2 * (base + nt) && go; ++seq) {
        go = wait_or_stop(&s.op_full[seq % P::kOperands], seq / P::kOperands & 1, abort);
        if (go) mbar_arrive(&s.op_empty[seq % P::kOperands]);
      }
      if (!go) break;
      mbar_arrive(&s.q_free);
      base += nt;
      continue;
    }
    const uint64_t q = desc_kmajor_sw128(smem_addr(s.q) + (both ? st * kTerms * P::kQTerm : 0));
    const int first = kPair ? 0 : (base ^ st) & 1;  // the unit's first page of this stream
    const int mine = nt > first ? (nt - first - 1) / kStep + 1 : 0;
    // What is ready goes first, weighted values before scores: a page's operands come in order, so
    // waiting for a key page while weights are there would hold up the pages before it.
    int si = 0, pi = 0;
    long long since = 0;
#pragma unroll 1
    while (pi < mine) {
      bool did = false;
      if (pi < si) {  // the weighted values of page pi
        const int b = np & 1, seq = 2 * (base + first + pi * kStep) + 1, slot = seq % P::kOperands;
        // (the first weights of a unit come when O of the unit before has been read)
        if (test_bar(&s.p_full[st][b], np >> 1 & 1) &&
            test_bar(&s.op_full[slot], seq / P::kOperands & 1)) {
          tc_fence_after();
          const uint64_t v = desc_mn_sw128(smem_addr(s.op[slot]), P::kHalf);
          const uint32_t w = s.tmem + s_col(st, b);
#pragma unroll
          for (int kk = 0; kk < kPageRows / 16; ++kk)
#pragma unroll
            for (int term = 0; term < kTerms; ++term)
              mma_ts(oc, w + kk / 2 * 32 + term * 16 + kk % 2 * 8, v + kk * (16 * 128 >> 4), kValues,
                     pi > 0 || kk > 0 || term > 0);
          umma_commit(&s.pv_done[st][b]);
          umma_commit(&s.op_empty[slot]);
          ++np;
          ++pi;
          did = true;
        }
      }
      if (si < mine && si < pi + 2) {  // the scores of page si
        const int b = ns & 1, seq = 2 * (base + first + si * kStep), slot = seq % P::kOperands;
        if (test_bar(&s.op_full[slot], seq / P::kOperands & 1) &&
            (ns < 2 || test_bar(&s.pv_done[st][b], ((ns >> 1) - 1) & 1))) {
          tc_fence_after();
          const uint64_t kd = desc_kmajor_sw128(smem_addr(s.op[slot]));
          const uint32_t sc = s.tmem + s_col(st, b);
#pragma unroll
          for (int term = 0; term < kTerms; ++term)
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              mma_ss(sc, q + term * (P::kQTerm >> 4) + kk / 4 * (P::kQHalf >> 4) + kk % 4 * 2,
                     kd + kk / 4 * (P::kHalf >> 4) + kk % 4 * 2, kScores, term > 0 || kk > 0);
          umma_commit(&s.s_full[st][b]);
          umma_commit(&s.op_empty[slot]);
          ++ns;
          ++si;
          did = true;
        }
      }
      if (did) {
        since = 0;
      } else {  // bounded like every other wait
        if (since == 0) since = clock64();
        if (clock64() - since > (1ll << 31)) *abort = 1;
        if (*abort) {
          go = false;
          break;
        }
      }
    }
    if (!go) break;
    mbar_arrive(&s.q_free);  // the weights were there, so the scores are complete
    base += nt;
  }
  if (asked) mbar_wait(&s.q_full, units & 1);  // (after a stop: nothing stays in flight)
  umma_commit(&s.drain[st]);  // every product issued is complete before the block ends
  mbar_wait(&s.drain[st], 0);
}

// A softmax warpgroup: stream st, a thread a query.
template <int D, int kTerms, bool kPair>
__device__ __forceinline__ void weights(Smem<D, kTerms, kPair>& s, const PagedDecodeArgs& n,
                                        const PrefixParts& px, int R, Walk wk) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int st = warp / 4, row = (warp & 3) * 32 + lane;
  volatile int* abort = &s.abort;
  const uint32_t lanes = s.tmem + ((uint32_t)((warp & 3) * 32) << 16);
  const uint32_t oc = lanes + o_col(st);
  int k = 0, mine = 0;  // pages of the block, those of this stream
  for (; wk.more(); wk.next()) {
    const int nt = wk.count();
    const bool both = wk.both();
    const int tile = wk.tile() + (kPair ? st : 0), j = tile * kTile + row;
    const int t = j < px.nq ? n.pos[j / R] : -1;
    const float fq = t < 0 ? 0.f : px.qf[((size_t)wk.c * px.tiles + tile) * kTile + row];
    // A key that does not count scores -inf, which its block's factor must leave alone: the exponent
    // of a block without a row may be any byte, and a query of zeros times a block of zeros has a
    // factor below what a float holds.  So no factor is below the least normal number: scores that
    // are that small (2^-96 at most) are as good as 0.  (Without a query: 0, whatever lies in S.)
    const float least = t < 0 ? 0.f : 1.17549435e-38f;
    const bool work = __any_sync(0xffffffffu, t >= 0);  // else no lane's result is asked for
    // the positions of the warp's queries lie from t_lo to t_hi
    const int t_lo = (int)__reduce_min_sync(0xffffffffu, t < 0 ? 0x7fffffffu : (uint32_t)t);
    const int t_hi = (int)__reduce_max_sync(0xffffffffu, t < 0 ? 0u : (uint32_t)t);
    float ms = kNoScore, mo = kNoScore, l = 0.f;  // reference of the scores; + V's exponent; sum
    int taken = 0;
#pragma unroll 1
    for (int i = 0; i < nt; ++i, ++k) {
      const int slot = k % kMetas;
      if (!warp_wait(&s.meta_full[slot], k / kMetas & 1, abort)) return;
      if (kPair ? st == 1 && !both : (k & 1) != st) {  // the other stream's
        if (lane == 0) mbar_arrive(&s.meta_empty[slot]);
        continue;
      }
      const PageMeta& m = s.meta[slot];
      const uint4 head = *reinterpret_cast<const uint4*>(&m);
      const int b2 = mine & 1;
      const uint32_t sc = lanes + s_col(st, b2);
      if (!warp_wait(&s.s_full[st][b2], mine >> 1 & 1, abort)) return;
      tc_fence_after();
      if (work) {
        const int cnt = (int)head.z, w = (int)head.w;
        if (cnt < kPageRows || w > 0) {
          // Which keys does any query of the warp see, as bits of the two columns of 32, and do
          // all of them see those?  (A ring also holds positions that no one sees any more.)
          uint32_t there[2];
          bool near = true;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const bool ok = x * 32 + lane < cnt;
            bool any = ok;
            if (w > 0) {
              const int p = m.pos[x * 32 + lane];
              any = ok && p >= 0 && p <= t_hi && t_lo - p < w;
              near &= any == (ok && p >= 0 && p <= t_lo && t_hi - p < w);
            }
            there[x] = __ballot_sync(0xffffffffu, any);
          }
          near = __all_sync(0xffffffffu, near);
          // keys that do not count score -inf
#pragma unroll 1
          for (int ch = 0; ch < 2; ++ch) {
            constexpr uint32_t kNone = 0xff800000u;
            const uint32_t bits = ch ? there[1] : there[0];
            if (near && bits == 0xffffffffu) continue;
            uint32_t r[32];
            tmem_ld32(sc + ch * 32, r);
            tmem_wait_ld(r);
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              if ((bits >> e & 15u) != 15u) {
#pragma unroll
                for (int x = 0; x < 4; ++x)
                  if (!(bits >> (e + x) & 1)) r[e + x] = kNone;
              }
            if (!near) {
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                const int4 p = *reinterpret_cast<const int4*>(m.pos + ch * 32 + e);
                const int p4[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
                for (int x = 0; x < 4; ++x)
                  if (p4[x] > t || (uint32_t)t - (uint32_t)p4[x] >= (uint32_t)w) r[e + x] = kNone;
              }
            }
            tmem_st16(sc + ch * 32, r);
            tmem_st16(sc + ch * 32 + 16, r + 16);
          }
          tmem_wait_st();
        }
        uint32_t r[2][32];  // the row of S
        tmem_ld32(sc, r[0]);
        tmem_ld32(sc + 32, r[1]);
        // factors of the blocks' scores and the exponents of their values
        float f[4], ev[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const uint32_t x = (b < 2 ? head.x : head.y) >> (16 * (b & 1));
          f[b] = fminf(fmaxf(fq * pow2f((int)(signed char)(x & 0xff)), least), 1.7e38f);
          ev[b] = (float)(signed char)(x >> 8 & 0xff);
        }
        tmem_wait_ld(r[0]);
        reg_barrier(r[1]);
        float smax = FG_NEG_INF, omax = FG_NEG_INF;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          float mx = FG_NEG_INF;
#pragma unroll
          for (int e = 0; e < 16; e += 2)
            mx = max3(mx, __uint_as_float(r[b / 2][b % 2 * 16 + e]),
                      __uint_as_float(r[b / 2][b % 2 * 16 + e + 1]));
          const float y = mx * f[b];
          smax = fmaxf(smax, y);
          omax = fmaxf(omax, y + ev[b]);
        }
        if (__any_sync(0xffffffffu, smax > ms + kSlack || omax > mo + kSlack)) {
          const float sn = fmaxf(ms, smax), on = fmaxf(mo, omax), z = ex2(mo - on);
          l *= ex2(ms - sn);
          ms = sn;
          mo = on;
          if (taken > 0) {  // O, when the product before is complete
            if (!warp_wait(&s.pv_done[st][b2 ^ 1], (mine - 1) >> 1 & 1, abort)) return;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              uint32_t o[16];
              tmem_ld16(oc + c, o);
              tmem_wait_ld16(o);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * z);
              tmem_st16(oc + c, o);
            }
          }
        }
        uint64_t sum2 = 0;  // (0, 0)
        const uint64_t nm2 = pack2(-ms, -ms);
        const float lift = ms - mo + kProdBits;
#pragma unroll
        for (int ch = 0; ch < 2; ++ch) {
          uint32_t hi[16], lo[16];
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const float g = ex2(fminf(ev[ch * 2 + b] + lift, 126.f));
            const uint64_t f2 = pack2(f[ch * 2 + b], f[ch * 2 + b]), g2 = pack2(g, g);
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              const int z = b * 16 + e;
              float x0, x1, p0, p1;
              unpack2(fma2(pack2(__uint_as_float(r[ch][z]), __uint_as_float(r[ch][z + 1])), f2, nm2),
                      x0, x1);
              const uint64_t w2 = pack2(ex2(x0), ex2(x1));
              sum2 = add2(sum2, w2);
              unpack2(mul2(w2, g2), p0, p1);
              hi[z / 2] = pack_f16x2(p0, p1);
              if constexpr (kTerms == 2) {
                const float2 y = unpack_f16x2(hi[z / 2]);
                lo[z / 2] = pack_f16x2(p0 - y.x, p1 - y.y);
              }
            }
          }
          tmem_st16(sc + ch * 32, hi);
          if constexpr (kTerms == 2) tmem_st16(sc + ch * 32 + 16, lo);
        }
        float x, y;
        unpack2(sum2, x, y);
        l += x + y;
        tmem_wait_st();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&s.p_full[st][b2]);
        mbar_arrive(&s.meta_empty[slot]);
      }
      ++mine;
      ++taken;
    }
    // the unit's partial result
    const size_t part = ((size_t)blockIdx.x + wk.unit()) * 2 + st;
    const bool write = row < px.rows && t >= 0;
    if (write)
      *reinterpret_cast<float2*>(px.ml + 2 * (part * px.rows + row)) = make_float2(ms, l);
    if (taken > 0) {
      if (!warp_wait(&s.pv_done[st][(mine - 1) & 1], (mine - 1) >> 1 & 1, abort)) return;
      tc_fence_after();
      if (work) {
        // O is in units of 2^(mo - kProdBits), l of 2^ms
        const float z = l == 0.f ? 0.f : exp2f(mo - ms - kProdBits) / l;
        // [d / 4][rows][4]: a warp's lanes write next to one another
        float4* out = reinterpret_cast<float4*>(px.acc + part * px.rows * D) + row;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          tmem_ld32(oc + c, o);
          tmem_wait_ld(o);
          if (write)
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              out[(size_t)((c + e) / 4) * px.rows] =
                  make_float4(__uint_as_float(o[e]) * z, __uint_as_float(o[e + 1]) * z,
                              __uint_as_float(o[e + 2]) * z, __uint_as_float(o[e + 3]) * z);
        }
      }
      tc_fence_before();
    }
  }
}

template <int D, int kTerms, bool kPair>
__global__ void __launch_bounds__(kPrefixThreads, 1)
    prefix_kernel(const PagedArgs a, const PagedDecodeArgs n, const PrefixParts px, int R) {
  extern __shared__ uint8_t smem_raw[];
  Smem<D, kTerms, kPair>& s = *reinterpret_cast<Smem<D, kTerms, kPair>*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  using P = Plan<D, kTerms, kPair>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0) {
    tmem_alloc(&s.tmem, kTmemCols);
    tmem_relinquish();
  }
  if (threadIdx.x == kLoadWarp * 32) {
    s.abort = 0;
    for (int i = 0; i < P::kRaw; ++i) {
      mbar_init(&s.raw_full[i], 1);
      mbar_init(&s.raw_empty[i], kUnpackWarps);
    }
    for (int i = 0; i < kMetas; ++i) {
      mbar_init(&s.meta_full[i], 1);
      mbar_init(&s.meta_empty[i], kUnpackWarps + kSoftWarps);
    }
    for (int i = 0; i < P::kOperands; ++i) {
      mbar_init(&s.op_full[i], kUnpackWarps);
      mbar_init(&s.op_empty[i], kPair ? 2 : 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&s.s_full[0][0] + i, 1);
      mbar_init(&s.p_full[0][0] + i, kSoftWarps / 2);
      mbar_init(&s.pv_done[0][0] + i, 1);
    }
    mbar_init(&s.drain[0], 1);
    mbar_init(&s.drain[1], 1);
    mbar_init(&s.q_full, 1);
    mbar_init(&s.q_free, 2);
    fence_barrier_init();
  }
  griddep_wait();
  griddep_launch_dependents();
  const long long total = px.cum[px.caches] * px.groups;
  const int ctas = prefix_ctas(total, px.ctas);
  const bool in = total > 0 && blockIdx.x < ctas;
  const long long x0 = in ? prefix_first(total, ctas, blockIdx.x) : 0;
  const long long x1 = in ? prefix_first(total, ctas, blockIdx.x + 1) : 0;
  for (int c = threadIdx.x; c < px.caches; c += kPrefixThreads)
    if (px.cum[c] * px.groups <= x0 && x0 < px.cum[c + 1] * px.groups) s.first_cache = c;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (x0 < x1) {
    const Walk wk(px, s.first_cache, x0, x1);
    if (warp < kSoftWarps)
      weights<D, kTerms, kPair>(s, n, px, R, wk);
    else if (warp < kLoadWarp)
      widen<D, kTerms, kPair>(s, warp - kSoftWarps, (int)(x1 - x0));
    else if (warp == kLoadWarp)
      load_pages<D, kTerms, kPair>(s, a, wk);
    else if (warp == kMetaWarp)
      load_metas<D, kTerms, kPair>(s, a, wk);
    else if (lane == 0)
      issue<D, kTerms, kPair>(s, px, warp - kMmaWarp, wk);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && s.abort) atomicOr(a.dev_err, kErrDevice);
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(s.tmem, kTmemCols);
  }
}

template <typename T, int D, bool kPair>
cudaError_t run_prefix(const ProfileDims& pd, const PagedDecodeArgs& n, const PagedArgs& pre,
                       const PrefixParts& px, cudaStream_t s) {
  constexpr int kTerms = sizeof(T) == 4 ? 2 : 1;
  const auto kernel = prefix_kernel<D, kTerms, kPair>;
  const int smem = (int)sizeof(Smem<D, kTerms, kPair>) + 1024;
  static_assert(sizeof(Smem<D, kTerms, kPair>) + 1024 <= kSmem, "shared memory of a block");
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess)
    e = launch_pdl(prefix_prep_kernel<T, D, kTerms>, cdiv(pd.G, kPrepThreads / 32) + 1,
                   kPrepThreads, 0, s, pre, n, px, pd.G, pd.H, pd.R, pd.HL, pd.sl2);
  if (e == cudaSuccess) e = launch_pdl(kernel, px.ctas, kPrefixThreads, smem, s, pre, n, px, pd.R);
  return e;
}

template <int D>
cudaError_t run_prefix(const ProfileDims& pd, const PagedDecodeArgs& n, const PagedArgs& pre,
                       const PrefixParts& px, cudaStream_t s) {
  if (pd.dtype == FG_FP32) return run_prefix<float, D, false>(pd, n, pre, px, s);
  return px.pair ? run_prefix<__nv_bfloat16, D, true>(pd, n, pre, px, s)
                 : run_prefix<__nv_bfloat16, D, false>(pd, n, pre, px, s);
}

}  // namespace

PrefixParts prefix_parts(const ProfileDims& pd, size_t (&bytes)[5]) {
  PrefixParts px = {};
  const int terms = pd.dtype == FG_FP32 ? 2 : 1;
  px.caches = pd.HLkv;
  px.nq = pd.B * pd.R;
  px.tiles = cdiv(px.nq, kTile);
  px.pair = terms == 1 && px.tiles > 1;
  px.groups = px.pair ? cdiv(px.tiles, 2) : px.tiles;
  px.rows = px.nq < kTile ? px.nq : kTile;
  const size_t tiles = (size_t)px.caches * px.tiles;
  const size_t parts = 2 * (kPrefixMaxCtas + (size_t)px.caches * px.groups) * px.rows;
  bytes[0] = (px.caches + 1) * sizeof(long long);
  bytes[1] = tiles * terms * kTile * pd.d * 2;
  bytes[2] = tiles * kTile * sizeof(float);
  bytes[3] = parts * 2 * sizeof(float);
  bytes[4] = parts * pd.d * sizeof(float);
  return px;
}

cudaError_t launch_prefix(const ProfileDims& pd, const PagedDecodeArgs& n, const PagedArgs& pre,
                          const PrefixParts& px, cudaStream_t s) {
  return pd.d == 64 ? run_prefix<64>(pd, n, pre, px, s) : run_prefix<128>(pd, n, pre, px, s);
}

}  // namespace fg
