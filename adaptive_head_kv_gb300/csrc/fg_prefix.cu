// Attention of a batch over the caches of a prompt that its sequences share:
// every query of sequence b and head h over cache h / R of the prompt, which is
// read once for all sequences.
//
// With B sequences and groups of R a cache meets B R queries, so both products
// are matrix products of the tensor cores:
//   S [128 queries x 128 keys] = Q K^T,  O [128 x d] += P V,
// accumulators and P in tensor memory, operands in shared memory.  The codes of
// a page are widened to f16, which holds them exactly, on their way; the
// exponents of a block of 16 keys are two numbers for 16 columns of S: K's
// scales the scores, V's goes into the weights that enter the product.
// Queries are f16 after the division by a power of two (11 bits; fp32 inputs two
// terms, 22 bits: Q = Qh + Ql along the product's depth, P = Ph + Pl likewise).
//
// A thread block per SM: a warp that loads pages (bulk copies of codes, 2 KB to
// 8 KB each), four that widen them into the swizzled layout the tensor cores
// read, one that issues the products, and two warpgroups of softmax, a thread a
// query.  The two work on separate streams with S and O of their own: two tiles
// of queries over the same key tiles, or, where there is one tile of queries,
// the even and the odd key tiles.  One stream's softmax runs while the tensor
// cores have the other's products.  P takes S's place in tensor memory.
//
// The softmax is one pass over the rows: sums and products are kept relative
// to reference maxima that follow the true ones when those get 2^kSlack ahead
// (then O is rescaled in tensor memory).  The sum's maximum is that of the
// scores, the product's that of score + V's exponent, as in the split kernel.
#include "fg_paged_decode.cuh"

namespace fg {
namespace {

using namespace sm100;

constexpr int kTile = kPrefixTile;
constexpr int kTilePages = kTile / kPageRows;
constexpr int kUnpackWarps = 4, kSoftWarps = 8;
// warps 0-7 softmax (warp w reads tensor memory lanes 32 (w % 4) ..), 8-11 widen
constexpr int kLoadWarp = kSoftWarps + kUnpackWarps, kMmaWarp = kLoadWarp + 1;
constexpr int kPrefixThreads = (kMmaWarp + 1) * 32;
constexpr int kMetas = 4;     // key tiles whose description is there
constexpr float kSlack = 4.f;
constexpr float kProdBits = 11.f;  // weights enter the product times 2^11, at most 2^15
constexpr int kSmem = 227 * 1024;

// A key tile: two pages of a segment or of a ring.
struct TileMeta {
  uint32_t exps[2 * kTilePages];  // of the pages' blocks: (K, V) bytes
  int cnt[kTilePages];            // rows of each page (0: no page)
  int ring;
  int w;
  int pos[kTile];                 // of a ring's rows
};

template <int D, int kTerms, bool kPair>
struct Plan {
  static constexpr int kHalf = kTile * 128;  // bytes of 64 dimensions of a tile
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kQTerm = kTileBytes;                           // one term of a tile of queries
  static constexpr int kQBytes = (kPair ? 2 : 1) * kTerms * kQTerm;   // the queries in shared memory
  static constexpr int kPiece = kPageRows * D;                        // codes of K or of V of a page
  // widened K or V tiles: K of the next tile beside K and V of this one at least
  static constexpr int kOperands = D == 64 ? 6 : kPair || kTerms == 2 ? 3 : 4;
  static constexpr int kRoom =
      (kSmem - 1024 - 3584 - kQBytes - kOperands * kTileBytes) / kPiece;
  static constexpr int kPieces = kRoom > 16 ? 16 : kRoom;
  static_assert(kPieces >= 2 * kTilePages, "a tile's codes are there together");
};

template <int D, int kTerms, bool kPair>
struct alignas(1024) Smem {
  using P = Plan<D, kTerms, kPair>;
  uint8_t q[P::kQBytes];
  uint8_t op[P::kOperands][P::kTileBytes];
  alignas(128) uint8_t raw[P::kPieces][P::kPiece];
  alignas(16) TileMeta meta[kMetas];
  uint64_t raw_full[P::kPieces], raw_empty[P::kPieces];
  uint64_t meta_full[kMetas], meta_empty[kMetas];
  uint64_t op_full[P::kOperands], op_empty[P::kOperands];
  uint64_t s_full[2], p_full[2], pv_done[2];
  uint64_t q_full, drain;
  int abort;
  uint32_t tmem;
  int first_cache;  // of this block's range
};

// tensor memory: S (and P) of the two streams, then O
constexpr uint32_t kTmemCols = 512;
__device__ __forceinline__ uint32_t s_col(int s) { return s * kTile; }
__device__ __forceinline__ uint32_t o_col(int s) { return 2 * kTile + s * 128; }

__device__ __forceinline__ bool wait_or_stop(uint64_t* bar, uint32_t parity, volatile int* abort) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  while (!*abort) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (global_timer_ns() - t0 > kWaitLimitNs) *abort = 1;
  }
  return false;
}
// The same by a whole warp.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  return __all_sync(0xffffffffu, wait_or_stop(bar, parity, abort));
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
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Key tiles of a cache: of its segment, of its ring.
__device__ __forceinline__ int2 key_tiles(const PagedArgs& a, const fg_paged_desc& hd, int rows) {
  return make_int2(cdiv(live_rows(hd, rows), kTile), cdiv(ring_slots(hd, a.max_w), kTile));
}

// ------------------------------------------------------------- before the products
// A CTA a tile of queries: rotated, divided by the power of two that brings the largest value to
// [2^13, 2^14), as f16 in the tensor cores' layout.  The last CTA counts the caches' key tiles.
constexpr int kPrepThreads = 256;

template <typename T, int D, int kTerms>
__global__ void __launch_bounds__(kPrepThreads)
    prefix_prep_kernel(const PagedArgs a, const PagedDecodeArgs n, const PrefixParts px, int H,
                       int R, int HL, float sl2) {
  constexpr int PER = D / 32;
  __shared__ long long scr[33];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  griddep_wait();
  griddep_launch_dependents();
  if (blockIdx.x == px.caches * px.tiles) {
    long long sum = 0, tot;
    for (int base = 0; base < px.caches; base += kPrepThreads) {
      const int c = base + threadIdx.x;
      long long x = 0;
      if (c < px.caches) {
        const fg_paged_desc hd = a.caches[c];
        const int rows = a.rows[c];
        if (live_rows(hd, rows) != rows || ring_slots(hd, a.max_w) != hd.w)
          atomicOr(a.dev_err, kErrInvalid);
        const int2 k = key_tiles(a, hd, rows);
        x = (long long)k.x + k.y;
      }
      const long long at = sum + block_exclusive_scan(x, scr, &tot);
      if (c < px.caches) px.cum[c] = at;
      sum += tot;
    }
    if (threadIdx.x == 0) px.cum[px.caches] = sum;
    return;
  }
  const int c = blockIdx.x / px.tiles, tile = blockIdx.x % px.tiles;
  uint8_t* dst = px.q + (size_t)blockIdx.x * kTerms * kTile * D * 2;
  float* qf = px.qf + (size_t)blockIdx.x * kTile;
  float2 cs[PER];
  int cs_of = -1;
  for (int r = warp; r < kTile; r += kPrepThreads / 32) {
    const int j = tile * kTile + r, b = j / R;
    const int t = j < px.nq ? n.pos[b] : -1;
    float x[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) x[k] = 0.f;
    float f = 0.f, inv = 0.f;
    if (t >= 0) {
      const size_t g = (size_t)b * HL + (size_t)(c / (H / R)) * H + (size_t)(c % (H / R)) * R + j % R;
      load_row<PER>((const T*)n.q + g * D, x);
      if (n.rope.rot > 0) {
        if (cs_of != b)
          row_angles<PER>(cs, n.rope.rot, n.rope.style, [&](int p) {
            float2 y;
            rope_cos_sin((unsigned)t, n.rope.turns[p], y.x, y.y);
            return y;
          });
        cs_of = b;
        rotate_row<PER>(x, cs, n.rope.rot, n.rope.style);
      }
      uint32_t top = 0;
#pragma unroll
      for (int k = 0; k < PER; ++k) top = max(top, finite_bits(x[k]));
      top = __reduce_max_sync(0xffffffffu, top);
      const int eq = max(-110, (int)(top >> 23) - 127 - 13);
      inv = pow2f(-eq);
      f = pow2f(eq) * sl2;
    }
    const int e = lane * PER;
    uint8_t* p = dst + e / 64 * (kTile * 128) + r * 128 + ((((e % 64) / 8) ^ (r & 7)) << 4) + e % 8 * 2;
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
    if (lane == 0) qf[r] = f;
  }
}

// ------------------------------------------------------------------- the products
// The part of a unit's key tiles that a thread block takes.
struct Walk {
  const PrefixParts& px;
  long long x, end;  // of the block's range
  int c, grp;
  long long c0, tiles;  // of the cache
  __device__ Walk(const PrefixParts& p, int first_cache, long long x0, long long x1)
      : px(p), x(x0), end(x1), c(first_cache) {
    c0 = px.cum[c];
    tiles = px.cum[c + 1] - c0;
    grp = tiles > 0 ? (int)((x - c0 * px.groups) / tiles) : 0;
  }
  __device__ bool more() const { return x < end; }
  __device__ int first() const { return (int)(x - c0 * px.groups - grp * tiles); }  // key tile
  __device__ int count() const { return (int)min(tiles - first(), end - x); }
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
      tiles = px.cum[c + 1] - c0;
    } while (tiles == 0);
  }
};

template <int D, int kTerms, bool kPair>
__device__ __forceinline__ void load_pages(Smem<D, kTerms, kPair>& s, const PagedArgs& a, Walk wk) {
  using P = Plan<D, kTerms, kPair>;
  const int lane = threadIdx.x & 31;
  volatile int* abort = &s.abort;
  int k = 0, pieces = 0, metas = 0;  // key tiles of this block; copies asked for so far
  bool stop = false;
  for (; wk.more() && !stop; wk.next()) {
    const fg_paged_desc hd = a.caches[wk.c];
    const int rows = live_rows(hd, a.rows[wk.c]), w = ring_slots(hd, a.max_w);
    const int seg = cdiv(rows, kTile), t0 = wk.first(), nt = wk.count();
    int page_l = -1;
    uint2 exp_l = make_uint2(0, 0);
    for (int i = 0; i < nt; ++i, ++k) {
      if ((i & 15) == 0) {  // pages of the next 16 tiles: lane l holds one and its exponents
        const int t = t0 + i + lane / 2, e = (t < seg ? t : t - seg) * kTilePages + lane % 2;
        page_l = -1;
        if (i + lane / 2 < nt && e * kPageRows < (t < seg ? rows : w)) {
          page_l = t < seg ? page_at(a, hd.first_page, hd.max_pages, e)
                           : page_at(a, hd.ring_page, hd.ring_pages, e);
          if (page_l < 0)
            atomicOr(a.dev_err, kErrInvalid);
          else
            exp_l = *reinterpret_cast<const uint2*>(a.exps + (size_t)page_l * kPageBlocks * 2);
        }
      }
      const int t = t0 + i, ring = t >= seg, row0 = (ring ? t - seg : t) * kTile;
      const int left = (ring ? w : rows) - row0;
      int page[kTilePages];
      uint2 ex[kTilePages];
#pragma unroll
      for (int g = 0; g < kTilePages; ++g) {
        page[g] = __shfl_sync(0xffffffffu, page_l, (i & 15) * 2 + g);
        ex[g].x = __shfl_sync(0xffffffffu, exp_l.x, (i & 15) * 2 + g);
        ex[g].y = __shfl_sync(0xffffffffu, exp_l.y, (i & 15) * 2 + g);
      }
      if (lane == 0) {
        const int ms = k % kMetas;
        if (k >= kMetas && !wait_or_stop(&s.meta_empty[ms], (k / kMetas - 1) & 1, abort)) stop = true;
        TileMeta& m = s.meta[ms];
        uint32_t bytes = 0;
        if (!stop) {
#pragma unroll
          for (int g = 0; g < kTilePages; ++g) {
            m.exps[2 * g] = ex[g].x;
            m.exps[2 * g + 1] = ex[g].y;
            m.cnt[g] = page[g] < 0 ? 0 : max(0, min(kPageRows, left - g * kPageRows));
            if (ring && page[g] >= 0) bytes += kPageRows * 4;
          }
          m.ring = ring;
          m.w = w;
          mbar_expect_tx(&s.meta_full[ms], bytes);
          ++metas;
#pragma unroll
          for (int g = 0; g < kTilePages; ++g)
            if (ring && page[g] >= 0)
              bulk_load(m.pos + g * kPageRows, a.pos + (size_t)page[g] * kPageRows, kPageRows * 4,
                        &s.meta_full[ms]);
        }
        for (int z = 0; z < 2 * kTilePages && !stop; ++z) {
          const int seq = 2 * kTilePages * k + z, slot = seq % P::kPieces, g = z % kTilePages;
          if (seq >= P::kPieces &&
              !wait_or_stop(&s.raw_empty[slot], (seq / P::kPieces - 1) & 1, abort)) {
            stop = true;
          } else if (page[g] < 0) {
            mbar_arrive(&s.raw_full[slot]);
            ++pieces;
          } else {
            ++pieces;
            mbar_expect_tx(&s.raw_full[slot], P::kPiece);
            bulk_load(s.raw[slot], (z < kTilePages ? a.kp : a.vp) + (size_t)page[g] * P::kPiece,
                      P::kPiece, &s.raw_full[slot]);
          }
        }
      }
      stop = __shfl_sync(0xffffffffu, stop, 0);
      if (stop) break;
    }
    if (stop) break;
  }
  if (*abort && lane == 0) {  // what is in flight lands before the block ends
    for (int i = max(0, pieces - P::kPieces); i < pieces; ++i)
      mbar_wait(&s.raw_full[i % P::kPieces], i / P::kPieces & 1);
    for (int i = max(0, metas - kMetas); i < metas; ++i)
      mbar_wait(&s.meta_full[i % kMetas], i / kMetas & 1);
  }
}

// One of the four warps that widen codes: rows 16 w .. of every page, where an operand row that is
// not there is zero.  A lane's 16 bytes and the 32 it makes of them are chosen so that the eight
// lanes of a phase meet eight different banks, in the codes and in the swizzled tile.
template <int D, int kTerms, bool kPair>
__device__ __forceinline__ void widen(Smem<D, kTerms, kPair>& s, int uw, int total) {
  using P = Plan<D, kTerms, kPair>;
  constexpr int kIter = kBlockRows * (D / 16) / 32;  // 16-byte pieces of a lane
  const int lane = threadIdx.x & 31, lr = lane & 7;
  volatile int* abort = &s.abort;
  for (int k = 0; k < total; ++k) {
    const int ms = k % kMetas;
    if (!warp_wait(&s.meta_full[ms], k / kMetas & 1, abort)) return;
    const TileMeta& m = s.meta[ms];
    const int ring = m.ring;
    uint32_t there[kTilePages], poison[kTilePages] = {};
#pragma unroll
    for (int g = 0; g < kTilePages; ++g) {
      const int row = uw * kBlockRows + lane;
      bool ok = lane < kBlockRows && row < m.cnt[g];
      if (ok && ring) ok = m.pos[g * kPageRows + row] >= 0;
      there[g] = __ballot_sync(0xffffffffu, ok);
    }
    if (ring) {
      // A ring's row may be seen by some queries and not by others, and 0 times a NaN value is
      // NaN: its NaN values become zeros, and its key NaN, which only who sees it takes.
#pragma unroll
      for (int g = 0; g < kTilePages; ++g) {
        const int seq = 2 * kTilePages * k + kTilePages + g;
        if (!warp_wait(&s.raw_full[seq % P::kPieces], seq / P::kPieces & 1, abort)) return;
        const uint8_t* v = s.raw[seq % P::kPieces] + uw * kBlockRows * D;
        if (m.cnt[g] > 0)
          for (int r = 0; r < kBlockRows; r += 8) {
            bool nan = false;
#pragma unroll
            for (int z = 0; z < D / 64; ++z) {
              const uint4 x = *reinterpret_cast<const uint4*>(v + (r + lane / 4) * D +
                                                              (lane % 4 * (D / 64) + z) * 16);
              nan |= (__vcmpeq4(x.x & 0x7f7f7f7fu, 0x7f7f7f7fu) | __vcmpeq4(x.y & 0x7f7f7f7fu, 0x7f7f7f7fu) |
                      __vcmpeq4(x.z & 0x7f7f7f7fu, 0x7f7f7f7fu) | __vcmpeq4(x.w & 0x7f7f7f7fu, 0x7f7f7f7fu)) != 0;
            }
            const uint32_t hit = __ballot_sync(0xffffffffu, nan);
            for (int i = 0; i < 8; ++i)
              if (hit >> (4 * i) & 15u) poison[g] |= 1u << (r + i);
          }
      }
    }
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const int oseq = 2 * k + side, slot = oseq % P::kOperands;
      if (oseq >= P::kOperands && !warp_wait(&s.op_empty[slot], (oseq / P::kOperands - 1) & 1, abort))
        return;
#pragma unroll
      for (int g = 0; g < kTilePages; ++g) {
        const int seq = 2 * kTilePages * k + side * kTilePages + g, raw = seq % P::kPieces;
        if (!warp_wait(&s.raw_full[raw], seq / P::kPieces & 1, abort)) return;
        const uint8_t* src = s.raw[raw] + uw * kBlockRows * D;
        uint8_t* dst = s.op[slot] + (g * kPageRows + uw * kBlockRows) * 128;
#pragma unroll
        for (int i = 0; i < kIter; ++i) {
          const int r = lr + (i & 1) * 8;
          const int c = D == 128 ? ((lane >> 3) + 4 * (i >> 1) + lr) & 7
                                 : (((((lr >> 2) ^ (lr >> 1)) & 1) << 1 | (lr >> 2)) ^ (lane >> 3)) & 3;
          uint4 x = *reinterpret_cast<const uint4*>(src + r * D + c * 16);
          uint32_t y[8];
          const uint32_t w4[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            y[2 * z] = decode2(w4[z]);
            y[2 * z + 1] = decode2(w4[z] >> 16);
          }
          if (!(there[g] >> r & 1)) {
#pragma unroll
            for (int z = 0; z < 8; ++z) y[z] = 0;
          } else if (poison[g] >> r & 1) {
#pragma unroll
            for (int z = 0; z < 8; ++z) {
              const uint32_t nan = __vcmpgtu2(y[z] & 0x7fff7fffu, 0x7c007c00u);
              y[z] = side == 0 ? 0x7fff7fffu : y[z] & ~nan;
            }
          }
          uint8_t* p = dst + c / 4 * P::kHalf + r * 128;
          const int z = c % 4 * 2;
          *reinterpret_cast<uint4*>(p + ((z ^ lr) << 4)) = make_uint4(y[0], y[1], y[2], y[3]);
          *reinterpret_cast<uint4*>(p + (((z + 1) ^ lr) << 4)) = make_uint4(y[4], y[5], y[6], y[7]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.raw_empty[raw]);
      }
      fence_async_shared();  // the tensor cores read what the lanes have written
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.op_full[slot]);
    }
    if (lane == 0) mbar_arrive(&s.meta_empty[ms]);
  }
}

template <int D, int kTerms, bool kPair>
__device__ __forceinline__ void issue(Smem<D, kTerms, kPair>& s, const PrefixParts& px, Walk wk) {
  using P = Plan<D, kTerms, kPair>;
  constexpr uint32_t kScores = idesc_f16(kTile, kTile, false), kValues = idesc_f16(kTile, D, true);
  volatile int* abort = &s.abort;
  const uint32_t tmem = s.tmem;
  int base = 0, units = 0;    // key tiles and units done
  int done[2] = {0, 0};       // P V products issued of each stream
  bool stop = false;
  for (; wk.more() && !stop; wk.next(), ++units) {
    const int nt = wk.count();
    const bool both = wk.both();
    const int n[2] = {both ? nt : (nt + 1) / 2, both ? nt : nt / 2};
    // the scores of the unit before are complete (their weights were formed)
    const uint32_t bytes = (both ? 2 : 1) * kTerms * P::kQTerm;
    mbar_expect_tx(&s.q_full, bytes);
    bulk_load(s.q, px.q + ((size_t)wk.c * px.tiles + wk.tile()) * kTerms * P::kQTerm, bytes, &s.q_full);
    if (!mbar_wait(&s.q_full, units & 1)) {
      *abort = 1;
      break;
    }
    int si[2] = {0, 0}, pi[2] = {0, 0};
    int idle = 0;
    uint64_t t0 = global_timer_ns();
    while (pi[0] < n[0] || pi[1] < n[1]) {
      bool did = false;
#pragma unroll
      for (int st = 0; st < 2; ++st) {
        if (pi[st] < si[st]) {  // the weighted values of a tile whose weights are there
          const int t = both ? pi[st] : 2 * pi[st] + st, oseq = 2 * (base + t) + 1;
          const int slot = oseq % P::kOperands;
          // (the first weights of a unit come when O of the unit before has been read)
          if (test_bar(&s.p_full[st], done[st] & 1) &&
              test_bar(&s.op_full[slot], oseq / P::kOperands & 1)) {
            tc_fence_after();
            const uint32_t v = smem_addr(s.op[slot]);
#pragma unroll
            for (int kk = 0; kk < kTile / 16; ++kk)
#pragma unroll
              for (int term = 0; term < kTerms; ++term)
                mma_ts(tmem + o_col(st), tmem + s_col(st) + kk / 2 * 32 + term * 16 + kk % 2 * 8,
                       desc_mn_sw128(v + kk * 16 * 128, P::kHalf), kValues,
                       pi[st] > 0 || kk > 0 || term > 0);
            umma_commit(&s.pv_done[st]);
            ++pi[st];
            ++done[st];
            if (!both || pi[st ^ 1] > t) umma_commit(&s.op_empty[slot]);
            did = true;
          }
        }
        if (si[st] < n[st] && si[st] == pi[st]) {  // the scores of a tile: P of the one before is read
          const int t = both ? si[st] : 2 * si[st] + st, oseq = 2 * (base + t);
          const int slot = oseq % P::kOperands;
          if ((done[st] == 0 || test_bar(&s.pv_done[st], (done[st] - 1) & 1)) &&
              test_bar(&s.op_full[slot], oseq / P::kOperands & 1)) {
            tc_fence_after();
            const uint32_t q = smem_addr(s.q) + (both ? st * kTerms * P::kQTerm : 0);
            const uint32_t kt = smem_addr(s.op[slot]);
#pragma unroll
            for (int term = 0; term < kTerms; ++term)
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t off = kk / 4 * P::kHalf + kk % 4 * 32;
                mma_ss(tmem + s_col(st), desc_kmajor_sw128(q + term * P::kQTerm + off),
                       desc_kmajor_sw128(kt + off), kScores, term > 0 || kk > 0);
              }
            umma_commit(&s.s_full[st]);
            ++si[st];
            if (!both || si[st ^ 1] > t) umma_commit(&s.op_empty[slot]);
            did = true;
          }
        }
      }
      if (did) {
        idle = 0;
        t0 = global_timer_ns();
        continue;
      }
      if (*abort) {
        stop = true;
        break;
      }
      if (++idle >= 64) {  // bounded like every other wait
        idle = 0;
        if (global_timer_ns() - t0 > kWaitLimitNs) *abort = 1;
      }
    }
    base += nt;
  }
  umma_commit(&s.drain);  // every product issued is complete before the block ends
  mbar_wait(&s.drain, 0);
}

// A softmax warpgroup: stream st, a thread a query.
template <int D, int kTerms, bool kPair>
__device__ __forceinline__ void weights(Smem<D, kTerms, kPair>& s, const PagedDecodeArgs& n,
                                        const PrefixParts& px, int R, Walk wk) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int st = warp / 4, row = (warp & 3) * 32 + lane;
  volatile int* abort = &s.abort;
  const uint32_t lanes = s.tmem + ((uint32_t)((warp & 3) * 32) << 16);
  const uint32_t sc = lanes + s_col(st), oc = lanes + o_col(st);
  int k = 0, mine = 0, cta = blockIdx.x;  // key tiles of the block, those of this stream
  for (; wk.more(); wk.next()) {
    const int nt = wk.count();
    const bool both = wk.both();
    const int tile = wk.tile() + (both ? st : 0), j = tile * kTile + row;
    const int t = j < px.nq ? n.pos[j / R] : -1;
    const float fq = px.qf[((size_t)wk.c * px.tiles + tile) * kTile + row];
    const bool work = __any_sync(0xffffffffu, t >= 0);  // else no lane's result is asked for
    float ms = kNoScore, mo = kNoScore, l = 0.f;  // reference of the scores; + V's exponent; sum
    int taken = 0;
    for (int i = 0; i < nt; ++i, ++k) {
      const int slot = k % kMetas;
      if (!both && (i & 1) != st) {  // the other stream's
        if (!warp_wait(&s.meta_full[slot], k / kMetas & 1, abort)) return;
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.meta_empty[slot]);
        continue;
      }
      if (!warp_wait(&s.meta_full[slot], k / kMetas & 1, abort)) return;
      const TileMeta& m = s.meta[slot];
      if (!warp_wait(&s.s_full[st], mine & 1, abort)) return;
      tc_fence_after();
      if (work) {
        const bool ring = m.ring, whole = !ring && m.cnt[0] == kPageRows && m.cnt[1] == kPageRows;
        const uint4 e4 = *reinterpret_cast<const uint4*>(m.exps);
        const uint32_t ew[4] = {e4.x, e4.y, e4.z, e4.w};
        auto ek = [&](int b) { return (int)(signed char)(ew[b / 2] >> (16 * (b & 1)) & 0xff); };
        auto ev = [&](int b) { return (float)(signed char)(ew[b / 2] >> (16 * (b & 1) + 8) & 0xff); };
        // does this query see key x of the tile?
        auto sees = [&](int x) {
          bool ok = x % kPageRows < m.cnt[x / kPageRows];
          if (ring) {
            const int p = m.pos[x];
            ok = ok && p >= 0 && (unsigned)t - (unsigned)p < (unsigned)m.w;
          }
          return ok;
        };
        float smax = FG_NEG_INF, omax = FG_NEG_INF;
        uint32_t seen[4] = {~0u, ~0u, ~0u, ~0u};
        if (!whole)
#pragma unroll
          for (int ch = 0; ch < 4; ++ch) {
            uint32_t bits = 0;
#pragma unroll 8
            for (int e = 0; e < 32; ++e) bits |= (sees(ch * 32 + e) ? 1u : 0u) << e;
            seen[ch] = bits;
          }
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) {
          uint32_t r[32];
          tmem_ld32(sc + ch * 32, r);
          tmem_wait_ld(r);
          if (!whole)
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!(seen[ch] >> e & 1)) r[e] = 0xff800000u;
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            float mx = FG_NEG_INF;
#pragma unroll
            for (int e = 0; e < 16; e += 2)
              mx = max3(mx, __uint_as_float(r[b * 16 + e]), __uint_as_float(r[b * 16 + e + 1]));
            const float y = mx * fminf(fq * pow2f(ek(ch * 2 + b)), 1.7e38f);
            smax = fmaxf(smax, y);
            omax = fmaxf(omax, y + ev(ch * 2 + b));
          }
        }
        if (__any_sync(0xffffffffu, smax > ms + kSlack || omax > mo + kSlack)) {
          const float sn = fmaxf(ms, smax), on = fmaxf(mo, omax), f = ex2(mo - on);
          l *= ex2(ms - sn);
          ms = sn;
          mo = on;
          if (taken > 0) {
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              uint32_t r[32];
              tmem_ld32(oc + c, r);
              tmem_wait_ld(r);
#pragma unroll
              for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * f);
              tmem_st16(oc + c, r);
              tmem_st16(oc + c + 16, r + 16);
            }
          }
        }
        uint64_t sum2 = 0;  // (0, 0)
        const uint64_t nm2 = pack2(-ms, -ms);
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) {
          uint32_t r[32], hi[16], lo[16];
          tmem_ld32(sc + ch * 32, r);
          tmem_wait_ld(r);
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const float f = fminf(fq * pow2f(ek(ch * 2 + b)), 1.7e38f);
            const float g = ex2(fminf(ev(ch * 2 + b) + ms - mo + kProdBits, 126.f));
            const uint64_t f2 = pack2(f, f), g2 = pack2(g, g);
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              const int z = b * 16 + e;
              float x0, x1, p0, p1;
              unpack2(fma2(pack2(__uint_as_float(r[z]), __uint_as_float(r[z + 1])), f2, nm2), x0, x1);
              x0 = ex2(x0);
              x1 = ex2(x1);
              if (!whole) {
                if (!(seen[ch] >> z & 1)) x0 = 0.f;
                if (!(seen[ch] >> (z + 1) & 1)) x1 = 0.f;
              }
              const uint64_t w2 = pack2(x0, x1);
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
        float a, b;
        unpack2(sum2, a, b);
        l += a + b;
        tmem_wait_st();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&s.p_full[st]);
        mbar_arrive(&s.meta_empty[slot]);
      }
      ++mine;
      ++taken;
    }
    // the unit's partial result
    const size_t part = ((size_t)cta + wk.unit()) * 2 + st;
    const bool write = row < px.rows && t >= 0;
    if (write)
      *reinterpret_cast<float2*>(px.ml + 2 * (part * px.rows + row)) = make_float2(ms, l);
    if (taken > 0) {
      if (!warp_wait(&s.pv_done[st], (mine - 1) & 1, abort)) return;
      tc_fence_after();
      if (work) {
        // O is in units of 2^(mo - kProdBits), l of 2^ms
        const float f = l == 0.f ? 0.f : exp2f(mo - ms - kProdBits) / l;
        float* out = px.acc + (part * px.rows + row) * D;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t r[32];
          tmem_ld32(oc + c, r);
          tmem_wait_ld(r);
          if (write)
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<float4*>(out + c + e) =
                  make_float4(__uint_as_float(r[e]) * f, __uint_as_float(r[e + 1]) * f,
                              __uint_as_float(r[e + 2]) * f, __uint_as_float(r[e + 3]) * f);
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
    for (int i = 0; i < P::kPieces; ++i) {
      mbar_init(&s.raw_full[i], 1);
      mbar_init(&s.raw_empty[i], kUnpackWarps);
    }
    for (int i = 0; i < kMetas; ++i) {
      mbar_init(&s.meta_full[i], 1);
      mbar_init(&s.meta_empty[i], kUnpackWarps + kSoftWarps);
    }
    for (int i = 0; i < P::kOperands; ++i) {
      mbar_init(&s.op_full[i], kUnpackWarps);
      mbar_init(&s.op_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.s_full[i], 1);
      mbar_init(&s.p_full[i], kSoftWarps / 2);
      mbar_init(&s.pv_done[i], 1);
    }
    mbar_init(&s.q_full, 1);
    mbar_init(&s.drain, 1);
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
    if (warp == kLoadWarp)
      load_pages<D, kTerms, kPair>(s, a, wk);
    else if (warp == kMmaWarp) {
      if (lane == 0) issue<D, kTerms, kPair>(s, px, wk);
    } else if (warp >= kSoftWarps)
      widen<D, kTerms, kPair>(s, warp - kSoftWarps, (int)(x1 - x0));
    else
      weights<D, kTerms, kPair>(s, n, px, R, wk);
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
    e = launch_pdl(prefix_prep_kernel<T, D, kTerms>, px.caches * px.tiles + 1, kPrepThreads, 0, s,
                   pre, n, px, pd.H, pd.R, pd.HL, pd.sl2);
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
