// One generation step over paged 8-bit caches (Model Tells You What to
// Discard, Method: head-specific caches, the prompt-time policy reused).
//
// Split-K over the work list: an item is up to rpw rows of one cache's
// never-evicted segment (the last one also every row appended later) or of
// its ring.  A CTA of 4 warps takes an item, warp v its blocks of 16 rows v,
// v + 4, ...; the CTA whose item holds the new token's row codes it into the
// page first.  A warp's blocks reach a ring of kStages blocks in shared memory by
// cp.async (each code is read once, and loads stay in flight without holding
// registers), and both products run as warp MMAs in f16, which holds every
// e4m3 code exactly:
//   S[16 x 16 keys] = Q[16 x d] . K^T    queries in rows 0-7; rows 8-15 hold
//                                        what f16 loses of fp32 queries
//   O^T[d x 8]     += V^T[d x 16 keys] . P^T
// The dimension order inside a product is free as long as both operands agree,
// so a lane's operand fragments are 16 consecutive bytes of a row; S's
// accumulators are P^T's operand fragment as they stand.  The order of the
// keys is free as well: with 16-byte pieces swizzled by the row, slot_key
// puts the rows that a load phase touches on different banks.  The exponents
// of a block are two numbers for the whole MMA: K's scales the scores, V's is
// added to them in base 2, so that the weight carries it and the sum divides
// it out again.  A weight enters the product in f16, times 2^15: 11 bits (22
// in two terms for fp32), and nothing below 2^-40 of the largest weight times
// 2^exponent.
//
// Bound by HBM: 2 d bytes a row.  Unpacking costs one conversion per two
// codes; scoring on the SIMT lanes would cost four instructions per two
// codes and query, past the row stream's pace at two queries already.
#include <type_traits>

#include "fg_paged.cuh"

namespace fg {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxR = 8;
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

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

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
__device__ __forceinline__ int lds4(uint32_t p) {
  int v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(p) : "memory");
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

// The ring: per stage a block's K and V codes, its rows' positions and its
// exponents.  Row r's 16-byte piece c sits at piece c ^ swizzle(r).  A load
// phase (8 lanes of 16 bytes, 16 of 8) of the K fragments touches all pieces
// of one half (d = 128) or all pieces (d = 64) of two rows, one of the V
// fragments two adjacent pieces of four rows; slot_key orders the 8 keys of a
// tile so that these fall on different banks.
template <int D>
struct Ring {
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr int kV = kBlockRows * D, kPos = 2 * kV, kMeta = kPos + kBlockRows * 4;
  static constexpr int kStride = kMeta + 64;  // a multiple of 128
  static constexpr int kWarpBytes = kStages * kStride;
  __device__ static int swizzle(int r) { return D == 128 ? r & 7 : r & 2; }
  __device__ static int slot_key(int n) {
    const int k = n >> 1;
    return D == 128 ? (n & 1 ? (n + 4) & 7 : n) : (n & 1 ? 4 + (k ^ 1) : k);
  }
};
static_assert(Ring<128>::kStride % 128 == 0 && Ring<64>::kStride % 128 == 0, "bank phase");

__device__ __forceinline__ uint32_t word4(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 4 : 3)
    q8_split_kernel(const PagedArgs a, const PagedDecodeArgs n, int H, int R, int HLkv, float sl2) {
  using RG = Ring<D>;
  constexpr bool kWide = sizeof(T) == 4;  // fp32: queries and weights in two f16 terms
  constexpr int KI = D / 64;   // 16-byte pieces of a K row per lane
  constexpr int PW = D / 32;   // words of a lane's V piece
  constexpr int MT = D / 16;   // 16-row tiles of O^T
  constexpr int PER = D / 32;
  extern __shared__ __align__(128) uint8_t ring_smem[];
  __shared__ float sm_m[kWarps][kMaxR], sm_l[kWarps][kMaxR], sm_f[kWarps][kMaxR];
  __shared__ float qs[kMaxR][D];
  __shared__ int sm_page;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t4 = lane & 3;
  const int2 it = a.work[blockIdx.x];
  const int c = it.x;
  const int b = c / HLkv;
  const fg_paged_desc hd = a.caches[c];
  const int2 range = a.ranges[c];
  const int rpw = a.rpw;
  const int nsc = range.y - cdiv(max(hd.w, 0), rpw);  // items of the never-evicted segment
  const bool ring = it.y >= nsc;
  const int r0 = (ring ? it.y - nsc : it.y) * rpw;
  const int first = ring ? hd.ring_page : hd.first_page;
  const int entries = ring ? hd.ring_pages : hd.max_pages;
  griddep_wait();
  griddep_launch_dependents();
  const int t = n.pos[b];
  const int had = a.rows[c];
  // pages of the item, 32 at a time: lane l holds page l
  int page_l = page_at(a, first, entries, r0 / kPageRows + lane);
  if (t < 0) return;

  // rows of the item, and the new token's place
  const int old = (int)max(0LL, min((long long)had, (long long)hd.max_pages * kPageRows));
  if (old != had && it.y == 0 && threadIdx.x == 0) atomicOr(a.dev_err, kErrInvalid);
  int r1, put = -1;  // put: row (or slot) of the new token if this item holds it
  if (!ring) {
    r1 = it.y == nsc - 1 ? old : min(r0 + rpw, old);
    if (min(old / rpw, nsc - 1) == it.y) put = old;
  } else {
    r1 = min(r0 + rpw, hd.w);
    const int slot = t % hd.w;
    if (hd.policy == FG_POLICY_SPFL && slot >= r0 && slot < r1) put = slot;
  }
  if (n.k_new && put >= 0) {
    const int tau = n.ids[b];
    const bool s = warp_id_in(tau, n.special, n.ns);
    const bool sp = s || warp_id_in(tau, n.punct, n.np);
    if (joins_static(hd.policy, s, sp) == ring) put = -1;
  } else {
    put = -1;
  }
  if (put >= 0) {  // uniform over the CTA
    if (threadIdx.x == 0) {
      const int i = put / kPageRows;
      int page = page_at(a, first, entries, i);
      if (page < 0) {
        int err = kErrInvalid;
        if (!ring && i >= entries) {
          err = kErrCapacity;
        } else if (!ring && first >= 0 && first <= a.table_len - 1 - i && a.table[first + i] < 0) {
          page = atomicAdd(a.next_page, 1);
          if (page >= 0 && page < a.n_pages) {
            a.table[first + i] = page;
          } else {
            page = -1;
            err = kErrCapacity;
          }
        }
        if (page < 0) atomicOr(a.dev_err, err);
      }
      sm_page = page;
    }
    __syncthreads();
    const int page = sm_page;
    if (page >= 0) {
      if (warp < 2) {
        float x[1][PER];
        load_row<PER>((const T*)(warp ? n.v_new : n.k_new) + (size_t)c * D, x[0]);
        if (warp == 0 && n.rope.rot > 0) {
          float2 cs[PER];
          row_angles<PER>(cs, n.rope.rot, n.rope.style, [&](int p) {
            float2 y;
            rope_cos_sin((unsigned)t, n.rope.turns[p], y.x, y.y);
            return y;
          });
          rotate_row<PER>(x[0], cs, n.rope.rot, n.rope.style);
        }
        const int r = put % kPageRows, blk = r / kBlockRows;
        put_rows<D, 1>(x, 1u, r % kBlockRows, !ring && r % kBlockRows == 0,
                       (warp ? a.vp : a.kp) + ((size_t)page * kPageRows + blk * kBlockRows) * D,
                       a.exps + ((size_t)page * kPageBlocks + blk) * 2 + warp);
        if (warp == 0 && lane == 0) a.pos[(size_t)page * kPageRows + r] = t;
      }
      if (!ring) r1 = put + 1;
    }
    __syncthreads();  // the row, its exponents and its position are visible to the CTA
    page_l = page_at(a, first, entries, r0 / kPageRows + lane);
  }

  // this warp's blocks: warp, warp + 4, ... of the item, i.e. block `warp` of each page
  static_assert(kPageBlocks == kWarps, "a warp takes one block of every page");
  const int blocks = r1 > r0 ? cdiv(r1 - r0, kBlockRows) : 0;
  const int mine = blocks > warp ? cdiv(blocks - warp, kWarps) : 0;
  const uint32_t stages =
      (uint32_t)__cvta_generic_to_shared(ring_smem) + (uint32_t)(warp * RG::kWarpBytes);
  uint32_t exp_l = 0;
  auto fetch = [&](int group) {  // pages group * 32 + lane of the item, and their exponents
    const int i = r0 / kPageRows + group * 32 + lane;
    const bool in = i * kPageRows < r1;
    if (group > 0) page_l = page_at(a, first, entries, i);
    if (!in) page_l = -1;
    else if (page_l < 0) atomicOr(a.dev_err, kErrInvalid);
    if (page_l >= 0)
      exp_l = *reinterpret_cast<const volatile unsigned short*>(
          a.exps + ((size_t)page_l * kPageBlocks + warp) * 2);
  };
  constexpr int kNoPage = 1 << 30;
  auto issue = [&](int j) {
    if ((j & 31) == 0) fetch(j >> 5);
    const int pg = __shfl_sync(0xffffffffu, page_l, j & 31);
    const int ex = (int)__shfl_sync(0xffffffffu, exp_l, j & 31);
    const uint32_t st = stages + (uint32_t)((j % RG::kStages) * RG::kStride);
    if (lane == 0)
      asm volatile("st.shared.u32 [%0], %1;" ::"r"(st + RG::kMeta), "r"(pg < 0 ? kNoPage : ex)
                   : "memory");
    if (pg >= 0) {
      const size_t row = (size_t)pg * kPageRows + warp * kBlockRows;
      const uint8_t* kb = a.kp + row * D + lane * 16;
      const uint8_t* vb = a.vp + row * D + lane * 16;
      constexpr int CPR = D / 16;  // pieces per row
#pragma unroll
      for (int i = 0; i < kBlockRows * CPR / 32; ++i) {
        const int r = i * (32 / CPR) + lane / CPR;
        const uint32_t dst = st + (uint32_t)(r * D + (((lane % CPR) ^ RG::swizzle(r)) << 4));
        cp_async16(dst, kb + i * 512);
        cp_async16(dst + RG::kV, vb + i * 512);
      }
      if (ring && lane < 4) cp_async16(st + RG::kPos + lane * 16, a.pos + row + lane * 4);
    }
  };
#pragma unroll
  for (int j = 0; j < RG::kStages - 1; ++j) {
    if (j < mine) issue(j);
    cp_async_commit();
  }

  // the group's queries, rotated, in shared memory
  {
    const int Hkv = H / R;
    const size_t g0 = (size_t)(c / Hkv) * H + (size_t)(c % Hkv) * R;
    float2 cs[PER];
    if (n.rope.rot > 0 && warp < R)
      row_angles<PER>(cs, n.rope.rot, n.rope.style, [&](int p) {
        float2 y;
        rope_cos_sin((unsigned)t, n.rope.turns[p], y.x, y.y);
        return y;
      });
    for (int qi = warp; qi < R; qi += kWarps) {
      float x[PER];
      load_row<PER>((const T*)n.q + (g0 + qi) * D, x);
      if (n.rope.rot > 0) rotate_row<PER>(x, cs, n.rope.rot, n.rope.style);
      uint32_t top = 0;
#pragma unroll
      for (int k = 0; k < PER; ++k) {
        qs[qi][lane * PER + k] = x[k];
        top = max(top, finite_bits(x[k]));
      }
      top = __reduce_max_sync(0xffffffffu, top);
      // the exponent that brings the largest value to [2^13, 2^14)
      if (lane == 0) sm_m[0][qi] = (float)max(-110, (int)(top >> 23) - 127 - 13);
    }
  }
  __syncthreads();
  // operand fragments: k-step 4 i + w takes dimensions 64 i + 16 t4 + 4 w + 0..3
  uint32_t qa[4 * KI][kWide ? 4 : 2];
  int eq = 0;
  if (g < R) {
    eq = (int)sm_m[0][g];
    const float inv = pow2f(-eq);
#pragma unroll
    for (int i = 0; i < KI; ++i)
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        float x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = qs[g][64 * i + 16 * t4 + 4 * w + k] * inv;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t hi = pack_f16x2(x[2 * k], x[2 * k + 1]);
          qa[4 * i + w][k] = hi;
          if constexpr (kWide) {  // what is left, times 2^11
            const float2 f = unpack_f16x2(hi);
            qa[4 * i + w][2 + k] =
                pack_f16x2((x[2 * k] - f.x) * 2048.f, (x[2 * k + 1] - f.y) * 2048.f);
          }
        }
      }
  } else {
#pragma unroll
    for (int i = 0; i < 4 * KI; ++i)
#pragma unroll
      for (int k = 0; k < (kWide ? 4 : 2); ++k) qa[i][k] = 0;
  }

  // this lane's rows of a block and their places in a stage: key kr (and + 8) for the scores,
  // keys va, vb (and + 8) for the values and the weights
  const int kr = RG::slot_key(g), va = RG::slot_key(2 * t4), vb = RG::slot_key(2 * t4 + 1);
  uint32_t k_off[KI];
#pragma unroll
  for (int i = 0; i < KI; ++i)
    k_off[i] = (uint32_t)(kr * D + (((t4 + 4 * i) ^ RG::swizzle(kr)) << 4));
  const int vp = D == 128 ? g : g >> 1, vo = D == 128 ? 0 : (g & 1) * 8;
  const uint32_t va_off = (uint32_t)(RG::kV + va * D + ((vp ^ RG::swizzle(va)) << 4) + vo);
  const uint32_t vb_off = (uint32_t)(RG::kV + vb * D + ((vp ^ RG::swizzle(vb)) << 4) + vo);

  // lanes without a query keep a maximum that no score passes: weight 0
  float m = g < R ? FG_NEG_INF : 1e30f, l = 0.f;
  float o[MT][4];
#pragma unroll
  for (int j = 0; j < MT; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;

#pragma unroll 1
  for (int j = 0; j < mine; ++j) {
    cp_async_wait<RG::kStages - 2>();
    __syncwarp();  // the stage has landed for every lane; the one before it is free
    if (j + RG::kStages - 1 < mine) issue(j + RG::kStages - 1);
    cp_async_commit();
    const uint32_t st = stages + (uint32_t)((j % RG::kStages) * RG::kStride);
    const int meta = lds4(st + RG::kMeta);
    const int ek = (int)(signed char)(meta & 0xff), ev = (int)(signed char)((meta >> 8) & 0xff);
    float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < KI; ++i) {
      const uint4 k0 = lds16(st + k_off[i]), k1 = lds16(st + k_off[i] + 8 * D);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t x = word4(k0, w), y = word4(k1, w);
        const uint32_t(&q)[kWide ? 4 : 2] = qa[4 * i + w];
        const uint32_t q2 = kWide ? q[kWide ? 2 : 0] : 0u, q3 = kWide ? q[kWide ? 3 : 0] : 0u;
        mma_f16_16816(s0, q[0], q2, q[1], q3, decode2(x), decode2(x >> 16));
        mma_f16_16816(s1, q[0], q2, q[1], q3, decode2(y), decode2(y >> 16));
      }
    }
    Piece<D> v[4];  // keys va, vb, va + 8, vb + 8
    v[0].load(st + va_off);
    v[1].load(st + vb_off);
    v[2].load(st + va_off + 8 * D);
    v[3].load(st + vb_off + 8 * D);
    // scores in base 2, V's exponent added: those keys and query g
    const int e = max(-126, min(127, ek + eq));
    const float kf = pow2f(e) * sl2, fv = (float)ev;
    float x[4] = {s0[0], s0[1], s1[0], s1[1]};
    if constexpr (kWide) {
      x[0] += s0[2] * (1.f / 2048.f);
      x[1] += s0[3] * (1.f / 2048.f);
      x[2] += s1[2] * (1.f / 2048.f);
      x[3] += s1[3] * (1.f / 2048.f);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = fmaf(x[i], kf, fv);
    const int row = r0 + (warp + j * kWarps) * kBlockRows;
    if (ring || row + kBlockRows > r1 || meta == kNoPage) {  // uniform: rows may be missing
      const unsigned w = (unsigned)hd.w;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = (i & 1 ? vb : va) + (i & 2 ? 8 : 0);
        bool ok = row + key < r1 && meta != kNoPage;
        if (ring) {  // in the window: position in (t - w, t]
          const int p = lds4(st + RG::kPos + key * 4);
          ok = ok && p >= 0 && (unsigned)t - (unsigned)p < w;
        }
        if (!ok) {
          x[i] = FG_NEG_INF;
          v[i].zero();  // such a row may hold anything, also NaN
        }
      }
    }
    float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    if (__any_sync(0xffffffffu, top > m)) {
      const float mn = fmaxf(m, top);
      const float corr = m == FG_NEG_INF ? 0.f : ex2(m - mn);
      m = mn;
      l *= corr;
      const float c0 = __shfl_sync(0xffffffffu, corr, 8 * t4);
      const float c1 = __shfl_sync(0xffffffffu, corr, 8 * t4 + 4);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        o[i][0] *= c0;
        o[i][1] *= c1;
        o[i][2] *= c0;
        o[i][3] *= c1;
      }
    }
    const float base = (m == FG_NEG_INF ? 0.f : m) - kPBits;
    float p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = ex2(x[i] - base);
    const uint32_t p01 = pack_f16x2(p[0], p[1]), p23 = pack_f16x2(p[2], p[3]);
    // the sum takes the weights in 32 bits: f16 would lose those that a small
    // exponent of V makes small
    l = fmaf((p[0] + p[1]) + (p[2] + p[3]), pow2f(-ev), l);
    uint32_t r01 = 0, r23 = 0;
    if constexpr (kWide) {
      const float2 f01 = unpack_f16x2(p01), f23 = unpack_f16x2(p23);
      r01 = pack_f16x2(p[0] - f01.x, p[1] - f01.y);
      r23 = pack_f16x2(p[2] - f23.x, p[3] - f23.y);
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
  cp_async_wait<0>();
  l += __shfl_xor_sync(0xffffffffu, l, 1);
  l += __shfl_xor_sync(0xffffffffu, l, 2);

  // O^T: rows 16 j + g, + 8 are dimensions (D / 8) g + 2 j, + 1; columns queries 2 t4, 2 t4 + 1
  __syncthreads();  // every warp is done with its ring: the warps' sums take its place
  float* sums = reinterpret_cast<float*>(ring_smem);  // [kWarps][R][D]
  static_assert(kWarps * kMaxR * D * 4 <= kWarps * RG::kWarpBytes, "the sums fit the rings");
  if (t4 == 0 && g < R) {
    sm_m[warp][g] = m;
    sm_l[warp][g] = l;
  }
#pragma unroll
  for (int qc = 0; qc < 2; ++qc) {
    const int qi = 2 * t4 + qc;
    if (qi < R) {
#pragma unroll
      for (int j = 0; j < MT; ++j)
        *reinterpret_cast<float2*>(&sums[(warp * R + qi) * D + (D / 8) * g + 2 * j]) =
            make_float2(o[j][qc], o[j][qc + 2]);
    }
  }
  __syncthreads();
  if (threadIdx.x < R) {
    const int qi = threadIdx.x;
    float M = FG_NEG_INF;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm_m[w][qi]);
    float L = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = sm_m[w][qi] == FG_NEG_INF ? 0.f : exp2f(sm_m[w][qi] - M);
      sm_f[w][qi] = f;
      L += sm_l[w][qi] * f;
    }
    const size_t slot = (size_t)blockIdx.x * R + qi;
    n.part_ml[2 * slot] = M;
    n.part_ml[2 * slot + 1] = L;
  }
  __syncthreads();
  for (int x = threadIdx.x; x < R * D; x += kThreads) {
    const int qi = x / D, dd = x % D;
    float A = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) A = fmaf(sm_f[w][qi], sums[(w * R + qi) * D + dd], A);
    n.part_acc[((size_t)blockIdx.x * R + qi) * D + dd] = A;
  }
}

// One CTA of D threads per query head: merges its items and writes the output;
// one member of a group also writes the cache's new row count.
template <typename T, int D>
__global__ void __launch_bounds__(D) q8_combine_kernel(const PagedArgs a, const PagedDecodeArgs n,
                                                       int H, int R, int HLkv) {
  const int gq = blockIdx.x, t = threadIdx.x;
  const int c = kv_head(gq, H, R), qi = (gq % H) % R;
  const int b = c / HLkv;
  const fg_paged_desc hd = a.caches[c];
  const int2 range = a.ranges[c];
  griddep_wait();
  griddep_launch_dependents();
  const bool bump = t == 0 && qi == 0;
  if (n.pos[b] < 0) {
    if (bump) a.rows_out[c] = a.rows[c];
    return;
  }
  bool stored = false;  // the new token belongs to the never-evicted segment
  if (n.k_new && qi == 0 && t < 32) {
    const int tau = n.ids[b];
    const bool s = warp_id_in(tau, n.special, n.ns);
    const bool sp = s || warp_id_in(tau, n.punct, n.np);
    stored = joins_static(hd.policy, s, sp);
  }
  float M = FG_NEG_INF, L = 0.f, acc = 0.f;
  for (int i0 = 0; i0 < range.y; i0 += 8) {
    float m[8], l[8], x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const bool ok = i0 + j < range.y;
      const size_t slot = ((size_t)range.x + i0 + j) * R + qi;
      m[j] = ok ? n.part_ml[2 * slot] : FG_NEG_INF;
      l[j] = ok ? n.part_ml[2 * slot + 1] : 0.f;
      x[j] = ok ? n.part_acc[slot * D + t] : 0.f;
    }
    float mc = m[0];
#pragma unroll
    for (int j = 1; j < 8; ++j) mc = fmaxf(mc, m[j]);
    const float Mn = fmaxf(M, mc);
    const float f = M == FG_NEG_INF ? 0.f : exp2f(M - Mn);
    L *= f;
    acc *= f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      // an item without rows, or one whose scores are all NaN, has maximum -inf: its sums count
      // as they are (0, or NaN)
      const float wgt = m[j] == FG_NEG_INF ? 1.f : exp2f(m[j] - Mn);
      L = fmaf(wgt, l[j], L);
      acc = fmaf(wgt, x[j], acc);
    }
    M = Mn;
  }
  store_out((T*)n.out + (size_t)gq * D + t, L == 0.f ? 0.f : acc / L);
  if (bump) {
    const int had = a.rows[c];
    const bool put =
        stored && had >= 0 && page_at(a, hd.first_page, hd.max_pages, had / kPageRows) >= 0;
    a.rows_out[c] = had + (put ? 1 : 0);
  }
}

template <typename T, int D>
cudaError_t run_decode_q8(const ProfileDims& pd, const PagedArgs& a, const PagedDecodeArgs& n,
                          cudaStream_t s) {
  constexpr int smem = kWarps * Ring<D>::kWarpBytes;
  cudaError_t e = cudaFuncSetAttribute(q8_split_kernel<T, D>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess)
    e = launch_pdl(q8_split_kernel<T, D>, a.n_work, kThreads, smem, s, a, n, pd.H, pd.R, pd.HLkv,
                   pd.sl2);
  if (e == cudaSuccess)
    e = launch_pdl(q8_combine_kernel<T, D>, pd.G, D, 0, s, a, n, pd.H, pd.R, pd.HLkv);
  return e;
}

}  // namespace

cudaError_t launch_decode_q8(const ProfileDims& pd, const PagedArgs& a, const PagedDecodeArgs& n,
                             cudaStream_t s) {
  if (pd.dtype == FG_FP32)
    return pd.d == 64 ? run_decode_q8<float, 64>(pd, a, n, s)
                      : run_decode_q8<float, 128>(pd, a, n, s);
  return pd.d == 64 ? run_decode_q8<__nv_bfloat16, 64>(pd, a, n, s)
                    : run_decode_q8<__nv_bfloat16, 128>(pd, a, n, s);
}

}  // namespace fg
