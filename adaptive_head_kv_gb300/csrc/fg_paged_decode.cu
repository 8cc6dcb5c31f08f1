// One generation step over paged 8-bit caches (Model Tells You What to
// Discard, Method: head-specific caches, the prompt-time policy reused).
//
// Split-K over the work list: an item is up to rpw rows of one cache's
// never-evicted segment (the last one also every row appended later) or of
// its ring.  A CTA of 4 warps takes an item, warp v its blocks of 16 rows v,
// v + 4, ...; the CTA whose item holds the new token's row codes it into the
// page first.  A block's K and V codes go from HBM to registers in 16-byte
// pieces, each read once, and both products run as warp MMAs in f16, which
// holds every e4m3 code exactly:
//   S[16 x 16 keys] = Q[16 x d] . K^T    queries in rows 0-7; rows 8-15 hold
//                                        what f16 loses of fp32 queries
//   O^T[d x 8]     += V^T[d x 16 keys] . P^T
// The dimension order inside a product is free as long as both operands agree,
// so every lane's operand fragments are consecutive bytes of a row and
// nothing passes through shared memory; S's accumulators are P^T's operand
// fragment as they stand.  The exponents of a block are two numbers for the
// whole MMA: K's scales the scores, V's is added to them in base 2, so that
// the weight carries it and the sum divides it out again.  A weight enters the
// product in f16, times 2^15: 11 bits (22 in two terms for fp32), and nothing
// below 2^-40 of the largest weight times 2^exponent.
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

__device__ __forceinline__ uint2 ld8(const void* p) {
  uint2 v;
  asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];"
               : "=r"(v.x), "=r"(v.y)
               : "l"(p)
               : "memory");
  return v;
}

template <int D>
struct Piece;  // a lane's D / 8 codes of a V row
template <>
struct Piece<128> {
  uint4 v;
  __device__ void load(const uint8_t* p) { v = ld16(p); }
  __device__ void zero() { v = make_uint4(0, 0, 0, 0); }
  __device__ uint32_t word(int i) const { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
};
template <>
struct Piece<64> {
  uint2 v;
  __device__ void load(const uint8_t* p) { v = ld8(p); }
  __device__ void zero() { v = make_uint2(0, 0); }
  __device__ uint32_t word(int i) const { return i == 0 ? v.x : v.y; }
};

__device__ __forceinline__ uint32_t word4(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 4 : 3)
    q8_split_kernel(const PagedArgs a, const PagedDecodeArgs n, int H, int R, int HLkv, float sl2) {
  constexpr bool kWide = sizeof(T) == 4;  // fp32: queries and weights in two f16 terms
  constexpr int KI = D / 64;   // 16-byte pieces of a K row per lane
  constexpr int PW = D / 32;   // words of a lane's V piece
  constexpr int MT = D / 16;   // 16-row tiles of O^T
  constexpr int PER = D / 32;
  __shared__ float sm_m[kWarps][kMaxR], sm_l[kWarps][kMaxR], sm_f[kWarps][kMaxR];
  __shared__ float sm_acc[kWarps][kMaxR][D];  // first the rotated queries, then the warps' sums
  __shared__ int sm_put;

  const int2 it = a.work[blockIdx.x];
  const int c = it.x;
  const int b = c / HLkv;
  const fg_paged_desc hd = a.caches[c];
  const int2 range = a.ranges[c];
  griddep_wait();
  griddep_launch_dependents();
  const int t = n.pos[b];
  if (t < 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t4 = lane & 3;
  const int rpw = a.rpw;
  const int nsc = range.y - cdiv(max(hd.w, 0), rpw);  // items of the never-evicted segment
  const bool ring = it.y >= nsc;

  // rows of the item, and the new token's place
  const int had = a.rows[c];
  const int old = (int)max(0LL, min((long long)had, (long long)hd.max_pages * kPageRows));
  if (old != had && it.y == 0 && threadIdx.x == 0) atomicOr(a.dev_err, kErrInvalid);
  int put = -1;  // row (or slot) of the new token if this item holds it
  int r0, r1, first, entries;
  bool is_static = false;
  if (n.k_new) {
    const int tau = n.ids[b];
    const bool s = id_in(tau, n.special, n.ns);
    is_static = joins_static(hd.policy, s, s || id_in(tau, n.punct, n.np));
  }
  if (!ring) {
    r0 = it.y * rpw;
    const bool last = it.y == nsc - 1;
    r1 = last ? old : min(r0 + rpw, old);
    first = hd.first_page;
    entries = hd.max_pages;
    if (is_static && min(old / rpw, nsc - 1) == it.y) put = old;
  } else {
    r0 = (it.y - nsc) * rpw;
    r1 = min(r0 + rpw, hd.w);
    first = hd.ring_page;
    entries = hd.ring_pages;
    if (n.k_new && !is_static && hd.policy == FG_POLICY_SPFL) {
      const int slot = t % hd.w;
      if (slot >= r0 && slot < r1) put = slot;
    }
  }
  if (put >= 0) {  // uniform over the CTA
    if (threadIdx.x == 0) {
      int page = page_at(a, first, entries, put / kPageRows);
      if (page < 0) {
        const int i = put / kPageRows;
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
      sm_put = page;
    }
    __syncthreads();
    const int page = sm_put;
    if (page >= 0) {
      if (warp < 2) {
        float x[1][PER];
        load_row<PER>((const T*)(warp ? n.v_new : n.k_new) + (size_t)c * D, x[0]);
        if (warp == 0 && n.rope.rot > 0)
          rotate_row<PER>(x[0], n.rope.rot, n.rope.style, [&](int p) {
            float2 cs;
            rope_cos_sin((unsigned)t, n.rope.turns[p], cs.x, cs.y);
            return cs;
          });
        const int r = put % kPageRows, blk = r / kBlockRows;
        put_rows<D, 1>(x, 1u, r % kBlockRows, !ring && r % kBlockRows == 0,
                       (warp ? a.vp : a.kp) + ((size_t)page * kPageRows + blk * kBlockRows) * D,
                       a.exps + ((size_t)page * kPageBlocks + blk) * 2 + warp);
        if (warp == 0 && lane == 0) a.pos[(size_t)page * kPageRows + r] = t;
      }
      if (!ring) r1 = put + 1;
    }
    __syncthreads();  // the row, its exponents and its position are visible to the CTA
  }

  // the group's queries, rotated, in shared memory
  float(*qs)[D] = sm_acc[0];
  {
    const int Hkv = H / R;
    const size_t g0 = (size_t)(c / Hkv) * H + (size_t)(c % Hkv) * R;
    for (int qi = warp; qi < R; qi += kWarps) {
      float x[PER];
      load_row<PER>((const T*)n.q + (g0 + qi) * D, x);
      if (n.rope.rot > 0)
        rotate_row<PER>(x, n.rope.rot, n.rope.style, [&](int p) {
          float2 cs;
          rope_cos_sin((unsigned)t, n.rope.turns[p], cs.x, cs.y);
          return cs;
        });
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
  __syncthreads();  // the queries' place becomes the warps' sums

  // pages of the item: lane l holds page l (of 32 at a time) and its exponents
  int page_l = -1;
  uint2 exp_l = make_uint2(0, 0);
  auto fetch_pages = [&](int group) {
    const int i = r0 / kPageRows + group * 32 + lane;
    const bool in = i * kPageRows < r1;
    page_l = in ? page_at(a, first, entries, i) : -1;
    if (in && page_l < 0) atomicOr(a.dev_err, kErrInvalid);
    if (page_l >= 0)
      exp_l = ld8(a.exps + (size_t)page_l * kPageBlocks * 2);
  };

  uint4 k0[KI], k1[KI];  // keys g and g + 8 of the block
  Piece<D> v[4];         // keys 2 t4, 2 t4 + 1, 2 t4 + 8, 2 t4 + 9
  int4 kp;               // their positions (ring)
  int page = -1, page_next = -1, ek = 0, ev = 0, ek_next = 0, ev_next = 0;
  const int blocks = r1 > r0 ? cdiv(r1 - r0, kBlockRows) : 0;
  // page and exponents of block `blk` of the item (all lanes call)
  auto look = [&](int blk, int& pg, int& e_k, int& e_v) {
    const int i = blk / kPageBlocks;
    if ((i & 31) == 0 && blk % kPageBlocks == warp) fetch_pages(i >> 5);
    pg = __shfl_sync(0xffffffffu, page_l, i & 31);
    const uint32_t lo = __shfl_sync(0xffffffffu, exp_l.x, i & 31);
    const uint32_t hi = __shfl_sync(0xffffffffu, exp_l.y, i & 31);
    const uint32_t w = (blk & 2 ? hi : lo) >> (blk & 1 ? 16 : 0);
    e_k = (int)(signed char)(w & 0xff);
    e_v = (int)(signed char)((w >> 8) & 0xff);
  };
  auto load_k = [&](int blk, int pg) {
    if (pg < 0) return;
    const uint8_t* p = a.kp + ((size_t)pg * kPageRows + (blk % kPageBlocks) * kBlockRows) * D;
#pragma unroll
    for (int i = 0; i < KI; ++i) {
      k0[i] = ld16(p + g * D + 64 * i + 16 * t4);
      k1[i] = ld16(p + (g + 8) * D + 64 * i + 16 * t4);
    }
  };
  auto load_v = [&](int blk, int pg) {
    if (pg < 0) return;
    const size_t row = (size_t)pg * kPageRows + (blk % kPageBlocks) * kBlockRows;
    const uint8_t* p = a.vp + row * D + g * (D / 8);
    v[0].load(p + (2 * t4) * D);
    v[1].load(p + (2 * t4 + 1) * D);
    v[2].load(p + (2 * t4 + 8) * D);
    v[3].load(p + (2 * t4 + 9) * D);
    if (ring) {
      const uint2 x = ld8(a.pos + row + 2 * t4), y = ld8(a.pos + row + 2 * t4 + 8);
      kp = make_int4((int)x.x, (int)x.y, (int)y.x, (int)y.y);
    }
  };

  // lanes without a query keep a maximum that no score passes: weight 0
  float m = g < R ? FG_NEG_INF : 1e30f, l = 0.f;
  float o[MT][4];
#pragma unroll
  for (int j = 0; j < MT; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
#pragma unroll
  for (int i = 0; i < KI; ++i) k0[i] = k1[i] = make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i].zero();
  kp = make_int4(-1, -1, -1, -1);

  if (warp < blocks) {
    look(warp, page, ek, ev);
    load_k(warp, page);
    load_v(warp, page);
  }
#pragma unroll 1
  for (int blk = warp; blk < blocks; blk += kWarps) {
    const int nxt = blk + kWarps;
    if (nxt < blocks) look(nxt, page_next, ek_next, ev_next);
    float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < KI; ++i)
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t x = word4(k0[i], w), y = word4(k1[i], w);
        const uint32_t(&q)[kWide ? 4 : 2] = qa[4 * i + w];
        const uint32_t q2 = kWide ? q[kWide ? 2 : 0] : 0u, q3 = kWide ? q[kWide ? 3 : 0] : 0u;
        mma_f16_16816(s0, q[0], q2, q[1], q3, decode2(x), decode2(x >> 16));
        mma_f16_16816(s1, q[0], q2, q[1], q3, decode2(y), decode2(y >> 16));
      }
    if (nxt < blocks) load_k(nxt, page_next);  // the K registers are free now
    // scores in base 2, V's exponent added: keys 2 t4, 2 t4 + 1, + 8, + 9 of query g
    const int e = max(-126, min(127, ek + eq));
    const float kf = pow2f(e) * sl2, fv = (float)ev;
    float x[4] = {s0[0], s0[1], s1[0], s1[1]};
    if constexpr (kWide) {
      x[0] += s0[2] * (1.f / 2048.f);
      x[1] += s0[3] * (1.f / 2048.f);
      x[2] += s1[2] * (1.f / 2048.f);
      x[3] += s1[3] * (1.f / 2048.f);
    }
    const int row = r0 + blk * kBlockRows + 2 * t4;
    bool ok[4];
    ok[0] = row < r1;
    ok[1] = row + 1 < r1;
    ok[2] = row + 8 < r1;
    ok[3] = row + 9 < r1;
    if (ring) {  // in the window: position in (t - w, t]
      const unsigned w = (unsigned)hd.w;
      ok[0] = ok[0] && kp.x >= 0 && (unsigned)t - (unsigned)kp.x < w;
      ok[1] = ok[1] && kp.y >= 0 && (unsigned)t - (unsigned)kp.y < w;
      ok[2] = ok[2] && kp.z >= 0 && (unsigned)t - (unsigned)kp.z < w;
      ok[3] = ok[3] && kp.w >= 0 && (unsigned)t - (unsigned)kp.w < w;
    }
    if (page < 0) ok[0] = ok[1] = ok[2] = ok[3] = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = ok[i] ? fmaf(x[i], kf, fv) : FG_NEG_INF;
      if (!ok[i]) v[i].zero();  // such a row may hold anything, also NaN
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
      for (int j = 0; j < MT; ++j) {
        o[j][0] *= c0;
        o[j][1] *= c1;
        o[j][2] *= c0;
        o[j][3] *= c1;
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
    if (nxt < blocks) load_v(nxt, page_next);
    page = page_next;
    ek = ek_next;
    ev = ev_next;
  }
  l += __shfl_xor_sync(0xffffffffu, l, 1);
  l += __shfl_xor_sync(0xffffffffu, l, 2);

  // O^T: rows 16 j + g, + 8 are dimensions (D / 8) g + 2 j, + 1; columns queries 2 t4, 2 t4 + 1
  if (t4 == 0 && g < R) {
    sm_m[warp][g] = m;
    sm_l[warp][g] = l;
  }
#pragma unroll
  for (int qc = 0; qc < 2; ++qc) {
    const int qi = 2 * t4 + qc;
    if (qi < R) {
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        sm_acc[warp][qi][(D / 8) * g + 2 * j] = o[j][qc];
        sm_acc[warp][qi][(D / 8) * g + 2 * j + 1] = o[j][qc + 2];
      }
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
    for (int w = 0; w < kWarps; ++w) A = fmaf(sm_f[w][qi], sm_acc[w][qi][dd], A);
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
    int put = 0;
    if (n.k_new) {
      const int tau = n.ids[b];
      const bool s = id_in(tau, n.special, n.ns);
      if (joins_static(hd.policy, s, s || id_in(tau, n.punct, n.np)) && had >= 0)
        put = page_at(a, hd.first_page, hd.max_pages, had / kPageRows) >= 0;
    }
    a.rows_out[c] = had + put;
  }
}

template <typename T, int D>
cudaError_t run_decode_q8(const ProfileDims& pd, const PagedArgs& a, const PagedDecodeArgs& n,
                          cudaStream_t s) {
  cudaError_t e = launch_pdl(q8_split_kernel<T, D>, a.n_work, kThreads, 0, s, a, n, pd.H, pd.R,
                             pd.HLkv, pd.sl2);
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
