// Paged 8-bit caches: the layout, the e4m3 coding of rows and the position
// rotation, shared by the kernels that fill, extend and read them.
//
// A page holds kPageRows rows of one cache; every kBlockRows rows share one
// power-of-two exponent for K and one for V, so that a row's value is
// code * 2^exponent.  Powers of two make the coding exact to reproduce (the
// scaling itself never rounds) and let a block's exponent grow when a larger
// row arrives: e4m3 keeps its fraction bits, only codes that fall among the
// subnormals are rounded again (an error of 2^-10 in units of the new exponent,
// 2^-17.8 of the block's largest value at most, each time it grows).
#pragma once

#include "fg_common.cuh"
#include "fg_internal.h"

namespace fg {

constexpr int kPageRows = FG_PAGE_ROWS;
constexpr int kBlockRows = FG_BLOCK_ROWS;
constexpr int kPageBlocks = kPageRows / kBlockRows;
// Pages of a decode work item when each item has a thread block of its own.
constexpr int kItemPages = 4;
constexpr int kExpMin = -100;  // exponent of a block without finite non-zero values

// Bits of |x| as an unsigned integer, 0 for infinities and NaN: the order of
// finite magnitudes is the order of these integers.
__device__ __forceinline__ uint32_t finite_bits(float x) {
  const uint32_t b = __float_as_uint(x) & 0x7fffffffu;
  return b < 0x7f800000u ? b : 0u;
}

// Least e >= kExpMin with amax <= 448 * 2^e (448 = 1.75 * 2^8, the largest
// e4m3 value), from the bits of amax.
__device__ __forceinline__ int block_exponent(uint32_t amax_bits) {
  const int e = (int)(amax_bits >> 23) - 127 - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(e, kExpMin);
}

// 2^e for a normal result (-126 <= e <= 127).
__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }

// e4m3 codes of a (low byte) and b, nearest even; magnitudes past 448 and
// infinities become 448, NaN stays NaN.
__device__ __forceinline__ uint32_t code2(float a, float b) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ uint32_t code4(float a, float b, float c, float d) {
  return code2(a, b) | (code2(c, d) << 16);
}

// Two e4m3 codes (bits 0-15 of w) as f16x2; exact.
__device__ __forceinline__ uint32_t decode2(uint32_t w) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((unsigned short)w));
  return r;
}

// Four codes times the f16x2 factor f (two equal powers of two <= 1), rounded
// again.  The f16 product of a 4-bit fraction is exact above 2^-24, far below
// the code's last place, so only the final conversion rounds.
__device__ __forceinline__ uint32_t recode4(uint32_t w, uint32_t f) {
  uint32_t lo = decode2(w), hi = decode2(w >> 16);
  asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(lo) : "r"(f));
  asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(hi) : "r"(f));
  unsigned short a, b;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(a) : "r"(lo));
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(b) : "r"(hi));
  return (uint32_t)a | ((uint32_t)b << 16);
}

// f16x2 of 2^-k, k >= 1.  From k = 19 on every code (at most 448 = 2^8.8)
// falls below half of the smallest one (2^-10) and becomes zero, so larger k
// may stand for 24, the last one f16 holds.
__device__ __forceinline__ uint32_t half2_pow2_neg(int k) {
  k = min(k, 24);
  const uint32_t h = k <= 14 ? (uint32_t)(15 - k) << 10 : 1u << (24 - k);
  return h | (h << 16);
}

// cos and sin of 2 pi * pos * turns / 2^64.  The product keeps the fraction
// of the turn exactly (modulo one turn, at any position), so nothing of the
// angle is lost at far positions.  The fraction's top 32 bits, as a signed
// number of half turns in [-1, 1), do not fit a float: what its rounding leaves
// over (at most 2^-25 half turns) is added to first order (kFull), so that the
// result is off by little more than sincospif itself.  Without it an angle is
// off by up to 2^-23, enough where the rotated value is rounded to 11 bits.
template <bool kFull = true>
__device__ __forceinline__ void rope_cos_sin(uint32_t pos, unsigned long long turns, float& c,
                                             float& s) {
  const int frac = (int)((unsigned long long)pos * turns >> 32);
  const float most = (float)frac;
  sincospif(most * 4.656612873077393e-10f, &s, &c);
  if constexpr (kFull) {
    const float rest = (float)(frac - __float2int_rn(most)) * 1.46291808e-9f;  // pi 2^-31
    const float c0 = c;
    c = fmaf(-s, rest, c);
    s = fmaf(c0, rest, s);
  }
}

// Streaming 16-byte load of memory that the kernel also writes (not the
// read-only path).
__device__ __forceinline__ uint4 ld16(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

// Is `id` one of the `cnt` ids of `set`?  All lanes of a warp call with the
// same id: each looks at every 32nd entry.
__device__ __forceinline__ bool warp_id_in(int id, const int32_t* __restrict__ set, int cnt) {
  bool hit = false;
  for (int i = threadIdx.x & 31; i < cnt; i += 32) hit |= __ldg(set + i) == id;
  return __any_sync(0xffffffffu, hit);
}

// A small id set over the lanes of a warp, read ahead of its use: lane l holds
// entry l; entries past 32 are looked up when asked.
struct LaneSet {
  const int32_t* set;
  int cnt, id;
  __device__ __forceinline__ LaneSet(const int32_t* s, int n) : set(s), cnt(n) {
    const int lane = threadIdx.x & 31;
    id = lane < n ? __ldg(s + lane) : 0;
  }
  // Is this lane's x an entry?  All lanes of the warp call, so never behind a
  // condition that differs between them (nor the right side of || or &&).
  __device__ __forceinline__ bool has_mine(int x) const {
    bool hit = false;
    for (int i = 0; i < min(cnt, 32); ++i) hit |= __shfl_sync(0xffffffffu, id, i) == x;
    return hit || (cnt > 32 && id_in(x, set + 32, cnt - 32));
  }
  // Is x, the same in every lane, an entry?  All lanes call.
  __device__ __forceinline__ bool has(int x) const {
    const int lane = threadIdx.x & 31;
    if (__any_sync(0xffffffffu, lane < cnt && id == x)) return true;
    return cnt > 32 && warp_id_in(x, set + 32, cnt - 32);
  }
};

// 16-byte global -> shared copy in the background.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

struct RopeArgs {
  const unsigned long long* turns;  // [rot / 2]
  int rot;                          // 0: no rotation
  int style;                        // FG_ROPE_*
};

// A decode work item: pages [seg0, seg1) of a cache's never-evicted segment
// and [ring0, ring1) of its ring.  The item with `last` set also takes the
// segment's pages from seg1 on (rows appended after the schedule).
struct PagedItem {
  int cache, last, seg0, seg1, ring0, ring1;
};

struct PagedArgs {
  uint8_t* kp;
  uint8_t* vp;
  int8_t* exps;
  int32_t* pos;
  int32_t* table;
  const fg_paged_desc* caches;
  const int32_t* rows;
  int32_t* rows_out;
  int32_t* next_page;
  const int4* ranges;      // [Gkv] x, y: first work item and items of each cache
  const PagedItem* items;  // [n_work]
  const int32_t* cta_first;  // [n_ctas + 1] first item of each thread block
  const long long* totals;   // [3], [4]: the list's items and thread blocks
  int n_pages, table_len, n_work, n_ctas;
  int max_w;  // ring slots of the call's parameters
  int32_t* dev_err;
};

// Bits of dev_err.
constexpr int kErrCapacity = 1, kErrDevice = 2, kErrInvalid = 4;

// Slots of a cache's ring.  Of one that the parameters do not allow no row is
// read or written: it has none, and who sees d.w differ flags it.
__device__ __forceinline__ int ring_slots(const fg_paged_desc& d, int max_w) {
  return (unsigned)d.w <= (unsigned)max_w ? d.w : 0;
}

// Page of entry `i` of a segment with `entries` entries from `first`; -1 when
// the entry does not exist or holds no page of the pool.
__device__ __forceinline__ int page_at(const PagedArgs& a, int first, int entries, int i) {
  if (i < 0 || i >= entries || first < 0 || first > a.table_len - 1 - i) return -1;
  const int page = a.table[first + i];
  return page >= 0 && page < a.n_pages ? page : -1;
}

// Takes `want` pages of the pool: the first one's number, of which those below n_pages are the
// caller's (a negative number: none).  What the pool does not have goes back to the counter, so
// that it ends at n_pages and a larger pool goes on from there.
__device__ __forceinline__ int take_pages(const PagedArgs& a, int want) {
  const int first = atomicAdd(a.next_page, want);
  const int got = first < 0 ? 0 : max(0, min(want, a.n_pages - first));
  if (got < want) atomicSub(a.next_page, want - got);
  return first;
}

// ------------------------------------------------- rows held by one warp
// A row of D values over the 32 lanes: lane l has values l * PER ..

// (cos, sin) of the pair of each of the lane's values; angle(i) gives pair i's.
template <int PER, typename Angle>
__device__ __forceinline__ void row_angles(float2 (&cs)[PER], int rot, int style, Angle angle) {
  const int e0 = (threadIdx.x & 31) * PER, h = rot / 2;
#pragma unroll
  for (int k = 0; k < PER; ++k) cs[k] = make_float2(1.f, 0.f);
  if (e0 >= rot) return;
  if (style == FG_ROPE_INTERLEAVED) {
#pragma unroll
    for (int k = 0; k < PER; k += 2) cs[k] = cs[k + 1] = angle((e0 + k) / 2);
  } else {
#pragma unroll
    for (int k = 0; k < PER; ++k) cs[k] = angle(e0 + k - (e0 < h ? 0 : h));
  }
}

// Rotates a row by its angles (all lanes call).
template <int PER>
__device__ __forceinline__ void rotate_row(float (&x)[PER], const float2 (&cs)[PER], int rot,
                                           int style) {
  const int lane = threadIdx.x & 31, e0 = lane * PER;
  if (style == FG_ROPE_INTERLEAVED) {
#pragma unroll
    for (int k = 0; k < PER; k += 2) {
      const float u = x[k], v = x[k + 1];
      if (e0 < rot) {
        x[k] = u * cs[k].x - v * cs[k].y;
        x[k + 1] = v * cs[k].x + u * cs[k].y;
      }
    }
  } else {
    const int h = rot / 2;  // a multiple of 8: the two halves of a pair sit in two lanes
    const bool first = e0 < h;
    const int other = e0 >= rot ? lane : first ? lane + h / PER : lane - h / PER;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const float y = __shfl_sync(0xffffffffu, x[k], other);
      if (e0 < rot) x[k] = first ? x[k] * cs[k].x - y * cs[k].y : x[k] * cs[k].x + y * cs[k].y;
    }
  }
}

// The warp's values of one row of bf16 or fp32.
template <int PER>
__device__ __forceinline__ void load_row(const __nv_bfloat16* p, float (&x)[PER]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int k = 0; k < PER; k += 2) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(p + lane * PER + k);
    x[k] = bf16_lo(w);
    x[k + 1] = bf16_hi(w);
  }
}
template <int PER>
__device__ __forceinline__ void load_row(const float* p, float (&x)[PER]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int k = 0; k < PER; k += 2) {
    const float2 w = *reinterpret_cast<const float2*>(p + lane * PER + k);
    x[k] = w.x;
    x[k + 1] = w.y;
  }
}

// ------------------------------------------ 16-byte pieces of rows in lanes
// The arithmetic on bf16 stays packed as long as it can (the largest
// magnitude as two 16-bit integers a word, the scaling as one product a
// pair): unpacked it took more of an SM's time than the loads.

// Codes of a lane's 16 bytes of values times the power of two `inv`.
__device__ __forceinline__ void code16(const uint4& x, float inv, uint8_t* p, const float*) {
  *reinterpret_cast<uint32_t*>(p) =
      code4(__uint_as_float(x.x) * inv, __uint_as_float(x.y) * inv, __uint_as_float(x.z) * inv,
            __uint_as_float(x.w) * inv);
}
__device__ __forceinline__ uint32_t code_bf16x4(uint32_t a, uint32_t b, uint32_t inv2) {
  // the products are exact: a power of two, and what underflows is far below half a code
  asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(inv2));
  asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(b) : "r"(inv2));
  return code4(bf16_lo(a), bf16_hi(a), bf16_lo(b), bf16_hi(b));
}
__device__ __forceinline__ void code16(const uint4& x, float inv, uint8_t* p,
                                       const __nv_bfloat16*) {
  const uint32_t h = __float_as_uint(inv) >> 16, inv2 = h | (h << 16);
  *reinterpret_cast<uint2*>(p) =
      make_uint2(code_bf16x4(x.x, x.y, inv2), code_bf16x4(x.z, x.w, inv2));
}

// Bits of the largest finite magnitude among N values: one maximum a value,
// which passes over NaN; an infinity is rare and costs a second look.
template <int N>
__device__ __forceinline__ uint32_t top_bits(const float (&x)[N]) {
  float top = 0.f;
#pragma unroll
  for (int k = 0; k < N; ++k) top = fmaxf(top, fabsf(x[k]));
  uint32_t bits = __float_as_uint(top);
  if (bits >= 0x7f800000u) {
    bits = 0;
#pragma unroll
    for (int k = 0; k < N; ++k) bits = max(bits, finite_bits(x[k]));
  }
  return bits;
}

// Bits of the largest magnitude (of finite values only) of the lane's N pieces.
template <int N>
__device__ __forceinline__ uint32_t lane_top(const uint4 (&x)[N], const float*) {
  float f[4 * N];
#pragma unroll
  for (int i = 0; i < N; ++i) unpack16(x[i], f + 4 * i, (const float*)nullptr);
  return top_bits<4 * N>(f);
}
template <int N>
__device__ __forceinline__ uint32_t lane_top(const uint4 (&x)[N], const __nv_bfloat16*) {
  constexpr uint32_t kAbs = 0x7fff7fffu;
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    top = __vmaxu2(top, __vmaxu2(x[i].x & kAbs, x[i].y & kAbs));
    top = __vmaxu2(top, __vmaxu2(x[i].z & kAbs, x[i].w & kAbs));
  }
  top = max(top & 0xffffu, top >> 16);
  if (top >= 0x7f80u) {  // an infinity or a NaN: again, one value at a time
    top = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k)
        top = max(top, max(finite_bits(bf16_lo(w[k])), finite_bits(bf16_hi(w[k]))) >> 16);
    }
  }
  return top << 16;
}

// Opens a block for new rows whose largest magnitude has the bits `top` (the
// lane's; all lanes call): its exponent, `had` so far (below kExpMin: the block
// starts with these rows), grows when they need it, and then its codes are
// rounded again.  Returns the factor of the new rows' values.
template <int D>
__device__ __forceinline__ float open_block(uint32_t top, int had, uint8_t* codes,
                                            int8_t* exp_at) {
  const int lane = threadIdx.x & 31;
  const int now = max(had, block_exponent(__reduce_max_sync(0xffffffffu, top)));
  if (had >= kExpMin && now > had) {
    const uint32_t f = half2_pow2_neg(now - had);
#pragma unroll
    for (int i = 0; i < kBlockRows * D / 512; ++i) {
      uint4* p = reinterpret_cast<uint4*>(codes) + i * 32 + lane;
      uint4 v = *p;
      v.x = recode4(v.x, f);
      v.y = recode4(v.y, f);
      v.z = recode4(v.z, f);
      v.w = recode4(v.w, f);
      *p = v;
    }
  }
  __syncwarp();  // the exponent has been read, the old codes are in place
  if (lane == 0) *exp_at = (int8_t)now;
  return pow2f(-now);
}

// Codes a row of an open block.
template <int PER>
__device__ __forceinline__ void code_row(const float (&x)[PER], float inv, uint8_t* row) {
  uint8_t* p = row + (threadIdx.x & 31) * PER;
  if constexpr (PER == 4)
    *reinterpret_cast<uint32_t*>(p) = code4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
  else
    *reinterpret_cast<unsigned short*>(p) = (unsigned short)code2(x[0] * inv, x[1] * inv);
}

// Rows of a never-evicted segment that its table can hold.
__device__ __forceinline__ int live_rows(const fg_paged_desc& hd, int rows) {
  return (int)max(0LL, min((long long)rows, (long long)hd.max_pages * kPageRows));
}

struct AppendArgs {
  const void* k_new;
  const void* v_new;
  const int32_t* ids;
  const int32_t* n_new;  // null: m tokens of every sequence
  const int32_t* pos;
  const int32_t* special;
  int ns;
  const int32_t* punct;
  int np;
  int m;
  RopeArgs rope;
  // workspace
  int32_t* lists;   // [B, 2, m]: indices of the special / special or punctuation tokens
  int32_t* old;     // [Gkv, 2]: rows before the call, rows stored
  float2* angles;   // [B, m, rot / 2]: (cos, sin)
};

struct PagedDecodeArgs {
  const void* q;
  const void* k_new;  // null: no token is appended
  const void* v_new;
  const int32_t* ids;
  const int32_t* pos;
  const int32_t* special;
  int ns;
  const int32_t* punct;
  int np;
  RopeArgs rope;
  void* out;
  float* part_ml;
  float* part_acc;
};

cudaError_t launch_rope(const ProfileDims& pd, const void* Q, const void* K, const int32_t* pos,
                        const RopeArgs& rope, void* Qo, void* Ko, cudaStream_t s);
// Layout of the caches after the prompt: descriptors, row counts and page
// table from cinfo (policy, never-evicted rows); totals = {pages, worst-case
// pages, table entries}.
cudaError_t launch_paged_plan(int Gkv, int w, int reserve, const int2* cinfo, fg_paged_desc* caches,
                              int32_t* rows, int32_t* table, int32_t* next_page,
                              long long* totals, cudaStream_t s);
// Decode work list of the current row counts; totals[3] = items, totals[4] =
// thread blocks.
cudaError_t launch_paged_schedule(int Gkv, int R, const fg_paged_desc* caches, const int32_t* rows,
                                  int max_w, int table_len, int max_work, int slots, int4* ranges,
                                  PagedItem* items, int32_t* cta_first, long long* totals,
                                  cudaStream_t s);
cudaError_t launch_compact_q8(const ProfileDims& pd, const void* K, const void* V,
                              const uint8_t* keep, const PagedArgs& a, cudaStream_t s);
cudaError_t launch_append_q8(const ProfileDims& pd, const PagedArgs& a, const AppendArgs& n,
                             cudaStream_t s);
cudaError_t launch_decode_q8(const ProfileDims& pd, const PagedArgs& a, const PagedDecodeArgs& n,
                             cudaStream_t s);
// Thread blocks of the decode kernel that a wave counts on.
int q8_slots(const ProfileDims& pd, int sms);

}  // namespace fg
