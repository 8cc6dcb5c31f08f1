// Attention of a batch over the caches of a prompt that its sequences share:
// every query of sequence b and head h over cache h / R of the prompt, which is
// read for all sequences at once.
//
// A thread block takes a chunk of a cache's rows and four queries; its warps
// take the rows in turn, a lane d / 32 dimensions.
#include "fg_paged_decode.cuh"

namespace fg {
namespace {

constexpr int kPrefixParts = 16;
constexpr int kQueries = 4;

template <typename T, int D>
__global__ void __launch_bounds__(128)
    prefix_kernel(const PagedArgs a, const PagedDecodeArgs n, const PrefixParts px, int H, int R,
                  int HL, float sl2) {
  constexpr int PER = D / 32;
  __shared__ float sm_m[4][kQueries], sm_l[4][kQueries], sm_o[4][kQueries][D];
  const int c = blockIdx.x, part = blockIdx.y, j0 = blockIdx.z * kQueries;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  griddep_wait();
  griddep_launch_dependents();
  const fg_paged_desc hd = a.caches[c];
  const int w = ring_slots(hd, a.max_w), rows = live_rows(hd, a.rows[c]);
  if ((w != hd.w || rows != a.rows[c]) && threadIdx.x == 0) atomicOr(a.dev_err, kErrInvalid);
  float q[kQueries][PER], o[kQueries][PER], m[kQueries], l[kQueries];
  int t[kQueries];
#pragma unroll
  for (int i = 0; i < kQueries; ++i) {
    const int j = j0 + i, b = j / R;
    m[i] = kNoScore;
    l[i] = 0.f;
    t[i] = j < px.nq ? n.pos[b] : -1;
#pragma unroll
    for (int k = 0; k < PER; ++k) q[i][k] = o[i][k] = 0.f;
    if (t[i] < 0) continue;
    const size_t g = (size_t)b * HL + (size_t)(c / (H / R)) * H + (size_t)(c % (H / R)) * R + j % R;
    load_row<PER>((const T*)n.q + g * D, q[i]);
    if (n.rope.rot > 0) {
      float2 cs[PER];
      row_angles<PER>(cs, n.rope.rot, n.rope.style, [&](int p) {
        float2 y;
        rope_cos_sin((unsigned)t[i], n.rope.turns[p], y.x, y.y);
        return y;
      });
      rotate_row<PER>(q[i], cs, n.rope.rot, n.rope.style);
    }
  }
  const long long all = (long long)rows + w;
  for (long long x = all * part / px.parts + warp; x < all * (part + 1) / px.parts; x += 4) {
    const bool ring = x >= rows;
    const int r = (int)(ring ? x - rows : x);
    const int page = ring ? page_at(a, hd.ring_page, hd.ring_pages, r / kPageRows)
                          : page_at(a, hd.first_page, hd.max_pages, r / kPageRows);
    if (page < 0) {
      if (lane == 0) atomicOr(a.dev_err, kErrInvalid);
      continue;
    }
    const size_t at = (size_t)page * kPageRows + r % kPageRows;
    const int p = ring ? a.pos[at] : 0;
    const int8_t* e = a.exps + ((size_t)page * kPageBlocks + r % kPageRows / kBlockRows) * 2;
    float kv[2][PER];
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int k = 0; k < PER; k += 2) {
        const uint8_t* z = (s ? a.vp : a.kp) + at * D + lane * PER + k;
        const float2 f = unpack_f16x2(decode2(z[0] | z[1] << 8));
        kv[s][k] = f.x * pow2f(e[s]);
        kv[s][k + 1] = f.y * pow2f(e[s]);
      }
#pragma unroll
    for (int i = 0; i < kQueries; ++i) {
      if (t[i] < 0) continue;
      if (ring && !(p >= 0 && (unsigned)t[i] - (unsigned)p < (unsigned)w)) continue;
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < PER; ++k) s = fmaf(q[i][k], kv[0][k], s);
#pragma unroll
      for (int z = 16; z; z >>= 1) s += __shfl_xor_sync(0xffffffffu, s, z);
      s *= sl2;
      const float mn = fmaxf(m[i], s), f = exp2f(m[i] - mn), y = exp2f(s - mn);
      l[i] = l[i] * f + y;
      m[i] = mn;
#pragma unroll
      for (int k = 0; k < PER; ++k) o[i][k] = o[i][k] * f + y * kv[1][k];
    }
  }
#pragma unroll
  for (int i = 0; i < kQueries; ++i) {
    if (lane == 0) {
      sm_m[warp][i] = m[i];
      sm_l[warp][i] = l[i];
    }
#pragma unroll
    for (int k = 0; k < PER; ++k) sm_o[warp][i][lane * PER + k] = o[i][k];
  }
  __syncthreads();
  const int i = warp;
  if (j0 + i >= px.nq) return;
  float M = kNoScore, L = 0.f;
  for (int z = 0; z < 4; ++z) M = fmaxf(M, sm_m[z][i]);
  for (int z = 0; z < 4; ++z) L += sm_l[z][i] * exp2f(sm_m[z][i] - M);
  const size_t slot = ((size_t)c * px.parts + part) * px.nq + j0 + i;
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    float y = 0.f;
    for (int z = 0; z < 4; ++z) y += sm_o[z][i][lane * PER + k] * exp2f(sm_m[z][i] - M);
    const_cast<float*>(px.acc)[slot * D + lane * PER + k] = L == 0.f ? 0.f : y / L;
  }
  if (lane == 0) {
    const_cast<float*>(px.ml)[2 * slot] = M;
    const_cast<float*>(px.ml)[2 * slot + 1] = L;
  }
}

}  // namespace

int prefix_parts(const ProfileDims&, int) { return kPrefixParts; }

template <typename T, int D>
static cudaError_t run_prefix(const ProfileDims& pd, const PagedDecodeArgs& n, const PagedArgs& pre,
                              const PrefixParts& px, cudaStream_t s) {
  prefix_kernel<T, D><<<dim3(px.caches, px.parts, cdiv(px.nq, kQueries)), 128, 0, s>>>(
      pre, n, px, pd.H, pd.R, pd.HL, pd.sl2);
  return cudaGetLastError();
}

cudaError_t launch_prefix(const ProfileDims& pd, const PagedDecodeArgs& n, const PagedArgs& pre,
                          const PrefixParts& px, cudaStream_t s) {
  if (pd.dtype == FG_FP32)
    return pd.d == 64 ? run_prefix<float, 64>(pd, n, pre, px, s)
                      : run_prefix<float, 128>(pd, n, pre, px, s);
  return pd.d == 64 ? run_prefix<__nv_bfloat16, 64>(pd, n, pre, px, s)
                    : run_prefix<__nv_bfloat16, 128>(pd, n, pre, px, s);
}

}  // namespace fg
