// Position rotation of a prompt's queries and keys (the Llama attention whose
// prompt encoding the Method profiles rotates both by position).
//
// A thread owns one 16-byte piece of a row at one position: it forms the
// piece's (cos, sin) once and applies them to that piece of kHeads heads, so
// the angles cost nothing beside the row stream.  Pairs in halves of the row
// sit in two lanes, which exchange their pieces by shuffle, so a rotation in
// place reads nothing that another thread has written.  Bound by HBM: every
// value is read and written once.  Measured (device time): 512 heads of 2048 x
// 128 bf16 (537 MB) 82 us, 6.6 TB/s, fp32 157 us, 6.8 TB/s; 320 heads of 1531 x
// 128 (251 MB, half of each row rotated) 43 us, 5.8 TB/s.
#include "fg_paged.cuh"

namespace fg {
namespace {

constexpr int kThreads = 256;
constexpr int kHeads = 16;  // heads per CTA
constexpr int kUnroll = 4;  // heads with loads in flight

__device__ __forceinline__ uint4 pack16(const float* f, const float*) {
  return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                    __float_as_uint(f[3]));
}
__device__ __forceinline__ uint4 pack16(const float* f, const __nv_bfloat16*) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

// heads of one sequence: hq query heads, then hk key heads (0 leaves a side out)
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) rope_kernel(const T* Q,
                                                        const T* K,
                                                        const int32_t* __restrict__ pos,
                                                        const RopeArgs rope, T* Qo, T* Ko, int n,
                                                        int hq, int hk, int tiles, int chunks) {
  constexpr int E = Vec16<T>::kElems;
  constexpr int LPR = D / E;             // lanes per row
  constexpr int ROWS = kThreads / LPR;   // positions per CTA
  const int tile = blockIdx.x % tiles, rest = blockIdx.x / tiles;
  const int chunk = rest % chunks, b = rest / chunks;
  const int gl = threadIdx.x % LPR, i = tile * ROWS + threadIdx.x / LPR;
  const int e0 = gl * E, rot = rope.rot, h = rot / 2;
  const bool in = i < n;
  const bool inter = rope.style == FG_ROPE_INTERLEAVED, first = e0 < h;
  griddep_wait();
  griddep_launch_dependents();
  // cos and sin of the pair of each value (sin signed: first value of a pair minus)
  float cs[E], sn[E];
#pragma unroll
  for (int k = 0; k < E; ++k) {
    cs[k] = 1.f;
    sn[k] = 0.f;
  }
  if (in && e0 < rot) {
    const unsigned p = pos ? (unsigned)pos[(size_t)b * n + i] : (unsigned)i;
    if (inter) {
#pragma unroll
      for (int k = 0; k < E; k += 2) {
        float c, s;
        rope_cos_sin(p, rope.turns[(e0 + k) / 2], c, s);
        cs[k] = cs[k + 1] = c;
        sn[k] = -s;
        sn[k + 1] = s;
      }
    } else {
#pragma unroll
      for (int k = 0; k < E; ++k) {
        float c, s;
        rope_cos_sin(p, rope.turns[e0 + k - (first ? 0 : h)], c, s);
        cs[k] = c;
        sn[k] = first ? -s : s;
      }
    }
  }
  // the lane that holds the other half of this lane's pairs (same row, same warp)
  const int lane = threadIdx.x & 31;
  const int other = inter || e0 >= rot ? lane : first ? lane + h / E : lane - h / E;
  const int h0 = chunk * kHeads, h1 = min(h0 + kHeads, hq + hk);
  for (int hb = h0; hb < h1; hb += kUnroll) {
    uint4 x[kUnroll];
    size_t at[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int head = hb + u;
      const bool key = head >= hq;
      at[u] = (((size_t)b * (key ? hk : hq) + (key ? head - hq : head)) * n + i) * D + e0;
      x[u] = in && head < h1 ? ld16((key ? K : Q) + at[u]) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int head = hb + u;
      float f[E], y[E];
      unpack16(x[u], f, (const T*)nullptr);
      if (inter) {
#pragma unroll
        for (int k = 0; k < E; ++k) y[k] = f[k ^ 1];
      } else {
        uint4 z;
        z.x = __shfl_sync(0xffffffffu, x[u].x, other);
        z.y = __shfl_sync(0xffffffffu, x[u].y, other);
        z.z = __shfl_sync(0xffffffffu, x[u].z, other);
        z.w = __shfl_sync(0xffffffffu, x[u].w, other);
        unpack16(z, y, (const T*)nullptr);
      }
#pragma unroll
      for (int k = 0; k < E; ++k)
        if (e0 < rot) f[k] = f[k] * cs[k] + y[k] * sn[k];
      if (in && head < h1)
        *reinterpret_cast<uint4*>((head >= hq ? Ko : Qo) + at[u]) = pack16(f, (const T*)nullptr);
    }
  }
}

template <typename T, int D>
cudaError_t run_rope(const ProfileDims& pd, const void* Q, const void* K, const int32_t* pos,
                     const RopeArgs& rope, void* Qo, void* Ko, cudaStream_t s) {
  constexpr int ROWS = kThreads / (D / Vec16<T>::kElems);
  const int hq = Q ? pd.HL : 0, hk = K ? pd.HLkv : 0;
  const int tiles = cdiv(pd.n, ROWS), chunks = cdiv(hq + hk, kHeads);
  const long long grid = (long long)tiles * chunks * pd.B;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  return launch_pdl(rope_kernel<T, D>, (unsigned)grid, kThreads, 0, s, (const T*)Q, (const T*)K,
                    pos, rope, (T*)Qo, (T*)Ko, pd.n, hq, hk, tiles, chunks);
}

}  // namespace

cudaError_t launch_rope(const ProfileDims& pd, const void* Q, const void* K, const int32_t* pos,
                        const RopeArgs& rope, void* Qo, void* Ko, cudaStream_t s) {
  if (pd.dtype == FG_FP32)
    return pd.d == 64 ? run_rope<float, 64>(pd, Q, K, pos, rope, Qo, Ko, s)
                      : run_rope<float, 128>(pd, Q, K, pos, rope, Qo, Ko, s);
  return pd.d == 64 ? run_rope<__nv_bfloat16, 64>(pd, Q, K, pos, rope, Qo, Ko, s)
                    : run_rope<__nv_bfloat16, 128>(pd, Q, K, pos, rope, Qo, Ko, s);
}

}  // namespace fg
