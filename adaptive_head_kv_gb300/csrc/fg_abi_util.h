// Argument checks and sizes shared by the C-ABI translation units.
#pragma once

#include <math.h>
#include <stdint.h>

#include "fg_common.cuh"
#include "fg_internal.h"

namespace {

using fg::cdiv;

constexpr size_t kAlign = 256;
constexpr int kMaxIdSet = 4096;

inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

inline int ratio_count(float r, int n) { return (int)ceil((double)r * (double)n); }

inline fg_status check_params(const fg_params* p) {
  if (!p) return FG_EINVAL;
  if (p->B < 1 || p->L < 1 || p->H < 1 || p->n < 1) return FG_EINVAL;
  const long long G = (long long)p->B * p->L * p->H;
  if (G > 0x7fffffffLL || (long long)G * p->n > (1LL << 40)) return FG_EINVAL;
  if (p->d != 64 && p->d != 128) return FG_EDTYPE;
  if (p->dtype != FG_BF16 && p->dtype != FG_FP32) return FG_EDTYPE;
  if (!(p->T > 0.f && p->T <= 1.f)) return FG_EINVAL;
  if (!(p->r_l >= 0.f && p->r_l <= 1.f) || !(p->r_f >= 0.f && p->r_f <= 1.f)) return FG_EINVAL;
  if (!(p->scale >= 0.f) || isinf(p->scale)) return FG_EINVAL;
  if (p->Hkv < 0 || (p->Hkv > 0 && p->H % p->Hkv != 0)) return FG_EINVAL;
  const int R = p->Hkv > 0 ? p->H / p->Hkv : 1;
  if (R != 1 && R != 2 && R != 4 && R != 8) return FG_EDTYPE;
  return FG_OK;
}

inline fg::ProfileDims dims(const fg_params* p) {
  fg::ProfileDims pd;
  pd.B = p->B;
  pd.HL = p->L * p->H;
  pd.G = p->B * pd.HL;
  pd.H = p->H;
  pd.Hkv = p->Hkv > 0 ? p->Hkv : p->H;
  pd.R = p->H / pd.Hkv;
  pd.HLkv = p->L * pd.Hkv;
  pd.Gkv = p->B * pd.HLkv;
  pd.n = p->n;
  pd.d = p->d;
  pd.dtype = p->dtype;
  pd.w = ratio_count(p->r_l, p->n);
  pd.k = ratio_count(p->r_f, p->n);
  pd.T = p->T;
  const float s = p->scale > 0.f ? p->scale : (float)(1.0 / sqrt((double)p->d));
  pd.sl2 = s * fg::kLog2e;
  return pd;
}

inline fg_status check_ids(const int32_t* set, int32_t cnt) {
  if (cnt < 0 || cnt > kMaxIdSet) return FG_EINVAL;
  if (cnt > 0 && !set) return FG_EINVAL;
  return FG_OK;
}

inline fg_status cuda_status(cudaError_t e) { return e == cudaSuccess ? FG_OK : FG_ECUDA; }

inline int kv_count(const fg_params* p) { return p->B * p->L * (p->Hkv > 0 ? p->Hkv : p->H); }
inline int group_size(const fg_params* p) { return p->Hkv > 0 ? p->H / p->Hkv : 1; }

}  // namespace
