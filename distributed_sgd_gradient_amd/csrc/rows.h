// rows.h - what the norms' kernels share: sums over a row's lanes, the inverse
// root, and the join of the columns' partial sums.  Device code only.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "elem.h"

namespace adasum {
namespace {

using namespace elem;

// Sums of N values over the LPR lanes of a row, the same in every lane.
// `slot` alternates between two LDS areas, so that one barrier a call is
// enough: an area is written again only after the barrier of the call between.
template <int LPR, int N, typename F>
__device__ __forceinline__ void row_sum(F (&s)[N], F (*lds)[N][LPR / 64 > 0 ? LPR / 64 : 1], int slot) {
#pragma unroll
  for (int i = 0; i < N; ++i) s[i] = LPR == 16 ? sum16(s[i]) : wave_sum(s[i]);
  if constexpr (LPR > 64) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) lds[slot][i][wave] = s[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      F t = 0;
#pragma unroll
      for (int w = 0; w < LPR / 64; ++w) t += lds[slot][i][w];
      s[i] = t;
    }
  }
}

// 1 / sqrt(v) for v > 0: the hardware's estimate and one Newton step, within
// one unit of the last place (v above fp32's range: 0).
__device__ __forceinline__ float inverse_root(float v) {
  const float r = __builtin_amdgcn_rsqf(v);
  const float e = __builtin_fmaf(-v * r, r, 1.f);
  const float n = __builtin_fmaf(0.5f * r, e, r);
  return v < __builtin_inff() ? n : r;
}

// Joins the workgroups' partial sums of `width` columns: 32 columns a
// workgroup, eight runs of consecutive partials a column, added in fp64 in the
// order of the partials.  The first `first` columns go to out0, the others to
// out1 (either may be NULL).
__global__ __launch_bounds__(256) void join_columns_kernel(const float* partials, int parts, int64_t width, void* out0,
                                                           int64_t first, void* out1, int dtype, int accumulate) {
  __shared__ double part[8][32];
  const int col = threadIdx.x & 31, run = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + col;
  const int per = (parts + 7) / 8;
  double s = 0.0;
  if (c < width) {
    const int lo = run * per, hi = min(parts, lo + per);
#pragma unroll 8
    for (int i = lo; i < hi; ++i) s += (double)partials[i * width + c];
  }
  part[run][col] = s;
  __syncthreads();
  if (run == 0 && c < width) {
#pragma unroll
    for (int q = 1; q < 8; ++q) s += part[q][col];
    void* dst = c < first ? out0 : out1;
    const int64_t i = c < first ? c : c - first;
    if (dst) store_any(dst, dtype, i, accumulate ? s + (double)load_any(dst, dtype, i) : s);
  }
}

}  // namespace
}  // namespace adasum
