// layer_norm.hip - layer norm over the rows of a matrix, forward and backward.
//
//   forward    m = mean(x), v = mean((x - m)^2), r = 1 / sqrt(v + eps),
//              y = (x - m) r w + b; optionally the normalised row (x - m) r
//              is kept in 8 bits for the backward pass
//   backward   g = dy w, n = (x - m) r (or the kept row),
//              dx = r (g - mean(g) - n mean(g n)),
//              dw = sum over rows of dy n, db = sum over rows of dy
//
// Bound by HBM: a row is held in registers by `LPR` lanes, NV vectors of 16
// bytes each, so it is read once, and the next row's loads are on their way
// while one is worked on.  LPR is 16 lanes or one wave for rows of up to 16
// values per lane (no LDS, no barrier), else a workgroup of 256 or 1024 lanes.
// 524288 x 128 bf16, forward: 54 us with 16 lanes a row, 152 with 64.
//
// Measured, bf16 (fp32 parameters): forward of 65536 x 1024 with kept rows 79
// us (4.3 TB/s), 524288 x 128 54 us (5.0), 8192 x 16384 115 us (4.7); backward
// of 65536 x 1024 from x 75 + 5 us (5.1), from kept rows 63 + 5 us (4.9),
// 524288 x 128 81 us (5.0), 8192 x 16384 162 us (5.0).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "elem.h"
#include "layer_ops.h"
#include "rows.h"

namespace adasum {
namespace {

using namespace elem;

template <typename T, int LPR, int NV, bool KEEP>
__global__ __launch_bounds__(LPR < 256 ? 256 : LPR) void norm_kernel(NormArgs a) {
  constexpr int VEC = Type<T>::kVec;
  constexpr int ROWS = LPR < 256 ? 256 / LPR : 1;
  __shared__ float lds1[2][1][LPR / 64 > 0 ? LPR / 64 : 1];
  __shared__ float lds2[2][2][LPR / 64 > 0 ? LPR / 64 : 1];
  const int lane = threadIdx.x & (LPR - 1);
  const int64_t step = (int64_t)gridDim.x * ROWS;
  int64_t r = (int64_t)blockIdx.x * ROWS + threadIdx.x / LPR;
  const int H = a.hidden;
  const float inv_h = 1.f / (float)H;
  int valid[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) valid[j] = H - (j * LPR + lane) * VEC;
  float w[NV][VEC], b[NV][VEC];
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const int c = (j * LPR + lane) * VEC + i;
      w[j][i] = i < valid[j] ? (a.weight ? load_any(a.weight, a.param_dtype, c) : 1.f) : 0.f;
      b[j][i] = i < valid[j] && a.bias ? load_any(a.bias, a.param_dtype, c) : 0.f;
    }
  const T* x = static_cast<const T*>(a.x);
  T* y = static_cast<T*>(a.y);
  const int64_t nb = (H + kScaleBlock - 1) / kScaleBlock;
  v4u raw[NV];
  if (r < a.rows) {
#pragma unroll
    for (int j = 0; j < NV; ++j) raw[j] = load_raw(x + r * a.x_stride + (j * LPR + lane) * VEC, valid[j]);
  }
  int slot = 0;
  for (; r < a.rows; r += step) {
    float v[NV][VEC];
#pragma unroll
    for (int j = 0; j < NV; ++j) widen<T>(raw[j], v[j]);
    if (r + step < a.rows) {  // the next row's loads, in flight behind this row's arithmetic
#pragma unroll
      for (int j = 0; j < NV; ++j) raw[j] = load_raw(x + (r + step) * a.x_stride + (j * LPR + lane) * VEC, valid[j]);
    }
    float s1[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < VEC; ++i) s1[0] += v[j][i];
    row_sum<LPR, 1>(s1, lds1, slot);
    const float m = s1[0] / (float)H;  // divided, so that a constant row's mean is the constant
    // squares around the mean; the sum of the deviations is what rounding
    // left out of m, and is taken out of both
    float s2[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        v[j][i] = i < valid[j] ? v[j][i] - m : 0.f;
        s2[0] += v[j][i];
        s2[1] = __builtin_fmaf(v[j][i], v[j][i], s2[1]);
      }
    row_sum<LPR, 2>(s2, lds2, slot);
    slot ^= 1;
    const float rest = s2[0] * inv_h;
    const float var = __builtin_fmaf(-rest, rest, s2[1] * inv_h);
    const float rstd = inverse_root((var < 0.f ? 0.f : var) + a.eps);  // NaN where the row holds one, or an infinity
    if (lane == 0) {
      if (a.mean) a.mean[r] = m + rest;
      a.rstd[r] = rstd;
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * LPR + lane) * VEC;
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[j][i] = i < valid[j] ? (v[j][i] - rest) * rstd : 0.f;
      if constexpr (KEEP)
        pack_vec<VEC>(v[j], valid[j], 248u, lane, a.codes + r * H + c, a.scales + r * nb + c / kScaleBlock);
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[j][i] = __builtin_fmaf(v[j][i], w[j][i], b[j][i]);
      store_vec(y + r * a.y_stride + c, v[j], valid[j]);
    }
  }
}

// The rows of a backward pass: dy and either x or the kept codes, one row
// ahead of the arithmetic.
template <typename T, int LPR, int NV, bool KEPT>
__global__ __launch_bounds__(LPR < 256 ? 256 : LPR) void norm_grad_kernel(NormGradArgs a) {
  constexpr int VEC = Type<T>::kVec;
  constexpr int ROWS = LPR < 256 ? 256 / LPR : 1;
  __shared__ float lds[2][2][LPR / 64 > 0 ? LPR / 64 : 1];
  const int lane = threadIdx.x & (LPR - 1);
  const int64_t step = (int64_t)gridDim.x * ROWS;
  int64_t r = (int64_t)blockIdx.x * ROWS + threadIdx.x / LPR;
  const int H = a.hidden;
  const float inv_h = 1.f / (float)H;
  const int64_t nb = (H + kScaleBlock - 1) / kScaleBlock;
  int valid[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) valid[j] = H - (j * LPR + lane) * VEC;
  // 1024 lanes have 128 registers each: there the weights, and for fp32 the
  // sums of dy, lie in LDS, every lane its own (8192 x 16384 bf16: 164 us
  // against 230 with spilled registers; 4096 x 16384 fp32: 177, with only the
  // weights 241, with neither 310)
  constexpr bool LDS_W = LPR == 1024, LDS_B = LDS_W && sizeof(T) == 4;
  __shared__ float far[LDS_W ? NV * LPR * VEC : 1], far_b[LDS_B ? NV * LPR * VEC : 1];
  float w[LDS_W ? 1 : NV][VEC], aw[NV][VEC], ab[LDS_B ? 1 : NV][VEC];
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const int c = (j * LPR + lane) * VEC + i;
      const float v = i < valid[j] ? (a.weight ? load_any(a.weight, a.param_dtype, c) : 1.f) : 0.f;
      if constexpr (LDS_W)
        far[c] = v;
      else
        w[j][i] = v;
      aw[j][i] = 0.f;
      if constexpr (LDS_B)
        far_b[c] = 0.f;
      else
        ab[j][i] = 0.f;
    }
  const T* dy = static_cast<const T*>(a.dy);
  const T* x = static_cast<const T*>(a.x);
  T* dx = static_cast<T*>(a.dx);
  v4u rdy[NV], rx[NV];
  uint32_t rc[NV][VEC / 4], rb[NV];
  float mean = 0.f, rstd = 0.f;
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * LPR + lane) * VEC;
      rdy[j] = load_raw(dy + row * a.dy_stride + c, valid[j]);
      if constexpr (KEPT) {
        load_codes<VEC>(a.codes + row * H + c, valid[j], rc[j]);
        rb[j] = valid[j] > 0 ? a.scales[row * nb + c / kScaleBlock] : 127u;
      } else {
        rx[j] = load_raw(x + row * a.x_stride + c, valid[j]);
      }
    }
    if constexpr (!KEPT) mean = a.mean[row];
    rstd = a.rstd[row];
  };
  if (r < a.rows) fetch(r);
  int slot = 0;
  for (; r < a.rows; r += step) {
    float g[NV][VEC], n[NV][VEC];
    const float rs = rstd;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      widen<T>(rdy[j], g[j]);
      if constexpr (KEPT) {
        const float s = scale_value(rb[j]);
#pragma unroll
        for (int q = 0; q < VEC / 4; ++q) {
          float t[4];
          widen_codes(rc[j][q], t);
#pragma unroll
          for (int i = 0; i < 4; ++i) n[j][4 * q + i] = t[i] * s;
        }
      } else {
        widen<T>(rx[j], n[j]);
#pragma unroll
        for (int i = 0; i < VEC; ++i) n[j][i] = i < valid[j] ? (n[j][i] - mean) * rs : 0.f;
      }
    }
    if (r + step < a.rows) fetch(r + step);
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float d = g[j][i];
        aw[j][i] = __builtin_fmaf(d, n[j][i], aw[j][i]);
        if constexpr (LDS_B)
          far_b[(j * LPR + lane) * VEC + i] += d;
        else
          ab[j][i] += d;
        g[j][i] = d * (LDS_W ? far[LDS_W ? (j * LPR + lane) * VEC + i : 0] : w[LDS_W ? 0 : j][i]);
        s[0] += g[j][i];
        s[1] = __builtin_fmaf(g[j][i], n[j][i], s[1]);
      }
    row_sum<LPR, 2>(s, lds, slot);
    slot ^= 1;
    const float mg = s[0] * inv_h, mgn = s[1] * inv_h;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) g[j][i] = __builtin_fmaf(-n[j][i], mgn, g[j][i] - mg) * rs;
      store_vec(dx + r * a.dx_stride + (j * LPR + lane) * VEC, g[j], valid[j]);
    }
  }
  if (a.partials == nullptr) return;
  // The workgroup's sums: its waves' rows added in wave order through LDS,
  // one wave's columns at a time.
  float* out = a.partials + (int64_t)blockIdx.x * 2 * H;
  if constexpr (LPR <= 64) {
    __shared__ float part[3][2][LPR * VEC];
    const int wave = threadIdx.x >> 6;
    if constexpr (LPR == 16) {  // the wave's four rows first
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i)
#pragma unroll
          for (int d = 16; d < 64; d *= 2) {
            aw[j][i] += __shfl_xor(aw[j][i], d);
            ab[j][i] += __shfl_xor(ab[j][i], d);
          }
    }
    const bool first = (threadIdx.x & 63) < LPR;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (j > 0) __syncthreads();
      if (wave > 0 && first) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          part[wave - 1][0][i * LPR + lane] = aw[j][i];
          part[wave - 1][1][i * LPR + lane] = ab[j][i];
        }
      }
      __syncthreads();
      if (wave == 0 && first) {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
#pragma unroll
          for (int q = 0; q < 3; ++q) {
            aw[j][i] += part[q][0][i * LPR + lane];
            ab[j][i] += part[q][1][i * LPR + lane];
          }
        store_row<float, VEC>(out + (j * LPR + lane) * VEC, aw[j], valid[j]);
        store_row<float, VEC>(out + H + (j * LPR + lane) * VEC, ab[j], valid[j]);
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * LPR + lane) * VEC;
      if constexpr (LDS_B) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) ab[0][i] = far_b[c + i];
      }
      store_row<float, VEC>(out + c, aw[j], valid[j]);
      store_row<float, VEC>(out + H + c, ab[LDS_B ? 0 : j], valid[j]);
    }
  }
}

template <typename T, int LPR, int NV>
hipError_t norm_launch(const NormArgs& a, hipStream_t st) {
  constexpr int ROWS = LPR < 256 ? 256 / LPR : 1;
  constexpr int THREADS = LPR < 256 ? 256 : LPR;
  // eight waves per SIMD's worth of workgroups at most: each then walks
  // several rows with the weights in registers
  const int64_t blocks = std::min<int64_t>(ceil_div(a.rows, ROWS), (int64_t)kCUs * 2048 / THREADS);
  if (a.codes)
    norm_kernel<T, LPR, NV, true><<<(unsigned)blocks, THREADS, 0, st>>>(a);
  else
    norm_kernel<T, LPR, NV, false><<<(unsigned)blocks, THREADS, 0, st>>>(a);
  return hipGetLastError();
}

// Lanes per row and vectors per lane of the backward pass; at most 16 values
// per lane, which keeps its two sums, the weights and two rows in registers.
struct GradShape {
  int lanes, threads, rows;
};
GradShape grad_shape(int hidden) {
  const int per_wave = 64 * 16;
  if (hidden <= 16 * 16) return {16, 256, 16};
  if (hidden <= per_wave) return {64, 256, 4};
  if (hidden <= 4 * per_wave) return {256, 256, 1};
  return {1024, 1024, 1};
}

template <typename T, int LPR, int NV>
hipError_t norm_grad_launch(const NormGradArgs& a, int blocks, hipStream_t st) {
  constexpr int THREADS = LPR < 256 ? 256 : LPR;
  if (a.x == nullptr)
    norm_grad_kernel<T, LPR, NV, true><<<blocks, THREADS, 0, st>>>(a);
  else
    norm_grad_kernel<T, LPR, NV, false><<<blocks, THREADS, 0, st>>>(a);
  return hipGetLastError();
}

template <typename T>
hipError_t norm_grad_width(const NormGradArgs& a, int lanes, int blocks, hipStream_t st) {
  constexpr int NV = 16 / Type<T>::kVec;
  const int64_t nvec = ceil_div(a.hidden, Type<T>::kVec);
  const bool half = nvec <= (int64_t)lanes * NV / 2;
  if (lanes == 16)
    return half ? norm_grad_launch<T, 16, NV / 2>(a, blocks, st) : norm_grad_launch<T, 16, NV>(a, blocks, st);
  if (lanes == 64)
    return half ? norm_grad_launch<T, 64, NV / 2>(a, blocks, st) : norm_grad_launch<T, 64, NV>(a, blocks, st);
  if (lanes == 256)
    return half ? norm_grad_launch<T, 256, NV / 2>(a, blocks, st) : norm_grad_launch<T, 256, NV>(a, blocks, st);
  return half ? norm_grad_launch<T, 1024, NV / 2>(a, blocks, st) : norm_grad_launch<T, 1024, NV>(a, blocks, st);
}

template <typename T>
hipError_t norm_width(const NormArgs& a, hipStream_t st) {
  constexpr int VEC = Type<T>::kVec;
  constexpr int NV = 16 / VEC;
  const int64_t nvec = ceil_div(a.hidden, VEC);
  if (nvec <= 16 * NV / 2) return norm_launch<T, 16, NV / 2>(a, st);
  if (nvec <= 16 * NV) return norm_launch<T, 16, NV>(a, st);
  if (nvec <= 64 * NV / 2) return norm_launch<T, 64, NV / 2>(a, st);
  if (nvec <= 64 * NV) return norm_launch<T, 64, NV>(a, st);
  if (nvec <= 256 * NV / 2) return norm_launch<T, 256, NV / 2>(a, st);
  if (nvec <= 256 * NV) return norm_launch<T, 256, NV>(a, st);
  if (nvec <= 1024 * NV / 2) return norm_launch<T, 1024, NV / 2>(a, st);
  return norm_launch<T, 1024, NV>(a, st);
}

}  // namespace

hipError_t launch_norm(int dtype, const NormArgs& a, hipStream_t st) {
  return with_dtype(dtype, [&](auto t) { return norm_width<decltype(t)>(a, st); });
}

namespace {

// Workgroups of one launch over `rows`.
int grad_blocks(int64_t rows, const GradShape& s) {
  // Two workgroups of 256 lanes per CU, or as many waves in wider ones, but
  // one per CU at least; and no more than leaves a wave four rows, or 16 lanes
  // two: every workgroup leaves a row of partial sums for the join.  65536 x
  // 1024 bf16: 75 us whether 512 or 1024 workgroups, the join 5 against 8 us.
  return (int)std::min<int64_t>(ceil_div(rows, s.rows * (s.lanes == 16 ? 2 : 4)),
                                std::max<int64_t>(kCUs, (int64_t)kCUs * 512 / s.threads));
}

// Rows of one launch: as many as leave the fp32 sums of dweight and dbias
// kNormGradRows long in a full one.  (More workgroups in one launch instead:
// 1048576 x 4096 bf16 5450 us against 4900.)
int64_t grad_rows(const GradShape& s) {
  return (int64_t)grad_blocks(kMaxDim, s) * s.rows * kNormGradRows;
}

}  // namespace

int64_t norm_grad_parts(int64_t rows, int hidden) {
  const GradShape s = grad_shape(hidden);
  const int64_t full = grad_rows(s);
  return rows / full * grad_blocks(full, s) + grad_blocks(rows % full, s);
}

hipError_t launch_norm_grad(int dtype, const NormGradArgs& a, hipStream_t st) {
  const GradShape s = grad_shape(a.hidden);
  const int64_t full = grad_rows(s), size = dtype == 0 ? 4 : 2;
  int64_t parts = 0;
  for (int64_t first = 0; first < a.rows; first += full) {
    NormGradArgs b = a;
    b.rows = std::min(full, a.rows - first);
    b.dy = static_cast<const char*>(a.dy) + first * a.dy_stride * size;
    b.dx = static_cast<char*>(a.dx) + first * a.dx_stride * size;
    b.rstd = a.rstd + first;
    if (a.x) {
      b.x = static_cast<const char*>(a.x) + first * a.x_stride * size;
      b.mean = a.mean + first;
    } else {
      b.codes = a.codes + first * a.hidden;
      b.scales = a.scales + first * ceil_div(a.hidden, kScaleBlock);
    }
    if (a.partials) b.partials = a.partials + parts * 2 * a.hidden;
    const int blocks = grad_blocks(b.rows, s);
    parts += blocks;
    const hipError_t e =
        with_dtype(dtype, [&](auto t) { return norm_grad_width<decltype(t)>(b, s.lanes, blocks, st); });
    if (e != hipSuccess) return e;
  }
  if (a.dweight || a.dbias) {
    const int64_t cols = 2 * (int64_t)a.hidden;
    join_columns_kernel<<<(unsigned)ceil_div(cols, 32), 256, 0, st>>>(a.partials, (int)parts, cols, a.dweight, a.hidden,
                                                                    a.dbias, a.grad_dtype, a.accumulate);
    return hipGetLastError();
  }
  return hipSuccess;
}

}  // namespace adasum
