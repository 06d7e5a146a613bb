// rms.hip - root-mean-square norm of a residual stream's rows, forward and
// backward.
//
//   forward    h = x + residual (rounded to the stream's type),
//              r = 1 / sqrt(mean(h^2) + eps), y = h r w; optionally the rows y
//              are given in 8 bits too, or only so
//   backward   g = dy w, n = h r,
//              dx = dh + r (g - n mean(g n)), dw = sum over rows of dy n
//
// dx is the gradient of x and of the residual alike.  Bound by HBM, and built
// like the layer norm: `LPR` lanes hold a row in registers, NV pieces of a
// vector of x each, so every operand is read once, and the next row's loads are
// on their way while one is worked on.  bf16, 65536 x 1024: forward with the rows
// in 8 bits too 120 us (606 MB, 5.1 TB/s), backward with dh 102 + 5 us (537 MB, 5.3
// TB/s); fp16 beside an fp32 stream, 8191 x 4096: 85 us (403 MB, 4.7 TB/s).  One
// row: 4.7 us, its call 13.
//
// The forward pass has time for more than fp32 beside its loads: squares are
// summed in fp64 and y carries what its first product leaves out, so rstd and y
// are rounded once, and the codes are those of the exact rows (in fp32 alone: 120
// us against 121, 83 against 85; one of some 10^5 codes differs).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cfloat>

#include "elem.h"
#include "layer_ops.h"
#include "rows.h"

namespace adasum {
namespace {

// A lane's piece of a row of R: N values, N that of another type's vector.
template <typename R, int N>
struct Piece {
  static constexpr int K = Type<R>::kVec;
  v4u raw[N / K];
  __device__ __forceinline__ void load(const R* p, int valid) {
#pragma unroll
    for (int q = 0; q < N / K; ++q) raw[q] = load_raw(p + q * K, valid - q * K);
  }
  __device__ __forceinline__ void values(float (&v)[N]) const {
#pragma unroll
    for (int q = 0; q < N / K; ++q) {
      float t[K];
      widen<R>(raw[q], t);
#pragma unroll
      for (int i = 0; i < K; ++i) v[q * K + i] = t[i];
    }
  }
};

// v as an fp32 number: gfx950 can round a product straight to fp16, which the
// compiler uses here and there, and y would differ with the place of a row.
__device__ __forceinline__ float rounded(float v) {
  asm("" : "+v"(v));
  return v;
}

// v (r + rest) w, rounded once: what the first product leaves out is added to
// the second, where an infinite w times it must not be of the other sign.
__device__ __forceinline__ float scaled(float v, float r, float rest, float w) {
  const float n = v * r, out = __builtin_fmaf(v, rest, __builtin_fmaf(v, r, -n));
  return __builtin_fmaf(n, w, __builtin_amdgcn_fmed3f(out * w, -FLT_MAX, FLT_MAX));
}

template <typename T, typename R, int LPR, int NV, bool PACK>
__global__ __launch_bounds__(LPR < 256 ? 256 : LPR) void rms_kernel(RmsArgs a) {
  constexpr int VEC = Type<T>::kVec;
  constexpr int ROWS = LPR < 256 ? 256 / LPR : 1;
  __shared__ double lds[2][1][LPR / 64 > 0 ? LPR / 64 : 1];
  const int lane = threadIdx.x & (LPR - 1);
  const int64_t step = (int64_t)gridDim.x * ROWS;
  int64_t r = (int64_t)blockIdx.x * ROWS + threadIdx.x / LPR;
  const int H = a.hidden;
  const double inv_h = 1.0 / (double)H;
  int valid[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) valid[j] = H - (j * LPR + lane) * VEC;
  const T* x = static_cast<const T*>(a.x);
  const R* residual = static_cast<const R*>(a.residual);
  T* y = static_cast<T*>(a.y);
  R* h = static_cast<R*>(a.h);
  const int64_t nb = (H + kScaleBlock - 1) / kScaleBlock;
  Piece<T, VEC> px[NV];
  Piece<R, VEC> pr[NV];
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int j = 0; j < NV; ++j) px[j].load(x + row * a.x_stride + (j * LPR + lane) * VEC, valid[j]);
    if (residual) {
#pragma unroll
      for (int j = 0; j < NV; ++j) pr[j].load(residual + row * a.residual_stride + (j * LPR + lane) * VEC, valid[j]);
    }
  };
  if (r < a.rows) fetch(r);
  float w[NV][VEC];
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      w[j][i] = i < valid[j] ? (a.weight ? load_any(a.weight, a.param_dtype, (j * LPR + lane) * VEC + i) : 1.f) : 0.f;
  int slot = 0;
  for (; r < a.rows; r += step) {
    float v[NV][VEC];
#pragma unroll
    for (int j = 0; j < NV; ++j) px[j].values(v[j]);
    if (residual) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float t[VEC];
        pr[j].values(t);
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[j][i] = (float)(R)(v[j][i] + t[i]);
        if (h) store_row<R, VEC>(h + r * a.h_stride + (j * LPR + lane) * VEC, v[j], valid[j]);
      }
    }
    if (r + step < a.rows) fetch(r + step);  // in flight behind this row's arithmetic
    double s[1] = {0.0}, odd = 0.0;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < VEC; i += 2) {  // zeros outside the row
        s[0] = __builtin_fma((double)v[j][i], (double)v[j][i], s[0]);
        odd = __builtin_fma((double)v[j][i + 1], (double)v[j][i + 1], odd);
      }
    s[0] += odd;
    row_sum<LPR, 1>(s, lds, slot);
    slot ^= 1;
    // rstd + rest: the estimate's Newton step in fp64 (a sum above fp32's range: 0)
    const double mean = s[0] * inv_h + (double)a.eps;
    const float near = inverse_root(s[0] > (double)FLT_MAX ? __builtin_inff() : (float)mean);
    const double root = __builtin_fma(0.5 * near, __builtin_fma(-mean * near, (double)near, 1.0), (double)near);
    const bool some = near != 0.f;
    const float rstd = some ? (float)root : near, rest = some ? (float)(root - (double)rstd) : 0.f;
    if (lane == 0) a.rstd[r] = rstd;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * LPR + lane) * VEC;
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[j][i] = i < valid[j] ? rounded(scaled(v[j][i], rstd, rest, w[j][i])) : 0.f;
      if (y) store_vec(y + r * a.y_stride + c, v[j], valid[j]);
      if constexpr (PACK) {
        // the codes are those of y as it is stored
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[j][i] = (float)(T)v[j][i];
        pack_vec<VEC>(v[j], valid[j], __is_same(T, _Float16) ? 136u : 248u, lane, a.codes + r * H + c,
                      a.scales + r * nb + c / kScaleBlock);
      }
    }
  }
}

template <typename T, typename R, int LPR, int NV>
__global__ __launch_bounds__(LPR < 256 ? 256 : LPR) void rms_grad_kernel(RmsGradArgs a) {
  constexpr int VEC = Type<T>::kVec;
  constexpr int ROWS = LPR < 256 ? 256 / LPR : 1;
  __shared__ float lds[2][1][LPR / 64 > 0 ? LPR / 64 : 1];
  const int lane = threadIdx.x & (LPR - 1);
  const int64_t step = (int64_t)gridDim.x * ROWS;
  int64_t r = (int64_t)blockIdx.x * ROWS + threadIdx.x / LPR;
  const int H = a.hidden;
  const float inv_h = 1.f / (float)H;
  int valid[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) valid[j] = H - (j * LPR + lane) * VEC;
  const T* dy = static_cast<const T*>(a.dy);
  const R* h = static_cast<const R*>(a.h);
  const R* dh = static_cast<const R*>(a.dh);
  R* dx = static_cast<R*>(a.dx);
  Piece<T, VEC> py[NV];
  Piece<R, VEC> ph[NV], pd[NV];
  float rstd = 0.f;
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * LPR + lane) * VEC;
      py[j].load(dy + row * a.dy_stride + c, valid[j]);
      ph[j].load(h + row * a.h_stride + c, valid[j]);
    }
    if (dh) {
#pragma unroll
      for (int j = 0; j < NV; ++j) pd[j].load(dh + row * a.dh_stride + (j * LPR + lane) * VEC, valid[j]);
    }
    rstd = a.rstd[row];
  };
  if (r < a.rows) fetch(r);
  // 1024 lanes have 128 registers each: there the weights lie in LDS, every
  // lane its own
  constexpr bool LDS_W = LPR == 1024;
  __shared__ float far[LDS_W ? NV * LPR * VEC : 1];
  float w[LDS_W ? 1 : NV][VEC], aw[NV][VEC];
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
    }
  int slot = 0;
  for (; r < a.rows; r += step) {
    float g[NV][VEC], n[NV][VEC], d[NV][VEC];
    const float rs = rstd;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      py[j].values(g[j]);
      ph[j].values(n[j]);
      if (dh) pd[j].values(d[j]);
    }
    if (r + step < a.rows) fetch(r + step);
    float s[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        n[j][i] *= rs;
        aw[j][i] = __builtin_fmaf(g[j][i], n[j][i], aw[j][i]);
        g[j][i] *= LDS_W ? far[LDS_W ? (j * LPR + lane) * VEC + i : 0] : w[LDS_W ? 0 : j][i];
        s[0] = __builtin_fmaf(g[j][i], n[j][i], s[0]);
      }
    row_sum<LPR, 1>(s, lds, slot);
    slot ^= 1;
    const float m = s[0] * inv_h;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        g[j][i] = __builtin_fmaf(-n[j][i], m, g[j][i]) * rs;
        if (dh) g[j][i] += d[j][i];
      }
      store_row<R, VEC>(dx + r * a.dx_stride + (j * LPR + lane) * VEC, g[j], valid[j]);
    }
  }
  if (a.partials == nullptr) return;
  // the workgroup's sums: its waves' added in wave order through LDS
  float* out = a.partials + (int64_t)blockIdx.x * H;
  if constexpr (LPR <= 64) {
    __shared__ float part[3][LPR * VEC];
    const int wave = threadIdx.x >> 6;
    if constexpr (LPR == 16) {  // the wave's four rows first
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i)
#pragma unroll
          for (int e = 16; e < 64; e *= 2) aw[j][i] += __shfl_xor(aw[j][i], e);
    }
    const bool first = (threadIdx.x & 63) < LPR;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (j > 0) __syncthreads();
      if (wave > 0 && first) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) part[wave - 1][i * LPR + lane] = aw[j][i];
      }
      __syncthreads();
      if (wave == 0 && first) {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
#pragma unroll
          for (int q = 0; q < 3; ++q) aw[j][i] += part[q][i * LPR + lane];
        store_row<float, VEC>(out + (j * LPR + lane) * VEC, aw[j], valid[j]);
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j) store_row<float, VEC>(out + (j * LPR + lane) * VEC, aw[j], valid[j]);
  }
}

template <typename T, typename R, int LPR, int NV>
hipError_t rms_launch(const RmsArgs& a, hipStream_t st) {
  constexpr int ROWS = LPR < 256 ? 256 / LPR : 1;
  constexpr int THREADS = LPR < 256 ? 256 : LPR;
  // eight waves per SIMD's worth of workgroups at most: each then walks
  // several rows with the weights in registers
  const int64_t blocks = std::min<int64_t>(ceil_div(a.rows, ROWS), (int64_t)kCUs * 2048 / THREADS);
  if (a.codes)
    rms_kernel<T, R, LPR, NV, true><<<(unsigned)blocks, THREADS, 0, st>>>(a);
  else
    rms_kernel<T, R, LPR, NV, false><<<(unsigned)blocks, THREADS, 0, st>>>(a);
  return hipGetLastError();
}

// Lanes per row and pieces per lane: at most 16 values a lane.
template <typename T, typename R>
hipError_t rms_width(const RmsArgs& a, hipStream_t st) {
  constexpr int VEC = Type<T>::kVec, NV = 16 / VEC;
  const int64_t pieces = ceil_div(a.hidden, VEC);
  if (pieces <= 16 * NV / 2) return rms_launch<T, R, 16, NV / 2>(a, st);
  if (pieces <= 16 * NV) return rms_launch<T, R, 16, NV>(a, st);
  if (pieces <= 64 * NV / 2) return rms_launch<T, R, 64, NV / 2>(a, st);
  if (pieces <= 64 * NV) return rms_launch<T, R, 64, NV>(a, st);
  if (pieces <= 256 * NV / 2) return rms_launch<T, R, 256, NV / 2>(a, st);
  if (pieces <= 256 * NV) return rms_launch<T, R, 256, NV>(a, st);
  if (pieces <= 1024 * NV / 2) return rms_launch<T, R, 1024, NV / 2>(a, st);
  return rms_launch<T, R, 1024, NV>(a, st);
}

struct RmsGradShape {
  int lanes, threads, rows;
};
RmsGradShape rms_grad_shape(int hidden) {
  if (hidden <= 16 * 16) return {16, 256, 16};
  if (hidden <= 64 * 16) return {64, 256, 4};
  if (hidden <= 256 * 16) return {256, 256, 1};
  return {1024, 1024, 1};
}

template <typename T, typename R, int LPR, int NV>
hipError_t rms_grad_launch(const RmsGradArgs& a, int blocks, hipStream_t st) {
  constexpr int THREADS = LPR < 256 ? 256 : LPR;
  rms_grad_kernel<T, R, LPR, NV><<<blocks, THREADS, 0, st>>>(a);
  return hipGetLastError();
}

template <typename T, typename R>
hipError_t rms_grad_width(const RmsGradArgs& a, int lanes, int blocks, hipStream_t st) {
  constexpr int NV = 16 / Type<T>::kVec;
  const bool half = ceil_div(a.hidden, Type<T>::kVec) <= (int64_t)lanes * NV / 2;
  if (lanes == 16)
    return half ? rms_grad_launch<T, R, 16, NV / 2>(a, blocks, st) : rms_grad_launch<T, R, 16, NV>(a, blocks, st);
  if (lanes == 64)
    return half ? rms_grad_launch<T, R, 64, NV / 2>(a, blocks, st) : rms_grad_launch<T, R, 64, NV>(a, blocks, st);
  if (lanes == 256)
    return half ? rms_grad_launch<T, R, 256, NV / 2>(a, blocks, st) : rms_grad_launch<T, R, 256, NV>(a, blocks, st);
  return half ? rms_grad_launch<T, R, 1024, NV / 2>(a, blocks, st) : rms_grad_launch<T, R, 1024, NV>(a, blocks, st);
}

// f(x's type, the stream's type): the stream is fp32 or of x's type.
template <typename F>
hipError_t with_stream(int dtype, int stream_dtype, F f) {
  return with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    if constexpr (sizeof(T) == 4) {
      return f(t, t);
    } else {
      return stream_dtype == 0 ? f(t, float()) : f(t, t);
    }
  });
}

// Workgroups of one launch over `rows`: two of 256 lanes per CU, or as many
// waves in wider ones, but one per CU at least; and no more than leaves a wave
// four rows, or 16 lanes two, since every workgroup leaves a row of partial
// sums for the join.
int rms_grad_blocks(int64_t rows, const RmsGradShape& s) {
  return (int)std::min<int64_t>(ceil_div(rows, s.rows * (s.lanes == 16 ? 2 : 4)),
                                std::max<int64_t>(kCUs, (int64_t)kCUs * 512 / s.threads));
}

// Rows of one launch: as many as leave the fp32 sums of dweight kNormGradRows
// long in a full one.
int64_t rms_grad_rows(const RmsGradShape& s) {
  return (int64_t)rms_grad_blocks(kMaxDim, s) * s.rows * kNormGradRows;
}

}  // namespace

hipError_t launch_rms(int dtype, int stream_dtype, const RmsArgs& a, hipStream_t st) {
  return with_stream(dtype, stream_dtype, [&](auto t, auto r) { return rms_width<decltype(t), decltype(r)>(a, st); });
}

int64_t rms_grad_parts(int64_t rows, int hidden) {
  const RmsGradShape s = rms_grad_shape(hidden);
  const int64_t full = rms_grad_rows(s);
  return rows / full * rms_grad_blocks(full, s) + rms_grad_blocks(rows % full, s);
}

hipError_t launch_rms_grad(int dtype, int stream_dtype, const RmsGradArgs& a, hipStream_t st) {
  const RmsGradShape s = rms_grad_shape(a.hidden);
  const int64_t full = rms_grad_rows(s), size = dtype == 0 ? 4 : 2, wide = stream_dtype == 0 ? 4 : 2;
  int64_t parts = 0;
  for (int64_t first = 0; first < a.rows; first += full) {
    RmsGradArgs b = a;
    b.rows = std::min(full, a.rows - first);
    b.dy = static_cast<const char*>(a.dy) + first * a.dy_stride * size;
    b.h = static_cast<const char*>(a.h) + first * a.h_stride * wide;
    if (a.dh) b.dh = static_cast<const char*>(a.dh) + first * a.dh_stride * wide;
    b.dx = static_cast<char*>(a.dx) + first * a.dx_stride * wide;
    b.rstd = a.rstd + first;
    if (a.partials) b.partials = a.partials + parts * a.hidden;
    const int blocks = rms_grad_blocks(b.rows, s);
    parts += blocks;
    const hipError_t e = with_stream(dtype, stream_dtype, [&](auto t, auto r) {
      return rms_grad_width<decltype(t), decltype(r)>(b, s.lanes, blocks, st);
    });
    if (e != hipSuccess) return e;
  }
  if (a.dweight == nullptr) return hipSuccess;
  join_columns_kernel<<<(unsigned)ceil_div(a.hidden, 32), 256, 0, st>>>(a.partials, (int)parts, (int64_t)a.hidden,
                                                                      a.dweight, (int64_t)a.hidden, nullptr,
                                                                      a.grad_dtype, a.accumulate);
  return hipGetLastError();
}

}  // namespace adasum
