// orthogonal.hip - an update's matrices made orthogonal by Newton-Schulz
// products: with X the matrix over its Frobenius norm, rows <= columns (else
// its transpose),
//
//   A = X X^T,  B = b A + c A A,  X <- a X + B X      steps times
//
// which takes every singular value s to a s + b s^3 + c s^5.  Bound by the
// matrix cores.
//
// Products take fp16 operands and sum in fp32.  X is kept as hi + lo, two fp16
// of 22 bits together, and a X is added in fp32 from both: rounding X itself to
// 16 bits would put noise into the directions of small singular values, which
// the steps then raise as if it were signal (a matrix of rank 8: 4e-2 of the
// result's norm; with hi + lo 4e-4).  What an operand of a product loses is
// scaled down by the product.  Of bf16 results (PARTS 1) the products take the
// hi parts only: off by 1.4e-3 of the norm for normally distributed matrices,
// where the rounding of the result itself costs 1.7e-3.  B's diagonal, its
// largest values, is kept in fp32 beside its fp16 copy (without: 1.7e-3).
// fp16 and fp32 results (PARTS 2) take hi hi + hi lo + lo hi: off by less than
// products in fp32 are.
//
// Values are scaled by powers of two so that neither part leaves fp16's normal
// range: the host admits coefficients only that keep singular values below 2
// and B below 31.
//
// Everything is padded with zeros to whole tiles in the workspace, so the
// products have no edges.  X and its transpose are both kept: each product then
// takes rows of both operands along the sum.  A and B are symmetric: half of
// their tiles are computed, and written twice.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "elem.h"
#include "layer_ops.h"

namespace adasum {
namespace {

using namespace elem;

typedef _Float16 v4h __attribute__((ext_vector_type(4)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));

constexpr float kScaleX = 16384.f, kScaleA = 8192.f, kScaleB = 2048.f;
constexpr int kSumParts = 64;  // workgroups that sum a matrix's squares
// bf16 results of sides above this take one part of each operand.  Narrower
// ones are bound by the launches, and in the smallest the roundings of few
// values do not average out (5 x 3: 4.9e-3 of the norm).
constexpr int kOnePartSide = 256;

enum Kind { kGramX, kSquareA, kApplyB };

// A workgroup's tile of T x T, and a wave's part of it.
template <int T>
struct Tile;
template <>
struct Tile<64> {
  static constexpr int kThreads = 256, kWavesP = 2, kWavesQ = 2;
};
template <>
struct Tile<128> {
  static constexpr int kThreads = 256, kWavesP = 2, kWavesQ = 2;
};
template <>
struct Tile<256> {
  static constexpr int kThreads = 512, kWavesP = 2, kWavesQ = 4;
};

__device__ __forceinline__ void split(float v, _Float16* hi, _Float16* lo) {
  *hi = (_Float16)v;
  *lo = (_Float16)(v - (float)*hi);
}

// ---------------------------------------------------------------- norm and first X

// Squares in fp64: neither over- nor underflow, whatever the update's scale.
template <typename T>
__global__ __launch_bounds__(256) void square_sum_kernel(OrthoArgs a, OrthoLayout l) {
  constexpr int VEC = Type<T>::kVec;
  const int64_t per_row = (a.cols + VEC - 1) / VEC, total = a.rows * per_row;
  const T* x = static_cast<const T*>(a.x[blockIdx.y]);
  double s = 0.0;
  for (int64_t p = (int64_t)blockIdx.x * 256 + threadIdx.x; p < total; p += kSumParts * 256) {
    const int64_t r = p / per_row, c = (p - r * per_row) * VEC;
    float v[VEC];
    widen<T>(load_raw(x + r * a.x_stride + c, (int)min<int64_t>(a.cols - c, VEC)), v);
#pragma unroll
    for (int i = 0; i < VEC; ++i) s = __builtin_fma((double)v[i], (double)v[i], s);
  }
  __shared__ double sums[256];
  sums[threadIdx.x] = s;
  __syncthreads();
  for (int w = 128; w > 0; w /= 2) {
    if ((int)threadIdx.x < w) sums[threadIdx.x] += sums[threadIdx.x + w];
    __syncthreads();
  }
  if (threadIdx.x == 0) reinterpret_cast<double*>(a.ws + blockIdx.y * l.per_matrix + l.sums)[blockIdx.x] = sums[0];
}

// X and its transpose, 64 x 64 values a workgroup.
template <typename T, int PARTS>
__global__ __launch_bounds__(256) void first_kernel(OrthoArgs a, OrthoLayout l) {
  __shared__ float tile[64][65];
  __shared__ double factor;
  char* ws = a.ws + blockIdx.y * l.per_matrix;
  if (threadIdx.x == 0) {
    const double* sums = reinterpret_cast<const double*>(ws + l.sums);
    double s = 0.0;
    for (int i = 0; i < kSumParts; ++i) s += sums[i];
    factor = (double)kScaleX / (sqrt(s) + a.eps);
  }
  __syncthreads();
  const double f = factor;
  const int64_t tiles_m = l.m / 64, ti = blockIdx.x / tiles_m, tk = blockIdx.x - ti * tiles_m;
  const int64_t i0 = ti * 64, k0 = tk * 64;
  const T* x = static_cast<const T*>(a.x[blockIdx.y]);
  const bool tall = a.rows > a.cols;
  const int fast = threadIdx.x & 63, slow = threadIdx.x >> 6;
  for (int s = slow; s < 64; s += 4) {
    // rows of the matrix as it lies: along k, or along i where it is tall
    const int64_t r = (tall ? k0 : i0) + s, c = (tall ? i0 : k0) + fast;
    float v = 0.f;
    if (r < a.rows && c < a.cols) v = (float)((double)(float)x[r * a.x_stride + c] * f);
    if (tall)
      tile[fast][s] = v;
    else
      tile[s][fast] = v;
  }
  __syncthreads();
  _Float16* xh = reinterpret_cast<_Float16*>(ws + l.x[0]);
  _Float16* xl = reinterpret_cast<_Float16*>(ws + l.x[1]);
  _Float16* th = reinterpret_cast<_Float16*>(ws + l.xt[0][0]);
  _Float16* tl = reinterpret_cast<_Float16*>(ws + l.xt[0][1]);
  for (int s = slow; s < 64; s += 4) {
    _Float16 hi, lo;
    split(tile[s][fast], &hi, &lo);
    const int64_t at = (i0 + s) * l.m + k0 + fast;
    xh[at] = hi;
    xl[at] = lo;
    split(tile[fast][s], &hi, &lo);
    const int64_t turned = (k0 + s) * l.n + i0 + fast;
    th[turned] = hi;
    if constexpr (PARTS == 2) tl[turned] = lo;
  }
}

// ---------------------------------------------------------------- products

constexpr int kLoadsDone = 0x0f70;  // wait for all loads, and for nothing else

typedef __attribute__((address_space(1))) const void* global_pointer;
typedef __attribute__((address_space(3))) void* lds_pointer;

// C = P Q^T over rows of P and Q of `ld` values: a tile of T x T, its sums over
// kStep values at a time.  The loads go straight to LDS, one step ahead; 16-byte
// pieces are permuted within a row by the row's number, so that 16 lanes that
// read the same piece of 16 rows find them in different banks.
template <int KIND, int PARTS, int T>
__global__ __launch_bounds__(Tile<T>::kThreads) void product_kernel(OrthoArgs a, OrthoLayout l, OrthoStep step) {
  constexpr int kWaves = Tile<T>::kThreads / 64;
  constexpr int WP = T / Tile<T>::kWavesP, WQ = T / Tile<T>::kWavesQ, MP = WP / 16, MQ = WQ / 16;
  constexpr int kStep = T == 256 && PARTS == 2 ? 32 : 64, kChunks = kStep / 8;
  constexpr int kKeyShift = kChunks == 8 ? 1 : 2;
  // operands of a buffer: P's parts, then Q's
  __shared__ v4u lds[2][2 * PARTS][T * kChunks];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  char* ws = a.ws + blockIdx.y * l.per_matrix;
  // tiles of the upper triangle, row by row, or all
  int64_t tp, tq;
  if constexpr (KIND == kApplyB) {
    const int64_t across = l.m / T;
    tp = blockIdx.x / across;
    tq = blockIdx.x - tp * across;
  } else {
    int64_t rest = blockIdx.x, width = l.n / T;
    tp = 0;
    while (rest >= width) {
      rest -= width;
      --width;
      ++tp;
    }
    tq = tp + rest;
  }
  const int64_t p0 = tp * T, q0 = tq * T;
  const int64_t ld = KIND == kGramX ? l.m : l.n;
  const _Float16* operand[2 * PARTS];
#pragma unroll
  for (int h = 0; h < PARTS; ++h) {
    const size_t p = KIND == kGramX ? l.x[h] : KIND == kSquareA ? l.a[h] : l.b[h];
    const size_t q = KIND == kGramX ? l.x[h] : KIND == kSquareA ? l.a[h] : l.xt[step.from][h];
    operand[h] = reinterpret_cast<const _Float16*>(ws + p) + p0 * ld;
    operand[PARTS + h] = reinterpret_cast<const _Float16*>(ws + q) + q0 * ld;
  }
  // A wave fills 64 consecutive pieces of an operand at a time: this lane's
  // row among them and the piece of that row which belongs there.
  constexpr int kRowsAtOnce = 64 / kChunks, kFills = T * kChunks / 64 / kWaves;
  static_assert(kFills * kWaves * 64 == T * kChunks, "whole waves");
  const int in_row = lane / kChunks;
  auto fetch = [&](int buffer, int64_t k0) __attribute__((always_inline)) {
#pragma unroll
    for (int o = 0; o < 2 * PARTS; ++o)
#pragma unroll
      for (int f = 0; f < kFills; ++f) {
        const int first = (f * kWaves + wave) * kRowsAtOnce, row = first + in_row;
        const int piece = (lane % kChunks) ^ ((row >> kKeyShift) & (kChunks - 1));
        __builtin_amdgcn_global_load_lds((global_pointer)(operand[o] + row * ld + k0 + piece * 8),
                                         (lds_pointer)&lds[buffer][o][first * kChunks], 16, 0, 0);
      }
  };
  const int wp = (wave / Tile<T>::kWavesQ) * WP, wq = (wave % Tile<T>::kWavesQ) * WQ;
  auto read = [&](int buffer, int o, int row, int half) __attribute__((always_inline)) {
    row += lane & 15;
    const int piece = (half * 4 + (lane >> 4)) ^ ((row >> kKeyShift) & (kChunks - 1));
    return __builtin_bit_cast(v8h, lds[buffer][o][row * kChunks + piece]);
  };
  v4f acc[MP][MQ];
#pragma unroll
  for (int i = 0; i < MP; ++i)
#pragma unroll
    for (int j = 0; j < MQ; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  const int64_t steps = ld / kStep;
  fetch(0, 0);
  for (int64_t t = 0; t < steps; ++t) {
    const int buffer = (int)(t & 1);
    // this step's loads have arrived, everyone's; and everyone has read the
    // other buffer
    __builtin_amdgcn_s_waitcnt(kLoadsDone);
    __syncthreads();
    if (t + 1 < steps) fetch(buffer ^ 1, (t + 1) * kStep);
#pragma unroll
    for (int half = 0; half < kStep / 32; ++half) {
      v8h fp[PARTS][MP], fq[PARTS][MQ];
#pragma unroll
      for (int h = 0; h < PARTS; ++h) {
#pragma unroll
        for (int i = 0; i < MP; ++i) fp[h][i] = read(buffer, h, wp + i * 16, half);
#pragma unroll
        for (int j = 0; j < MQ; ++j) fq[h][j] = read(buffer, PARTS + h, wq + j * 16, half);
      }
#pragma unroll
      for (int i = 0; i < MP; ++i)
#pragma unroll
        for (int j = 0; j < MQ; ++j) {
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(fq[0][j], fp[0][i], acc[i][j], 0, 0, 0);
          if constexpr (PARTS == 2) {
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(fq[1][j], fp[0][i], acc[i][j], 0, 0, 0);
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(fq[0][j], fp[1][i], acc[i][j], 0, 0, 0);
          }
        }
    }
  }

  // a lane: four consecutive columns q of row p
#pragma unroll
  for (int i = 0; i < MP; ++i)
#pragma unroll
    for (int j = 0; j < MQ; ++j) {
      const int64_t p = p0 + wp + i * 16 + (lane & 15), q = q0 + wq + j * 16 + (lane >> 4) * 4;
      float v[4];
      if constexpr (KIND == kGramX) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = acc[i][j][e] * (kScaleA / (kScaleX * kScaleX));
      } else if constexpr (KIND == kSquareA) {
        const v4h hi = *reinterpret_cast<const v4h*>(ws + l.a[0] + (p * l.n + q) * 2);
        v4h lo = {};
        if constexpr (PARTS == 2) lo = *reinterpret_cast<const v4h*>(ws + l.a[1] + (p * l.n + q) * 2);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float one = ((float)hi[e] + (float)lo[e]) * (kScaleB / kScaleA);
          v[e] = __builtin_fmaf(step.c, acc[i][j][e] * (kScaleB / (kScaleA * kScaleA)), step.b * one);
        }
        if constexpr (PARTS == 1) {  // what fp16 leaves out of the diagonal
          float* rest = reinterpret_cast<float*>(ws + l.rest);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (p == q + e) rest[p] = (v[e] - (float)(_Float16)v[e]) * (1.f / kScaleB);
        }
      } else {
        const v4h hi = *reinterpret_cast<const v4h*>(ws + l.x[0] + (p * l.m + q) * 2);
        const v4h lo = *reinterpret_cast<const v4h*>(ws + l.x[1] + (p * l.m + q) * 2);
        float f = step.a;
        if constexpr (PARTS == 1) f += reinterpret_cast<const float*>(ws + l.rest)[p];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = __builtin_fmaf(f, (float)hi[e] + (float)lo[e], acc[i][j][e] * (1.f / kScaleB));
      }
      if (KIND == kApplyB && step.last) {
        const bool tall = a.rows > a.cols;
        const int64_t n = tall ? a.cols : a.rows, m = tall ? a.rows : a.cols;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (p < n && q + e < m) {
            const int64_t at = tall ? (q + e) * a.out_stride + p : p * a.out_stride + q + e;
            const float r = v[e] * (1.f / kScaleX) * a.scale;
            void* out = a.out[blockIdx.y];
            if (a.out_dtype == 0)
              static_cast<float*>(out)[at] = r;
            else if (a.out_dtype == 1)
              static_cast<_Float16*>(out)[at] = (_Float16)r;
            else
              static_cast<__bf16*>(out)[at] = (__bf16)r;
          }
        continue;
      }
      v4h hi, lo;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        _Float16 h, r;
        split(v[e], &h, &r);
        hi[e] = h;
        lo[e] = r;
      }
      // the tile, and for A and B its mirror image, for X the transpose
      const size_t* whole = KIND == kGramX ? l.a : KIND == kSquareA ? l.b : l.x;
      const size_t* mirror = KIND == kApplyB ? l.xt[step.from ^ 1] : whole;
      const int64_t width = KIND == kApplyB ? l.m : l.n;
      *reinterpret_cast<v4h*>(ws + whole[0] + (p * width + q) * 2) = hi;
      if (PARTS == 2 || KIND == kApplyB) *reinterpret_cast<v4h*>(ws + whole[1] + (p * width + q) * 2) = lo;
      if (KIND == kApplyB || tp != tq) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          reinterpret_cast<_Float16*>(ws + mirror[0])[(q + e) * l.n + p] = hi[e];
          if constexpr (PARTS == 2) reinterpret_cast<_Float16*>(ws + mirror[1])[(q + e) * l.n + p] = lo[e];
        }
      }
    }
}

size_t align256(size_t b) { return (b + 255) & ~size_t(255); }

template <int PARTS, int T>
hipError_t steps_of(const OrthoArgs& a, const OrthoLayout& l, int count, hipStream_t st) {
  const unsigned side = (unsigned)(l.n / T), triangle = side * (side + 1) / 2, all = side * (unsigned)(l.m / T);
  constexpr int kThreads = Tile<T>::kThreads;
  for (int s = 0; s < a.steps; ++s) {
    const OrthoStep step{a.coefficients[3 * s], a.coefficients[3 * s + 1], a.coefficients[3 * s + 2], s & 1,
                         s + 1 == a.steps};
    product_kernel<kGramX, PARTS, T><<<dim3(triangle, count), kThreads, 0, st>>>(a, l, step);
    product_kernel<kSquareA, PARTS, T><<<dim3(triangle, count), kThreads, 0, st>>>(a, l, step);
    product_kernel<kApplyB, PARTS, T><<<dim3(all, count), kThreads, 0, st>>>(a, l, step);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

OrthoLayout ortho_layout(int64_t count, int64_t rows, int64_t cols, int out_dtype) {
  OrthoLayout l{};
  const int64_t n = std::min(rows, cols), m = std::max(rows, cols);
  l.parts = out_dtype == 2 && n > kOnePartSide ? 1 : 2;
  l.tile = 128;
  l.n = ceil_div(n, l.tile) * l.tile;
  l.m = ceil_div(m, l.tile) * l.tile;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += align256(bytes);
    return here;
  };
  const size_t x = (size_t)l.n * l.m * 2, s = (size_t)l.n * l.n * 2;
  l.x[0] = take(x);
  l.x[1] = take(x);
  for (int h = 0; h < l.parts; ++h) {
    l.xt[0][h] = take(x);
    l.xt[1][h] = take(x);
    l.a[h] = take(s);
    l.b[h] = take(s);
  }
  l.rest = take((size_t)l.n * 4);
  l.sums = take(kSumParts * 8);
  l.per_matrix = at;
  l.together = (int)std::min<int64_t>(count, kOrthoTogether);
  l.total = at * l.together;
  return l;
}

hipError_t launch_ortho(int dtype, const OrthoCall& call, hipStream_t st) {
  const OrthoLayout l = ortho_layout(call.count, call.args.rows, call.args.cols, call.args.out_dtype);
  for (int64_t first = 0; first < call.count; first += l.together) {
    OrthoArgs a = call.args;
    const int count = (int)std::min<int64_t>(l.together, call.count - first);
    for (int i = 0; i < count; ++i) {
      a.x[i] = call.x[first + i];
      a.out[i] = call.out[first + i];
    }
    hipError_t e = with_dtype(dtype, [&](auto t) {
      using T = decltype(t);
      const dim3 tiles((unsigned)(l.n / 64 * (l.m / 64)), count);
      square_sum_kernel<T><<<dim3(kSumParts, count), 256, 0, st>>>(a, l);
      if (l.parts == 1)
        first_kernel<T, 1><<<tiles, 256, 0, st>>>(a, l);
      else
        first_kernel<T, 2><<<tiles, 256, 0, st>>>(a, l);
      return hipGetLastError();
    });
    if (e == hipSuccess) e = l.parts == 1 ? steps_of<1, 128>(a, l, count, st) : steps_of<2, 128>(a, l, count, st);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace adasum
