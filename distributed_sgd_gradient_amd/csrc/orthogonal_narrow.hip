// orthogonal_narrow.hip - orthogonal updates of matrices with a side of at most
// 64 (see orthogonal.hip for the steps).
//
// Every X of the steps is a polynomial in G = X0 X0^T times X0, so narrow
// matrices take their steps on G alone: with P = a I + b G + c G G,
//
//   Q <- P Q,  G <- P G P      steps times;   result Q X0
//
// All of these commute and are symmetric, so half of their tiles are computed.
// G holds the squares of the singular values, so everything is in fp64, where
// those that fp32 can tell from zero keep their digits.  Three launches instead
// of three a step: partial sums of G over the long side, the steps in one
// workgroup a matrix on the fp64 matrix cores, and the product with X0.  Bound by
// the latency of the steps: 17 products of 64 x 64 one after another.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "elem.h"
#include "layer_ops.h"

namespace adasum {
namespace {

using namespace elem;

typedef double v4d __attribute__((ext_vector_type(4)));

constexpr int kSide = kOrthoNarrow, kChunk = 64;  // columns of X at a time
constexpr int kPitch = kSide + 2;                 // of a matrix in LDS, in doubles
constexpr int kThreads = 640, kWaves = kThreads / 64;  // a wave for each tile on or above the diagonal
constexpr int kTilesOfWave = 1;
static_assert(kTilesOfWave * kWaves >= 10, "all tiles of 64 x 64");

// 64 columns from k0 on of X (the shorter side being its rows) as tile[k][i];
// zeros outside.  All of a lane's loads are on their way before the first is
// used.
template <typename T>
__device__ __forceinline__ void load_chunk(const OrthoArgs& a, int matrix, int64_t k0, float (*tile)[kSide + 4]) {
  const T* x = static_cast<const T*>(a.x[matrix]);
  const bool tall = a.rows > a.cols;
  const int fast = threadIdx.x & 63, slow = threadIdx.x >> 6;
  T v[16];
#pragma unroll
  for (int u = 0; u < 16; ++u) {
    // a place outside reads the last row or column
    const int64_t r = min(tall ? k0 + slow + 4 * u : slow + 4 * u, a.rows - 1);
    const int64_t c = min(tall ? fast : k0 + fast, a.cols - 1);
    v[u] = x[r * a.x_stride + c];
  }
#pragma unroll
  for (int u = 0; u < 16; ++u) {
    const int s = slow + 4 * u;
    const bool there = tall ? k0 + s < a.rows && fast < a.cols : s < a.rows && k0 + fast < a.cols;
    (tall ? tile[s][fast] : tile[fast][s]) = there ? (float)v[u] : 0.f;
  }
}

// A part of G: products of fp32 values are exact in fp64.
template <typename T>
__global__ __launch_bounds__(256) void narrow_gram_kernel(OrthoArgs a, OrthoLayout l) {
  __shared__ float tile[kChunk][kSide + 4];
  const int i0 = (threadIdx.x >> 4) * 4, j0 = (threadIdx.x & 15) * 4;
  const int64_t m = max(a.rows, a.cols);
  double acc[4][4] = {};
  for (int64_t k0 = (int64_t)blockIdx.x * kChunk; k0 < m; k0 += (int64_t)l.splits * kChunk) {
    load_chunk<T>(a, blockIdx.y, k0, tile);
    __syncthreads();
#pragma unroll 4
    for (int k = 0; k < kChunk; ++k) {
      double u[4], v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        u[e] = tile[k][i0 + e];
        v[e] = tile[k][j0 + e];
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int f = 0; f < 4; ++f) acc[e][f] = __builtin_fma(u[e], v[f], acc[e][f]);
    }
    __syncthreads();
  }
  double* out = reinterpret_cast<double*>(a.ws + blockIdx.y * l.per_matrix + l.partials) + blockIdx.x * kSide * kSide;
#pragma unroll
  for (int e = 0; e < 4; ++e)
#pragma unroll
    for (int f = 0; f < 4; ++f) out[(i0 + e) * kSide + j0 + f] = acc[e][f];
}

// A tile of 16 x 16 of A B, of symmetric matrices that commute, `side` wide:
// tile t of those on and above the diagonal, row by row.
struct Place {
  int i, j;  // of the tile
};
__device__ __forceinline__ Place place_of(int t, int blocks) {
  int i = 0;
  while (t >= blocks - i) {
    t -= blocks - i;
    ++i;
  }
  return {i * 16, (i + t) * 16};
}
__device__ __forceinline__ v4d tile_product(const double* a, const double* b, Place at, int side) {
  const int lane = threadIdx.x & 63;
  const double* u = a + (at.i + (lane & 15)) * kPitch + (lane >> 4);
  const double* v = b + (at.j + (lane & 15)) * kPitch + (lane >> 4);  // a column of B is its row
  v4d acc[2] = {{0.0, 0.0, 0.0, 0.0}, {0.0, 0.0, 0.0, 0.0}};  // two chains, added at the end
  for (int k = 0; k < side; k += 16)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      acc[e & 1] = __builtin_amdgcn_mfma_f64_16x16x4f64(u[k + 4 * e], v[k + 4 * e], acc[e & 1], 0, 0, 0);
  return acc[0] + acc[1];
}
// f(place in a matrix, value) for the tile's values and their mirror images.
template <typename F>
__device__ __forceinline__ void each_place(Place at, v4d c, F f) {
  const int lane = threadIdx.x & 63, j = at.j + (lane & 15);
#pragma unroll
  for (int r = 0; r < 4; ++r) {  // a lane: rows 4 r + lane / 16 of column lane % 16
    const int i = at.i + 4 * r + (lane >> 4);
    f(i, j, i * kPitch + j, c[r]);
    if (at.i != at.j) f(j, i, j * kPitch + i, c[r]);
  }
}

__global__ __launch_bounds__(kThreads) void narrow_steps_kernel(OrthoArgs a, OrthoLayout l) {
  __shared__ double space[4][kSide * kPitch];
  char* ws = a.ws + blockIdx.x * l.per_matrix;
  const double* parts = reinterpret_cast<const double*>(ws + l.partials);
  const int n = (int)min(a.rows, a.cols), blocks = (n + 15) / 16, side = blocks * 16;
  const int wave = threadIdx.x >> 6, tiles = blocks * (blocks + 1) / 2;
  double *g = space[0], *p = space[1], *q = space[2], *t = space[3];
  constexpr int kOwn = (kSide * kSide + kThreads - 1) / kThreads;  // of a lane
  double sum[kOwn] = {};
  for (int first = 0; first < l.splits; first += 4) {
    double v[kOwn][4];  // parts past the last are read at the last: all loads at once
#pragma unroll
    for (int u = 0; u < kOwn; ++u)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        v[u][k] = parts[(int64_t)min(first + k, l.splits - 1) * kSide * kSide +
                        min((int)threadIdx.x + u * kThreads, kSide * kSide - 1)];
#pragma unroll
    for (int u = 0; u < kOwn; ++u)
#pragma unroll
      for (int k = 0; k < 4; ++k) sum[u] += first + k < l.splits ? v[u][k] : 0.0;
  }
#pragma unroll
  for (int u = 0; u < kOwn; ++u) {
    const int e = threadIdx.x + u * kThreads;
    if (e < kSide * kSide) g[e / kSide * kPitch + e % kSide] = sum[u];
  }
  __syncthreads();
  double squares = 0.0;
#pragma unroll 8
  for (int i = 0; i < n; ++i) squares += g[i * kPitch + i];
  const double f = 1.0 / (sqrt(squares) + a.eps);
  __syncthreads();
  for (int e = threadIdx.x; e < side * side; e += kThreads) g[e / side * kPitch + e % side] *= f * f;
  __syncthreads();
  for (int s = 0; s < a.steps; ++s) {
    const double ca = a.coefficients[3 * s], cb = a.coefficients[3 * s + 1], cc = a.coefficients[3 * s + 2];
    for (int k = wave; k < tiles; k += kWaves) {
      const Place at = place_of(k, blocks);
      each_place(at, tile_product(g, g, at, side), [&](int i, int j, int where, double v) {
        v = cb * g[where] + cc * v + (i == j ? ca : 0.0);
        p[where] = v;
        if (s == 0) q[where] = v;
      });
    }
    __syncthreads();
    if (s == 0) {  // Q = P; T = P G
      if (a.steps == 1) break;
      for (int k = wave; k < tiles; k += kWaves) {
        const Place at = place_of(k, blocks);
        each_place(at, tile_product(p, g, at, side), [&](int, int, int where, double v) { t[where] = v; });
      }
      __syncthreads();
      for (int k = wave; k < tiles; k += kWaves) {
        const Place at = place_of(k, blocks);
        each_place(at, tile_product(t, p, at, side), [&](int, int, int where, double v) { g[where] = v; });
      }
      __syncthreads();
      continue;
    }
    // T = P Q and, but for the last step, P G: each wave keeps its tiles of the
    // latter until everyone has read G
    const bool last = s + 1 == a.steps;
    v4d kept[kTilesOfWave];
#pragma unroll
    for (int u = 0; u < kTilesOfWave; ++u) {
      const int k = wave + u * kWaves;
      if (k < tiles) {
        const Place at = place_of(k, blocks);
        each_place(at, tile_product(p, q, at, side), [&](int, int, int where, double v) { t[where] = v; });
        if (!last) kept[u] = tile_product(p, g, at, side);
      }
    }
    __syncthreads();
    double* const free = q;
    q = t;
    t = free;
    if (last) break;
#pragma unroll
    for (int u = 0; u < kTilesOfWave; ++u) {
      const int k = wave + u * kWaves;
      if (k < tiles) each_place(place_of(k, blocks), kept[u], [&](int, int, int where, double v) { t[where] = v; });
    }
    __syncthreads();
    for (int k = wave; k < tiles; k += kWaves) {
      const Place at = place_of(k, blocks);
      each_place(at, tile_product(t, p, at, side), [&](int, int, int where, double v) { g[where] = v; });
    }
    __syncthreads();
  }
  double* out = reinterpret_cast<double*>(ws + l.rest);
  for (int e = threadIdx.x; e < kSide * kSide; e += kThreads) {
    const int i = e / kSide, j = e % kSide;
    out[e] = i < side && j < side ? q[i * kPitch + j] * (f * (double)a.scale) : 0.0;
  }
}

// Q X: 64 columns a workgroup, 16 rows of a column a lane.
template <typename T>
__global__ __launch_bounds__(256) void narrow_apply_kernel(OrthoArgs a, OrthoLayout l) {
  __shared__ float tile[kChunk][kSide + 4];
  __shared__ double q[kSide][kSide];
  const int64_t k0 = (int64_t)blockIdx.x * kChunk;
  const int n = (int)min(a.rows, a.cols), side = (n + 15) / 16 * 16;
  const int64_t m = max(a.rows, a.cols);
  const double* from = reinterpret_cast<const double*>(a.ws + blockIdx.y * l.per_matrix + l.rest);
  load_chunk<T>(a, blockIdx.y, k0, tile);
  double v[kSide * kSide / 256];
#pragma unroll
  for (int u = 0; u < kSide * kSide / 256; ++u) v[u] = from[u * 256 + threadIdx.x];
#pragma unroll
  for (int u = 0; u < kSide * kSide / 256; ++u) q[(u * 256 + threadIdx.x) / kSide][threadIdx.x % kSide] = v[u];
  __syncthreads();
  const int column = threadIdx.x & 63, i0 = (threadIdx.x >> 6) * 16;
  if (i0 >= side) return;
  double acc[16] = {};
  for (int j = 0; j < n; ++j) {
    const double x = tile[column][j];
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[e] = __builtin_fma(q[j][i0 + e], x, acc[e]);  // Q is symmetric
  }
  if (k0 + column >= m) return;
  const bool tall = a.rows > a.cols;
#pragma unroll
  for (int e = 0; e < 16; ++e)
    if (i0 + e < n)
      store_any(a.out[blockIdx.y], a.out_dtype, tall ? (k0 + column) * a.out_stride + i0 + e
                                                     : (int64_t)(i0 + e) * a.out_stride + k0 + column, acc[e]);
}

}  // namespace

OrthoLayout ortho_narrow_layout(int64_t count, int64_t rows, int64_t cols) {
  OrthoLayout l{};
  l.together = (int)std::min<int64_t>(count, kOrthoTogether);
  // every part is read by one workgroup: no more than 32
  l.splits = (int)std::min<int64_t>(ceil_div(std::max(rows, cols), kChunk), 32);
  l.rest = 0;
  l.partials = kSide * kSide * sizeof(double);
  l.per_matrix = l.partials * (1 + l.splits);
  l.total = l.per_matrix * l.together;
  return l;
}

hipError_t launch_ortho_narrow(int dtype, const OrthoArgs& a, const OrthoLayout& l, int count, hipStream_t st) {
  const unsigned chunks = (unsigned)ceil_div(std::max(a.rows, a.cols), kChunk);
  return with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    narrow_gram_kernel<T><<<dim3((unsigned)l.splits, count), 256, 0, st>>>(a, l);
    narrow_steps_kernel<<<(unsigned)count, kThreads, 0, st>>>(a, l);
    narrow_apply_kernel<T><<<dim3(chunks, count), 256, 0, st>>>(a, l);
    return hipGetLastError();
  });
}

}  // namespace adasum
