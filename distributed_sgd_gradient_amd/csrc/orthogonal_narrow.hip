// orthogonal_narrow.hip - orthogonal updates of matrices with a side of at most
// 64 (see orthogonal.hip for the steps).
//
// Every X of the steps is a polynomial in G = X0 X0^T times X0, so narrow
// matrices take their steps on G alone: with P = a I + b G + c G G,
//
//   Q <- P Q,  G <- P G P      steps times;   result Q X0
//
// All of these commute and are symmetric, so half of their tiles are computed.
// G holds the squares of the singular values, so everything is in fp64, and after
// as many steps as raise G's rounding to 2^-20 (8 by default) G is formed again,
// from Q X0: small singular values have grown by then, and where X has none G is
// zero again.  Three launches instead of three a step, and two more each time G is
// formed again: partial sums of G over the long side, the steps in one workgroup a
// matrix on the fp64 matrix cores, a wave for each tile of 16 x 16 on and above the
// diagonal, and the product with X0.  Bound by the latency of the steps, in which
// three products follow one another: 61 x 769 fp32 in 5 steps takes 9 + 40 + 11 us
// (the steps with a product's sum in one chain of matrix instructions, and LDS read
// between them: 48; with fp32 steps through the products of orthogonal.hip: 254 a
// call against 61); 8 steps 82 us a call, 9 steps, with G formed again, 113.
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

// Q, turned, from the workspace to LDS; everyone's after the next barrier.
__device__ __forceinline__ void load_q(const OrthoArgs& a, const OrthoLayout& l, double (*q)[kSide]) {
  const double* from = reinterpret_cast<const double*>(a.ws + blockIdx.y * l.per_matrix + l.rest);
  double v[kSide * kSide / 256];
#pragma unroll
  for (int u = 0; u < kSide * kSide / 256; ++u) v[u] = from[u * 256 + threadIdx.x];
#pragma unroll
  for (int u = 0; u < kSide * kSide / 256; ++u) q[(u * 256 + threadIdx.x) / kSide][threadIdx.x % kSide] = v[u];
}

// Rows i0 to i0 + 15 of a column of Q X0, the column being n values at x.
__device__ __forceinline__ void times_q(const double (*q)[kSide], const float* x, int n, int i0, double (&acc)[16]) {
#pragma unroll
  for (int e = 0; e < 16; ++e) acc[e] = 0.0;
  for (int j = 0; j < n; ++j) {
    const double v = x[j];
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[e] = __builtin_fma(q[j][i0 + e], v, acc[e]);
  }
}

// A chunk's share of 4 x 4 values of G, from X as tile[k][i].
template <typename F>
__device__ __forceinline__ void add_gram(const F* tile, int pitch, int i0, int j0, double (&acc)[4][4]) {
#pragma unroll 4
  for (int k = 0; k < kChunk; ++k) {
    double u[4], v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      u[e] = tile[k * pitch + i0 + e];
      v[e] = tile[k * pitch + j0 + e];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int f = 0; f < 4; ++f) acc[e][f] = __builtin_fma(u[e], v[f], acc[e][f]);
  }
}

// A part of G: of X0, whose products are exact in fp64, or (AGAIN) of the X that
// the steps up to here have made of it, Q X0.
template <typename T, bool AGAIN>
__global__ __launch_bounds__(256) void narrow_gram_kernel(OrthoArgs a, OrthoLayout l) {
  __shared__ float tile[kChunk][kSide + 4];
  __shared__ double q[AGAIN ? kSide : 1][kSide], made[AGAIN ? kChunk : 1][kPitch];
  const int i0 = (threadIdx.x >> 4) * 4, j0 = (threadIdx.x & 15) * 4;
  const int64_t m = max(a.rows, a.cols);
  double acc[4][4] = {};
  if constexpr (AGAIN) load_q(a, l, q);
  for (int64_t k0 = (int64_t)blockIdx.x * kChunk; k0 < m; k0 += (int64_t)l.splits * kChunk) {
    load_chunk<T>(a, blockIdx.y, k0, tile);
    __syncthreads();
    if constexpr (AGAIN) {
      const int column = threadIdx.x & 63, first = (threadIdx.x >> 6) * 16;
      double x[16];
      times_q(q, tile[column], (int)min(a.rows, a.cols), first, x);
#pragma unroll
      for (int e = 0; e < 16; ++e) made[column][first + e] = x[e];
      __syncthreads();
      add_gram(&made[0][0], kPitch, i0, j0, acc);
    } else {
      add_gram(&tile[0][0], kSide + 4, i0, j0, acc);
    }
    __syncthreads();
  }
  double* out = reinterpret_cast<double*>(a.ws + blockIdx.y * l.per_matrix + l.partials) + blockIdx.x * kSide * kSide;
#pragma unroll
  for (int e = 0; e < 4; ++e)
#pragma unroll
    for (int f = 0; f < 4; ++f) out[(i0 + e) * kSide + j0 + f] = acc[e][f];
}

// The steps of a matrix whose narrow side is B blocks of 16: a wave for each of
// the tiles of 16 x 16 on and above the diagonal.
template <int B>
constexpr int tiles_of = B * (B + 1) / 2;

// The wave's tile of U V^T.
template <int B>
__device__ __forceinline__ v4d tile_product(const double* u, const double* v, int ti, int tj) {
  const int lane = threadIdx.x & 63;
  const double* from_u = u + (ti + (lane & 15)) * kPitch + (lane >> 4);
  const double* from_v = v + (tj + (lane & 15)) * kPitch + (lane >> 4);
  double x[4 * B], y[4 * B];
#pragma unroll
  for (int k = 0; k < 4 * B; ++k) {
    x[k] = from_u[4 * k];
    y[k] = from_v[4 * k];
  }
  v4d acc[2] = {{0.0, 0.0, 0.0, 0.0}, {0.0, 0.0, 0.0, 0.0}};  // two chains, added at the end
#pragma unroll
  for (int k = 0; k < 4 * B; ++k) acc[k & 1] = __builtin_amdgcn_mfma_f64_16x16x4f64(x[k], y[k], acc[k & 1], 0, 0, 0);
  return acc[0] + acc[1];
}

// Steps `begin` to `end` - 1, on the G of the X before them.
template <int B>
__global__ __launch_bounds__((64 * tiles_of<B>)) void narrow_steps_kernel(OrthoArgs a, OrthoLayout l, int begin,
                                                                          int end) {
  constexpr int kThreads = 64 * tiles_of<B>, kWidth = 16 * B;
  __shared__ double space[4][kWidth * kPitch];
  char* ws = a.ws + blockIdx.x * l.per_matrix;
  const double* parts = reinterpret_cast<const double*>(ws + l.partials);
  const int n = (int)min(a.rows, a.cols), lane = threadIdx.x & 63;
  int ti = 0, tj = threadIdx.x >> 6;  // the wave's tile, row by row
  while (tj >= B - ti) {
    tj -= B - ti;
    ++ti;
  }
  tj = (tj + ti) * 16;
  ti *= 16;
  double *g = space[0], *p = space[1], *q = space[2], *t = space[3];
  constexpr int kOwn = (kWidth * kWidth + kThreads - 1) / kThreads;  // values of G of a lane
  double sum[kOwn] = {};
  for (int first = 0; first < l.splits; first += 4) {
    double v[kOwn][4];  // parts past the last are read at the last: all loads at once
#pragma unroll
    for (int u = 0; u < kOwn; ++u)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int e = min((int)threadIdx.x + u * kThreads, kWidth * kWidth - 1);
        v[u][k] = parts[(int64_t)min(first + k, l.splits - 1) * kSide * kSide + e / kWidth * kSide + e % kWidth];
      }
#pragma unroll
    for (int u = 0; u < kOwn; ++u)
#pragma unroll
      for (int k = 0; k < 4; ++k) sum[u] += first + k < l.splits ? v[u][k] : 0.0;
  }
#pragma unroll
  for (int u = 0; u < kOwn; ++u) {
    const int e = threadIdx.x + u * kThreads;
    if (e < kWidth * kWidth) g[e / kWidth * kPitch + e % kWidth] = sum[u];
  }
  __syncthreads();
  double squares = lane < n ? g[lane * kPitch + lane] : 0.0;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) squares += __shfl_xor(squares, d);
  const double f = begin > 0 ? 1.0 : 1.0 / (sqrt(squares) + a.eps);
  __syncthreads();
#pragma unroll
  for (int u = 0; u < kOwn; ++u) {
    const int e = threadIdx.x + u * kThreads;
    if (e < kWidth * kWidth) g[e / kWidth * kPitch + e % kWidth] = sum[u] * (f * f);
  }
  __syncthreads();
  // A lane's places of its wave's tile: rows 4 r + lane / 16 of column lane % 16,
  // and their mirror images.  Of a tile on the diagonal, too, the upper half is
  // both halves' source: two roundings of one value would differ, and every step
  // takes rows for columns and raises the difference some 30 times (32 x 300 of
  // rank 4 in 12 steps: off by 0.5 of the norm).  The lower half goes where nobody
  // reads, behind the row.
  const int row = ti + (lane >> 4), column = tj + (lane & 15);
  int place[4], mirror[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int i = row + 4 * r;
    place[r] = i * kPitch + (i > column ? kSide : column);
    mirror[r] = i > column ? place[r] : column * kPitch + i;
  }
  auto put = [&](double* to, v4d v) __attribute__((always_inline)) {
#pragma unroll
    for (int r = 0; r < 4; ++r) to[place[r]] = to[mirror[r]] = v[r];
  };
  for (int s = begin; s < end; ++s) {
    const double ca = a.coefficients[3 * s], cb = a.coefficients[3 * s + 1], cc = a.coefficients[3 * s + 2];
    v4d v = tile_product<B>(g, g, ti, tj);
#pragma unroll
    for (int r = 0; r < 4; ++r)
      v[r] = cb * g[(row + 4 * r) * kPitch + column] + cc * v[r] + (row + 4 * r == column ? ca : 0.0);
    put(p, v);
    if (s == begin) put(q, v);
    __syncthreads();
    const bool last = s + 1 == end;
    if (s > begin) {
      v = tile_product<B>(p, q, ti, tj);
      put(t, v);
    }
    if (!last) v = tile_product<B>(p, g, ti, tj);
    __syncthreads();
    if (s > begin) {  // T is the new Q, and Q's place is free
      double* const free = q;
      q = t;
      t = free;
    }
    if (last) break;
    put(t, v);
    __syncthreads();
    v = tile_product<B>(t, p, ti, tj);
    put(g, v);
    __syncthreads();
  }
  double* out = reinterpret_cast<double*>(ws + l.rest);
  const double scale = f * (end == a.steps ? (double)a.scale : 1.0);
  if (begin == 0) {
    for (int e = threadIdx.x; e < kSide * kSide; e += kThreads) {
      const int i = e / kSide, j = e % kSide;
      out[e] = i < kWidth && j < kWidth ? q[i * kPitch + j] * scale : 0.0;
    }
    return;
  }
  // behind the steps before: of the product Q P, turned, P^T Q, where P need not be
  // symmetric to the last bit
  for (int e = threadIdx.x; e < kWidth * kWidth; e += kThreads)
    g[e / kWidth * kPitch + e % kWidth] = out[e / kWidth * kSide + e % kWidth];
  __syncthreads();
  for (int tile = threadIdx.x >> 6; tile < B * B; tile += tiles_of<B>) {
    const int i0 = tile / B * 16, j0 = tile % B * 16;
    const v4d v = tile_product<B>(g, q, i0, j0);
#pragma unroll
    for (int r = 0; r < 4; ++r) out[(i0 + 4 * r + (lane >> 4)) * kSide + j0 + (lane & 15)] = v[r] * scale;
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
  load_chunk<T>(a, blockIdx.y, k0, tile);
  load_q(a, l, q);
  __syncthreads();
  const int column = threadIdx.x & 63, i0 = (threadIdx.x >> 6) * 16;
  if (i0 >= side) return;
  double acc[16];
  times_q(q, tile[column], n, i0, acc);
  if (k0 + column >= m) return;
  const bool tall = a.rows > a.cols;
#pragma unroll
  for (int e = 0; e < 16; ++e)
    if (i0 + e < n)
      store_any(a.out[blockIdx.y], a.out_dtype, tall ? (k0 + column) * a.out_stride + i0 + e
                                                     : (int64_t)(i0 + e) * a.out_stride + k0 + column, acc[e]);
}

// Steps from `begin` on that one G can take.  Where X has no direction, G's
// rounding (2^-50 or so) stands for a singular value's square, of either sign, and
// a step raises it by a^2; far below zero it would grow without end.  2^30 leave it
// below 2^-20, and directions whose singular value they bring to 1 have digits to
// 5e-6 at least.  The default coefficients take 8 steps at once.
int steps_at_once(const OrthoArgs& a, int begin) {
  double raised = 1.0;
  int s = begin;
  for (; s < a.steps; ++s) {
    const double k = a.coefficients[3 * s];
    raised *= std::max(1.0, k * k);
    if (raised > 1073741824.0 && s > begin) break;
  }
  return s - begin;
}

template <typename T>
void launch_gram(bool again, const OrthoArgs& a, const OrthoLayout& l, int count, hipStream_t st) {
  if (again)
    narrow_gram_kernel<T, true><<<dim3((unsigned)l.splits, count), 256, 0, st>>>(a, l);
  else
    narrow_gram_kernel<T, false><<<dim3((unsigned)l.splits, count), 256, 0, st>>>(a, l);
}

template <int B>
void launch_steps(const OrthoArgs& a, const OrthoLayout& l, int begin, int end, int count, hipStream_t st) {
  narrow_steps_kernel<B><<<(unsigned)count, 64 * tiles_of<B>, 0, st>>>(a, l, begin, end);
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
    const int64_t blocks = ceil_div(std::min(a.rows, a.cols), 16);
    for (int begin = 0, end; begin < a.steps; begin = end) {
      end = begin + steps_at_once(a, begin);
      launch_gram<T>(begin > 0, a, l, count, st);
      if (blocks == 1)
        launch_steps<1>(a, l, begin, end, count, st);
      else if (blocks == 2)
        launch_steps<2>(a, l, begin, end, count, st);
      else if (blocks == 3)
        launch_steps<3>(a, l, begin, end, count, st);
      else
        launch_steps<4>(a, l, begin, end, count, st);
    }
    narrow_apply_kernel<T><<<dim3(chunks, count), 256, 0, st>>>(a, l);
    return hipGetLastError();
  });
}

}  // namespace adasum
