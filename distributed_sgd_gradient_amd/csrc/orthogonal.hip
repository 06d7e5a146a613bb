// orthogonal.hip - an update's matrices made orthogonal by Newton-Schulz
// products: with X the matrix over its Frobenius norm, rows <= columns (else
// its transpose),
//
//   A = X X^T,  B = b A + c A A,  X <- a X + B X      steps times
//
// which takes every singular value s to a s + b s^3 + c s^5.
//
// Bound by the matrix cores and X's traffic: 24 matrices of 1024 x 1024 in bf16
// take 820 to 850 us, 620 TFLOP/s with half of the symmetric products (a library
// product of 8192^3 in fp16 reaches 1127).  A step there is 41 us of A, 42 of B and
// 96 of X.  The loops alone take 28, 25 and 70 (1.1, 1.3 and 0.74 PFLOP/s, A's and
// B's what a library product reaches); in A and B the results are written when the
// loops of all workgroups have ended, in X beside loads, which wait for them (with
// the loads of the first steps only X takes 69 too).  Matrices with a side of at
// most 64 are in orthogonal_narrow.hip.
//
// Products take fp16 operands and sum in fp32.  X is kept as hi + lo, two fp16
// of 22 bits together, and a X is added in fp32 from both: rounding X itself to
// 16 bits would put noise into the directions of small singular values, which
// the steps then raise as if it were signal (a matrix of rank 8: 4e-2 of the
// result's norm; with hi + lo 4e-4).  What an operand of a product loses is
// scaled down by the product.  Of bf16 results (PARTS 1) the products take the
// hi parts only: off by 1.1e-3 of the norm for normally distributed matrices of
// 1024 x 1024 in 5 steps, 3.4e-3 in 12, where the rounding of the result itself
// costs 1.7e-3.  B's diagonal, its largest values, is kept in fp32 beside its fp16
// copy (without it the error grows by a fifth).  fp16 and fp32 results (PARTS 2)
// take hi hi + hi lo + lo hi: off by less than products in fp32 are.
//
// Values are scaled by powers of two so that neither part leaves fp16's normal
// range: the host admits coefficients only that keep singular values below 2
// and B below 31, and a matrix that is far smaller than eps, or that the steps
// shrink, has powers of its own (65 x 66 fp32, eps 10^8 of its norm: off by 1e-7
// of the result's norm, without them by 2e-2).
//
// Everything is padded with zeros to whole tiles in the workspace, so the
// products have no edges.  A and B are symmetric: half of their tiles are
// computed, and written twice.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <map>
#include <mutex>
#include <tuple>
#include <type_traits>
#include <vector>

#include "elem.h"
#include "layer_ops.h"

namespace adasum {
namespace {

using namespace elem;

typedef _Float16 v4h __attribute__((ext_vector_type(4)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));

constexpr float kScaleX = 16384.f, kScaleA = 8192.f, kScaleB = 2048.f;
// Workgroups that sum a matrix's squares (4096 x 1024 fp32: 6 us, with 64 of them
// 14; 24 x 1024 x 1024 bf16 17 against 15).
constexpr int kSumParts = 256;
// bf16 results of sides above this take one part of each operand.  Narrower
// ones are bound by the launches, and in the smallest the roundings of few
// values do not average out (5 x 3: 4.9e-3 of the norm).
constexpr int kOnePartSide = 256;

// A = X X^T, B = b A + c A A, a X + B X, and that of the last step.
enum Kind { kGramX, kSquareA, kApplyB, kLastB };

// A workgroup's tile of T x T: its waves along both sides, and the steps of the
// sum that LDS holds.
template <int T, int PARTS>
struct Tile {  // 64
  static constexpr int kWavesP = 2, kWavesQ = 2, kStages = 4 / PARTS;
};
template <int PARTS>
struct Tile<128, PARTS> {
  static constexpr int kWavesP = 2, kWavesQ = 2 * PARTS, kStages = 2;
};
template <int PARTS>
struct Tile<256, PARTS> {
  static constexpr int kWavesP = 2, kWavesQ = 4, kStages = 2;
};
template <int T, int PARTS>
constexpr int threads_of = 64 * Tile<T, PARTS>::kWavesP * Tile<T, PARTS>::kWavesQ;
constexpr int kStep = 64;  // of the sum: rows of 128 bytes, a line of the L2
constexpr int kXCDs = 8;

// X is held as 2^e X, where its singular values are below 1/2 at most (an update
// far smaller than eps, coefficients that shrink it): of a step's e to the next
// one's, and B as 2^f B.  All powers are 1 else.
struct Scale {
  float b, c;  // of A as it is held, and of its square
  float own;   // a 2^f
  int out;     // the exponent that the sum of both is raised by
};
typedef __attribute__((address_space(4))) const Scale* constant_scales;  // read into scalar registers

// v has arrived here, not where it is used first.
__device__ __forceinline__ void arrived(float& v) {
  int bits = __builtin_bit_cast(int, v);
  asm volatile("" : "+r"(bits));
  v = __builtin_bit_cast(float, bits);
}

// The least e from 0 on that leaves 2^e s in [1/2, 1).
__device__ __forceinline__ int room_above(double s) {
  int k = 0;
  if (s > 0 && s < 0.5) frexp(s, &k);
  return -k;
}

// The first e, from the exponents alone: norm / (norm + eps) is below 2^-e.
__device__ __forceinline__ int first_room(const OrthoArgs& a, double norm) {
  int of_norm, of_sum;
  frexp(norm, &of_norm);
  frexp(norm + a.eps, &of_sum);
  return max(0, of_sum - of_norm - 1);
}

// The powers of all steps.
__device__ void write_scales(const OrthoArgs& a, double norm, Scale* to) {
  int e = first_room(a, norm);
  double most = norm / (norm + a.eps) * 1.001;  // that a singular value is, with room for rounding
  for (int s = 0; s < a.steps; ++s) {
    const double ca = a.coefficients[3 * s], cb = a.coefficients[3 * s + 1], cc = a.coefficients[3 * s + 2];
    const OrthoBound bound = ortho_bound(ca, cb, cc, most);
    most = bound.value * 1.01;
    const int next = s + 1 < a.steps ? room_above(most) : 0;
    // B is raised no further than it counts beside a, nor above its range
    int f = room_above(bound.added / 30);
    if (ca != 0) f = min(f, room_above(fabs(ca)));
    to[s] = Scale{(float)ldexp(cb, f - 2 * e), (float)ldexp(cc, f - 4 * e), (float)ldexp(ca, f), next - e - f};
    e = next;
  }
}

__device__ __forceinline__ void split(float v, _Float16* hi, _Float16* lo) {
  *hi = (_Float16)v;
  *lo = (_Float16)(v - (float)*hi);
}

// ---------------------------------------------------------------- norm and first X

// Squares in fp64: neither over- nor underflow, whatever the update's scale.
template <typename T>
__global__ __launch_bounds__(256) void square_sum_kernel(OrthoArgs a, OrthoLayout l) {
  constexpr int VEC = Type<T>::kVec, AHEAD = 4;
  const uint32_t per_row = (uint32_t)(a.cols + VEC - 1) / VEC, total = (uint32_t)a.rows * per_row;  // below 2^28
  const T* x = static_cast<const T*>(a.x[blockIdx.y]);
  double s = 0.0;
  for (uint32_t first = blockIdx.x * 256 + threadIdx.x; first < total; first += AHEAD * gridDim.x * 256) {
    v4u raw[AHEAD];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      const uint32_t p = first + u * gridDim.x * 256, r = p / per_row, c = (p - r * per_row) * VEC;
      raw[u] = load_raw(x + r * a.x_stride + c, p < total ? (int)(a.cols - c) : 0);
    }
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      float v[VEC];
      widen<T>(raw[u], v);
#pragma unroll
      for (int i = 0; i < VEC; ++i) s = __builtin_fma((double)v[i], (double)v[i], s);
    }
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

// The norm, from its parts, in every lane.
__device__ __forceinline__ double norm_of(const char* ws, const OrthoLayout& l) {
  const double* sums = reinterpret_cast<const double*>(ws + l.sums) + (threadIdx.x & 63);
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < kSumParts / 64; ++i) s += sums[i * 64];
  return sqrt(wave_sum(s));
}
// All powers are 1 (also of a norm that is NaN).
__device__ __forceinline__ bool usual(const OrthoArgs& a, double norm) { return a.plain && !(norm < 100 * a.eps); }

// X, 64 x 64 values a workgroup: a vector of four values of each of four rows a
// lane, turned in LDS where the matrix is tall.  The last workgroup of a matrix
// leaves the steps' powers.
template <typename T>
__global__ __launch_bounds__(256) void first_kernel(OrthoArgs a, OrthoLayout l) {
  __shared__ float tile[64][65];
  char* ws = a.ws + blockIdx.y * l.per_matrix;
  if (blockIdx.x == gridDim.x - 1) {
    Scale* const scales = reinterpret_cast<Scale*>(ws + l.scales);
    const double norm = norm_of(ws, l);
    if (!usual(a, norm)) {
      if (threadIdx.x == 0) write_scales(a, norm, scales);
    } else if ((int)threadIdx.x < a.steps) {
      const double* k = a.coefficients + 3 * threadIdx.x;
      scales[threadIdx.x] = Scale{(float)k[1], (float)k[2], (float)k[0], 0};
    }
    return;
  }
  const uint32_t tiles_m = (uint32_t)(l.m / 64), ti = blockIdx.x / tiles_m, tk = blockIdx.x - ti * tiles_m;
  const int64_t i0 = (int64_t)ti * 64, k0 = (int64_t)tk * 64;
  const T* x = static_cast<const T*>(a.x[blockIdx.y]);
  const bool tall = a.rows > a.cols;
  const int c = (threadIdx.x & 15) * 4, row = threadIdx.x >> 4;
  // rows of the matrix as it lies: along k, or along i where it is tall
  T raw[4][4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int64_t r = (tall ? k0 : i0) + row + 16 * u, from = (tall ? i0 : k0) + c;
    const T* p = x + r * a.x_stride + from;
    typedef T Four __attribute__((ext_vector_type(4)));
    if (r < a.rows && from + 4 <= a.cols) {
      const Four v = load_at<Four, sizeof(T)>(p);
#pragma unroll
      for (int e = 0; e < 4; ++e) raw[u][e] = v[e];
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) raw[u][e] = r < a.rows && from + e < a.cols ? p[e] : (T)0.f;
    }
  }
  const double norm = norm_of(ws, l);
  const double f = ldexp((double)kScaleX / (norm + a.eps), first_room(a, norm));
  float v[4][4];
#pragma unroll
  for (int u = 0; u < 4; ++u)
#pragma unroll
    for (int e = 0; e < 4; ++e) v[u][e] = (float)((double)(float)raw[u][e] * f);
  if (tall) {
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e) tile[c + e][row + 16 * u] = v[u][e];
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e) v[u][e] = tile[row + 16 * u][c + e];
  }
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    v4h hi, lo;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      _Float16 h, r;
      split(v[u][e], &h, &r);
      hi[e] = h;
      lo[e] = r;
    }
    const int64_t at = (i0 + row + 16 * u) * l.m + k0 + c;
    *reinterpret_cast<v4h*>(ws + l.x[0][0] + at * 2) = hi;
    *reinterpret_cast<v4h*>(ws + l.x[0][1] + at * 2) = lo;
  }
}

// ---------------------------------------------------------------- products

// N values (2, 4 or 8) rounded to a type and stored from element `at` on, the
// first `valid` of them.
template <typename T, int N>
__device__ __forceinline__ void store_as(T* p, const float (&v)[N], int64_t valid) {
  if (valid >= N) {
    typedef T Row __attribute__((ext_vector_type(N)));
    Row r;
#pragma unroll
    for (int i = 0; i < N; ++i) r[i] = (T)v[i];
    store_at<Row, sizeof(T)>(p, r);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < valid) p[i] = (T)v[i];
  }
}
template <int N>
__device__ __forceinline__ void store_out(void* out, int dtype, int64_t at, const float (&v)[N], int64_t valid) {
  if (dtype == 0)
    store_as(static_cast<float*>(out) + at, v, valid);
  else if (dtype == 1)
    store_as(static_cast<_Float16*>(out) + at, v, valid);
  else
    store_as(static_cast<__bf16*>(out) + at, v, valid);
}

typedef __attribute__((address_space(1))) const void* global_pointer;
typedef __attribute__((address_space(3))) void* lds_pointer;
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s* lds_v4s;

// Wait until at most `loads` of this wave's loads are on their way.
template <int loads>
__device__ __forceinline__ void wait_for_loads() {
  static_assert(loads < 63, "six bits, all of which mean no limit");
  __builtin_amdgcn_s_waitcnt(0x0f70 | (loads & 15) | (loads >> 4) << 14);
}
// Wait for this wave's LDS reads.
__device__ __forceinline__ void wait_for_reads() { __builtin_amdgcn_s_waitcnt(0xc07f); }
// All waves have come here; unlike __syncthreads, loads stay on their way.
__device__ __forceinline__ void meet() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Rows along the sum, of 64 values, in 16-byte pieces permuted within a row.
// The LDS serves lanes 0-3, 12-15 and 20-27 of a 16-byte read together, and the
// other 16 of each 32: with these keys each set finds different banks (no
// conflicts counted; where rows 0-3 and 4-7 met, every read took twice as long).
__device__ __forceinline__ int along_key(int row) { return (row >> 1) & 7; }
// Rows across the sum, of T values, in segments of 32 permuted within a row: a
// transposing read takes half of the same segment of 16 rows.
template <int T>
__device__ __forceinline__ int across_key(int row) {
  return ((row & 3) | ((row >> 1) & 4)) & (T / 32 - 1);
}

// A tile of T x T of C = P Q, summed over kStep values at a time; P's rows lie
// along the sum, and Q's columns (kGramX, kSquareA: C = P Q^T, rows of one
// symmetric matrix) or, of a product with X, Q's rows across it, which transposing
// reads turn.  Loads go straight to LDS, kStages steps ahead, and LDS is read half
// a step ahead of the products.  Rows of 128 bytes, not of 64 (24 x 1024 x 1024
// bf16: A 39 us against 45, X 110 against 121); tiles of X written from the
// registers, 64 bytes a row, not through LDS: X 100 us against 96.
template <int KIND, int PARTS, int T, int DEEP>
__global__ __launch_bounds__((threads_of<T, PARTS>), 2) void product_kernel(OrthoArgs a, OrthoLayout l, OrthoStep step) {
  using S = Tile<T, PARTS>;
  constexpr bool APPLY = KIND == kApplyB || KIND == kLastB;
  constexpr int kWaves = S::kWavesP * S::kWavesQ;
  constexpr int WP = T / S::kWavesP, WQ = T / S::kWavesQ, MP = WP / 16, MQ = WQ / 16;
  constexpr int kPieces = T * kStep / 8;  // 16-byte pieces of an operand's part
  constexpr int kStages = S::kStages * DEEP;
  constexpr int kFills = kPieces / 64 / kWaves, kLoads = 2 * PARTS * kFills;
  static_assert(kFills * kWaves * 64 == kPieces, "whole waves");
  __shared__ v4u lds[kStages][2 * PARTS][kPieces];  // of each step P's parts, then Q's
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);

  // Workgroups are dealt to the eight XCDs in turn: each takes a run of
  // consecutive tiles, which share their operands in its L2.
  const uint32_t xcd = blockIdx.x % kXCDs, whole = gridDim.x / kXCDs, rest = gridDim.x % kXCDs;
  uint32_t block = xcd * whole + min(xcd, rest) + blockIdx.x / kXCDs;
  const uint32_t matrix = block / step.blocks;
  block -= matrix * step.blocks;
  const uint32_t part = block / step.tiles;
  block -= part * step.tiles;
  char* ws = a.ws + matrix * l.per_matrix;
  const constant_scales scales = (constant_scales)(ws + l.scales) + step.index;
  float scale_a = 0.f, scale_b = 0.f, scale_c = 0.f;
  int raise = 0;
  if constexpr (KIND == kSquareA) {
    scale_b = scales->b;
    scale_c = scales->c;
  }
  if constexpr (APPLY) {
    scale_a = scales->own;
    raise = scales->out;
  }
  // tiles of the upper triangle, row by row, or all
  uint32_t tp = 0, tq = block;
  if constexpr (APPLY) {
    const uint32_t across = (uint32_t)(l.m / T);
    tp = block / across;
    tq = block - tp * across;
  } else {
    uint32_t width = (uint32_t)(l.n / T);
    while (tq >= width) {
      tq -= width;
      --width;
      ++tp;
    }
    tq += tp;
  }
  const int64_t p0 = (int64_t)tp * T, q0 = (int64_t)tq * T;
  const int64_t ld = KIND == kGramX ? l.m : l.n;
  int begin = 0, end = (int)(ld / kStep);
  if constexpr (KIND == kGramX) {
    begin = part * step.part_steps;
    end = min(end, begin + step.part_steps);
  }

  // Where this lane's pieces of a step lie, from the step's first: kFills of
  // each operand, 64 consecutive places of LDS a wave.
  uint32_t from_p[kFills], from_q[kFills];
#pragma unroll
  for (int f = 0; f < kFills; ++f) {
    const int place = (f * kWaves + wave) * 64 + lane;
    const int row = place / 8, piece = (place % 8) ^ along_key(row);
    // row 16 i + r of a wave's part holds its row MP r + i: a lane's sums are
    // then of MP consecutive rows of P
    const int of_p = row / WP * WP + row % 16 * MP + row % WP / 16;
    from_p[f] = (uint32_t)(of_p * ld + piece * 8) * 2;
    if constexpr (APPLY) {
      const int k = place / (T / 8), across = (place % (T / 8)) ^ (across_key<T>(k) * 4);
      from_q[f] = (uint32_t)(k * l.m + across * 8) * 2;
    } else {
      // and those of two neighbouring groups of 16 of eight consecutive of Q
      const int of_q = row / 32 * 32 + row % 16 / 4 * 8 + row % 32 / 16 * 4 + row % 4;
      from_q[f] = (uint32_t)(of_q * ld + piece * 8) * 2;
    }
  }
  const char* operand[2 * PARTS];
#pragma unroll
  for (int h = 0; h < PARTS; ++h) {
    const size_t p = KIND == kGramX ? l.x[step.from][h] : KIND == kSquareA ? l.a[h] : l.b[h];
    operand[h] = ws + p + p0 * ld * 2;
    operand[PARTS + h] = APPLY ? ws + l.x[step.from][h] + q0 * 2 : ws + p + q0 * ld * 2;
  }
  const int64_t next_p = kStep * 2, next_q = APPLY ? kStep * l.m * 2 : kStep * 2;
  auto fetch = [&](int buffer, int t) __attribute__((always_inline)) {
#pragma unroll
    for (int o = 0; o < 2 * PARTS; ++o) {
      const char* base = operand[o] + t * (o < PARTS ? next_p : next_q);
#pragma unroll
      for (int f = 0; f < kFills; ++f)
        __builtin_amdgcn_global_load_lds((global_pointer)(base + (o < PARTS ? from_p[f] : from_q[f])),
                                         (lds_pointer)&lds[buffer][o][(f * kWaves + wave) * 64], 16, 0, 0);
    }
  };

  const int wp = (wave / S::kWavesQ) * WP, wq = (wave % S::kWavesQ) * WQ;
  // this lane's piece of 16 rows along the sum, from a step's first
  const int at = (lane & 15) * 8 + ((lane >> 4) ^ along_key(lane & 15));
  const int at_p = wp * 8 + at, at_q = PARTS * kPieces + wq * 8 + at;
  // Eight rows of a lane's column: lane i of 16 names four columns of row i / 4
  // and gets value i of four rows; the columns are those of of_q above.
  const int turn_row = (lane >> 4) * 8 + ((lane & 15) >> 2), turn_key = across_key<T>(turn_row);
  auto turned = [&](const v4u* stage, int h, int column, int half) __attribute__((always_inline)) {
    const char* p = reinterpret_cast<const char*>(stage + (PARTS + h) * kPieces) + (half * 32 + turn_row) * T * 2 +
                    ((column / 32) ^ turn_key) * 64 + (lane & 3) * 16 + column % 32 / 16 * 8;
    const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)(p));
    const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)(p + 4 * T * 2));
    return __builtin_bit_cast(v8h, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  };
  v4f acc[MP][MQ];
#pragma unroll
  for (int i = 0; i < MP; ++i)
#pragma unroll
    for (int j = 0; j < MQ; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  // A lane holds rows p .. p + MP - 1 of columns q + 32 j .. q + 32 j + 7.  What
  // the products are added to, b A or a X, is read before them where there are
  // registers for it, else kGroup rows ahead of the stores.  With one part an
  // operand the high part of X is taken from LDS instead, in the step that holds
  // it; with two that would cost digits: every sum behind it rounds a X too (rank
  // 3, fp32: 6.8e-5 of the norm against 4.5e-5).
  constexpr bool kBase = KIND != kGramX, kOwn = APPLY && PARTS == 1;
  constexpr int kGroup = MP < 4 ? MP : 4, kGroups = MP / kGroup * (MQ / 2);
  constexpr bool kEarly = kGroups <= 2;
  const int64_t p = p0 + wp + (lane & 15) * MP, q = q0 + wq + (lane >> 4) * 8;
  const int64_t width = APPLY ? l.m : l.n;
  const char* base[2];
  char* to[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    base[h] = ws + (APPLY ? l.x[step.from][kOwn ? 1 : h] : l.a[h]) + (p * width + q) * 2;
    to[h] = ws + (KIND == kGramX ? l.a[h] : KIND == kSquareA ? l.b[h] : l.x[step.from ^ 1][h]);
  }
  v8h had[2][kGroup][PARTS];
  auto read_base = [&](int set, int g) __attribute__((always_inline)) {
#pragma unroll
    for (int r = 0; r < kGroup; ++r)
#pragma unroll
      for (int h = 0; h < PARTS; ++h)
        had[set][r][h] = *reinterpret_cast<const v8h*>(
            base[h] + ((g % (MP / kGroup) * kGroup + r) * width + g / (MP / kGroup) * 32) * 2);
  };
  if constexpr (kBase && kEarly) {
#pragma unroll
    for (int g = 0; g < kGroups; ++g) read_base(g, g);
  }
  float factor[MP];  // of a X
#pragma unroll
  for (int i = 0; i < MP; ++i) {
    factor[i] = scale_a;
    if constexpr (kOwn) factor[i] += reinterpret_cast<const float*>(ws + l.rest)[p + i];
  }
  // A step is two halves of 32 terms: the products of one from one set of
  // registers, while the other set is filled for the next.
  v8h fp[2][PARTS][MP], fq[2][PARTS][MQ];
  auto read = [&](auto half_of, int buffer) __attribute__((always_inline)) {
    constexpr int half = decltype(half_of)::value;
    const v4u* stage = &lds[buffer][0][0];
#pragma unroll
    for (int h = 0; h < PARTS; ++h) {
#pragma unroll
      for (int i = 0; i < MP; ++i)
        fp[half][h][i] = __builtin_bit_cast(v8h, stage[(at_p ^ (half * 4)) + h * kPieces + i * 128]);
#pragma unroll
      for (int j = 0; j < MQ; ++j) {
        if constexpr (APPLY)
          fq[half][h][j] = turned(stage, h, wq + j * 16, half);
        else
          fq[half][h][j] = __builtin_bit_cast(v8h, stage[(at_q ^ (half * 4)) + h * kPieces + j * 128]);
      }
    }
    // on their way before the products that follow, which do not need them
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  auto multiply = [&](auto half_of) __attribute__((always_inline)) {
    constexpr int half = decltype(half_of)::value;
#pragma unroll
    for (int i = 0; i < MP; ++i)
#pragma unroll
      for (int j = 0; j < MQ; ++j) {
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(fq[half][0][j], fp[half][0][i], acc[i][j], 0, 0, 0);
        if constexpr (PARTS == 2) {
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(fq[half][1][j], fp[half][0][i], acc[i][j], 0, 0, 0);
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(fq[half][0][j], fp[half][1][i], acc[i][j], 0, 0, 0);
        }
      }
  };
  // a X of the high part in LDS, the lane's rows being `row` .. of a step
  auto add_own = [&](int buffer, int row) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < MP; ++i)
#pragma unroll
      for (int j = 0; j < MQ / 2; ++j) {
        const int place = (row + i) * (T / 8) + (((wq + 32 * j) / 8 + (lane >> 4)) ^ (across_key<T>(row + i) * 4));
        const v8h x = __builtin_bit_cast(v8h, lds[buffer][PARTS][place]);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          acc[i][2 * j + e / 4][e % 4] = __builtin_fmaf(factor[i] * kScaleB, (float)x[e], acc[i][2 * j + e / 4][e % 4]);
      }
  };
  const std::integral_constant<int, 0> first_half;
  const std::integral_constant<int, 1> second_half;
#pragma unroll
  for (int t = 0; t < kStages; ++t)
    if (begin + t < end) fetch(t, begin + t);
  arrived(scale_a);
  arrived(scale_b);
  arrived(scale_c);
  // Between steps 2^8 at most either way: with p the larger of |a| and |b s^2 + c s^4|
  // a step takes the bound on s to p s / 10 at least and 2 p s at most, and f is
  // log2 1/p but for 30.  Behind the last as low as the result is, in two factors.
  const float raised = APPLY ? __builtin_ldexpf(1.f, max(raise, -100)) : 1.f;
  if (end - begin >= kStages)
    wait_for_loads<(kStages - 1) * kLoads>();
  else
    wait_for_loads<0>();
  meet();
  read(first_half, 0);
  int buffer = 0;
  for (int t = begin; t < end; ++t) {
    const int next = buffer + 1 == kStages ? 0 : buffer + 1;
    if constexpr (kOwn) {
      // the step that holds this lane's rows of X
      if (t >= (int)(p0 + wp) / kStep && t <= (int)(p0 + wp + WP - 1) / kStep) {
        if ((int)p / kStep == t) add_own(buffer, (int)p - t * kStep);
      }
    }
    wait_for_reads();
    read(second_half, buffer);
    multiply(first_half);
    // the next step's loads have arrived, everyone's; and everyone has read
    // this step's buffer, which is filled again
    wait_for_reads();
    if (end - t >= kStages)
      wait_for_loads<(kStages - 2) * kLoads>();
    else
      wait_for_loads<0>();
    meet();
    if (t + kStages < end) fetch(buffer, t + kStages);
    read(first_half, next);  // of the last step: what nobody uses
    multiply(second_half);
    buffer = next;
  }

  if (KIND == kGramX && step.parts > 1) {
    float* sums = reinterpret_cast<float*>(ws + l.partials) + part * l.n * l.n + p * l.n + q;
#pragma unroll
    for (int j = 0; j < MQ; ++j)
#pragma unroll
      for (int i = 0; i < MP; ++i) *reinterpret_cast<v4f*>(sums + i * l.n + j / 2 * 32 + j % 2 * 4) = acc[i][j];
    return;
  }
  if constexpr (kBase && !kEarly) read_base(0, 0);
  // Where LDS holds the tile, it goes there first and leaves in whole rows.  Every
  // wave is past its reads: the last barrier of the loop lies behind them.
  constexpr int kStored = PARTS == 2 || APPLY ? 2 : 1;
  constexpr bool kStash = KIND != kLastB && kStored * T * T * 2 <= (int)sizeof(lds);
  v4u* const stash = &lds[0][0][0];
  // 16-byte pieces permuted within a row, so that 16 lanes' rows, MP apart, find
  // different banks
  auto stash_at = [](int row, int piece) __attribute__((always_inline)) {
    return row * (T / 8) + (piece ^ (row / MP & (T / 8 - 1)));
  };
  const bool turn = KIND == kLastB ? a.rows > a.cols : tp != tq;
  v8h hi[MP], lo[MP];
  float v[MP][8];
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    if constexpr (kBase && !kEarly)
      if (g + 1 < kGroups) read_base((g + 1) & 1, g + 1);
    const int j = g / (MP / kGroup);
#pragma unroll
    for (int r = 0; r < kGroup; ++r) {
      const int i = g % (MP / kGroup) * kGroup + r;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float sum = acc[i][2 * j + e / 4][e % 4];
        if constexpr (KIND == kGramX) {
          v[i][e] = sum * (kScaleA / (kScaleX * kScaleX));
        } else {
          float was = (float)had[g & 1][r][0][e];
          if constexpr (PARTS == 2) was += (float)had[g & 1][r][1][e];
          if constexpr (KIND == kSquareA)
            v[i][e] = __builtin_fmaf(scale_c, sum * (kScaleB / (kScaleA * kScaleA)),
                                     scale_b * (was * (kScaleB / kScaleA)));
          else
            v[i][e] = __builtin_fmaf(factor[i] * raised, was, sum * (raised / kScaleB));
        }
        if constexpr (KIND == kSquareA && PARTS == 1) {  // what fp16 leaves out of the diagonal
          if (p + i == q + 32 * j + e)
            reinterpret_cast<float*>(ws + l.rest)[p + i] = (v[i][e] - (float)(_Float16)v[i][e]) * (1.f / kScaleB);
        }
      }
      if constexpr (KIND == kLastB) continue;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        _Float16 h, t;
        split(v[i][e], &h, &t);
        hi[i][e] = h;
        lo[i][e] = t;
      }
      if constexpr (kStash) {
        const int place = stash_at((int)(p - p0) + i, (int)(q - q0) / 8 + 4 * j);
        stash[place] = __builtin_bit_cast(v4u, hi[i]);
        if constexpr (kStored == 2) stash[T * T / 8 + place] = __builtin_bit_cast(v4u, lo[i]);
      } else {
        const int64_t at_out = ((p + i) * width + q + 32 * j) * 2;
        *reinterpret_cast<v8h*>(to[0] + at_out) = hi[i];
        if constexpr (kStored == 2) *reinterpret_cast<v8h*>(to[1] + at_out) = lo[i];
      }
    }
    if (g % (MP / kGroup) != MP / kGroup - 1) continue;
    // all MP rows of these columns are there
    if constexpr (KIND == kLastB) {
      const int64_t n = min(a.rows, a.cols), m = max(a.rows, a.cols), c = q + 32 * j;
      const float f = __builtin_ldexpf(a.scale * (1.f / kScaleX), min(raise + 100, 0));
      if (turn) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float t[MP];
#pragma unroll
          for (int i = 0; i < MP; ++i) t[i] = v[i][e] * f;
          if (c + e < m) store_out(a.out[matrix], a.out_dtype, (c + e) * a.out_stride + p, t, n - p);
        }
      } else {
#pragma unroll
        for (int i = 0; i < MP; ++i) {
          float t[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) t[e] = v[i][e] * f;
          if (p + i < n) store_out(a.out[matrix], a.out_dtype, (p + i) * a.out_stride + c, t, m - c);
        }
      }
    } else if (!APPLY && turn) {  // the mirror image
#pragma unroll
      for (int h = 0; h < PARTS; ++h)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          typedef _Float16 Column __attribute__((ext_vector_type(MP)));
          Column t;
#pragma unroll
          for (int i = 0; i < MP; ++i) t[i] = h == 0 ? hi[i][e] : lo[i][e];
          *reinterpret_cast<Column*>(to[h] + ((q + 32 * j + e) * l.n + p) * 2) = t;
        }
    }
  }
  if constexpr (kStash) {
    __syncthreads();
    constexpr int kThreads = kWaves * 64, kRow = T / 8;
#pragma unroll
    for (int h = 0; h < kStored; ++h)
#pragma unroll
      for (int u = 0; u < T * kRow / kThreads; ++u) {
        const int place = u * kThreads + tid, row = place / kRow, piece = place % kRow;
        *reinterpret_cast<v4u*>(to[h] + ((p0 + row) * width + q0 + piece * 8) * 2) =
            stash[h * T * kRow + stash_at(row, piece)];
      }
  }
}

// A from the sums of its parts, added in their order: a tile of 32 x 32 on or
// above the diagonal and its mirror image.
template <int PARTS>
__global__ __launch_bounds__(256) void join_kernel(OrthoArgs a, OrthoLayout l, int parts) {
  __shared__ float tile[32][33];
  char* ws = a.ws + blockIdx.y * l.per_matrix;
  uint32_t rest = blockIdx.x, width = (uint32_t)(l.n / 32), tp = 0;
  while (rest >= width) {
    rest -= width;
    --width;
    ++tp;
  }
  const int64_t p0 = (int64_t)tp * 32, q0 = (int64_t)(tp + rest) * 32;
  const int row = threadIdx.x >> 3, c = (threadIdx.x & 7) * 4;
  const float* sums = reinterpret_cast<const float*>(ws + l.partials) + (p0 + row) * l.n + q0 + c;
  float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int s = 0; s < parts; ++s) {
    const v4f t = *reinterpret_cast<const v4f*>(sums + s * l.n * l.n);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] += t[e];
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) tile[row][c + e] = v[e] * (kScaleA / (kScaleX * kScaleX));
  __syncthreads();
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    if (side == 1 && p0 == q0) break;
    v4h hi, lo;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      // within the tile on the diagonal the upper half is both halves' source
      const bool lower = side == 1 || (p0 == q0 && row > c + e);
      _Float16 h, r;
      split(lower ? tile[c + e][row] : tile[row][c + e], &h, &r);
      hi[e] = h;
      lo[e] = r;
    }
    const int64_t to = ((side ? q0 : p0) + row) * l.n + (side ? p0 : q0) + c;
    *reinterpret_cast<v4h*>(ws + l.a[0] + to * 2) = hi;
    if constexpr (PARTS == 2) *reinterpret_cast<v4h*>(ws + l.a[1] + to * 2) = lo;
  }
}

size_t align256(size_t b) { return (b + 255) & ~size_t(255); }

template <int KIND, int PARTS, int T>
hipError_t product(const OrthoArgs& a, const OrthoLayout& l, OrthoStep step, int count, hipStream_t st) {
  const uint32_t side = (uint32_t)(l.n / T);
  step.tiles = KIND == kGramX || KIND == kSquareA ? side * (side + 1) / 2 : side * (uint32_t)(l.m / T);
  step.blocks = step.tiles * step.parts;
  constexpr int kThreads = threads_of<T, PARTS>;
  // Two parts an operand leave LDS for two steps where two workgroups share a CU;
  // of one a CU, four hide the loads' way (1 x 1024 x 1024 fp32: 231 us against
  // 246.  One part has four already; with eight 160 against 152)
  if constexpr (T == 64 && PARTS == 2)
    if (step.blocks * count <= kCUs) {
      product_kernel<KIND, PARTS, T, 2><<<step.blocks * count, kThreads, 0, st>>>(a, l, step);
      return hipGetLastError();
    }
  product_kernel<KIND, PARTS, T, 1><<<step.blocks * count, kThreads, 0, st>>>(a, l, step);
  return hipGetLastError();
}

template <int KIND, int PARTS>
hipError_t product(int tile, const OrthoArgs& a, const OrthoLayout& l, const OrthoStep& step, int count,
                   hipStream_t st) {
  if constexpr (PARTS == 1)
    if (tile == 256) return product<KIND, PARTS, 256>(a, l, step, count, st);
  return tile == 128 ? product<KIND, PARTS, 128>(a, l, step, count, st)
                     : product<KIND, PARTS, 64>(a, l, step, count, st);
}

template <int PARTS>
hipError_t steps_of(const OrthoArgs& a, const OrthoLayout& l, int count, hipStream_t st) {
  for (int s = 0; s < a.steps; ++s) {
    OrthoStep step{};
    step.index = s;
    step.from = s & 1;
    step.parts = l.splits;
    step.part_steps = l.split_steps;
    hipError_t e = product<kGramX, PARTS>(l.tile_a, a, l, step, count, st);
    if (e == hipSuccess && l.splits > 1) {
      const uint32_t small = (uint32_t)(l.n / 32);
      join_kernel<PARTS><<<dim3(small * (small + 1) / 2, count), 256, 0, st>>>(a, l, l.splits);
      e = hipGetLastError();
    }
    step.parts = 1;
    if (e == hipSuccess) e = product<kSquareA, PARTS>(l.tile_b, a, l, step, count, st);
    if (e == hipSuccess)
      e = s + 1 < a.steps ? product<kApplyB, PARTS>(l.tile_x, a, l, step, count, st)
                          : product<kLastB, PARTS>(l.tile_x, a, l, step, count, st);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// What a product takes, in us: a round of `slots` workgroups at once starts and
// ends (fixed) and takes `steps` of 64 of the sum, each of `full` where the card
// is full, down to `alone` where it is nearly empty.  From measured products of 1
// to 24 matrices of 1024 x 1024 and 1 of 1024 x 4096 and 4096 x 4096.  Of 36 calls
// from 100 x 100 to 4096 x 4096, 1 to 24 matrices, 31 take at most 5 % longer than
// with the best of six fixed choices, the others up to 14 % (24 x 1024 x 1024 bf16:
// 854 us, with tiles of 64 alone 1322, of 128 alone 891; 1 x 1024 x 1024: 151, 152
// and 271).
struct Cost {
  int slots;
  double alone, full, fixed;
};
constexpr Cost kCosts[2][2][3] = {  // A and B, or X; one part or two; tiles of 64, 128, 256
    {{{512, 0.28, 0.45, 3}, {512, 0.72, 1.25, 5}, {256, 1.2, 1.75, 11}},
     {{512, 0.6, 0.95, 4}, {256, 1.3, 1.6, 4}, {256, 1e9, 1e9, 0}}},
    {{{512, 0.6, 0.7, 4}, {512, 0.8, 1.5, 8}, {256, 1.1, 2.4, 25}},
     {{512, 1.0, 1.35, 4}, {256, 1.5, 1.9, 5}, {256, 1e9, 1e9, 0}}}};

double cost_of(bool x, int parts, int index, int64_t blocks, int64_t steps) {
  const Cost& c = kCosts[x][parts - 1][index];
  const int64_t rounds = blocks / c.slots;
  const double rest = (double)(blocks - rounds * c.slots) / c.slots;
  return rounds * (c.fixed + steps * c.full) +
         (rest > 0 ? c.fixed + steps * (c.alone + (c.full - c.alone) * rest) : 0.0);
}

}  // namespace

namespace {

OrthoLayout layout_of(int64_t n, int64_t m, int parts, int together) {
  OrthoLayout l{};
  l.parts = parts;
  l.together = together;
  // the tiles of the three products, and the parts of A's sums, that take the
  // least time; all sides are padded to the largest tile
  double best = 1e30;
  for (int largest = 0; largest < 3; ++largest) {
    const int64_t pad = 64 << largest, pn = ceil_div(n, pad) * pad, pm = ceil_div(m, pad) * pad;
    double sum = 0;
    int tile[3] = {}, splits = 1;
    for (int kind = 0; kind < 3; ++kind) {
      double least = 1e30;
      for (int i = 0; i <= largest; ++i) {
        const int64_t side = pn / (64 << i);
        const int64_t tiles = (kind == 2 ? side * (pm / (64 << i)) : side * (side + 1) / 2) * l.together;
        const int64_t steps = (kind == 0 ? pm : pn) / kStep;
        for (int64_t s = 1; s <= (kind == 0 ? std::min<int64_t>(16, steps / 4) : 1) || s == 1; ++s) {
          // the parts are written, read, and waited for
          const double join = s == 1 ? 0 : 8 + 6e-7 * (double)(s * pn * pn * l.together);
          const double c = cost_of(kind == 2, l.parts, i, tiles * s, ceil_div(steps, s)) + join;
          if (c < least) {
            least = c;
            tile[kind] = 64 << i;
            if (kind == 0) splits = (int)s;
          }
        }
      }
      sum += least;
    }
    if (sum < best) {
      best = sum;
      l.tile_a = tile[0];
      l.tile_b = tile[1];
      l.tile_x = tile[2];
      l.n = pn;
      l.m = pm;
      l.splits = splits;
    }
  }
  const int64_t steps = l.m / kStep;
  l.split_steps = (int)ceil_div(steps, l.splits);
  l.splits = (int)ceil_div(steps, l.split_steps);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += align256(bytes);
    return here;
  };
  const size_t x = (size_t)l.n * l.m * 2, s = (size_t)l.n * l.n * 2;
  for (int h = 0; h < 2; ++h) {
    l.x[0][h] = take(x);
    l.x[1][h] = take(x);
  }
  for (int h = 0; h < l.parts; ++h) {
    l.a[h] = take(s);
    l.b[h] = take(s);
  }
  l.rest = take((size_t)l.n * 4);
  l.sums = take(kSumParts * 8);
  l.scales = take(kOrthoSteps * sizeof(Scale));
  l.partials = take(l.splits > 1 ? s * 2 * l.splits : 0);
  l.per_matrix = at;
  l.total = at * l.together;
  return l;
}

}  // namespace

OrthoLayout ortho_layout(int64_t count, int64_t rows, int64_t cols, int out_dtype) {
  const int64_t n = std::min(rows, cols), m = std::max(rows, cols);
  if (n <= kOrthoNarrow) return ortho_narrow_layout(count, rows, cols);
  const int parts = out_dtype == 2 && n > kOnePartSide ? 1 : 2;
  OrthoLayout l = layout_of(n, m, parts, (int)std::min<int64_t>(count, kOrthoWide));
  // fewer matrices may be padded further, or have A's sums in more parts
  while (l.total > kOrthoWorkspace && l.together > 1)
    l = layout_of(n, m, parts,
                  (int)std::max<size_t>(1, std::min<size_t>(l.together - 1, kOrthoWorkspace / l.per_matrix)));
  return l;
}

// A call of fewer matrices can take more: its tiles, and so its padding and the
// parts of A's sums, are others.  A workspace for many is for fewer too, so what
// `count` need is the most of all calls up to it; kept for each shape, since the 32
// layouts take some 60 us.
size_t ortho_workspace(int64_t count, int64_t rows, int64_t cols, int out_dtype) {
  const int64_t n = std::min(rows, cols), m = std::max(rows, cols);
  if (n <= kOrthoNarrow) return ortho_narrow_layout(count, rows, cols).total;
  constexpr size_t kShapes = 1024;
  static std::mutex mutex;
  static std::map<std::tuple<int64_t, int64_t, int>, std::vector<size_t>> kept;
  std::lock_guard<std::mutex> lock(mutex);
  if (kept.size() >= kShapes) kept.clear();
  std::vector<size_t>& most = kept[{n, m, out_dtype}];  // of one matrix, of two, ..
  const size_t together = (size_t)std::min<int64_t>(count, kOrthoWide);
  while (most.size() < together) {
    const size_t one = ortho_layout((int64_t)most.size() + 1, rows, cols, out_dtype).total;
    most.push_back(most.empty() ? one : std::max(one, most.back()));
  }
  return most[together - 1];
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
    hipError_t e;
    if (std::min(a.rows, a.cols) <= kOrthoNarrow) {
      e = launch_ortho_narrow(dtype, a, l, count, st);
    } else {
      e = with_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        square_sum_kernel<T><<<dim3(kSumParts, count), 256, 0, st>>>(a, l);
        first_kernel<T><<<dim3((unsigned)(l.n / 64 * (l.m / 64) + 1), count), 256, 0, st>>>(a, l);
        return hipGetLastError();
      });
      if (e == hipSuccess) e = l.parts == 1 ? steps_of<1>(a, l, count, st) : steps_of<2>(a, l, count, st);
    }
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace adasum
