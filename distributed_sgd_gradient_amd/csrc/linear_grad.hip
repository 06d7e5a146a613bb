// linear_grad.hip - gradient of a linear layer's weight and bias from kept
// 8-bit activations:
//
//   dweight[o][i] = sum over rows r of dy[r][o] x[r][i],  x = code * 2^e
//   dbias[o]      = sum over rows r of dy[r][o]
//
// on the matrix cores.  The sum runs over the slow axis of both operands, the
// rows, while a matrix instruction takes eight consecutive terms of the sum
// per lane.  So a thread loads the same few columns of eight rows and turns
// the 8 x 4 patch while it writes it to LDS, where a column's rows are then
// consecutive.
//
// Products are exact: a code times a power of two has 7 significant bits and
// is a bf16 value, and an fp16 value too where fp16 activations were packed.
// So 16-bit dy meets x in its own type; fp32 dy is cut into three bf16 parts
// of 8 bits each, hi + mid + lo = dy exactly, that meet x one after another.
// Sums are fp32 within a split of the rows; splits are joined in fp64.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "elem.h"
#include "layer_ops.h"

namespace adasum {
namespace {

using namespace elem;

constexpr int kTile = 128;  // outputs of a workgroup along either side
typedef short v8s __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef __bf16 v8b __attribute__((ext_vector_type(8)));

template <typename T>
struct Cut;  // how dy of type T meets the matrix cores
template <>
struct Cut<__bf16> {
  static constexpr int kParts = 1, kStep = 64;
};
template <>
struct Cut<_Float16> {
  static constexpr int kParts = 1, kStep = 64;
};
template <>
struct Cut<float> {
  static constexpr int kParts = 3, kStep = 32;
};

template <typename T>
__device__ __forceinline__ v4f multiply(v4u a, v4u b, v4f c) {
  if constexpr (__is_same(T, _Float16))
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8b, a), __builtin_bit_cast(v8b, b), c, 0, 0, 0);
}

// hi + mid + lo = v, each a bf16 (as the upper half of an fp32): cutting off
// the low bits leaves remainders that are exact.  An infinity or NaN stays in
// hi.
__device__ __forceinline__ void cut3(float v, uint32_t (&part)[3]) {
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  const bool finite = (u & 0x7f800000u) != 0x7f800000u;
  uint32_t h = u & 0xffff0000u;
  if (!finite && (u & 0x7fffffu) != 0u) h |= 0x400000u;  // a NaN whose payload is cut off
  part[0] = h;
  const float r1 = finite ? v - __builtin_bit_cast(float, h) : 0.f;
  part[1] = __builtin_bit_cast(uint32_t, r1) & 0xffff0000u;
  part[2] = __builtin_bit_cast(uint32_t, r1 - __builtin_bit_cast(float, part[1]));
}

// The upper halves of two words as one: a's in the low half.
__device__ __forceinline__ uint32_t upper_pair(uint32_t a, uint32_t b) {
  return __builtin_amdgcn_perm(b, a, 0x07060302u);
}
__device__ __forceinline__ uint32_t lower_pair(uint32_t a, uint32_t b) {
  return __builtin_amdgcn_perm(b, a, 0x05040100u);
}

// LDS holds, per part, 128 columns of kStep rows each as 16-byte chunks of
// eight rows.  A column's chunks are permuted by its number, so that the 16
// columns that a matrix instruction's lanes read side by side, and the columns
// that neighbouring threads write, lie in different banks.
template <int STEP>
__device__ __forceinline__ int chunk_at(int col, int chunk) {
  constexpr int N = STEP / 8;
  return col * N + (chunk ^ ((col >> 1) & (N - 1)));
}

template <typename T>
__global__ __launch_bounds__(256) void linear_grad_kernel(LinearGradArgs a, LinearGradLayout l) {
  constexpr int P = Cut<T>::kParts, STEP = Cut<T>::kStep, CH = STEP / 8;
  constexpr int COLS = kTile * CH / 256;  // columns of a thread's patch: 4, or 2 where a step is 32 rows
  __shared__ v4u lds_y[2][P][kTile * CH];
  __shared__ v4u lds_x[2][kTile * CH];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int64_t o0 = (int64_t)(blockIdx.x % l.tiles_out) * kTile;
  const int64_t i0 = (int64_t)(blockIdx.x / l.tiles_out) * kTile;
  const int64_t r_begin = (int64_t)blockIdx.y * l.split_rows;
  const int64_t r_end = std::min(r_begin + l.split_rows, a.rows);
  const int64_t nb = (a.in + kScaleBlock - 1) / kScaleBlock;

  // this thread's patch: columns c .. c + COLS - 1 of rows 8 k .. 8 k + 7
  const int c = (tid % (kTile / COLS)) * COLS, k = tid / (kTile / COLS);
  const int valid_y = (int)std::min<int64_t>(a.out - (o0 + c), COLS);
  const int valid_x = (int)std::min<int64_t>(a.in - (i0 + c), COLS);
  const T* dy = static_cast<const T*>(a.dy) + o0 + c;
  const int8_t* codes = a.codes + i0 + c;
  const uint8_t* scales = a.scales + (i0 + c) / kScaleBlock;
  const bool bias = i0 == 0 && a.dbias != nullptr;

  uint32_t py[8][COLS * sizeof(T) / 4];  // the patch of dy, as loaded
  uint32_t px[8];
  uint32_t ps[8];
  float sum[COLS];
#pragma unroll
  for (int q = 0; q < COLS; ++q) sum[q] = 0.f;

  auto fetch = [&](int64_t r0) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int64_t r = r0 + 8 * k + e;
      const bool in_rows = r < r_end;
      constexpr int W = COLS * sizeof(T) / 4;
#pragma unroll
      for (int w = 0; w < W; ++w) py[e][w] = 0u;
      px[e] = 0u;
      ps[e] = 127u;
      if (in_rows && valid_y == COLS) {
        if constexpr (W == 2) {
          const v2u t = load_at<v2u, sizeof(T)>(dy + r * a.dy_stride);
          py[e][0] = t.x;
          py[e][1] = t.y;
        } else {
          py[e][0] = load_at<uint32_t, sizeof(T)>(dy + r * a.dy_stride);
        }
      } else if (in_rows) {
#pragma unroll
        for (int q = 0; q < COLS; ++q)
          if (q < valid_y) {
            if constexpr (sizeof(T) == 4)
              py[e][q] = __builtin_bit_cast(uint32_t, dy[r * a.dy_stride + q]);
            else
              py[e][q / 2] |= (uint32_t)__builtin_bit_cast(uint16_t, dy[r * a.dy_stride + q]) << (16 * (q & 1));
          }
      }
      if (in_rows && valid_x == COLS) {
        if constexpr (COLS == 4)
          px[e] = load_at<uint32_t, 1>(codes + r * a.in);
        else
          px[e] = load_at<uint16_t, 1>(codes + r * a.in);
      } else if (in_rows) {
#pragma unroll
        for (int q = 0; q < COLS; ++q)
          if (q < valid_x) px[e] |= (uint32_t)(uint8_t)codes[r * a.in + q] << (8 * q);
      }
      if (in_rows && valid_x > 0) ps[e] = scales[r * nb];
    }
  };

  auto stage = [&](int buf) {
    // x: eight rows of a column, widened, scaled and paired
    float s[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] = scale_value(ps[e]);
#pragma unroll
    for (int q = 0; q < COLS; ++q) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const float x0 = (float)(int8_t)(px[e] >> (8 * q)) * s[e];
        const float x1 = (float)(int8_t)(px[e + 1] >> (8 * q)) * s[e + 1];
        if constexpr (__is_same(T, _Float16)) {
          w[e / 2] = (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)x0) |
                     ((uint32_t)__builtin_bit_cast(uint16_t, (_Float16)x1) << 16);
        } else {
          w[e / 2] = upper_pair(__builtin_bit_cast(uint32_t, x0), __builtin_bit_cast(uint32_t, x1));
        }
      }
      lds_x[buf][chunk_at<STEP>(c + q, k)] = v4u{w[0], w[1], w[2], w[3]};
    }
    // dy: the same columns turned, fp32 in three parts
#pragma unroll
    for (int q = 0; q < COLS; ++q) {
      uint32_t w[P][4];
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        if constexpr (P == 3) {
          uint32_t a3[3], b3[3];
          cut3(__builtin_bit_cast(float, py[e][q]), a3);
          cut3(__builtin_bit_cast(float, py[e + 1][q]), b3);
#pragma unroll
          for (int p = 0; p < 3; ++p) w[p][e / 2] = upper_pair(a3[p], b3[p]);
        } else {
          w[0][e / 2] = (q & 1) ? upper_pair(py[e][q / 2], py[e + 1][q / 2]) : lower_pair(py[e][q / 2], py[e + 1][q / 2]);
        }
      }
#pragma unroll
      for (int p = 0; p < P; ++p) lds_y[buf][p][chunk_at<STEP>(c + q, k)] = v4u{w[p][0], w[p][1], w[p][2], w[p][3]};
      if (bias) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if constexpr (P == 3)
            sum[q] += __builtin_bit_cast(float, py[e][q]);
          else
            sum[q] += (float)__builtin_bit_cast(T, (uint16_t)(py[e][q / 2] >> (16 * (q & 1))));
        }
      }
    }
  };

  // a wave's quarter: 64 columns of x by 64 columns of dy
  const int wx = (wave & 1) * 64, wy = (wave >> 1) * 64;
  v4f acc[4][4];
#pragma unroll
  for (int m = 0; m < 4; ++m)
#pragma unroll
    for (int n = 0; n < 4; ++n) acc[m][n] = v4f{0.f, 0.f, 0.f, 0.f};

  fetch(r_begin);
  int buf = 0;
  for (int64_t r = r_begin; r < r_end; r += STEP, buf ^= 1) {
    stage(buf);
    __syncthreads();
    if (r + STEP < r_end) fetch(r + STEP);
#pragma unroll
    for (int kk = 0; kk < STEP / 32; ++kk) {
      v4u fx[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) fx[m] = lds_x[buf][chunk_at<STEP>(wx + m * 16 + (lane & 15), kk * 4 + (lane >> 4))];
#pragma unroll
      for (int p = 0; p < P; ++p) {
        v4u fy[4];
#pragma unroll
        for (int n = 0; n < 4; ++n)
          fy[n] = lds_y[buf][p][chunk_at<STEP>(wy + n * 16 + (lane & 15), kk * 4 + (lane >> 4))];
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
          for (int n = 0; n < 4; ++n) acc[m][n] = multiply<T>(fx[m], fy[n], acc[m][n]);
      }
    }
    // one barrier a step: a buffer is written again only after the next
    // step's barrier, which every wave reaches past its reads of it
  }

  // lane: four consecutive columns of x for one column of dy
  const bool join = l.splits > 1;
  float* part = reinterpret_cast<float*>(a.ws + l.weight) + (int64_t)blockIdx.y * a.out * a.in;
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    const int64_t o = o0 + wy + n * 16 + (lane & 15);
    if (o >= a.out) continue;
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const int64_t i = i0 + wx + m * 16 + (lane >> 4) * 4;
      const int valid = (int)std::min<int64_t>(a.in - i, 4);
      const float v[4] = {acc[m][n][0], acc[m][n][1], acc[m][n][2], acc[m][n][3]};
      if (join) {
        store_row<float, 4>(part + o * a.in + i, v, valid);
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (q < valid) {
            const int64_t at = o * a.in + i + q;
            store_any(a.dweight, a.grad_dtype, at,
                      a.accumulate ? (double)v[q] + (double)load_any(a.dweight, a.grad_dtype, at) : (double)v[q]);
          }
      }
    }
  }
  if (bias) {
    // the row groups' sums, added in their order
    __syncthreads();
    float* sums = reinterpret_cast<float*>(&lds_x[0][0]);  // [CH][kTile]
#pragma unroll
    for (int q = 0; q < COLS; ++q) sums[k * kTile + c + q] = sum[q];
    __syncthreads();
    const int64_t o = o0 + tid;
    if (tid < kTile && o < a.out) {
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < CH; ++e) s += sums[e * kTile + tid];
      if (join)
        reinterpret_cast<float*>(a.ws + l.bias)[(int64_t)blockIdx.y * a.out + o] = s;
      else
        store_any(a.dbias, a.grad_dtype, o,
                  a.accumulate ? (double)s + (double)load_any(a.dbias, a.grad_dtype, o) : (double)s);
    }
  }
}

// The splits' partial sums, added in their order in fp64; count values each.
__global__ __launch_bounds__(256) void linear_join_kernel(const float* parts, int splits, int64_t count, void* out,
                                                          int dtype, int accumulate) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < count; i += (int64_t)gridDim.x * 256) {
    double s = 0.0;
#pragma unroll 8
    for (int p = 0; p < splits; ++p) s += (double)parts[p * count + i];
    store_any(out, dtype, i, accumulate ? s + (double)load_any(out, dtype, i) : s);
  }
}

size_t align256(size_t b) { return (b + 255) & ~size_t(255); }

}  // namespace

LinearGradLayout linear_grad_layout(int64_t rows, int64_t out, int64_t in, int dtype) {
  LinearGradLayout l{};
  l.tiles_out = ceil_div(out, kTile);
  l.tiles_in = ceil_div(in, kTile);
  const int step = dtype == 0 ? Cut<float>::kStep : Cut<__bf16>::kStep;
  const int64_t tiles = l.tiles_out * l.tiles_in;
  // two workgroups per CU, of at least four steps each
  const int64_t want = std::max<int64_t>(1, 2 * kCUs / tiles);
  const int64_t most = std::max<int64_t>(1, rows / (4 * step));
  const int64_t splits = std::min<int64_t>({want, most, 256});
  l.split_rows = std::max<int64_t>(step, ceil_div(ceil_div(rows, splits), step) * step);
  l.splits = (int)std::max<int64_t>(1, ceil_div(rows, l.split_rows));
  if (l.splits > 1) {
    l.weight = 0;
    l.bias = align256((size_t)l.splits * out * in * 4);
    l.total = l.bias + align256((size_t)l.splits * out * 4);
  }
  return l;
}

hipError_t launch_linear_grad(int dtype, const LinearGradArgs& a, hipStream_t st) {
  const LinearGradLayout l = linear_grad_layout(a.rows, a.out, a.in, dtype);
  const dim3 grid((unsigned)(l.tiles_out * l.tiles_in), (unsigned)l.splits);
  hipError_t e = with_dtype(dtype, [&](auto t) {
    linear_grad_kernel<decltype(t)><<<grid, 256, 0, st>>>(a, l);
    return hipGetLastError();
  });
  if (e != hipSuccess || l.splits == 1) return e;
  const int64_t count = a.out * a.in;
  linear_join_kernel<<<(unsigned)std::min<int64_t>(ceil_div(count, 256), 16 * kCUs), 256, 0, st>>>(
      reinterpret_cast<const float*>(a.ws + l.weight), l.splits, count, a.dweight, a.grad_dtype, a.accumulate);
  e = hipGetLastError();
  if (e != hipSuccess || a.dbias == nullptr) return e;
  linear_join_kernel<<<(unsigned)ceil_div(a.out, 256), 256, 0, st>>>(
      reinterpret_cast<const float*>(a.ws + l.bias), l.splits, a.out, a.dbias, a.grad_dtype, a.accumulate);
  return hipGetLastError();
}

}  // namespace adasum
