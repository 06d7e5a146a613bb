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
#include <type_traits>

#include "elem.h"
#include "layer_ops.h"

namespace adasum {
namespace {

using namespace elem;

typedef short v8s __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef __bf16 v8b __attribute__((ext_vector_type(8)));

// A workgroup of eight waves takes 256 columns of x by kTileY of dy and walks
// the rows 32 at a time; a wave holds 64 x kWaveY sums.  16-bit dy: 256 x 256
// outputs, 128 sums a lane.  fp32 dy, with three times the matrix
// instructions and LDS per column: half as many columns of dy.
constexpr int kStep = 32, kChunks = kStep / 8, kThreads = 512, kTileX = 256, kWaveX = 64, kColsX = 4;
template <typename T>
struct Shape {
  static constexpr int kParts = 1, kTileY = 256, kWaveY = 128, kColsY = 4;
};
template <>
struct Shape<float> {
  static constexpr int kParts = 3, kTileY = 128, kWaveY = 64, kColsY = 2;
};
constexpr int kAhead = 2;  // steps whose loads are in flight, and buffers in LDS

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

// LDS holds a column's 32 rows as four 16-byte chunks of eight.  Every four
// columns are a 256-byte line, whose 16 chunks are permuted by the line's
// number: then neither the 16 neighbouring columns that a matrix
// instruction's lanes read, nor the columns that neighbouring threads write
// (every second or fourth), meet in a bank.
__device__ __forceinline__ int chunk_at(int col, int chunk) { return (col * 4 + chunk) ^ ((col >> 2) & 15); }

// The first four waves load and stage x, the other four dy, each thread the
// same few columns of eight rows; all eight run the matrix instructions.  In
// step t a wave computes on one LDS buffer while it stages step t + 1 into
// the next and then asks for step t + 1 + kAhead: one barrier a step, and
// kAhead steps of loads on their way.
template <typename T, bool NARROW>
__global__ __launch_bounds__(kThreads, 2) void linear_grad_kernel(LinearGradArgs a, LinearGradLayout l) {
  using S = Shape<T>;
  constexpr int P = S::kParts, CX = kColsX, CY = S::kColsY;
  constexpr int MX = kWaveX / 16, NY = S::kWaveY / 16, WAVES_X = kTileX / kWaveX;
  static_assert(CY * sizeof(T) == 8, "a row of a thread's columns of dy is two words");
  __shared__ v4u lds_x[kAhead][kTileX * kChunks];
  __shared__ v4u lds_y[kAhead][P][S::kTileY * kChunks];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;

  const int64_t tiles = l.tiles_out * l.tiles_in;
  const int64_t split = blockIdx.x / tiles, tile = blockIdx.x - split * tiles;
  const int64_t tile_o = tile / l.tiles_in, tile_i = tile - tile_o * l.tiles_in;
  const int64_t o0 = tile_o * S::kTileY, i0 = tile_i * kTileX;
  const int64_t r_begin = split * l.split_rows;
  const int rows = (int)std::max<int64_t>(0, std::min(l.split_rows, a.rows - r_begin));  // of this split
  const int64_t nb = (a.in + kScaleBlock - 1) / kScaleBlock;
  const int steps = (rows + kStep - 1) / kStep;

  // This thread's patch: rows 8 k .. 8 k + 7 of columns c .. of x or of dy.
  // Past the edge any column will do, since its sums are not stored; a patch
  // across the edge loads the last whole patch of the row and moves it down
  // by `shift` bits.  (A matrix narrower than a patch is loaded value by
  // value.)
  const bool is_x = wave < 4;
  const int k = wave & 3;
  const int c = lane * (is_x ? CX : CY);
  const int64_t width = is_x ? a.in : a.out, col = (is_x ? i0 : o0) + c;
  const int cols = is_x ? CX : CY;
  const int64_t from = col + cols <= width ? col : width - cols;
  const int shift = !NARROW && col < width && col > from ? (int)(col - from) * (is_x ? 8 : 8 * (int)sizeof(T)) : 0;
  const bool shifts = __ballot(shift != 0) != 0;

  // x: eight rows of codes and one scale byte, of row lane / 8 and block
  // lane % 8 of the wave's eight rows; dy: eight rows of two words
  uint32_t set[kAhead][16];

  // Step t's loads.  A wave's rows are the same for all its lanes: row
  // pointers are scalars, and a lane adds one 32-bit offset, the same for
  // every row.  There is no branch around the loads (steps and rows past the
  // split's end read its last row; trim clears dy's), so that the waits for a
  // step's loads leave the later steps' on their way.
  const uint32_t off0 = (uint32_t)((NARROW ? 0 : from) * (is_x ? 1 : (int64_t)sizeof(T)));
  const uint32_t block = (uint32_t)std::min<int64_t>(i0 / kScaleBlock + (lane & 7), nb - 1);
  auto read = [&](auto x_wave, uint32_t (&w)[16], int t) __attribute__((always_inline)) {
    const int first = std::min(t * kStep + 8 * k, rows - 1), left = rows - 1 - first;
    uint32_t off = off0;
    asm("" : "+v"(off));  // opaque here, so that the address is a scalar and this offset
    if constexpr (decltype(x_wave)::value) {
      const int8_t* x0 = a.codes + (r_begin + first) * a.in;
      const uint8_t* s0 = a.scales + (r_begin + first) * nb;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int row = std::min(e, left);
        const int8_t* x = x0 + row * (int)a.in;
        if constexpr (NARROW) {
          w[e] = 0u;
#pragma unroll
          for (int q = 0; q < CX; ++q)
            w[e] |= (uint32_t)(uint8_t)x[std::min<int64_t>(col + q, width - 1)] << (8 * q);
        } else {
          w[e] = load_at<uint32_t, 1>(x + off);
        }
      }
      w[8] = s0[(uint32_t)(std::min(lane >> 3, left) * (int)nb) + block];
    } else {
      const T* y0 = static_cast<const T*>(a.dy) + (r_begin + first) * a.dy_stride;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const T* y = y0 + std::min(e, left) * (int)a.dy_stride;
        if constexpr (NARROW) {
          w[2 * e] = w[2 * e + 1] = 0u;
#pragma unroll
          for (int q = 0; q < CY; ++q) {
            const T v = y[std::min<int64_t>(col + q, width - 1)];
            if constexpr (sizeof(T) == 4)
              w[2 * e + q] = __builtin_bit_cast(uint32_t, v);
            else
              w[2 * e + q / 2] |= (uint32_t)__builtin_bit_cast(uint16_t, v) << (16 * (q & 1));
          }
        } else {
          const v2u u = load_at<v2u, sizeof(T)>(reinterpret_cast<const char*>(y) + off);
          w[2 * e] = u.x;
          w[2 * e + 1] = u.y;
        }
      }
    }
    __builtin_amdgcn_sched_barrier(0);  // the sets' loads in order: waits count them
  };

  float power[8];
  // column q of the patch of x: eight rows widened, scaled and paired
  auto stage_x = [&](const uint32_t (&s)[16], int buf, int q) __attribute__((always_inline)) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const float x0 = (float)(int8_t)(s[e] >> (8 * q)) * power[e];
      const float x1 = (float)(int8_t)(s[e + 1] >> (8 * q)) * power[e + 1];
      if constexpr (__is_same(T, _Float16)) {
        w[e / 2] = (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)x0) |
                   ((uint32_t)__builtin_bit_cast(uint16_t, (_Float16)x1) << 16);
      } else {
        w[e / 2] = upper_pair(__builtin_bit_cast(uint32_t, x0), __builtin_bit_cast(uint32_t, x1));
      }
    }
    lds_x[buf][chunk_at(c + q, k)] = v4u{w[0], w[1], w[2], w[3]};
  };
  // column q of the patch of dy, fp32 in three parts
  auto stage_y = [&](const uint32_t (&s)[16], int buf, int q) __attribute__((always_inline)) {
    uint32_t w[P][4];
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      if constexpr (P == 3) {
        uint32_t a3[3], b3[3];
        cut3(__builtin_bit_cast(float, s[2 * e + q]), a3);
        cut3(__builtin_bit_cast(float, s[2 * e + 2 + q]), b3);
#pragma unroll
        for (int p = 0; p < 3; ++p) w[p][e / 2] = upper_pair(a3[p], b3[p]);
      } else {
        const uint32_t u = s[2 * e + q / 2], v = s[2 * e + 2 + q / 2];
        w[0][e / 2] = (q & 1) ? upper_pair(u, v) : lower_pair(u, v);
      }
    }
#pragma unroll
    for (int p = 0; p < P; ++p) lds_y[buf][p][chunk_at(c + q, k)] = v4u{w[p][0], w[p][1], w[p][2], w[p][3]};
  };

  // a lane's chunk of column 16 m + (lane & 15) is at 64 m + place[m % 4]
  int place[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) place[j] = chunk_at(lane & 15, lane >> 4) ^ (4 * j);
  const int wx = (wave % WAVES_X) * kWaveX, wy = (wave / WAVES_X) * S::kWaveY;
  v4f acc[MX][NY];
#pragma unroll
  for (int m = 0; m < MX; ++m)
#pragma unroll
    for (int n = 0; n < NY; ++n) acc[m][n] = v4f{0.f, 0.f, 0.f, 0.f};
  // dbias: the tiles of one column of dy take the steps in turn
  float sum[CY];
#pragma unroll
  for (int q = 0; q < CY; ++q) sum[q] = 0.f;
  int turn = (int)tile_i;  // steps until this tile's next

  // step t's loads made ready to be staged
  auto settle = [&](auto x_wave, uint32_t (&w)[16], int t) __attribute__((always_inline)) {
    if constexpr (decltype(x_wave)::value) {
      if (shifts) {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] >>= shift;
      }
      // this lane's power of two, and those of its own columns in all rows
      // from the lanes that hold them
      const float own = w[8] == 255u ? __builtin_nanf("") : __builtin_amdgcn_ldexpf(1.f, (int)w[8] - 127);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        power[e] = __builtin_bit_cast(
            float, __builtin_amdgcn_ds_bpermute((e * 8 + (lane >> 3)) * 4, __builtin_bit_cast(int, own)));
    } else {
      if (shifts) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint64_t v = ((uint64_t)w[2 * e + 1] << 32 | w[2 * e]) >> shift;
          w[2 * e] = (uint32_t)v;
          w[2 * e + 1] = (uint32_t)(v >> 32);
        }
      }
      if ((t + 1) * kStep > rows) {  // trim: no row past the split's end counts
        const int left = rows - t * kStep - 8 * k;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (e >= left) w[2 * e] = w[2 * e + 1] = 0u;
      }
      if (turn == 0) {
#pragma unroll
        for (int q = 0; q < CY; ++q)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if constexpr (P == 3)
              sum[q] += __builtin_bit_cast(float, w[2 * e + q]);
            else
              sum[q] += (float)__builtin_bit_cast(T, (uint16_t)(w[2 * e + q / 2] >> (16 * (q & 1))));
          }
        turn = (int)l.tiles_in;
      }
      --turn;
    }
  };
  auto piece = [&](auto x_wave, const uint32_t (&w)[16], int buf, int q) __attribute__((always_inline)) {
    if constexpr (decltype(x_wave)::value)
      stage_x(w, buf, q);
    else
      stage_y(w, buf, q);
  };
  auto walk = [&](auto x_wave) __attribute__((always_inline)) {
    constexpr int PIECES = decltype(x_wave)::value ? CX : CY, GROUPS = P * NY;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) read(x_wave, set[u], u);
    settle(x_wave, set[0], 0);
#pragma unroll
    for (int q = 0; q < PIECES; ++q) piece(x_wave, set[0], 0, q);
    __builtin_amdgcn_sched_barrier(0);
    read(x_wave, set[0], kAhead);
    __syncthreads();
    // whole rounds of sets: a step past the last adds zeros, where a way out
    // inside the round would make every wait for loads one for all of them
    for (int t0 = 0; t0 < steps; t0 += kAhead) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int t = t0 + u, later = (u + 1) % kAhead;
        // The matrix instructions of this step, and between them the next
        // step's staging into the next buffer, in one basic block, so that
        // the vector unit works while the matrix unit is busy.  (Past the
        // last step the staging writes what nobody reads.)
        settle(x_wave, set[later], t + 1);
        v4u fx[MX], fy[2];
#pragma unroll
        for (int m = 0; m < MX; ++m) fx[m] = lds_x[u][wx * 4 + 64 * m + place[m % 4]];
        fy[0] = lds_y[u][0][wy * 4 + place[0]];
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
          const int n = g % NY, next = g + 1;
          if (next < GROUPS) fy[next % 2] = lds_y[u][next / NY][wy * 4 + 64 * (next % NY) + place[next % NY % 4]];
#pragma unroll
          for (int m = 0; m < MX; ++m) acc[m][n] = multiply<T>(fx[m], fy[g % 2], acc[m][n]);
          if ((g + 1) * PIECES / GROUPS > g * PIECES / GROUPS) piece(x_wave, set[later], later, g * PIECES / GROUPS);
        }
        read(x_wave, set[later], t + 1 + kAhead);
        __syncthreads();
      }
    }
  };
  if (steps > 0) {
    if (is_x)
      walk(std::true_type());
    else
      walk(std::false_type());
  }

  // lane: four consecutive columns of x for one column of dy
  float* part = l.direct ? static_cast<float*>(a.dweight)
                         : reinterpret_cast<float*>(a.ws + l.weight) + split * a.out * a.in;
#pragma unroll
  for (int n = 0; n < NY; ++n) {
    const int64_t o = o0 + wy + n * 16 + (lane & 15);
    if (o >= a.out) continue;
#pragma unroll
    for (int m = 0; m < MX; ++m) {
      const int64_t i = i0 + wx + m * 16 + (lane >> 4) * 4;
      const float v[4] = {acc[m][n][0], acc[m][n][1], acc[m][n][2], acc[m][n][3]};
      store_row<float, 4>(part + o * a.in + i, v, (int)std::min<int64_t>(a.in - i, 4));
    }
  }
  if (a.dbias) {
    // the row groups' sums, added in their order
    float* sums = reinterpret_cast<float*>(&lds_x[0][0]);  // [4][kTileY]; every wave is past its reads
    if (!is_x) {
#pragma unroll
      for (int q = 0; q < CY; ++q) sums[k * S::kTileY + c + q] = sum[q];
    }
    __syncthreads();
    const int64_t o = o0 + tid;
    if (tid < S::kTileY && o < a.out) {
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < kChunks; ++e) s += sums[e * S::kTileY + tid];
      reinterpret_cast<float*>(a.ws + l.bias)[(split * l.tiles_in + tile_i) * a.out + o] = s;
    }
  }
}

// Partial sums added in their order in fp64: of `count` values, `parts`
// arrays each, four values a thread.
struct JoinPart {
  const float* parts;
  int count_parts;
  int64_t count;
  void* out;
};
__device__ __forceinline__ void join_values(const JoinPart& j, int64_t i, int dtype, int accumulate) {
  const int valid = (int)std::min<int64_t>(j.count - i, 4);
  double s[4] = {0.0, 0.0, 0.0, 0.0};
#pragma unroll 4
  for (int p = 0; p < j.count_parts; ++p) {
    float v[4];
    load_row<float, 4>(j.parts + p * j.count + i, valid, v);
#pragma unroll
    for (int q = 0; q < 4; ++q) s[q] += (double)v[q];
  }
#pragma unroll
  for (int q = 0; q < 4; ++q)
    if (q < valid)
      store_any(j.out, dtype, i + q, accumulate ? s[q] + (double)load_any(j.out, dtype, i + q) : s[q]);
}
// dweight's blocks first, then dbias's
__global__ __launch_bounds__(256) void linear_join_kernel(JoinPart weight, JoinPart bias, int weight_blocks, int dtype,
                                                          int accumulate) {
  const bool is_bias = (int)blockIdx.x >= weight_blocks;
  const JoinPart& j = is_bias ? bias : weight;
  const int64_t first = ((int64_t)(is_bias ? blockIdx.x - weight_blocks : blockIdx.x) * 256 + threadIdx.x) * 4;
  const int64_t step = (int64_t)(is_bias ? gridDim.x - weight_blocks : weight_blocks) * 1024;
  for (int64_t i = first; i < j.count; i += step) join_values(j, i, dtype, accumulate);
}

size_t align256(size_t b) { return (b + 255) & ~size_t(255); }

}  // namespace

LinearGradLayout linear_grad_layout(int64_t rows, int64_t out, int64_t in, int dtype) {
  LinearGradLayout l{};
  l.tiles_out = ceil_div(out, dtype == 0 ? Shape<float>::kTileY : Shape<__bf16>::kTileY);
  l.tiles_in = ceil_div(in, kTileX);
  const int64_t tiles = l.tiles_out * l.tiles_in, steps = std::max<int64_t>(1, ceil_div(rows, kStep));
  // One workgroup per CU at a time.  The number of splits that takes the
  // fewest rounds of steps, where a workgroup's start and end count as four
  // steps, and every split's partial sums as a step of all tiles' outputs.
  int64_t best = 1, cost = INT64_MAX;
  for (int64_t s = 1; s <= std::min<int64_t>(steps, 256) && (s - 1) * tiles < 2 * kCUs; ++s) {
    const int64_t c = ceil_div(tiles * s, kCUs) * (ceil_div(steps, s) + 4) + (s > 1 ? 2 + ceil_div(s * tiles, kCUs) : 0);
    if (c < cost) {
      cost = c;
      best = s;
    }
  }
  l.split_rows = ceil_div(steps, best) * kStep;
  l.splits = (int)std::max<int64_t>(1, ceil_div(rows, l.split_rows));
  size_t at = 0;
  l.weight = at;
  at += align256((size_t)l.splits * out * in * 4);
  l.bias = at;
  at += align256((size_t)l.splits * l.tiles_in * out * 4);
  l.total = at;
  return l;
}

hipError_t launch_linear_grad(int dtype, const LinearGradArgs& a, hipStream_t st) {
  LinearGradLayout l = linear_grad_layout(a.rows, a.out, a.in, dtype);
  l.direct = l.splits == 1 && a.grad_dtype == 0 && !a.accumulate;
  const unsigned blocks = (unsigned)(l.tiles_out * l.tiles_in * l.splits);
  hipError_t e = with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    if (a.out < Shape<T>::kColsY || a.in < kColsX)
      linear_grad_kernel<T, true><<<blocks, kThreads, 0, st>>>(a, l);
    else
      linear_grad_kernel<T, false><<<blocks, kThreads, 0, st>>>(a, l);
    return hipGetLastError();
  });
  if (e != hipSuccess || (l.direct && !a.dbias)) return e;
  JoinPart weight{reinterpret_cast<const float*>(a.ws + l.weight), l.splits, a.out * a.in, a.dweight};
  JoinPart bias{reinterpret_cast<const float*>(a.ws + l.bias), (int)(l.splits * l.tiles_in), a.out, a.dbias};
  const int weight_blocks = l.direct ? 0 : (int)std::min<int64_t>(ceil_div(weight.count, 1024), 16 * kCUs);
  const int bias_blocks = a.dbias ? (int)ceil_div(bias.count, 1024) : 0;
  linear_join_kernel<<<weight_blocks + bias_blocks, 256, 0, st>>>(weight, bias, weight_blocks, a.grad_dtype,
                                                                  a.accumulate);
  e = hipGetLastError();
  return e;
}

}  // namespace adasum
