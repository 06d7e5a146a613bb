// linear_grad.hip - gradient of a linear layer's weight and bias from kept
// 8-bit activations:
//
//   dweight[o][i] = sum over rows r of dy[r][o] x[r][i],  x = code * 2^e
//   dbias[o]      = sum over rows r of dy[r][o]
//
// on the matrix cores.  The sum runs over the slow axis of both operands, the
// rows, while a matrix instruction takes eight consecutive terms of the sum
// per lane.  So rows are staged in LDS as they lie in memory, as 16-bit
// values, and turned by the transposing LDS reads, which give a lane four
// rows of its column.
//
// Products are exact: a code times a power of two has 7 significant bits and
// is a bf16 value, and an fp16 value too where fp16 activations were packed.
// So 16-bit dy meets x in its own type; fp32 dy is cut into three bf16 parts
// of 8 bits each, hi + mid + lo = dy exactly, that meet x one after another.
// Sums are fp32 within a split of the rows, of at most 65536; splits are joined
// in fp64.
//
// Bound by the matrix cores and what shares a CU with them: of 65536 x 4096 x
// 1024 in bf16, 485 to 508 us in all on different cards (1080 to 1130 TFLOP/s;
// a large library product reaches 1225), the matrix instructions and LDS reads alone take 330
// us, with the loads 340, with the staging (widening the codes, LDS writes)
// 430.  fp32 dy costs three times the matrix instructions: 16384 x 4096 x 1024
// in 370 us.  Tried and dropped: a patch of columns turned in registers before
// LDS (707 us against 590 of the transposing reads, under a profiler), 64 rows
// a step, three steps of loads ahead (registers spill), raised wave priority
// around the matrix instructions.
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
// instructions and LDS per column: half as many columns of dy.  A thread
// stages kVecX codes of each of two rows, or kVecY values of dy of kRowsY.
constexpr int kStep = 32, kThreads = 512, kTileX = 256, kWaveX = 64, kVecX = 16, kRowsX = 2, kVecY = 8;
template <typename T>
struct Shape {
  static constexpr int kParts = 1, kTileY = 256, kWaveY = 128;
};
template <>
struct Shape<float> {
  static constexpr int kParts = 3, kTileY = 128, kWaveY = 64;
};
constexpr int kXCDs = 8, kRunSteps = 128;
constexpr int kJoinRuns = 16, kManyParts = 32;
constexpr int kAhead = 2;  // steps whose loads are in flight, and buffers in LDS

template <typename T>
__device__ __forceinline__ v4f multiply(v4u a, v4u b, v4f c) {
  if constexpr (__is_same(T, _Float16))
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8b, a), __builtin_bit_cast(v8b, b), c, 0, 0, 0);
}

// hi + mid + lo = v, each a bf16 (as the upper half of an fp32): cutting off
// the low bits leaves remainders that are exact.  Bits of v below 2^-133, the
// least bf16, are lost.  An infinity or NaN stays in hi.
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

// LDS holds a step's rows of `cols` 16-bit values each, as segments of 16
// columns that are permuted within the row by the row's number: a transposing
// read takes the same segment of 16 rows, which would otherwise lie in the
// same eight banks.
__device__ __forceinline__ int segment_key(int row) { return (row & 3) | ((row >> 1) & 4); }
// 16-byte piece `piece` (eight columns) of a row, in units of 16 bytes
__device__ __forceinline__ int piece_at(int row, int piece, int cols) {
  return row * (cols / 8) + (piece ^ (segment_key(row) * 2));
}

typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s* lds_v4s;
// Eight rows of a lane's column: lane i of 16 names four columns of row i / 4,
// and gets column i of the four rows; `at` is the byte address for the first
// four of the eight rows, `pitch` a row's bytes.
__device__ __forceinline__ v4u turned(const v4u* base, uint32_t at, int pitch) {
  const char* p = reinterpret_cast<const char*>(base) + at;
  const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)(p));
  const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)(p + 4 * pitch));
  return __builtin_bit_cast(v4u, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// Four words moved down by `bits` below 128.
__device__ __forceinline__ void shift_down(uint32_t* w, int bits) {
  const uint64_t lo = (uint64_t)w[1] << 32 | w[0], hi = (uint64_t)w[3] << 32 | w[2];
  const int b = bits & 63;
  const uint64_t both = (lo >> b) | ((hi << 1) << (63 - b));
  const uint64_t l = bits >= 64 ? hi >> b : both, h = bits >= 64 ? 0u : hi >> b;
  w[0] = (uint32_t)l;
  w[1] = (uint32_t)(l >> 32);
  w[2] = (uint32_t)h;
  w[3] = (uint32_t)(h >> 32);
}

// The first four waves load and stage x, the other four dy, each thread the
// same columns of its rows; all eight run the matrix instructions.  In step t
// a wave computes on one LDS buffer while it stages step t + 1 into the next
// and then asks for step t + 1 + kAhead: one barrier a step, and kAhead steps
// of loads on their way.
template <typename T, bool NARROW_X, bool NARROW_Y>
__global__ __launch_bounds__(kThreads, 2) void linear_grad_kernel(LinearGradArgs a, LinearGradLayout l) {
  using S = Shape<T>;
  constexpr int P = S::kParts, TY = S::kTileY;
  constexpr int MX = kWaveX / 16, NY = S::kWaveY / 16, WAVES_X = kTileX / kWaveX;
  // four waves, each with 64 / (columns / a lane's) rows at a time
  constexpr int LANES_X = kTileX / kVecX, LANES_Y = TY / kVecY;  // lanes of a row
  constexpr int PASS_X = 4 * 64 / LANES_X, PASS_Y = 4 * 64 / LANES_Y, ROWS_Y = kStep / PASS_Y;
  static_assert(PASS_X * kRowsX == kStep && ROWS_Y * kVecY * sizeof(T) == 64, "16 words a thread and step");
  __shared__ v4u lds_x[kAhead][kStep * kTileX / 8];
  __shared__ v4u lds_y[kAhead][P][kStep * TY / 8];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;

  // Workgroups are dealt to the eight XCDs in turn.  Where splits are long,
  // each XCD takes a run of consecutive tiles, which share rows of dy and x in
  // its L2.  65536 x 4096 x 1024 bf16 (512 steps a split): 484 us against 533
  // without; 2047 x 769 x 1001 fp32 (8 steps): 36 against 32; equal at 64.
  const uint32_t xcd = blockIdx.x % kXCDs, whole = gridDim.x / kXCDs, rest = gridDim.x % kXCDs;
  const uint32_t block =
      l.split_rows >= kRunSteps * kStep ? xcd * whole + std::min(xcd, rest) + blockIdx.x / kXCDs : blockIdx.x;
  const int64_t tiles = l.tiles_out * l.tiles_in;
  const int64_t split = block / tiles, tile = block - split * tiles;
  const int64_t tile_o = tile / l.tiles_in, tile_i = tile - tile_o * l.tiles_in;
  const int64_t o0 = tile_o * TY, i0 = tile_i * kTileX;
  const int64_t r_begin = split * l.split_rows;
  const int rows = (int)std::max<int64_t>(0, std::min(l.split_rows, a.rows - r_begin));  // of this split
  const int64_t nb = (a.in + kScaleBlock - 1) / kScaleBlock;
  const int steps = (rows + kStep - 1) / kStep;

  // This thread's columns c .. of x or of dy, of the step's rows my_row +
  // PASS u.  Past the edge any column will do, since its sums are not stored;
  // columns across the edge are loaded as the last whole vector of the row
  // and moved down by `shift` bits.  (A matrix narrower than a vector is
  // loaded value by value.)
  const bool is_x = wave < 4, narrow = is_x ? NARROW_X : NARROW_Y;
  const int in_row = lane & ((is_x ? LANES_X : LANES_Y) - 1);
  const int my_row = ((wave & 3) * 64 + lane) / (is_x ? LANES_X : LANES_Y);
  const int cols = is_x ? kVecX : kVecY, c = in_row * cols;
  const int64_t width = is_x ? a.in : a.out, col = (is_x ? i0 : o0) + c;
  const int64_t from = col + cols <= width ? col : width - cols;
  const int shift = !narrow && col < width && col > from ? (int)(col - from) * (is_x ? 8 : 8 * (int)sizeof(T)) : 0;
  const bool shifts = __ballot(shift != 0) != 0;

  // x: two rows of 16 codes, and their scale bytes in `byte`; dy: 64 bytes of
  // ROWS_Y rows
  uint32_t set[kAhead][16], byte[kAhead][kRowsX];

  // Step t's loads.  There is no branch around them (steps and rows past the
  // split's end read its last row; trim clears dy's), so that the waits for a
  // step's loads leave the later steps' on their way.  A row's offset is 32 x
  // 32 bits.
  const char* const base = is_x ? reinterpret_cast<const char*>(a.codes + r_begin * a.in + (narrow ? 0 : from))
                                : reinterpret_cast<const char*>(static_cast<const T*>(a.dy) + r_begin * a.dy_stride +
                                                                (narrow ? 0 : from));
  const uint8_t* const scale_base = a.scales + r_begin * nb + std::min<int64_t>(col / kScaleBlock, nb - 1);
  const uint32_t pitch = is_x ? (uint32_t)a.in : (uint32_t)(a.dy_stride * sizeof(T));
  auto read = [&](auto x_wave, uint32_t (&w)[16], uint32_t (&b)[kRowsX], int t) __attribute__((always_inline)) {
    if constexpr (decltype(x_wave)::value) {
#pragma unroll
      for (int u = 0; u < kRowsX; ++u) {
        const uint32_t row = (uint32_t)std::min(t * kStep + PASS_X * u + my_row, rows - 1);
        const char* x = base + (uint64_t)row * pitch;
        if constexpr (NARROW_X) {
#pragma unroll
          for (int i = 0; i < 4; ++i) w[4 * u + i] = 0u;
#pragma unroll
          for (int i = 0; i < kVecX; ++i)
            w[4 * u + i / 4] |= (uint32_t)(uint8_t)x[std::min<int64_t>(col + i, width - 1)] << (8 * (i & 3));
        } else {
          const v4u v = load_at<v4u, 1>(x);
          w[4 * u] = v.x; w[4 * u + 1] = v.y; w[4 * u + 2] = v.z; w[4 * u + 3] = v.w;
        }
        b[u] = scale_base[(uint64_t)row * (uint32_t)nb];
      }
    } else {
      constexpr int W = 16 / ROWS_Y;  // words of a row
#pragma unroll
      for (int u = 0; u < ROWS_Y; ++u) {
        const uint32_t row = (uint32_t)std::min(t * kStep + PASS_Y * u + my_row, rows - 1);
        const char* y = base + (uint64_t)row * pitch;
        if constexpr (NARROW_Y) {
#pragma unroll
          for (int i = 0; i < W; ++i) w[W * u + i] = 0u;
#pragma unroll
          for (int i = 0; i < kVecY; ++i) {
            const T v = reinterpret_cast<const T*>(y)[std::min<int64_t>(col + i, width - 1)];
            if constexpr (sizeof(T) == 4)
              w[W * u + i] = __builtin_bit_cast(uint32_t, v);
            else
              w[W * u + i / 2] |= (uint32_t)__builtin_bit_cast(uint16_t, v) << (16 * (i & 1));
          }
        } else {
#pragma unroll
          for (int i = 0; i < W; i += 4) {
            const v4u v = load_at<v4u, sizeof(T)>(y + 4 * i);
            w[W * u + i] = v.x; w[W * u + i + 1] = v.y; w[W * u + i + 2] = v.z; w[W * u + i + 3] = v.w;
          }
        }
      }
    }
    __builtin_amdgcn_sched_barrier(0);  // the sets' loads in order: waits count them
  };

  float power[kRowsX];
  // Eight codes widened and scaled: piece q of the thread's four.  Every other
  // four lanes take a row's second half first, so that eight lanes' pieces
  // fill 128 bytes of banks (without: eight more cycles a write; 65536 x 4096
  // x 1024 in turns 516 us against 508).
  const int second = (lane >> 2) & 1;
  auto stage_x = [&](const uint32_t (&s)[16], int buf, int q) __attribute__((always_inline)) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const uint32_t four = (second ? s[(2 * q + e / 4) ^ 2] : s[2 * q + e / 4]) >> (8 * (e & 3));
      const float x0 = (float)(int8_t)four * power[q / 2], x1 = (float)(int8_t)(four >> 8) * power[q / 2];
      if constexpr (__is_same(T, _Float16)) {
        w[e / 2] = (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)x0) |
                   ((uint32_t)__builtin_bit_cast(uint16_t, (_Float16)x1) << 16);
      } else {
        w[e / 2] = upper_pair(__builtin_bit_cast(uint32_t, x0), __builtin_bit_cast(uint32_t, x1));
      }
    }
    const int at = piece_at(my_row + PASS_X * (q / 2), 2 * in_row + ((q & 1) ^ second), kTileX);
    lds_x[buf][at] = v4u{w[0], w[1], w[2], w[3]};
  };
  // eight values of row q of the thread's rows of dy, fp32 in three parts
  auto stage_y = [&](const uint32_t (&s)[16], int buf, int q) __attribute__((always_inline)) {
    const int at = piece_at(my_row + PASS_Y * q, in_row, TY);
    if constexpr (P == 1) {
      lds_y[buf][0][at] = v4u{s[4 * q], s[4 * q + 1], s[4 * q + 2], s[4 * q + 3]};
    } else {
      uint32_t w[P][4];
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        uint32_t a3[3], b3[3];
        cut3(__builtin_bit_cast(float, s[8 * q + e]), a3);
        cut3(__builtin_bit_cast(float, s[8 * q + e + 1]), b3);
#pragma unroll
        for (int p = 0; p < 3; ++p) w[p][e / 2] = upper_pair(a3[p], b3[p]);
      }
#pragma unroll
      for (int p = 0; p < P; ++p) lds_y[buf][p][at] = v4u{w[p][0], w[p][1], w[p][2], w[p][3]};
    }
  };

  // byte addresses of a lane's part of 16 columns, for its wave's m-th
  const int wx = (wave % WAVES_X) * kWaveX, wy = (wave / WAVES_X) * S::kWaveY;
  uint32_t at_x[MX], at_y[NY];
  {
    const int row = (lane >> 4) * 8 + ((lane & 15) >> 2), part = (lane & 3) * 8;
#pragma unroll
    for (int m = 0; m < MX; ++m)
      at_x[m] = (uint32_t)(row * kTileX * 2 + ((wx / 16 + m) ^ segment_key(row)) * 32 + part);
#pragma unroll
    for (int n = 0; n < NY; ++n)
      at_y[n] = (uint32_t)(row * TY * 2 + ((wy / 16 + n) ^ segment_key(row)) * 32 + part);
  }
  v4f acc[MX][NY];
#pragma unroll
  for (int m = 0; m < MX; ++m)
#pragma unroll
    for (int n = 0; n < NY; ++n) acc[m][n] = v4f{0.f, 0.f, 0.f, 0.f};
  // dbias: the tiles of one column of dy take the steps in turn
  float sum[kVecY];
#pragma unroll
  for (int q = 0; q < kVecY; ++q) sum[q] = 0.f;
  int turn = (int)tile_i;  // steps until this tile's next

  // step t's loads made ready to be staged
  auto settle = [&](auto x_wave, uint32_t (&w)[16], const uint32_t (&b)[kRowsX], int t) __attribute__((always_inline)) {
    if constexpr (decltype(x_wave)::value) {
      if (shifts) {
#pragma unroll
        for (int u = 0; u < kRowsX; ++u) shift_down(&w[4 * u], shift);
      }
#pragma unroll
      for (int u = 0; u < kRowsX; ++u) power[u] = scale_value(b[u]);
    } else {
      if (shifts) {
        if constexpr (sizeof(T) == 2) {
#pragma unroll
          for (int u = 0; u < ROWS_Y; ++u) shift_down(&w[4 * u], shift);
        } else {
#pragma unroll
          for (int u = 0; u < ROWS_Y; ++u)
#pragma unroll
            for (int bit = 0; bit < 3; ++bit)
              if ((shift >> (5 + bit)) & 1) {
#pragma unroll
                for (int i = 0; i + (1 << bit) < 8; ++i) w[8 * u + i] = w[8 * u + i + (1 << bit)];
              }
        }
      }
      if ((t + 1) * kStep > rows) {  // trim: no row past the split's end counts
#pragma unroll
        for (int u = 0; u < ROWS_Y; ++u)
          if (t * kStep + PASS_Y * u + my_row >= rows) {
#pragma unroll
            for (int i = 0; i < 16 / ROWS_Y; ++i) w[16 / ROWS_Y * u + i] = 0u;
          }
      }
      if (turn == 0) {
#pragma unroll
        for (int u = 0; u < ROWS_Y; ++u)
#pragma unroll
          for (int q = 0; q < kVecY; ++q) {
            if constexpr (P == 3)
              sum[q] += __builtin_bit_cast(float, w[8 * u + q]);
            else
              sum[q] += (float)__builtin_bit_cast(T, (uint16_t)(w[4 * u + q / 2] >> (16 * (q & 1))));
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
    constexpr int PIECES = decltype(x_wave)::value ? 2 * kRowsX : ROWS_Y, GROUPS = P * NY;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) read(x_wave, set[u], byte[u], u);
    settle(x_wave, set[0], byte[0], 0);
#pragma unroll
    for (int q = 0; q < PIECES; ++q) piece(x_wave, set[0], 0, q);
    __builtin_amdgcn_sched_barrier(0);
    read(x_wave, set[0], byte[0], kAhead);
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
        settle(x_wave, set[later], byte[later], t + 1);
        v4u fx[MX], fy[3];  // dy's columns are read two groups ahead
#pragma unroll
        for (int m = 0; m < MX; ++m) fx[m] = turned(lds_x[u], at_x[m], kTileX * 2);
#pragma unroll
        for (int g = 0; g < 2; ++g) fy[g] = turned(lds_y[u][g / NY], at_y[g % NY], TY * 2);
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
          const int n = g % NY, next = g + 2;
          if (next < GROUPS) fy[next % 3] = turned(lds_y[u][next / NY], at_y[next % NY], TY * 2);
#pragma unroll
          for (int m = 0; m < MX; ++m) acc[m][n] = multiply<T>(fx[m], fy[g % 3], acc[m][n]);
          if ((g + 1) * PIECES / GROUPS > g * PIECES / GROUPS) piece(x_wave, set[later], later, g * PIECES / GROUPS);
        }
        read(x_wave, set[later], byte[later], t + 1 + kAhead);
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
    float* sums = reinterpret_cast<float*>(&lds_x[0][0]);  // [PASS_Y][TY]; every wave is past its reads
    static_assert(PASS_Y * TY * sizeof(float) <= sizeof(lds_x), "fits");
    if (!is_x) {
#pragma unroll
      for (int q = 0; q < kVecY; ++q) sums[my_row * TY + c + q] = sum[q];
    }
    __syncthreads();
    const int64_t o = o0 + tid;
    if (tid < TY && o < a.out) {
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < PASS_Y; ++e) s += sums[e * TY + tid];
      reinterpret_cast<float*>(a.ws + l.bias)[(split * l.tiles_in + tile_i) * a.out + o] = s;
    }
  }
}

// Partial sums added in fp64: of `count` values, `count_parts` arrays each,
// four values a thread, in `runs` runs of consecutive parts whose sums are
// added in their order.  Many parts of few values would otherwise be waited
// for one after another (9 x 105 outputs of 217 parts: 6.5 us with 16 runs, 35
// with one; 256 x 1024 of 64: 14 and 31; but 1024 x 1024 of 16: 24 and 19).
struct JoinPart {
  const float* parts;
  int count_parts, runs;
  int64_t count;
  void* out;
};
__device__ __forceinline__ void join_values(const JoinPart& j, int64_t block, int64_t blocks, int dtype,
                                            int accumulate) {
  __shared__ double sums[256][4];
  const int quads = 256 / j.runs, run = threadIdx.x / quads, quad = threadIdx.x - run * quads;
  const int per = (j.count_parts + j.runs - 1) / j.runs;
  const int begin = run * per, end = min(j.count_parts, begin + per);
  for (int64_t first = block * quads * 4; first < j.count; first += blocks * quads * 4) {
    const int64_t i = first + quad * 4;
    const int valid = (int)std::max<int64_t>(0, std::min<int64_t>(j.count - i, 4));
    double s[4] = {0.0, 0.0, 0.0, 0.0};
#pragma unroll 8
    for (int p = begin; p < end; ++p) {
      float v[4];
      load_row<float, 4>(j.parts + p * j.count + i, valid, v);
#pragma unroll
      for (int q = 0; q < 4; ++q) s[q] += (double)v[q];
    }
    if (j.runs > 1) {
#pragma unroll
      for (int q = 0; q < 4; ++q) sums[threadIdx.x][q] = s[q];
      __syncthreads();
      if (run == 0) {
        for (int r = 1; r < j.runs; ++r)
#pragma unroll
          for (int q = 0; q < 4; ++q) s[q] += sums[r * quads + quad][q];
      }
      __syncthreads();
    }
    if (run == 0) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (q < valid)
          store_any(j.out, dtype, i + q, accumulate ? s[q] + (double)load_any(j.out, dtype, i + q) : s[q]);
    }
  }
}
// dweight's blocks first, then dbias's
__global__ __launch_bounds__(256) void linear_join_kernel(JoinPart weight, JoinPart bias, int weight_blocks, int dtype,
                                                          int accumulate) {
  const bool is_bias = (int)blockIdx.x >= weight_blocks;
  if (is_bias)
    join_values(bias, blockIdx.x - weight_blocks, gridDim.x - weight_blocks, dtype, accumulate);
  else
    join_values(weight, blockIdx.x, weight_blocks, dtype, accumulate);
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
    const int64_t c =
        ceil_div(tiles * s, kCUs) * (ceil_div(steps, s) + 4) + (s > 1 ? 2 + ceil_div(s * tiles, kCUs) : 0);
    if (c < cost) {
      cost = c;
      best = s;
    }
  }
  // and no fp32 sum longer than kMaxLinearRows
  best = std::max(best, ceil_div(steps, kMaxLinearRows / kStep));
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
    // 65536 rows, bf16: 2 x 1024 outputs 63 us, 1024 x 2 70 us; loading both
    // operands value by value would add 49 and 80
    const bool narrow_x = a.in < kVecX, narrow_y = a.out < kVecY;
    if (narrow_x && narrow_y)
      linear_grad_kernel<T, true, true><<<blocks, kThreads, 0, st>>>(a, l);
    else if (narrow_x)
      linear_grad_kernel<T, true, false><<<blocks, kThreads, 0, st>>>(a, l);
    else if (narrow_y)
      linear_grad_kernel<T, false, true><<<blocks, kThreads, 0, st>>>(a, l);
    else
      linear_grad_kernel<T, false, false><<<blocks, kThreads, 0, st>>>(a, l);
    return hipGetLastError();
  });
  if (e != hipSuccess || (l.direct && !a.dbias)) return e;
  auto runs = [](int parts) { return parts >= kManyParts ? kJoinRuns : 1; };
  const int bias_parts = (int)(l.splits * l.tiles_in);
  JoinPart weight{reinterpret_cast<const float*>(a.ws + l.weight), l.splits, runs(l.splits), a.out * a.in, a.dweight};
  JoinPart bias{reinterpret_cast<const float*>(a.ws + l.bias), bias_parts, runs(bias_parts), a.out, a.dbias};
  auto blocks_of = [](const JoinPart& j) { return (int)std::min<int64_t>(ceil_div(j.count * j.runs, 1024), 16 * kCUs); };
  const int weight_blocks = l.direct ? 0 : blocks_of(weight), bias_blocks = a.dbias ? blocks_of(bias) : 0;
  linear_join_kernel<<<weight_blocks + bias_blocks, 256, 0, st>>>(weight, bias, weight_blocks, a.grad_dtype,
                                                                  a.accumulate);
  e = hipGetLastError();
  return e;
}

}  // namespace adasum
