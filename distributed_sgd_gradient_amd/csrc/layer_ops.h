// layer_ops.h - the layer operators: arguments and launches of their kernels.
//
// Every launch_* function enqueues kernels on st and returns the launch's
// error.  Pointers are device pointers, strides are in elements, dtype codes
// are those of adasum_dtype_t.  The callers (layer_ops.hip) have checked the
// arguments: sizes >= 1 and below kMaxDim, extents inside 2^40 elements.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

namespace adasum {

constexpr int kCUs = 256;                 // compute units of an MI355X
constexpr int kScaleBlock = 32;           // values that share an 8-bit scale
constexpr int kMaxNormHidden = 16384;     // widest row of the layer norm kernels (held in registers)
constexpr int kNormGradRows = 1024;       // rows that one fp32 sum of the layer norm gradient takes at most
constexpr int64_t kMaxDim = int64_t(1) << 31;  // rows, tokens, vocabulary and widths stay below this
constexpr int64_t kMaxEmbeddingHidden = int64_t(1) << 23;  // a launch has 65536 workgroups along a row at most
// Rows that one fp32 sum of the linear gradient takes at most.  A split more of
// a dweight too large to be split otherwise costs the writing and reading of
// its partial sums, 8 bytes beside the 131072 operations of each: 262144,
// 30522 x 1024 bf16 15840 us in four splits, 15890 in one.
constexpr int64_t kMaxLinearRows = 65536;
// Row stride of the linear gradient's dy: a row's offset is the product of two
// 32-bit numbers, the row and the stride in bytes.
constexpr int64_t kMaxLinearStride = int64_t(1) << 28;

// f(value of the C++ type of a dtype code), for picking a kernel.
template <typename F>
hipError_t with_dtype(int dtype, F f) {
  switch (dtype) {
    case 0: return f(float());
    case 1: return f(_Float16());
    default: return f(__bf16());
  }
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// ---------------------------------------------------------------- layer norm

struct NormArgs {
  const void* x;
  int64_t rows, x_stride, y_stride;
  int hidden;
  const void* weight;  // NULL: 1
  const void* bias;    // NULL: 0
  int param_dtype;
  float eps;
  void* y;
  float* mean;     // may be NULL
  float* rstd;
  int8_t* codes;   // NULL: the normalised rows are not kept
  uint8_t* scales;
};
hipError_t launch_norm(int dtype, const NormArgs& a, hipStream_t st);

struct NormGradArgs {
  const void* dy;
  int64_t rows, dy_stride, x_stride, dx_stride;
  int hidden;
  const void* x;        // NULL: codes and scales hold the normalised rows
  const float* mean;
  const int8_t* codes;
  const uint8_t* scales;
  const float* rstd;
  const void* weight;   // NULL: 1
  int param_dtype;
  void* dx;
  void* dweight;        // NULL: not wanted
  void* dbias;          // NULL: not wanted
  int grad_dtype;
  int accumulate;
  float* partials;      // norm_grad_parts(...) x 2 x hidden
};
// Workgroups of the backward pass (in one launch or more), each with a row of
// partial sums.
int64_t norm_grad_parts(int64_t rows, int hidden);
hipError_t launch_norm_grad(int dtype, const NormGradArgs& a, hipStream_t st);

// ---------------------------------------------------------------- root-mean-square norm

// The residual stream (residual, h, dh, dx) is of x's type or fp32.
struct RmsArgs {
  const void* x;
  const void* residual;  // NULL: h = x, and R is x's type
  int64_t rows, x_stride, residual_stride, y_stride, h_stride;
  int hidden;
  const void* weight;  // NULL: 1
  int param_dtype;
  float eps;
  void* y;  // may be NULL with codes
  void* h;  // may be NULL
  float* rstd;
  int8_t* codes;  // NULL: y is not given in 8 bits
  uint8_t* scales;
};
hipError_t launch_rms(int dtype, int stream_dtype, const RmsArgs& a, hipStream_t st);

struct RmsGradArgs {
  const void* dy;
  const void* h;
  const void* dh;  // NULL: 0
  int64_t rows, dy_stride, h_stride, dh_stride, dx_stride;
  int hidden;
  const float* rstd;
  const void* weight;  // NULL: 1
  int param_dtype;
  void* dx;
  void* dweight;  // NULL: not wanted
  int grad_dtype;
  int accumulate;
  float* partials;  // rms_grad_parts(...) x hidden
};
int64_t rms_grad_parts(int64_t rows, int hidden);
hipError_t launch_rms_grad(int dtype, int stream_dtype, const RmsGradArgs& a, hipStream_t st);

// ---------------------------------------------------------------- relative bias

constexpr int kMaxBuckets = 256;
constexpr int64_t kMaxReach = int64_t(1) << 30;

// Where the buckets of one side begin: border[k] <= distance < border[k + 1],
// and no end behind the last.
struct BiasBuckets {
  int both;  // the keys behind the query have buckets of their own, side ..
  int side;  // buckets of a side
  uint32_t far;  // the last one's border
  uint32_t border[kMaxBuckets];
};
BiasBuckets bias_buckets(int buckets, int64_t reach, bool both);

struct BiasArgs {
  const void* table;  // buckets x heads
  int64_t table_stride;
  int table_dtype;
  BiasBuckets buckets;
  int64_t batch, heads, queries, keys, offset;
  const void* scores;  // NULL: the bias alone
  int64_t scores_stride, out_stride;
  void* out;
};
struct BiasLayout {
  int64_t row_tiles, col_tiles, part_batch, blocks;
};
BiasLayout bias_layout(int64_t batch, int64_t heads, int64_t queries, int64_t keys);
hipError_t launch_bias(int dtype, const BiasArgs& a, hipStream_t st);

struct BiasGradArgs {
  const void* dscores;
  int64_t stride;
  BiasBuckets buckets;
  int buckets_total;
  int64_t batch, heads, queries, keys, offset;
  void* dtable;
  int grad_dtype;
  int accumulate;
  float* partials;
};
// Workgroups of the gradient: tiles of diagonals, heads, and splits of the rows;
// and of the join, where a bucket is cut into pieces of `piece` diagonals.
struct BiasGradLayout {
  int lanes;  // that share a row
  int64_t tiles, splits, blocks, piece, piece_blocks;
  size_t sums, bytes;  // the pieces' sums begin at `sums`
};
BiasGradLayout bias_grad_layout(int64_t batch, int64_t heads, int64_t queries, int64_t keys, int dtype);
hipError_t launch_bias_grad(int dtype, const BiasGradArgs& a, hipStream_t st);

// ---------------------------------------------------------------- orthogonal updates

// Matrices of one launch at most.  A narrow one takes its steps in a workgroup,
// so more fill the card (96 of 64 x 1024 fp32: 114 us, 32 at a time 226); of wide
// ones 32 do, and their workspaces grow.
constexpr int kOrthoTogether = 128, kOrthoWide = 32;
constexpr size_t kOrthoWorkspace = size_t(4) << 30;  // and no more than this takes, if it is two or more
constexpr int kOrthoSteps = 16;
constexpr int64_t kMaxOrthoSide = int64_t(1) << 15;
constexpr int kOrthoNarrow = 64;  // a side of at most this takes its steps in fp64

// Where a matrix's pieces lie in its part of the workspace (byte offsets), n x
// m its sides, the shorter first, padded to whole tiles; [0] high parts, [1]
// low parts.
struct OrthoLayout {
  int64_t n, m;
  int parts, together;  // together: matrices of one launch
  int tile_a, tile_b, tile_x;  // of the three products of a step
  int splits, split_steps;    // of the sums of X X^T
  size_t x[2][2], a[2], b[2], rest, sums, scales, partials;  // x: of even and odd steps
  size_t per_matrix, total;
};
OrthoLayout ortho_layout(int64_t count, int64_t rows, int64_t cols, int out_dtype);
size_t ortho_workspace(int64_t count, int64_t rows, int64_t cols, int out_dtype);

// At most what a step makes of singular values s up to `most`, |a s + b s^3 + c
// s^5|, and what it adds to a, |b s^2 + c s^4|.
struct OrthoBound {
  double value, added;
};
__host__ __device__ inline OrthoBound ortho_bound(double a, double b, double c, double most) {
  const double t = most * most;
  auto image = [&](double u) { return fabs(sqrt(u) * (a + u * (b + u * c))); };  // of s^2 = u
  auto added = [&](double u) { return fabs(u * (b + u * c)); };
  OrthoBound most_of{image(t), added(t)};
  // where a + 3 b u + 5 c u^2 = 0, and where b + 2 c u = 0
  const double root = 9 * b * b - 20 * a * c;
  const double at[4] = {c != 0 && root >= 0 ? (-3 * b + sqrt(root)) / (10 * c) : 0,
                        c != 0 && root >= 0 ? (-3 * b - sqrt(root)) / (10 * c) : 0, b != 0 ? -a / (3 * b) : 0,
                        c != 0 ? -b / (2 * c) : 0};
  for (int i = 0; i < 4; ++i)
    if (at[i] > 0 && at[i] < t) {
      most_of.value = image(at[i]) > most_of.value ? image(at[i]) : most_of.value;
      most_of.added = added(at[i]) > most_of.added ? added(at[i]) : most_of.added;
    }
  return most_of;
}

struct OrthoArgs {
  const void* x[kOrthoTogether];
  void* out[kOrthoTogether];
  int64_t rows, cols, x_stride, out_stride;
  int out_dtype, steps;
  int plain;  // no step leaves all singular values of an X of norm 1 below 1/2
  double eps;
  float scale;
  double coefficients[3 * kOrthoSteps];
  char* ws;
};
struct OrthoStep {
  int index;
  int from;  // the X to read; the other one is written
  uint32_t tiles, blocks;  // of a matrix: tiles, and workgroups
  int parts, part_steps;
};
struct OrthoCall {
  OrthoArgs args;  // without x and out
  int64_t count;
  const void* const* x;
  void* const* out;
};
hipError_t launch_ortho(int dtype, const OrthoCall& call, hipStream_t st);
OrthoLayout ortho_narrow_layout(int64_t count, int64_t rows, int64_t cols);
hipError_t launch_ortho_narrow(int dtype, const OrthoArgs& a, const OrthoLayout& l, int count, hipStream_t st);

// ---------------------------------------------------------------- 8-bit activations

struct PackArgs {
  const void* x;
  int64_t rows, stride;
  int hidden;
  int8_t* codes;
  uint8_t* scales;
};
hipError_t launch_pack(int dtype, const PackArgs& a, hipStream_t st);

struct UnpackArgs {
  const int8_t* codes;
  const uint8_t* scales;
  int64_t rows, stride;
  int hidden;
  void* out;
};
hipError_t launch_unpack(int dtype, const UnpackArgs& a, hipStream_t st);

// ---------------------------------------------------------------- embedding

struct EmbeddingArgs {
  const void* table;
  int64_t vocab, table_stride, out_stride;
  int hidden;
  const void* tokens;
  int token_bytes;  // 4 or 8
  int64_t n;
  float scale;
  void* out;
};
hipError_t launch_embedding(int table_dtype, int out_dtype, const EmbeddingArgs& a, hipStream_t st);

// Where the pieces of an embedding gradient's workspace lie (byte offsets).
struct EmbeddingGradLayout {
  size_t rows, tokens, count, head, tail, total;
  int units;      // row groups of a workgroup of the summing kernel
  int lanes;      // lanes that share a row
  int span;       // consecutive grouped positions of a row group
  int64_t blocks; // workgroups along the grouped positions
  int tiles;      // workgroups along a row
};
EmbeddingGradLayout embedding_grad_layout(int64_t n, int hidden, int dtype);

struct EmbeddingGradArgs {
  const void* dy;
  int64_t n, dy_stride, vocab;
  int hidden;
  const void* tokens;
  int token_bytes;
  float scale;
  void* grad;
  int grad_dtype;
  int accumulate;
  char* ws;
};
hipError_t launch_embedding_grad(int dtype, const EmbeddingGradArgs& a, hipStream_t st);

// ---------------------------------------------------------------- linear gradient

// How the gradient's matrix is cut: tiles of the output, and the rows split
// over `splits` workgroups per tile whose partial sums are joined (those of
// dbias from every tile: the tiles of a column of dy share its rows).
struct LinearGradLayout {
  int64_t tiles_out, tiles_in;
  int splits;
  int64_t split_rows;  // rows of a split, a multiple of the kernel's step
  size_t weight, bias, total;  // byte offsets of the partial sums
  bool direct;                 // one split whose sums are the gradient as they are
};
LinearGradLayout linear_grad_layout(int64_t rows, int64_t out, int64_t in, int dtype);

struct LinearGradArgs {
  const void* dy;
  int64_t rows, dy_stride;
  int64_t out, in;
  const int8_t* codes;
  const uint8_t* scales;
  void* dweight;
  void* dbias;  // NULL: not wanted
  int grad_dtype;
  int accumulate;
  char* ws;
};
hipError_t launch_linear_grad(int dtype, const LinearGradArgs& a, hipStream_t st);

}  // namespace adasum
