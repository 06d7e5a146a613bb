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
