// layer_ops.hip - C ABI of the layer operators: argument checks and launches.
//
// Every entry point checks all of its arguments before anything is enqueued,
// on the host first and then with the runtime's pointer queries, allocates
// nothing, and lets no C++ exception out.
#include "layer_ops.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdio>
#include <exception>
#include <mutex>
#include <new>
#include <string>
#include <vector>

#include "../../include/adasum.h"
#include "library.h"

namespace adasum {
namespace {

bool known_dtype(int d) { return d == ADASUM_F32 || d == ADASUM_F16 || d == ADASUM_BF16; }
size_t size_of(int d) { return d == ADASUM_F32 ? 4 : 2; }

constexpr int64_t kMaxElements = int64_t(1) << 40;
constexpr int64_t kMaxVocab = int64_t(1) << 24;
constexpr int64_t kMaxOrthoCount = int64_t(1) << 16;

// One buffer argument: where it lies and what a call does with it.
struct Buffer {
  const void* p;
  size_t bytes;  // 0: not used by this call
  size_t align;
  const char* name;
  bool written;
};

int einval(const char* format, const char* name) {
  char buf[200];
  snprintf(buf, sizeof buf, format, name);
  return fail(ADASUM_EINVAL, buf);
}

template <size_t N>
int check_buffers(const Buffer (&b)[N]) {
  for (const Buffer& x : b) {
    if (x.bytes == 0) continue;
    if (x.p == nullptr) return einval("%s is NULL", x.name);
    if (reinterpret_cast<uintptr_t>(x.p) % x.align != 0) return einval("%s is not aligned to its elements", x.name);
  }
  for (size_t i = 0; i < N; ++i) {
    for (size_t j = i + 1; j < N; ++j) {
      if (b[i].bytes == 0 || b[j].bytes == 0 || (!b[i].written && !b[j].written)) continue;
      const uintptr_t x = reinterpret_cast<uintptr_t>(b[i].p), y = reinterpret_cast<uintptr_t>(b[j].p);
      if (x < y + b[j].bytes && y < x + b[i].bytes) {
        char buf[200];
        snprintf(buf, sizeof buf, "%s overlaps %s", b[i].name, b[j].name);
        return fail(ADASUM_EINVAL, buf);
      }
    }
  }
  int device = 0;
  const hipError_t e = hipGetDevice(&device);
  if (e != hipSuccess) return fail_hip(e, "hipGetDevice");
  // small tensors often lie in one allocation, which is asked for once a call
  uintptr_t lo[N], end[N];
  size_t known = 0;
  for (const Buffer& x : b) {
    if (x.bytes == 0) continue;
    const uintptr_t p = reinterpret_cast<uintptr_t>(x.p);
    bool inside = false;
    for (size_t i = 0; i < known; ++i) inside |= p >= lo[i] && p < end[i] && x.bytes <= end[i] - p;
    if (inside) continue;
    lo[known] = end[known] = 0;
    const int rc = check_device_range(x.p, x.bytes, x.name, device, &lo[known], &end[known]);
    if (rc != ADASUM_OK) return rc;
    ++known;
  }
  return ADASUM_OK;
}

// Sizes of a matrix argument; *bytes is what lies from its first to its last
// element.
int check_matrix(int64_t rows, int64_t cols, int64_t stride, int dtype, const char* name, size_t* bytes) {
  if (!known_dtype(dtype)) return einval("%s: unknown dtype", name);
  if (rows < 0 || rows >= kMaxDim) return einval("%s: the number of rows must be in [0, 2^31)", name);
  if (cols < 1 || cols >= kMaxDim) return einval("%s: the width must be in [1, 2^31)", name);
  if (stride < cols) return einval("%s: the row stride is below the width", name);
  if (rows > 1 && stride > kMaxElements / rows) return einval("%s: over 2^40 elements", name);
  *bytes = rows == 0 ? 0 : ((size_t)(rows - 1) * stride + cols) * size_of(dtype);
  return ADASUM_OK;
}

int check_workspace(const void* ws, size_t given, size_t needed) {
  if (needed == 0) return ADASUM_OK;
  if (ws == nullptr) return fail(ADASUM_EINVAL, "workspace is NULL but this call needs one");
  if (given < needed) {
    char buf[200];
    snprintf(buf, sizeof buf, "workspace too small: %zu bytes given, %zu needed", given, needed);
    return fail(ADASUM_EINVAL, buf);
  }
  return ADASUM_OK;
}

// The launches of one call, timed and traced as one record.
template <typename F>
int launch(int kind, const char* name, double bytes, hipStream_t st, F f) {
  std::lock_guard<std::mutex> lock(g_mu);
  if (log_enabled()) std::fprintf(stderr, "[adasum] %s %.0f bytes\n", name, bytes);
  const int pr = prof_start(kind, bytes, st);
  const hipError_t e = f();
  prof_stop(pr, st);
  return e == hipSuccess ? ADASUM_OK : fail_hip(e, name);
}

// No exception leaves a C entry point.
template <typename F>
auto guarded(F f) -> decltype(f()) {
  try {
    return f();
  } catch (const std::bad_alloc&) {
    return fail(ADASUM_ENOMEM, "out of host memory");
  } catch (const std::exception& e) {
    return fail(ADASUM_EHIP, e.what());
  } catch (...) {
    return fail(ADASUM_EHIP, "unknown exception");
  }
}

#define RETURN_IF(expr)                    \
  do {                                     \
    const int rc_ = (expr);                \
    if (rc_ != ADASUM_OK) return rc_;      \
  } while (0)

int embedding(const void* table, int64_t vocab, int64_t hidden, int64_t table_stride, int table_dtype,
              const void* tokens, int token_bytes, int64_t n, double scale, void* out, int64_t out_stride,
              int out_dtype, void* stream) {
  size_t table_bytes = 0, out_bytes = 0;
  RETURN_IF(check_matrix(vocab, hidden, table_stride, table_dtype, "table", &table_bytes));
  RETURN_IF(check_matrix(n, hidden, out_stride, out_dtype, "out", &out_bytes));
  if (hidden > kMaxEmbeddingHidden) return fail(ADASUM_EINVAL, "embedding: hidden must be at most 2^23");
  if (vocab < 1 || vocab > kMaxVocab) return fail(ADASUM_EINVAL, "vocab must be in [1, 2^24]");
  if (token_bytes != 4 && token_bytes != 8) return fail(ADASUM_EINVAL, "token_bytes must be 4 or 8");
  if (!std::isfinite((float)scale)) return fail(ADASUM_EINVAL, "scale must be finite in fp32");
  if (n == 0) return ADASUM_OK;
  const Buffer b[] = {{table, table_bytes, size_of(table_dtype), "table", false},
                      {tokens, (size_t)n * token_bytes, (size_t)token_bytes, "tokens", false},
                      {out, out_bytes, size_of(out_dtype), "out", true}};
  RETURN_IF(check_buffers(b));
  EmbeddingArgs a{};
  a.table = table;
  a.vocab = vocab;
  a.table_stride = table_stride;
  a.out_stride = out_stride;
  a.hidden = (int)hidden;
  a.tokens = tokens;
  a.token_bytes = token_bytes;
  a.n = n;
  a.scale = (float)scale;
  a.out = out;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const double bytes = (double)n * (token_bytes + (double)hidden * (size_of(table_dtype) + size_of(out_dtype)));
  return launch(kEmbedding, "embedding", bytes, st, [&] { return launch_embedding(table_dtype, out_dtype, a, st); });
}

int64_t embedding_grad_bytes(int64_t n, int64_t hidden, int dtype) {
  size_t bytes = 0;
  RETURN_IF(check_matrix(n, hidden, hidden, dtype, "dy", &bytes));
  if (hidden > kMaxEmbeddingHidden) return fail(ADASUM_EINVAL, "embedding: hidden must be at most 2^23");
  return (int64_t)embedding_grad_layout(n, (int)hidden, dtype).total;
}

int embedding_grad(const void* dy, int64_t n, int64_t hidden, int64_t dy_stride, int dtype, const void* tokens,
                   int token_bytes, int64_t vocab, double scale, void* grad, int grad_dtype, int accumulate,
                   void* workspace, size_t workspace_bytes, void* stream) {
  size_t dy_bytes = 0, grad_bytes = 0;
  RETURN_IF(check_matrix(n, hidden, dy_stride, dtype, "dy", &dy_bytes));
  RETURN_IF(check_matrix(vocab, hidden, hidden, grad_dtype, "grad", &grad_bytes));
  if (hidden > kMaxEmbeddingHidden) return fail(ADASUM_EINVAL, "embedding: hidden must be at most 2^23");
  if (vocab < 1 || vocab > kMaxVocab) return fail(ADASUM_EINVAL, "vocab must be in [1, 2^24]");
  if (token_bytes != 4 && token_bytes != 8) return fail(ADASUM_EINVAL, "token_bytes must be 4 or 8");
  if (!std::isfinite((float)scale)) return fail(ADASUM_EINVAL, "scale must be finite in fp32");
  if (n == 0 && accumulate) return ADASUM_OK;
  const size_t need = embedding_grad_layout(n, (int)hidden, dtype).total;
  RETURN_IF(check_workspace(workspace, workspace_bytes, need));
  const Buffer b[] = {{dy, dy_bytes, size_of(dtype), "dy", false},
                      {tokens, (size_t)n * token_bytes, (size_t)token_bytes, "tokens", false},
                      {grad, grad_bytes, size_of(grad_dtype), "grad", true},
                      {workspace, need, 16, "workspace", true}};
  RETURN_IF(check_buffers(b));
  EmbeddingGradArgs a{};
  a.dy = dy;
  a.n = n;
  a.dy_stride = dy_stride;
  a.vocab = vocab;
  a.hidden = (int)hidden;
  a.tokens = tokens;
  a.token_bytes = token_bytes;
  a.scale = (float)scale;
  a.grad = grad;
  a.grad_dtype = grad_dtype;
  a.accumulate = accumulate != 0;
  a.ws = static_cast<char*>(workspace);
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const double bytes = (double)n * (token_bytes + (double)hidden * size_of(dtype)) + (double)grad_bytes;
  return launch(kEmbedding, "embedding gradient", bytes, st, [&] { return launch_embedding_grad(dtype, a, st); });
}

int layer_norm(const void* x, int64_t rows, int64_t hidden, int64_t x_stride, int dtype, const void* weight,
               const void* bias, int param_dtype, double eps, void* y, int64_t y_stride, float* mean, float* rstd,
               int8_t* codes, uint8_t* scales, void* stream) {
  size_t x_bytes = 0, y_bytes = 0;
  RETURN_IF(check_matrix(rows, hidden, x_stride, dtype, "x", &x_bytes));
  RETURN_IF(check_matrix(rows, hidden, y_stride, dtype, "y", &y_bytes));
  if (hidden > kMaxNormHidden) return fail(ADASUM_EINVAL, "layer norm: hidden must be at most 16384");
  if (!known_dtype(param_dtype)) return fail(ADASUM_EINVAL, "unknown param_dtype");
  if (!std::isfinite((float)eps) || (float)eps < FLT_MIN)
    return fail(ADASUM_EINVAL, "eps must be a positive normal fp32 number");
  if ((codes == nullptr) != (scales == nullptr)) return fail(ADASUM_EINVAL, "codes and scales belong together");
  if (rows == 0) return ADASUM_OK;
  const size_t param = (size_t)hidden * size_of(param_dtype), stat = (size_t)rows * 4;
  const Buffer b[] = {{x, x_bytes, size_of(dtype), "x", false},
                      {weight, weight ? param : 0, size_of(param_dtype), "weight", false},
                      {bias, bias ? param : 0, size_of(param_dtype), "bias", false},
                      {y, y_bytes, size_of(dtype), "y", true},
                      {mean, mean ? stat : 0, 4, "mean", true},
                      {rstd, stat, 4, "rstd", true},
                      {codes, codes ? (size_t)(rows * hidden) : 0, 1, "codes", true},
                      {scales, codes ? (size_t)(rows * ceil_div(hidden, kScaleBlock)) : 0, 1, "scales", true}};
  RETURN_IF(check_buffers(b));
  NormArgs a{};
  a.x = x;
  a.rows = rows;
  a.x_stride = x_stride;
  a.y_stride = y_stride;
  a.hidden = (int)hidden;
  a.weight = weight;
  a.bias = bias;
  a.param_dtype = param_dtype;
  a.eps = (float)eps;
  a.y = y;
  a.mean = mean;
  a.rstd = rstd;
  a.codes = codes;
  a.scales = scales;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const double bytes = (double)rows * ((double)hidden * (2 * size_of(dtype) + (codes ? 33.0 / 32 : 0.0)) + 8);
  return launch(kNorm, "layer norm", bytes, st, [&] { return launch_norm(dtype, a, st); });
}

size_t norm_grad_workspace(int64_t rows, int64_t hidden) {
  return rows == 0 ? 0 : (size_t)norm_grad_parts(rows, (int)hidden) * 2 * hidden * sizeof(float);
}

int64_t layer_norm_grad_bytes(int64_t rows, int64_t hidden, int dtype) {
  size_t bytes = 0;
  RETURN_IF(check_matrix(rows, hidden, hidden, dtype, "dy", &bytes));
  if (hidden > kMaxNormHidden) return fail(ADASUM_EINVAL, "layer norm: hidden must be at most 16384");
  return (int64_t)norm_grad_workspace(rows, hidden);
}

int layer_norm_grad(const void* dy, int64_t rows, int64_t hidden, int64_t dy_stride, int dtype, const void* x,
                    int64_t x_stride, const float* mean, const int8_t* codes, const uint8_t* scales,
                    const float* rstd, const void* weight, int param_dtype, void* dx, int64_t dx_stride,
                    void* dweight, void* dbias, int grad_dtype, int accumulate, void* workspace,
                    size_t workspace_bytes, void* stream) {
  size_t dy_bytes = 0, x_bytes = 0, dx_bytes = 0;
  RETURN_IF(check_matrix(rows, hidden, dy_stride, dtype, "dy", &dy_bytes));
  RETURN_IF(check_matrix(rows, hidden, dx_stride, dtype, "dx", &dx_bytes));
  if (hidden > kMaxNormHidden) return fail(ADASUM_EINVAL, "layer norm: hidden must be at most 16384");
  if (!known_dtype(param_dtype)) return fail(ADASUM_EINVAL, "unknown param_dtype");
  if (!known_dtype(grad_dtype)) return fail(ADASUM_EINVAL, "unknown grad_dtype");
  const bool kept = x == nullptr;
  if (kept) {
    if (mean != nullptr) return fail(ADASUM_EINVAL, "mean belongs to x: with codes and scales both are NULL");
  } else {
    if (codes != nullptr || scales != nullptr)
      return fail(ADASUM_EINVAL, "either x and mean or codes and scales, not both");
    RETURN_IF(check_matrix(rows, hidden, x_stride, dtype, "x", &x_bytes));
  }
  const bool sums = dweight != nullptr || dbias != nullptr;
  if (rows == 0 && (accumulate || !sums)) return ADASUM_OK;
  const size_t need = sums ? norm_grad_workspace(rows, hidden) : 0;
  RETURN_IF(check_workspace(workspace, workspace_bytes, need));
  const size_t param = (size_t)hidden * size_of(param_dtype), grad = (size_t)hidden * size_of(grad_dtype);
  const size_t stat = (size_t)rows * 4;
  const Buffer b[] = {{dy, dy_bytes, size_of(dtype), "dy", false},
                      {x, x_bytes, size_of(dtype), "x", false},
                      {mean, kept ? 0 : stat, 4, "mean", false},
                      {codes, kept ? (size_t)(rows * hidden) : 0, 1, "codes", false},
                      {scales, kept ? (size_t)(rows * ceil_div(hidden, kScaleBlock)) : 0, 1, "scales", false},
                      {rstd, stat, 4, "rstd", false},
                      {weight, weight ? param : 0, size_of(param_dtype), "weight", false},
                      {dx, dx_bytes, size_of(dtype), "dx", true},
                      {dweight, dweight ? grad : 0, size_of(grad_dtype), "dweight", true},
                      {dbias, dbias ? grad : 0, size_of(grad_dtype), "dbias", true},
                      {workspace, need, 16, "workspace", true}};
  RETURN_IF(check_buffers(b));
  NormGradArgs a{};
  a.dy = dy;
  a.rows = rows;
  a.dy_stride = dy_stride;
  a.x_stride = x_stride;
  a.dx_stride = dx_stride;
  a.hidden = (int)hidden;
  a.x = x;
  a.mean = mean;
  a.codes = codes;
  a.scales = scales;
  a.rstd = rstd;
  a.weight = weight;
  a.param_dtype = param_dtype;
  a.dx = dx;
  a.dweight = dweight;
  a.dbias = dbias;
  a.grad_dtype = grad_dtype;
  a.accumulate = accumulate != 0;
  a.partials = sums ? static_cast<float*>(workspace) : nullptr;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const double bytes =
      (double)rows * ((double)hidden * (2 * size_of(dtype) + (kept ? 33.0 / 32 : (double)size_of(dtype))) + 8);
  return launch(kNorm, "layer norm gradient", bytes, st, [&] { return launch_norm_grad(dtype, a, st); });
}

int checkpoint_pack(const void* x, int64_t rows, int64_t hidden, int64_t x_stride, int dtype, int8_t* codes,
                    uint8_t* scales, void* stream) {
  size_t x_bytes = 0;
  RETURN_IF(check_matrix(rows, hidden, x_stride, dtype, "x", &x_bytes));
  if (rows == 0) return ADASUM_OK;
  const Buffer b[] = {{x, x_bytes, size_of(dtype), "x", false},
                      {codes, (size_t)(rows * hidden), 1, "codes", true},
                      {scales, (size_t)(rows * ceil_div(hidden, kScaleBlock)), 1, "scales", true}};
  RETURN_IF(check_buffers(b));
  PackArgs a{};
  a.x = x;
  a.rows = rows;
  a.stride = x_stride;
  a.hidden = (int)hidden;
  a.codes = codes;
  a.scales = scales;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const double bytes = (double)rows * hidden * (size_of(dtype) + 33.0 / 32);
  return launch(kPack, "pack", bytes, st, [&] { return launch_pack(dtype, a, st); });
}

int checkpoint_unpack(const int8_t* codes, const uint8_t* scales, int64_t rows, int64_t hidden, void* out,
                      int64_t out_stride, int dtype, void* stream) {
  size_t out_bytes = 0;
  RETURN_IF(check_matrix(rows, hidden, out_stride, dtype, "out", &out_bytes));
  if (rows == 0) return ADASUM_OK;
  const Buffer b[] = {{codes, (size_t)(rows * hidden), 1, "codes", false},
                      {scales, (size_t)(rows * ceil_div(hidden, kScaleBlock)), 1, "scales", false},
                      {out, out_bytes, size_of(dtype), "out", true}};
  RETURN_IF(check_buffers(b));
  UnpackArgs a{};
  a.codes = codes;
  a.scales = scales;
  a.rows = rows;
  a.stride = out_stride;
  a.hidden = (int)hidden;
  a.out = out;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const double bytes = (double)rows * hidden * (size_of(dtype) + 33.0 / 32);
  return launch(kPack, "unpack", bytes, st, [&] { return launch_unpack(dtype, a, st); });
}

int check_linear(int64_t rows, int64_t out, int64_t in, int64_t stride, int dtype, size_t* dy_bytes) {
  RETURN_IF(check_matrix(rows, out, stride, dtype, "dy", dy_bytes));
  if (in < 1 || in > kMaxVocab || out > kMaxVocab)
    return fail(ADASUM_EINVAL, "in_features and out_features must be in [1, 2^24]");
  if (rows > 1 && stride > kMaxLinearStride)
    return fail(ADASUM_EINVAL, "linear gradient: the row stride of dy must be at most 2^28 elements");
  if (in > kMaxElements / out || (rows > 0 && in > kMaxElements / rows))
    return fail(ADASUM_EINVAL, "linear gradient: over 2^40 elements");
  const LinearGradLayout l = linear_grad_layout(rows, out, in, dtype);
  // workgroups of a launch: 512 lanes each, 2^32 lanes at most
  if (l.tiles_out * l.tiles_in * l.splits >= (int64_t(1) << 23))
    return fail(ADASUM_EINVAL, "linear gradient: dweight is too large for one call");
  return ADASUM_OK;
}

int64_t linear_grad_bytes(int64_t rows, int64_t out, int64_t in, int dtype) {
  size_t bytes = 0;
  RETURN_IF(check_linear(rows, out, in, out, dtype, &bytes));
  return (int64_t)linear_grad_layout(rows, out, in, dtype).total;
}

int linear_grad(const void* dy, int64_t rows, int64_t out, int64_t dy_stride, int dtype, const int8_t* codes,
                const uint8_t* scales, int64_t in, void* dweight, void* dbias, int grad_dtype, int accumulate,
                void* workspace, size_t workspace_bytes, void* stream) {
  size_t dy_bytes = 0;
  RETURN_IF(check_linear(rows, out, in, dy_stride, dtype, &dy_bytes));
  if (!known_dtype(grad_dtype)) return fail(ADASUM_EINVAL, "unknown grad_dtype");
  if (rows == 0 && accumulate) return ADASUM_OK;
  const size_t need = linear_grad_layout(rows, out, in, dtype).total;
  RETURN_IF(check_workspace(workspace, workspace_bytes, need));
  const Buffer b[] = {{dy, dy_bytes, size_of(dtype), "dy", false},
                      {codes, (size_t)(rows * in), 1, "codes", false},
                      {scales, (size_t)(rows * ceil_div(in, kScaleBlock)), 1, "scales", false},
                      {dweight, (size_t)(out * in) * size_of(grad_dtype), size_of(grad_dtype), "dweight", true},
                      {dbias, dbias ? (size_t)out * size_of(grad_dtype) : 0, size_of(grad_dtype), "dbias", true},
                      {workspace, need, 16, "workspace", true}};
  RETURN_IF(check_buffers(b));
  LinearGradArgs a{};
  a.dy = dy;
  a.rows = rows;
  a.dy_stride = dy_stride;
  a.out = out;
  a.in = in;
  a.codes = codes;
  a.scales = scales;
  a.dweight = dweight;
  a.dbias = dbias;
  a.grad_dtype = grad_dtype;
  a.accumulate = accumulate != 0;
  a.ws = static_cast<char*>(workspace);
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const double bytes = (double)rows * ((double)out * size_of(dtype) + in * 33.0 / 32) +
                       (double)out * (in + 1) * size_of(grad_dtype);
  return launch(kLinear, "linear gradient", bytes, st, [&] { return launch_linear_grad(dtype, a, st); });
}

int check_params(int64_t hidden, int param_dtype, double eps) {
  if (hidden > kMaxNormHidden) return fail(ADASUM_EINVAL, "root-mean-square norm: hidden must be at most 16384");
  if (!known_dtype(param_dtype)) return fail(ADASUM_EINVAL, "unknown param_dtype");
  if (!std::isfinite((float)eps) || (float)eps < FLT_MIN)
    return fail(ADASUM_EINVAL, "eps must be a positive normal fp32 number");
  return ADASUM_OK;
}

// The residual stream is of x's type or fp32.
int check_stream(int dtype, int stream_dtype) {
  if (!known_dtype(dtype)) return fail(ADASUM_EINVAL, "unknown dtype");
  if (stream_dtype != dtype && stream_dtype != ADASUM_F32)
    return fail(ADASUM_EINVAL, "stream_dtype must be dtype or fp32");
  return ADASUM_OK;
}

int rms(const void* x, int64_t rows, int64_t hidden, int64_t x_stride, int dtype, const void* residual,
        int64_t residual_stride, int stream_dtype, const void* weight, int param_dtype, double eps, void* y,
        int64_t y_stride, void* h, int64_t h_stride, float* rstd, int8_t* codes, uint8_t* scales, void* stream) {
  size_t x_bytes = 0, residual_bytes = 0, y_bytes = 0, h_bytes = 0;
  RETURN_IF(check_stream(dtype, stream_dtype));
  RETURN_IF(check_matrix(rows, hidden, x_stride, dtype, "x", &x_bytes));
  if (residual) RETURN_IF(check_matrix(rows, hidden, residual_stride, stream_dtype, "residual", &residual_bytes));
  if (y || !codes) RETURN_IF(check_matrix(rows, hidden, y_stride, dtype, "y", &y_bytes));
  if (h) RETURN_IF(check_matrix(rows, hidden, h_stride, stream_dtype, "h", &h_bytes));
  RETURN_IF(check_params(hidden, param_dtype, eps));
  if ((codes == nullptr) != (scales == nullptr)) return fail(ADASUM_EINVAL, "codes and scales belong together");
  if (rows == 0) return ADASUM_OK;
  if (h && !residual) return fail(ADASUM_EINVAL, "without a residual there is no h: it is x");
  if (!residual && stream_dtype != dtype) return fail(ADASUM_EINVAL, "without a residual stream_dtype must be dtype");
  if (h && h == residual && h_stride == residual_stride) residual_bytes = 0;  // in place
  const Buffer b[] = {{x, x_bytes, size_of(dtype), "x", false},
                      {residual, residual_bytes, size_of(stream_dtype), "residual", false},
                      {weight, weight ? (size_t)hidden * size_of(param_dtype) : 0, size_of(param_dtype), "weight", false},
                      {y, y_bytes, size_of(dtype), "y", true},
                      {h, h_bytes, size_of(stream_dtype), "h", true},
                      {rstd, (size_t)rows * 4, 4, "rstd", true},
                      {codes, codes ? (size_t)(rows * hidden) : 0, 1, "codes", true},
                      {scales, codes ? (size_t)(rows * ceil_div(hidden, kScaleBlock)) : 0, 1, "scales", true}};
  RETURN_IF(check_buffers(b));
  RmsArgs a{};
  a.x = x;
  a.residual = residual;
  a.rows = rows;
  a.x_stride = x_stride;
  a.residual_stride = residual_stride;
  a.y_stride = y_stride;
  a.h_stride = h_stride;
  a.hidden = (int)hidden;
  a.weight = weight;
  a.param_dtype = param_dtype;
  a.eps = (float)eps;
  a.y = y;
  a.h = h;
  a.rstd = rstd;
  a.codes = codes;
  a.scales = scales;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const double wide = (residual ? 1 : 0) * size_of(stream_dtype) + (h ? 1 : 0) * size_of(stream_dtype);
  const double bytes =
      (double)rows * ((double)hidden * ((y ? 2 : 1) * size_of(dtype) + wide + (codes ? 33.0 / 32 : 0.0)) + 4);
  return launch(kNorm, "root-mean-square norm", bytes, st, [&] { return launch_rms(dtype, stream_dtype, a, st); });
}

size_t rms_grad_workspace(int64_t rows, int64_t hidden) {
  return rows == 0 ? 0 : (size_t)rms_grad_parts(rows, (int)hidden) * hidden * sizeof(float);
}

int64_t rms_grad_bytes(int64_t rows, int64_t hidden, int dtype) {
  size_t bytes = 0;
  RETURN_IF(check_matrix(rows, hidden, hidden, dtype, "dy", &bytes));
  if (hidden > kMaxNormHidden) return fail(ADASUM_EINVAL, "root-mean-square norm: hidden must be at most 16384");
  return (int64_t)rms_grad_workspace(rows, hidden);
}

int rms_grad(const void* dy, int64_t rows, int64_t hidden, int64_t dy_stride, int dtype, const void* h,
             int64_t h_stride, int stream_dtype, const void* dh, int64_t dh_stride, const float* rstd,
             const void* weight, int param_dtype, void* dx, int64_t dx_stride, void* dweight, int grad_dtype,
             int accumulate, void* workspace, size_t workspace_bytes, void* stream) {
  size_t dy_bytes = 0, h_bytes = 0, dh_bytes = 0, dx_bytes = 0;
  RETURN_IF(check_stream(dtype, stream_dtype));
  RETURN_IF(check_matrix(rows, hidden, dy_stride, dtype, "dy", &dy_bytes));
  RETURN_IF(check_matrix(rows, hidden, h_stride, stream_dtype, "h", &h_bytes));
  if (dh) RETURN_IF(check_matrix(rows, hidden, dh_stride, stream_dtype, "dh", &dh_bytes));
  RETURN_IF(check_matrix(rows, hidden, dx_stride, stream_dtype, "dx", &dx_bytes));
  RETURN_IF(check_params(hidden, param_dtype, 1.0));
  if (!known_dtype(grad_dtype)) return fail(ADASUM_EINVAL, "unknown grad_dtype");
  if (rows == 0 && (accumulate || !dweight)) return ADASUM_OK;
  const size_t need = dweight ? rms_grad_workspace(rows, hidden) : 0;
  RETURN_IF(check_workspace(workspace, workspace_bytes, need));
  if (dh && dx == dh && dx_stride == dh_stride) dh_bytes = 0;  // in place
  const Buffer b[] = {{dy, dy_bytes, size_of(dtype), "dy", false},
                      {h, h_bytes, size_of(stream_dtype), "h", false},
                      {dh, dh_bytes, size_of(stream_dtype), "dh", false},
                      {rstd, (size_t)rows * 4, 4, "rstd", false},
                      {weight, weight ? (size_t)hidden * size_of(param_dtype) : 0, size_of(param_dtype), "weight", false},
                      {dx, dx_bytes, size_of(stream_dtype), "dx", true},
                      {dweight, dweight ? (size_t)hidden * size_of(grad_dtype) : 0, size_of(grad_dtype), "dweight", true},
                      {workspace, need, 16, "workspace", true}};
  RETURN_IF(check_buffers(b));
  RmsGradArgs a{};
  a.dy = dy;
  a.h = h;
  a.dh = dh;
  a.rows = rows;
  a.dy_stride = dy_stride;
  a.h_stride = h_stride;
  a.dh_stride = dh_stride;
  a.dx_stride = dx_stride;
  a.hidden = (int)hidden;
  a.rstd = rstd;
  a.weight = weight;
  a.param_dtype = param_dtype;
  a.dx = dx;
  a.dweight = dweight;
  a.grad_dtype = grad_dtype;
  a.accumulate = accumulate != 0;
  a.partials = dweight ? static_cast<float*>(workspace) : nullptr;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const double bytes =
      (double)rows * ((double)hidden * (size_of(dtype) + (dh ? 3 : 2) * size_of(stream_dtype)) + 4);
  return launch(kNorm, "root-mean-square norm gradient", bytes, st,
                [&] { return launch_rms_grad(dtype, stream_dtype, a, st); });
}

int check_bias(int64_t heads, int64_t batch, int64_t queries, int64_t keys, int64_t offset, int64_t buckets,
               int64_t max_distance, int bidirectional) {
  if (heads < 1 || heads >= kMaxDim) return fail(ADASUM_EINVAL, "heads must be in [1, 2^31)");
  if (batch < 0 || batch >= kMaxDim) return fail(ADASUM_EINVAL, "batch must be in [0, 2^31)");
  if (queries < 0 || queries >= kMaxDim) return fail(ADASUM_EINVAL, "queries must be in [0, 2^31)");
  if (keys < 1 || keys >= kMaxDim) return fail(ADASUM_EINVAL, "keys must be in [1, 2^31)");
  if (batch * heads >= kMaxDim || batch * heads * queries >= kMaxDim)
    return fail(ADASUM_EINVAL, "relative bias: the number of rows must be below 2^31");
  if (queries + keys > kMaxReach) return fail(ADASUM_EINVAL, "queries and keys must be at most 2^30 together");
  if (offset <= -kMaxDim || offset >= kMaxDim) return fail(ADASUM_EINVAL, "offset must be within 2^31");
  if (buckets < (bidirectional ? 4 : 2) || buckets > kMaxBuckets || (bidirectional && buckets % 2 != 0))
    return fail(ADASUM_EINVAL, "buckets must be in [2, 256], in both directions even and at least 4");
  const int64_t exact = (bidirectional ? buckets / 2 : buckets) / 2;
  if (max_distance <= exact || max_distance > kMaxReach)
    return fail(ADASUM_EINVAL, "max_distance must be above half the buckets of a side, and at most 2^30");
  return ADASUM_OK;
}

// Workgroups of a launch: 256 lanes each, 2^32 lanes at most.
constexpr int64_t kMaxBlocks = int64_t(1) << 24;

int relative_bias(const void* table, int64_t buckets, int64_t heads, int64_t table_stride, int table_dtype,
                  int64_t max_distance, int bidirectional, int64_t batch, int64_t queries, int64_t keys,
                  int64_t offset, const void* scores, int64_t scores_stride, void* out, int64_t out_stride, int dtype,
                  void* stream) {
  size_t table_bytes = 0, scores_bytes = 0, out_bytes = 0;
  RETURN_IF(check_bias(heads, batch, queries, keys, offset, buckets, max_distance, bidirectional));
  RETURN_IF(check_matrix(buckets, heads, table_stride, table_dtype, "table", &table_bytes));
  const int64_t rows = batch * heads * queries;
  if (scores) RETURN_IF(check_matrix(rows, keys, scores_stride, dtype, "scores", &scores_bytes));
  RETURN_IF(check_matrix(rows, keys, out_stride, dtype, "out", &out_bytes));
  if (rows == 0) return ADASUM_OK;
  if (bias_layout(batch, heads, queries, keys).blocks >= kMaxBlocks)
    return fail(ADASUM_EINVAL, "relative bias: the scores are too large for one call");
  if (out == scores && out_stride == scores_stride) scores_bytes = 0;  // in place
  const Buffer b[] = {{table, table_bytes, size_of(table_dtype), "table", false},
                      {scores, scores_bytes, size_of(dtype), "scores", false},
                      {out, out_bytes, size_of(dtype), "out", true}};
  RETURN_IF(check_buffers(b));
  BiasArgs a{};
  a.table = table;
  a.table_stride = table_stride;
  a.table_dtype = table_dtype;
  a.buckets = bias_buckets((int)buckets, max_distance, bidirectional != 0);
  a.batch = batch;
  a.heads = heads;
  a.queries = queries;
  a.keys = keys;
  a.offset = offset;
  a.scores = scores;
  a.scores_stride = scores_stride;
  a.out_stride = out_stride;
  a.out = out;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const double bytes = (double)rows * keys * size_of(dtype) * (scores ? 2 : 1);
  return launch(kBias, "relative bias", bytes, st, [&] { return launch_bias(dtype, a, st); });
}

int check_bias_grad(int64_t batch, int64_t heads, int64_t queries, int64_t keys, int64_t stride, int dtype,
                    size_t* bytes) {
  const int64_t rows = batch * heads * queries;
  RETURN_IF(check_matrix(rows, keys, stride, dtype, "dscores", bytes));
  const BiasGradLayout l = bias_grad_layout(rows == 0 ? 0 : batch, heads, std::max<int64_t>(queries, 1), keys, dtype);
  if (l.blocks >= kMaxBlocks || l.piece_blocks >= kMaxBlocks || heads * kMaxBuckets >= kMaxBlocks)
    return fail(ADASUM_EINVAL, "relative bias: the scores are too large for one call");
  return ADASUM_OK;
}

int64_t relative_bias_grad_bytes(int64_t batch, int64_t heads, int64_t queries, int64_t keys, int dtype) {
  size_t bytes = 0;
  RETURN_IF(check_bias(heads, batch, queries, keys, 0, 4, 4, 1));
  RETURN_IF(check_bias_grad(batch, heads, queries, keys, keys, dtype, &bytes));
  return (int64_t)bias_grad_layout(bytes == 0 ? 0 : batch, heads, std::max<int64_t>(queries, 1), keys, dtype).bytes;
}

int relative_bias_grad(const void* dscores, int64_t batch, int64_t heads, int64_t queries, int64_t keys,
                       int64_t stride, int dtype, int64_t offset, int64_t buckets, int64_t max_distance,
                       int bidirectional, void* dtable, int grad_dtype, int accumulate, void* workspace,
                       size_t workspace_bytes, void* stream) {
  size_t in_bytes = 0, table_bytes = 0;
  RETURN_IF(check_bias(heads, batch, queries, keys, offset, buckets, max_distance, bidirectional));
  RETURN_IF(check_bias_grad(batch, heads, queries, keys, stride, dtype, &in_bytes));
  RETURN_IF(check_matrix(buckets, heads, heads, grad_dtype, "dtable", &table_bytes));
  if (in_bytes == 0) {  // no rows: a gradient of zeros
    if (accumulate) return ADASUM_OK;
    batch = 0;
    queries = std::max<int64_t>(queries, 1);
  }
  const BiasGradLayout l = bias_grad_layout(batch, heads, queries, keys, dtype);
  RETURN_IF(check_workspace(workspace, workspace_bytes, l.bytes));
  const Buffer b[] = {{dscores, in_bytes, size_of(dtype), "dscores", false},
                      {dtable, table_bytes, size_of(grad_dtype), "dtable", true},
                      {workspace, l.bytes, 16, "workspace", true}};
  RETURN_IF(check_buffers(b));
  BiasGradArgs a{};
  a.dscores = dscores;
  a.stride = stride;
  a.buckets = bias_buckets((int)buckets, max_distance, bidirectional != 0);
  a.buckets_total = (int)buckets;
  a.batch = batch;
  a.heads = heads;
  a.queries = queries;
  a.keys = keys;
  a.offset = offset;
  a.dtable = dtable;
  a.grad_dtype = grad_dtype;
  a.accumulate = accumulate != 0;
  a.partials = static_cast<float*>(workspace);
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const double bytes = (double)batch * heads * queries * keys * size_of(dtype);
  return launch(kBias, "relative bias gradient", bytes, st, [&] { return launch_bias_grad(dtype, a, st); });
}

// One of many buffers: rows of `width` bytes, `pitch` apart.
struct Rows {
  Buffer all;
  size_t width, pitch;
  int index;  // -1: there is one only
};

// Whether b, which begins within a's span, has a byte of it.  Rows of one pitch may
// lie between each other's, as column slices of one matrix do.
bool share_bytes(const Rows& a, const Rows& b) {
  if (a.all.bytes == a.width || (b.all.bytes != b.width && a.pitch != b.pitch)) return true;
  const size_t d = (reinterpret_cast<uintptr_t>(b.all.p) - reinterpret_cast<uintptr_t>(a.all.p)) % a.pitch;
  return d < a.width || d + b.width > a.pitch;
}

// The buffers of a call with any number of them, as check_buffers.
int check_many(const std::vector<Rows>& rows) {
  std::vector<size_t> order;
  std::vector<Buffer> given;
  for (const Rows& r : rows) given.push_back(r.all);
  auto name = [&](size_t i) {
    return std::string(given[i].name) + (rows[i].index < 0 ? "" : "[" + std::to_string(rows[i].index) + "]");
  };
  for (size_t i = 0; i < given.size(); ++i) {
    const Buffer& x = given[i];
    if (x.bytes == 0) continue;
    if (x.p == nullptr) return einval("%s is NULL", name(i).c_str());
    if (reinterpret_cast<uintptr_t>(x.p) % x.align != 0)
      return einval("%s is not aligned to its elements", name(i).c_str());
    order.push_back(i);
  }
  auto start = [&](size_t i) { return reinterpret_cast<uintptr_t>(given[i].p); };
  std::sort(order.begin(), order.end(), [&](size_t i, size_t j) { return start(i) < start(j); });
  std::vector<size_t> open[2];  // what is read, what is written, and reaches up to here
  for (size_t i : order) {
    for (int w = given[i].written ? 0 : 1; w < 2; ++w) {
      size_t left = 0;
      for (size_t j : open[w]) {
        if (start(j) + given[j].bytes <= start(i)) continue;
        if (share_bytes(rows[j], rows[i])) return einval("%s", (name(i) + " overlaps " + name(j)).c_str());
        open[w][left++] = j;
      }
      open[w].resize(left);
    }
    std::vector<size_t>& mine = open[given[i].written ? 1 : 0];
    if (mine.empty() || given[mine.back()].p != given[i].p) mine.push_back(i);  // read many times: once
  }
  int device = 0;
  const hipError_t e = hipGetDevice(&device);
  if (e != hipSuccess) return fail_hip(e, "hipGetDevice");
  uintptr_t lo = 0, last = 0;  // of the allocation that was asked for last
  for (size_t i : order) {
    if (start(i) >= lo && start(i) < last && given[i].bytes <= last - start(i)) continue;
    lo = last = 0;
    RETURN_IF(check_device_range(given[i].p, given[i].bytes, name(i).c_str(), device, &lo, &last));
  }
  return ADASUM_OK;
}

int check_ortho(int64_t count, int64_t rows, int64_t cols, int out_dtype) {
  if (count < 0 || count > kMaxOrthoCount) return fail(ADASUM_EINVAL, "count must be in [0, 2^16]");
  if (rows < 0 || rows > kMaxOrthoSide || cols < 1 || cols > kMaxOrthoSide)
    return fail(ADASUM_EINVAL, "orthogonalize: rows must be in [0, 2^15], cols in [1, 2^15]");
  if (!known_dtype(out_dtype)) return fail(ADASUM_EINVAL, "unknown out_dtype");
  return ADASUM_OK;
}

int64_t orthogonalize_bytes(int64_t count, int64_t rows, int64_t cols, int out_dtype) {
  RETURN_IF(check_ortho(count, rows, cols, out_dtype));
  return count == 0 || rows == 0 ? 0 : (int64_t)ortho_workspace(count, rows, cols, out_dtype);
}

// Follows the largest singular value through the steps: the kernels hold X and
// B in fp16 parts, whose range they must not leave.  *plain: it stays above 1/2.
int check_coefficients(int steps, const double* k, int* plain) {
  *plain = 1;
  if (steps < 1 || steps > kOrthoSteps) return fail(ADASUM_EINVAL, "steps must be in [1, 16]");
  if (k == nullptr) return fail(ADASUM_EINVAL, "coefficients is NULL");
  double most = 1.001;  // with room for rounding
  for (int s = 0; s < steps; ++s, k += 3) {
    const double a = k[0], b = k[1], c = k[2];
    if (!std::isfinite((float)a) || !std::isfinite((float)b) || !std::isfinite((float)c))
      return fail(ADASUM_EINVAL, "coefficients must be finite in fp32");
    const OrthoBound bound = ortho_bound(a, b, c, most);
    if (!(bound.value < 2.0) || !(bound.added <= 30.0))
      return fail(ADASUM_EINVAL, "coefficients must keep singular values below 2, and b A + c A^2 below 31");
    if (bound.value <= 0.5) *plain = 0;
    most = std::max(bound.value * 1.01, 1e-3);
  }
  return ADASUM_OK;
}

int orthogonalize(const void* const* x, int64_t count, int64_t rows, int64_t cols, int64_t x_stride, int dtype,
                  int steps, const double* coefficients, double eps, double scale, void* const* out,
                  int64_t out_stride, int out_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  size_t x_bytes = 0, out_bytes = 0;
  RETURN_IF(check_ortho(count, rows, cols, out_dtype));
  RETURN_IF(check_matrix(rows, cols, x_stride, dtype, "x", &x_bytes));
  RETURN_IF(check_matrix(rows, cols, out_stride, out_dtype, "out", &out_bytes));
  int plain = 0;
  RETURN_IF(check_coefficients(steps, coefficients, &plain));
  if (!std::isfinite((float)eps) || (float)eps < FLT_MIN)
    return fail(ADASUM_EINVAL, "eps must be a positive normal fp32 number");
  if (!std::isfinite((float)scale)) return fail(ADASUM_EINVAL, "scale must be finite in fp32");
  if (count == 0 || rows == 0) return ADASUM_OK;
  if (x == nullptr || out == nullptr) return einval("%s is NULL", x == nullptr ? "x" : "out");
  const size_t need = ortho_workspace(count, rows, cols, out_dtype);
  RETURN_IF(check_workspace(workspace, workspace_bytes, need));
  std::vector<Rows> b;
  const size_t x_size = size_of(dtype), out_size = size_of(out_dtype);
  for (int64_t i = 0; i < count; ++i) {
    const bool in_place = x[i] == out[i] && x_stride == out_stride && dtype == out_dtype;
    b.push_back({{x[i], in_place ? 0 : x_bytes, x_size, "x", false}, cols * x_size, x_stride * x_size, (int)i});
    b.push_back({{out[i], out_bytes, out_size, "out", true}, cols * out_size, out_stride * out_size, (int)i});
  }
  b.push_back({{workspace, need, 16, "workspace", true}, need, need, -1});
  RETURN_IF(check_many(b));
  OrthoCall call{};
  OrthoArgs& a = call.args;
  a.rows = rows;
  a.cols = cols;
  a.x_stride = x_stride;
  a.out_stride = out_stride;
  a.out_dtype = out_dtype;
  a.steps = steps;
  a.plain = plain;
  a.eps = eps;
  a.scale = (float)scale;
  for (int i = 0; i < 3 * steps; ++i) a.coefficients[i] = coefficients[i];
  a.ws = static_cast<char*>(workspace);
  call.count = count;
  call.x = x;
  call.out = out;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const double bytes = (double)count * rows * cols * (size_of(dtype) + size_of(out_dtype));
  return launch(kOrthogonal, "orthogonalize", bytes, st, [&] { return launch_ortho(dtype, call, st); });
}

}  // namespace
}  // namespace adasum

extern "C" {

int adasum_embedding(const void* table, int64_t vocab, int64_t hidden, int64_t table_stride, int table_dtype,
                     const void* tokens, int token_bytes, int64_t n, double scale, void* out, int64_t out_stride,
                     int out_dtype, void* stream) {
  return adasum::guarded([&] {
    return adasum::embedding(table, vocab, hidden, table_stride, table_dtype, tokens, token_bytes, n, scale, out,
                             out_stride, out_dtype, stream);
  });
}

int64_t adasum_embedding_grad_workspace_bytes(int64_t n, int64_t hidden, int dtype) {
  return adasum::guarded([&] { return adasum::embedding_grad_bytes(n, hidden, dtype); });
}

int adasum_embedding_grad(const void* dy, int64_t n, int64_t hidden, int64_t dy_stride, int dtype,
                          const void* tokens, int token_bytes, int64_t vocab, double scale, void* grad,
                          int grad_dtype, int accumulate, void* workspace, size_t workspace_bytes, void* stream) {
  return adasum::guarded([&] {
    return adasum::embedding_grad(dy, n, hidden, dy_stride, dtype, tokens, token_bytes, vocab, scale, grad,
                                  grad_dtype, accumulate, workspace, workspace_bytes, stream);
  });
}

int adasum_layer_norm(const void* x, int64_t rows, int64_t hidden, int64_t x_stride, int dtype, const void* weight,
                      const void* bias, int param_dtype, double eps, void* y, int64_t y_stride, float* mean,
                      float* rstd, int8_t* codes, uint8_t* scales, void* stream) {
  return adasum::guarded([&] {
    return adasum::layer_norm(x, rows, hidden, x_stride, dtype, weight, bias, param_dtype, eps, y, y_stride, mean,
                              rstd, codes, scales, stream);
  });
}

int64_t adasum_layer_norm_grad_workspace_bytes(int64_t rows, int64_t hidden, int dtype) {
  return adasum::guarded([&] { return adasum::layer_norm_grad_bytes(rows, hidden, dtype); });
}

int adasum_layer_norm_grad(const void* dy, int64_t rows, int64_t hidden, int64_t dy_stride, int dtype,
                           const void* x, int64_t x_stride, const float* mean, const int8_t* codes,
                           const uint8_t* scales, const float* rstd, const void* weight, int param_dtype, void* dx,
                           int64_t dx_stride, void* dweight, void* dbias, int grad_dtype, int accumulate,
                           void* workspace, size_t workspace_bytes, void* stream) {
  return adasum::guarded([&] {
    return adasum::layer_norm_grad(dy, rows, hidden, dy_stride, dtype, x, x_stride, mean, codes, scales, rstd,
                                   weight, param_dtype, dx, dx_stride, dweight, dbias, grad_dtype, accumulate,
                                   workspace, workspace_bytes, stream);
  });
}

int adasum_checkpoint_pack(const void* x, int64_t rows, int64_t hidden, int64_t x_stride, int dtype, int8_t* codes,
                           uint8_t* scales, void* stream) {
  return adasum::guarded(
      [&] { return adasum::checkpoint_pack(x, rows, hidden, x_stride, dtype, codes, scales, stream); });
}

int adasum_checkpoint_unpack(const int8_t* codes, const uint8_t* scales, int64_t rows, int64_t hidden, void* out,
                             int64_t out_stride, int dtype, void* stream) {
  return adasum::guarded(
      [&] { return adasum::checkpoint_unpack(codes, scales, rows, hidden, out, out_stride, dtype, stream); });
}

int64_t adasum_linear_grad_workspace_bytes(int64_t rows, int64_t out_features, int64_t in_features, int dtype) {
  return adasum::guarded([&] { return adasum::linear_grad_bytes(rows, out_features, in_features, dtype); });
}

int adasum_linear_grad(const void* dy, int64_t rows, int64_t out_features, int64_t dy_stride, int dtype,
                       const int8_t* codes, const uint8_t* scales, int64_t in_features, void* dweight, void* dbias,
                       int grad_dtype, int accumulate, void* workspace, size_t workspace_bytes, void* stream) {
  return adasum::guarded([&] {
    return adasum::linear_grad(dy, rows, out_features, dy_stride, dtype, codes, scales, in_features, dweight, dbias,
                               grad_dtype, accumulate, workspace, workspace_bytes, stream);
  });
}

int adasum_rms(const void* x, int64_t rows, int64_t hidden, int64_t x_stride, int dtype, const void* residual,
               int64_t residual_stride, int stream_dtype, const void* weight, int param_dtype, double eps, void* y,
               int64_t y_stride, void* h, int64_t h_stride, float* rstd, int8_t* codes, uint8_t* scales,
               void* stream) {
  return adasum::guarded([&] {
    return adasum::rms(x, rows, hidden, x_stride, dtype, residual, residual_stride, stream_dtype, weight, param_dtype,
                       eps, y, y_stride, h, h_stride, rstd, codes, scales, stream);
  });
}

int64_t adasum_rms_grad_workspace_bytes(int64_t rows, int64_t hidden, int dtype) {
  return adasum::guarded([&] { return adasum::rms_grad_bytes(rows, hidden, dtype); });
}

int adasum_rms_grad(const void* dy, int64_t rows, int64_t hidden, int64_t dy_stride, int dtype, const void* h,
                    int64_t h_stride, int stream_dtype, const void* dh, int64_t dh_stride, const float* rstd,
                    const void* weight, int param_dtype, void* dx, int64_t dx_stride, void* dweight, int grad_dtype,
                    int accumulate, void* workspace, size_t workspace_bytes, void* stream) {
  return adasum::guarded([&] {
    return adasum::rms_grad(dy, rows, hidden, dy_stride, dtype, h, h_stride, stream_dtype, dh, dh_stride, rstd, weight,
                            param_dtype, dx, dx_stride, dweight, grad_dtype, accumulate, workspace, workspace_bytes,
                            stream);
  });
}

int adasum_relative_bias(const void* table, int64_t buckets, int64_t heads, int64_t table_stride, int table_dtype,
                         int64_t max_distance, int bidirectional, int64_t batch, int64_t queries, int64_t keys,
                         int64_t offset, const void* scores, int64_t scores_stride, void* out, int64_t out_stride,
                         int dtype, void* stream) {
  return adasum::guarded([&] {
    return adasum::relative_bias(table, buckets, heads, table_stride, table_dtype, max_distance, bidirectional, batch,
                                 queries, keys, offset, scores, scores_stride, out, out_stride, dtype, stream);
  });
}

int64_t adasum_relative_bias_grad_workspace_bytes(int64_t batch, int64_t heads, int64_t queries, int64_t keys,
                                                  int dtype) {
  return adasum::guarded([&] { return adasum::relative_bias_grad_bytes(batch, heads, queries, keys, dtype); });
}

int adasum_relative_bias_grad(const void* dscores, int64_t batch, int64_t heads, int64_t queries, int64_t keys,
                              int64_t stride, int dtype, int64_t offset, int64_t buckets, int64_t max_distance,
                              int bidirectional, void* dtable, int grad_dtype, int accumulate, void* workspace,
                              size_t workspace_bytes, void* stream) {
  return adasum::guarded([&] {
    return adasum::relative_bias_grad(dscores, batch, heads, queries, keys, stride, dtype, offset, buckets,
                                      max_distance, bidirectional, dtable, grad_dtype, accumulate, workspace,
                                      workspace_bytes, stream);
  });
}

int64_t adasum_orthogonalize_workspace_bytes(int64_t count, int64_t rows, int64_t cols, int out_dtype) {
  return adasum::guarded([&] { return adasum::orthogonalize_bytes(count, rows, cols, out_dtype); });
}

int adasum_orthogonalize(const void* const* x, int64_t count, int64_t rows, int64_t cols, int64_t x_stride, int dtype,
                         int steps, const double* coefficients, double eps, double scale, void* const* out,
                         int64_t out_stride, int out_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  return adasum::guarded([&] {
    return adasum::orthogonalize(x, count, rows, cols, x_stride, dtype, steps, coefficients, eps, scale, out,
                                 out_stride, out_dtype, workspace, workspace_bytes, stream);
  });
}

}  // extern "C"
