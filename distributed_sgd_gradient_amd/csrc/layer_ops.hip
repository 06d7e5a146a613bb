// layer_ops.hip - C ABI of the layer operators: argument checks and launches.
//
// Every entry point checks all of its arguments before anything is enqueued,
// on the host first and then with the runtime's pointer queries, allocates
// nothing, and lets no C++ exception out.
#include "layer_ops.h"

#include <hip/hip_runtime.h>

#include <cfloat>
#include <cmath>
#include <cstdio>
#include <exception>
#include <mutex>
#include <new>

#include "../../include/adasum.h"
#include "library.h"

namespace adasum {
namespace {

bool known_dtype(int d) { return d == ADASUM_F32 || d == ADASUM_F16 || d == ADASUM_BF16; }
size_t size_of(int d) { return d == ADASUM_F32 ? 4 : 2; }

constexpr int64_t kMaxElements = int64_t(1) << 40;
constexpr int64_t kMaxVocab = int64_t(1) << 24;

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

}  // extern "C"
