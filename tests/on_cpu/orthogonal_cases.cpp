// The orthogonal update's kernels on the CPU against the definition in long
// double: rows cols dtype out_dtype steps rank rounded eps limit, and a b c for
// each step (or once for all).  rank 0: whole numbers / 64 at every place; else
// a product of that rank, of whole numbers, or (rounded) of such a product that
// does not fit its type.  The largest singular value of the update is about 1
// where it is divided by its norm, so eps says how small the matrix is beside it.
#include "orthogonal.inc"
#include "orthogonal_narrow.inc"
#include "values.h"

using namespace adasum;
typedef long double Real;

int main(int count, char** arg) {
  std::setvbuf(stdout, nullptr, _IONBF, 0);
  on_cpu::may_divide = true;
  int v[7];
  for (int i = 0; i < 7; ++i) v[i] = std::atoi(arg[i + 1]);
  const int64_t rows = v[0], cols = v[1], stride = cols + 3, out_stride = cols + 1;
  const int dtype = v[2], out_dtype = v[3], steps = v[4], rank = v[5];
  const double eps = std::atof(arg[8]), limit = std::atof(arg[9]);
  const int given = (count - 10) / 3;
  std::srand(7);
  char* x = rows_of(rows, cols, stride, dtype);
  char* out = rows_of(rows, cols, out_stride, out_dtype);
  if (rank > 0) {
    std::vector<double> left(rows * rank), right(rank * cols);
    for (double& t : left) t = std::rand() % 15 - 7 + (v[6] ? std::rand() / 3e9 : 0.);
    for (double& t : right) t = std::rand() % 15 - 7 + (v[6] ? std::rand() / 3e9 : 0.);
    for (int64_t i = 0; i < rows; ++i)
      for (int64_t j = 0; j < cols; ++j) {
        double sum = 0;
        for (int r = 0; r < rank; ++r) sum += left[i * rank + r] * right[r * cols + j];
        put(x, dtype, i * stride + j, sum);
      }
  }
  const OrthoLayout l = ortho_layout(1, rows, cols, out_dtype);
  OrthoCall call{};
  OrthoArgs& a = call.args;
  a.rows = rows;
  a.cols = cols;
  a.x_stride = stride;
  a.out_stride = out_stride;
  a.out_dtype = out_dtype;
  a.steps = steps;
  a.eps = eps;
  a.scale = 1.f;
  for (int i = 0; i < 3 * steps; ++i) a.coefficients[i] = std::atof(arg[10 + i % (3 * given)]);
  a.ws = on_cpu::guarded(l.total);
  const void* const from[] = {x};
  void* const to[] = {out};
  call.count = 1;
  call.x = from;
  call.out = to;
  launch_ortho(dtype, call, nullptr);

  // the shorter side's products
  const bool tall = rows > cols;
  const int64_t n = std::min(rows, cols), m = std::max(rows, cols);
  std::vector<Real> y(n * m);
  Real norm = 0;
  for (int64_t i = 0; i < n; ++i)
    for (int64_t j = 0; j < m; ++j) {
      y[i * m + j] = value(x, dtype, tall ? j * stride + i : i * stride + j);
      norm += y[i * m + j] * y[i * m + j];
    }
  norm = std::sqrt(norm);
  for (Real& t : y) t /= norm + eps;
  for (int s = 0; s < steps; ++s) {
    const double* k = a.coefficients + 3 * s;
    std::vector<Real> g(n * n), p(n * n), z(n * m);
    for (int64_t i = 0; i < n; ++i)
      for (int64_t j = i; j < n; ++j) {
        Real sum = 0;
        for (int64_t q = 0; q < m; ++q) sum += y[i * m + q] * y[j * m + q];
        g[i * n + j] = g[j * n + i] = sum;
      }
    for (int64_t i = 0; i < n; ++i)
      for (int64_t j = 0; j < n; ++j) {
        Real sum = 0;
        for (int64_t q = 0; q < n; ++q) sum += g[i * n + q] * g[j * n + q];
        p[i * n + j] = k[1] * g[i * n + j] + k[2] * sum + (i == j ? k[0] : 0.);
      }
    for (int64_t i = 0; i < n; ++i)
      for (int64_t q = 0; q < n; ++q)
        for (int64_t j = 0; j < m; ++j) z[i * m + j] += p[i * n + q] * y[q * m + j];
    y.swap(z);
  }
  Real off = 0, all = 0, got_all = 0;
  for (int64_t i = 0; i < n; ++i)
    for (int64_t j = 0; j < m; ++j) {
      const Real got = value(out, out_dtype, tall ? j * out_stride + i : i * out_stride + j), want = y[i * m + j];
      off += (got - want) * (got - want);
      all += want * want;
      got_all += got * got;
    }
  const double far = (double)std::sqrt(off / all);
  std::printf("off by %.3g of the norm %.6Lg (is %.6Lg), limit %.3g\n", far, std::sqrt(all), std::sqrt(got_all), limit);
  if (!(far <= limit)) on_cpu::stop("too far off");
  std::printf("done\n");
}
