// The orthogonal update's kernels on the CPU: count rows cols dtype out_dtype
// steps.
#include "orthogonal.inc"
#include "orthogonal_narrow.inc"
#include "values.h"

using namespace adasum;

int main(int, char** arg) {
  std::setvbuf(stdout, nullptr, _IONBF, 0);
  on_cpu::may_divide = true;
  int v[6];
  for (int i = 0; i < 6; ++i) v[i] = std::atoi(arg[i + 1]);
  const int64_t count = v[0], rows = v[1], cols = v[2], stride = cols + 3, out_stride = cols + 1;
  const int dtype = v[3], out_dtype = v[4], steps = v[5];
  std::srand(4);
  std::vector<const void*> x;
  std::vector<void*> out;
  for (int i = 0; i < count; ++i) {
    x.push_back(rows_of(rows, cols, stride, dtype));
    out.push_back(rows_of(rows, cols, out_stride, out_dtype));
  }
  const OrthoLayout l = ortho_layout(count, rows, cols, out_dtype);
  OrthoCall call{};
  call.args.rows = rows;
  call.args.cols = cols;
  call.args.x_stride = stride;
  call.args.out_stride = out_stride;
  call.args.out_dtype = out_dtype;
  call.args.steps = steps;
  call.args.eps = 1e-7;
  call.args.scale = 1.5f;
  const double k[3] = {3.4445, -4.775, 2.0315};
  for (int i = 0; i < 3 * steps; ++i) call.args.coefficients[i] = k[i % 3];
  call.args.ws = on_cpu::guarded(l.total);
  call.count = count;
  call.x = x.data();
  call.out = out.data();
  launch_ortho(dtype, call, nullptr);
  for (int c = 0; c < count; ++c) {
    std::vector<double> a(rows * cols), b;
    double s = 0;
    for (int64_t i = 0; i < rows * cols; ++i) {
      a[i] = value(x[c], dtype, i / cols * stride + i % cols);
      s += a[i] * a[i];
    }
    s = std::sqrt(s) + 1e-7;
    for (double& t : a) t /= s;
    for (int t = 0; t < steps; ++t) {
      // a X + b (X X^T) X + c (X X^T) (X X^T) X, whichever side is shorter
      auto gram_times = [&](const std::vector<double>& y) {
        std::vector<double> g(rows * rows), z(rows * cols);
        for (int64_t i = 0; i < rows; ++i)
          for (int64_t j = 0; j < rows; ++j)
            for (int64_t q = 0; q < cols; ++q) g[i * rows + j] += a[i * cols + q] * a[j * cols + q];
        for (int64_t i = 0; i < rows; ++i)
          for (int64_t j = 0; j < rows; ++j)
            for (int64_t q = 0; q < cols; ++q) z[i * cols + q] += g[i * rows + j] * y[j * cols + q];
        return z;
      };
      const std::vector<double> one = gram_times(a), two = gram_times(one);
      for (int64_t i = 0; i < rows * cols; ++i) a[i] = k[0] * a[i] + k[1] * one[i] + k[2] * two[i];
    }
    double off = 0, all = 0;
    for (int64_t i = 0; i < rows * cols; ++i) {
      const double got = value(out[c], out_dtype, i / cols * out_stride + i % cols);
      off += std::pow(got - 1.5 * a[i], 2);
      all += std::pow(1.5 * a[i], 2);
    }
    for (int64_t r = 0; r + 1 < rows; ++r)
      if (value(out[c], out_dtype, r * out_stride + cols) == value(out[c], out_dtype, r * out_stride + cols))
        on_cpu::stop("a gap was written");
    const double far = std::sqrt(off / all);
    std::printf("off by %.3g of the norm\n", far);
    if (!(far <= (out_dtype == 2 ? 6e-3 : out_dtype == 1 ? 6e-4 : 2e-5))) on_cpu::stop("too far off");
  }
  std::printf("done\n");
}
