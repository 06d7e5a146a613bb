// The root-mean-square norm's kernels on the CPU: rows hidden dtype wide
// (an fp32 stream) more (a residual, 8-bit rows, dh, and accumulation).
#include "rms.inc"
#include "values.h"

using namespace adasum;

static void close_to(double got, double want, double bound, const char* what) {
  if (!(std::abs(got - want) <= bound)) {
    std::printf("%s: %.9g, not %.9g within %.3g\n", what, got, want, bound);
    on_cpu::stop(what);
  }
}

int main(int, char** arg) {
  std::setvbuf(stdout, nullptr, _IONBF, 0);
  on_cpu::may_divide = true;  // 16 lanes have a row of their own, which others may not
  const int64_t rows = std::atoll(arg[1]);
  const int H = std::atoi(arg[2]), dtype = std::atoi(arg[3]), wide = std::atoi(arg[4]), more = std::atoi(arg[5]);
  const int of = wide ? 0 : dtype;
  const int64_t stride = H + 3, nb = (H + 31) / 32;
  std::srand(2);
  char* x = rows_of(rows, H, stride, dtype);
  char* residual = rows_of(rows, H, H + 1, of);
  char* y = rows_of(rows, H, stride, dtype);
  char* h = rows_of(rows, H, stride, of);
  char* dy = rows_of(rows, H, H + 1, dtype);
  char* dh = rows_of(rows, H, H + 2, of);
  char* dx = rows_of(rows, H, stride, of);
  char* w = rows_of(1, H, H, 0);
  float* rstd = reinterpret_cast<float*>(on_cpu::guarded(rows * 4));
  int8_t* codes = reinterpret_cast<int8_t*>(on_cpu::guarded(rows * H));
  uint8_t* scales = reinterpret_cast<uint8_t*>(on_cpu::guarded(rows * nb));
  const double eps = 1e-3;
  const bool add = more || of != dtype;

  RmsArgs f{x, add ? residual : nullptr, rows, stride, H + 1, stride, stride, H, w, 0, (float)eps, y,
            add ? h : nullptr, rstd, more ? codes : nullptr, more ? scales : nullptr};
  launch_rms(dtype, of, f, nullptr);
  if (!add) h = x;

  const int64_t parts = rms_grad_parts(rows, H);
  float* partials = reinterpret_cast<float*>(on_cpu::guarded(parts * H * 4));
  char* dw = rows_of(1, H, H, dtype);
  std::vector<double> sw(H), aw(H);
  for (int c = 0; c < H; ++c) sw[c] = more ? value(dw, dtype, c) : 0.0;
  RmsGradArgs g{dy, h, more ? dh : nullptr, rows, H + 1, stride, H + 2, stride, H, rstd, w, 0, dx, dw, dtype, more,
                partials};
  launch_rms_grad(dtype, of, g, nullptr);

  // loose bounds: this looks for accesses and for columns or rows mixed up
  const double e = 1e-4, u = half_step(dtype), v = half_step(of);
  for (int64_t r = 0; r < rows; ++r) {
    double s = 0, m = 0;
    std::vector<double> n(H);
    for (int c = 0; c < H; ++c) {
      const double t = value(x, dtype, r * stride + c) + (add ? value(residual, of, r * (H + 1) + c) : 0.0);
      n[c] = value(h, of, r * stride + c);
      close_to(n[c], t, v * std::abs(t), "h");
      s += n[c] * n[c] / H;
    }
    s = 1 / std::sqrt(s + eps);
    close_to(rstd[r], s, e * s, "rstd");
    for (int c = 0; c < H; ++c) {
      n[c] *= s;
      const double t = n[c] * value(w, 0, c);
      close_to(value(y, dtype, r * stride + c), t, (e + u) * std::abs(t), "y");
      m += value(dy, dtype, r * (H + 1) + c) * value(w, 0, c) * n[c] / H;
    }
    for (int b = 0; more && b < nb; ++b) {
      double most = 0;
      for (int c = 32 * b; c < std::min(H, 32 * b + 32); ++c)
        most = std::max(most, std::abs(value(y, dtype, r * stride + c)));
      for (int c = 32 * b; c < std::min(H, 32 * b + 32); ++c)
        close_to(codes[r * H + c] * std::exp2(scales[r * nb + b] - 127.), value(y, dtype, r * stride + c),
                 most / 127 + 1e-38, "codes");
    }
    for (int c = 0; c < H; ++c) {
      const double d = value(dy, dtype, r * (H + 1) + c);
      const double along = more ? value(dh, of, r * (H + 2) + c) : 0.0;
      const double t = along + s * (d * value(w, 0, c) - n[c] * m);
      close_to(value(dx, of, r * stride + c), t, e * (s * (1 + std::abs(n[c])) + std::abs(along)) + v * std::abs(t),
               "dx");
      sw[c] += d * n[c];
      aw[c] += std::abs(d * n[c]);
    }
    for (int64_t c = H; r + 1 < rows && c < stride; ++c)
      if (value(y, dtype, r * stride + c) == value(y, dtype, r * stride + c) ||
          value(dx, of, r * stride + c) == value(dx, of, r * stride + c) ||
          (add && value(h, of, r * stride + c) == value(h, of, r * stride + c)))
        on_cpu::stop("a gap between rows was written");
  }
  for (int c = 0; c < H; ++c) close_to(value(dw, dtype, c), sw[c], e * aw[c] + u * std::abs(sw[c]), "dweight");
  std::printf("done\n");
}
