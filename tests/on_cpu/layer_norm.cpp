// The layer norm kernels on the CPU: rows hidden dtype kept accumulate.
#include "layer_norm.inc"
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
  const int H = std::atoi(arg[2]), dtype = std::atoi(arg[3]), kept = std::atoi(arg[4]), add = std::atoi(arg[5]);
  const int64_t gap = 3, stride = H + gap, nb = (H + 31) / 32;
  std::srand(2);
  char* x = rows_of(rows, H, stride, dtype);
  char* dy = rows_of(rows, H, H + 1, dtype);
  char* y = rows_of(rows, H, stride, dtype);
  char* dx = rows_of(rows, H, stride, dtype);
  char* w = rows_of(1, H, H, 0);
  char* b = rows_of(1, H, H, 0);
  float* mean = reinterpret_cast<float*>(on_cpu::guarded(rows * 4));
  float* rstd = reinterpret_cast<float*>(on_cpu::guarded(rows * 4));
  int8_t* codes = reinterpret_cast<int8_t*>(on_cpu::guarded(rows * H));
  uint8_t* scales = reinterpret_cast<uint8_t*>(on_cpu::guarded(rows * nb));
  const double eps = 1e-3;

  NormArgs f{x, rows, stride, stride, H, w, b, 0, (float)eps, y, kept ? nullptr : mean, rstd,
             kept ? codes : nullptr, kept ? scales : nullptr};
  launch_norm(dtype, f, nullptr);

  const int64_t parts = norm_grad_parts(rows, H);
  float* partials = reinterpret_cast<float*>(on_cpu::guarded(parts * 2 * H * 4));
  char* dw = rows_of(1, H, H, dtype);
  char* db = rows_of(1, H, H, dtype);
  std::vector<double> sw(H), sb(H), aw(H), ab(H);
  for (int c = 0; c < H; ++c) {
    sw[c] = add ? value(dw, dtype, c) : 0.0;
    sb[c] = add ? value(db, dtype, c) : 0.0;
  }
  NormGradArgs g{dy, rows, H + 1, stride, stride, H, kept ? nullptr : x, kept ? nullptr : mean,
                 kept ? codes : nullptr, kept ? scales : nullptr, rstd, w, 0, dx, dw, db, dtype, add, partials};
  launch_norm_grad(dtype, g, nullptr);

  // loose bounds: the values are checked closely elsewhere, this looks for
  // accesses and for columns or rows that are mixed up
  const double e = 1e-4, u = half_step(dtype);
  for (int64_t r = 0; r < rows; ++r) {
    double m = 0, v = 0, mg = 0, mgn = 0;
    for (int c = 0; c < H; ++c) m += value(x, dtype, r * stride + c) / H;
    for (int c = 0; c < H; ++c) v += std::pow(value(x, dtype, r * stride + c) - m, 2) / H;
    const double s = 1 / std::sqrt(v + eps);
    close_to(rstd[r], s, e * s, "rstd");
    if (!kept) close_to(mean[r], m, e, "mean");
    std::vector<double> n(H);
    for (int c = 0; c < H; ++c) {
      n[c] = (value(x, dtype, r * stride + c) - m) * s;
      const double t = n[c] * value(w, 0, c) + value(b, 0, c);
      close_to(value(y, dtype, r * stride + c), t, e * 40 + u * std::abs(t), "y");
      if (kept) n[c] = codes[r * H + c] * std::exp2(scales[r * nb + c / 32] - 127.);
      const double gr = value(dy, dtype, r * (H + 1) + c) * value(w, 0, c);
      mg += gr / H;
      mgn += gr * n[c] / H;
    }
    for (int c = 0; c < H; ++c) {
      const double d = value(dy, dtype, r * (H + 1) + c);
      const double t = s * (d * value(w, 0, c) - mg - n[c] * mgn);
      close_to(value(dx, dtype, r * stride + c), t, e * s * (1 + std::abs(n[c])) + u * std::abs(t), "dx");
      sw[c] += d * n[c];
      sb[c] += d;
      aw[c] += std::abs(d * n[c]);
      ab[c] += std::abs(d);
    }
    for (int64_t c = H; r + 1 < rows && c < stride; ++c)
      if (value(y, dtype, r * stride + c) == value(y, dtype, r * stride + c) ||
          value(dx, dtype, r * stride + c) == value(dx, dtype, r * stride + c))
        on_cpu::stop("a gap between rows was written");
  }
  for (int c = 0; c < H; ++c) {
    close_to(value(dw, dtype, c), sw[c], e * aw[c] + u * std::abs(sw[c]), "dweight");
    close_to(value(db, dtype, c), sb[c], e * ab[c] + u * std::abs(sb[c]), "dbias");
  }
  std::printf("done\n");
}
