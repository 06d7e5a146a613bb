// The linear gradient's kernels on the CPU: rows out in dtype grad_dtype
// accumulate.
#include "linear_grad.inc"
#include "values.h"

using namespace adasum;

int main(int, char** arg) {
  std::setvbuf(stdout, nullptr, _IONBF, 0);
  const int64_t rows = std::atoll(arg[1]), out = std::atoll(arg[2]), in = std::atoll(arg[3]);
  const int dtype = std::atoi(arg[4]), grad = std::atoi(arg[5]), add = std::atoi(arg[6]);
  const int64_t stride = out + 5, nb = (in + 31) / 32;
  std::srand(3);
  char* dy = rows_of(rows, out, stride, dtype);
  int8_t* codes = reinterpret_cast<int8_t*>(on_cpu::guarded(rows * in));
  uint8_t* scales = reinterpret_cast<uint8_t*>(on_cpu::guarded(rows * nb));
  for (int64_t i = 0; i < rows * in; ++i) codes[i] = (int8_t)(std::rand() % 255 - 127);
  for (int64_t i = 0; i < rows * nb; ++i) scales[i] = (uint8_t)(119 + std::rand() % 3);
  char* dw = rows_of(1, out * in, out * in, grad);
  char* db = rows_of(1, out, out, grad);
  const LinearGradLayout l = linear_grad_layout(rows, out, in, dtype);
  char* ws = on_cpu::guarded(l.total);
  for (size_t i = 0; i < l.total; ++i) ws[i] = (char)0xff;  // NaN

  std::vector<double> sw(out * in), sb(out);
  for (int64_t i = 0; i < out * in; ++i) sw[i] = add ? value(dw, grad, i) : 0.0;
  for (int64_t o = 0; o < out; ++o) sb[o] = add ? value(db, grad, o) : 0.0;
  LinearGradArgs a{dy, rows, stride, out, in, codes, scales, dw, db, grad, add, ws};
  launch_linear_grad(dtype, a, nullptr);

  for (int64_t r = 0; r < rows; ++r)
    for (int64_t o = 0; o < out; ++o) {
      const double d = value(dy, dtype, r * stride + o);
      sb[o] += d;
      for (int64_t i = 0; i < in; ++i) sw[o * in + i] += d * codes[r * in + i] * std::exp2(scales[r * nb + i / 32] - 127.);
    }
  // products are 13-bit multiples of 2^-14 below 1: sums of up to 1024 are
  // exact in fp32, and rounded once
  const double u = grad == 0 ? 0.0 : half_step(grad);
  for (int64_t i = 0; i < out * in; ++i)
    if (!(std::abs(value(dw, grad, i) - sw[i]) <= u * std::abs(sw[i]))) on_cpu::stop("a wrong value of dweight");
  for (int64_t o = 0; o < out; ++o)
    if (!(std::abs(value(db, grad, o) - sb[o]) <= u * std::abs(sb[o]))) on_cpu::stop("a wrong value of dbias");
  std::printf("done\n");
}
