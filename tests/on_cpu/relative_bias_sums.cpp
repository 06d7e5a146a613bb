// The relative bias's gradient on the CPU: queries keys dtype.  One diagonal has
// 2^25 in its first rows and ones further down, which a sum in fp32 would lose.
#include "relative_bias.inc"
#include "values.h"

using namespace adasum;

int main(int, char** arg) {
  std::setvbuf(stdout, nullptr, _IONBF, 0);
  on_cpu::may_divide = true;
  const int64_t queries = std::atoll(arg[1]), keys = std::atoll(arg[2]);
  const int dtype = std::atoi(arg[3]);
  const double large = dtype == 1 ? 32768. : 33554432., one = dtype == 1 ? 1. / 1024 : 1.;  // 2^25 apart
  char* scores = rows_of(queries, keys, keys, dtype);
  for (int64_t i = 0; i < queries * keys; ++i) put(scores, dtype, i, 0.);
  // on the diagonal, 16 rows apart: every group of lanes has one
  put(scores, dtype, 2 * keys + 2, large);
  int ones = 0;
  for (int64_t i = 16; i < queries && i < keys; i += 16, ++ones) put(scores, dtype, i * keys + i, one);
  const BiasBuckets k = bias_buckets(32, 128, true);
  const BiasGradLayout l = bias_grad_layout(1, 1, queries, keys, dtype);
  char* grad = rows_of(32, 1, 1, 0);
  BiasGradArgs g{scores, keys, k, 32, 1, 1, queries, keys, 0, grad, 0, 0,
                 reinterpret_cast<float*>(on_cpu::guarded(l.bytes))};
  launch_bias_grad(dtype, g, nullptr);
  const float got = (float)value(grad, 0, 0), want = (float)(large + ones * one);
  std::printf("%d ones: %.9g, not %.9g\n", ones, got, want);
  if (got != want || ones < 3) on_cpu::stop("sum");
  std::printf("done\n");
}
