// The relative bias's kernels on the CPU: batch heads queries keys offset
// buckets reach both dtype.  Values are whole numbers / 64, so sums are exact.
#include "relative_bias.inc"
#include "values.h"

using namespace adasum;

int main(int, char** arg) {
  std::setvbuf(stdout, nullptr, _IONBF, 0);
  on_cpu::may_divide = true;
  int64_t v[9];
  for (int i = 0; i < 9; ++i) v[i] = std::atoll(arg[i + 1]);
  const int64_t batch = v[0], heads = v[1], queries = v[2], keys = v[3], offset = v[4];
  const int buckets = (int)v[5], both = (int)v[7], dtype = (int)v[8];
  const int64_t rows = batch * heads * queries, stride = keys + 2;
  std::srand(3);
  const BiasBuckets k = bias_buckets(buckets, v[6], both != 0);
  auto bucket = [&](int64_t d) {
    const int64_t n = both ? std::abs(d) : std::max<int64_t>(-d, 0);
    int b = 0;
    while (b + 1 < k.side && k.border[b + 1] <= n) ++b;
    return both && d > 0 ? b + k.side : b;
  };
  char* table = rows_of(buckets, heads, heads + 1, 0);
  char* scores = rows_of(rows, keys, stride, dtype);
  char* out = rows_of(rows, keys, stride, dtype);
  BiasArgs f{table, heads + 1, 0, k, batch, heads, queries, keys, offset, scores, stride, stride, out};
  launch_bias(dtype, f, nullptr);
  std::vector<double> sums(buckets * heads);
  for (int64_t r = 0; r < rows; ++r)
    for (int64_t j = 0; j < keys; ++j) {
      const int64_t i = r % queries, h = r / queries % heads;
      const int b = bucket(j - i - offset);
      const double s = value(scores, dtype, r * stride + j), t = s + value(table, 0, b * (heads + 1) + h);
      if (std::abs(value(out, dtype, r * stride + j) - t) > half_step(dtype) * std::abs(t)) on_cpu::stop("out");
      sums[b * heads + h] += s;
    }
  for (int64_t r = 0; r + 1 < rows; ++r)
    for (int64_t j = keys; j < stride; ++j)
      if (value(out, dtype, r * stride + j) == value(out, dtype, r * stride + j)) on_cpu::stop("a gap was written");
  BiasArgs alone = f;
  alone.batch = 1;
  alone.scores = nullptr;
  char* line = rows_of(heads * queries, keys, stride, 0);
  alone.out = line;
  launch_bias(0, alone, nullptr);
  for (int64_t r = 0; r < heads * queries; ++r)
    for (int64_t j = 0; j < keys; ++j)
      if (value(line, 0, r * stride + j) != value(table, 0, bucket(j - r % queries - offset) * (heads + 1) + r / queries))
        on_cpu::stop("bias");

  const BiasGradLayout l = bias_grad_layout(batch, heads, queries, keys, dtype);
  float* partials = reinterpret_cast<float*>(on_cpu::guarded(l.bytes));
  char* grad = rows_of(buckets, heads, heads, 0);
  std::vector<double> before(buckets * heads);
  for (int i = 0; i < buckets * heads; ++i) before[i] = value(grad, 0, i);
  BiasGradArgs g{scores, stride, k, buckets, batch, heads, queries, keys, offset, grad, 0, 1, partials};
  launch_bias_grad(dtype, g, nullptr);
  for (int i = 0; i < buckets * heads; ++i)
    if (value(grad, 0, i) != before[i] + sums[i]) {
      std::printf("bucket %d head %d: %.9g, not %.9g\n", i / (int)heads, i % (int)heads, value(grad, 0, i),
                  before[i] + sums[i]);
      on_cpu::stop("dtable");
    }
  std::printf("done\n");
}
