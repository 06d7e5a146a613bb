// The embedding kernels on the CPU: n vocab hidden kind dtype grad_dtype
// token_bytes accumulate.  The grouped list has to be right at every position,
// so that no bound the kernels put on it is ever met, and the sums within
// rounding of 64 bits.
#include <hip/hip_runtime.h>

namespace adasum {
namespace {
thread_local int32_t counts[16 * 512];  // the grouping kernel's dynamic LDS
}
}  // namespace adasum

#include "embedding.inc"
#include "values.h"

using namespace adasum;

int main(int, char** arg) {
  std::setvbuf(stdout, nullptr, _IONBF, 0);
  const int64_t n = std::atoll(arg[1]), vocab = std::atoll(arg[2]);
  const int hidden = std::atoi(arg[3]), kind = std::atoi(arg[4]), dtype = std::atoi(arg[5]), out = std::atoi(arg[6]);
  const int token_bytes = std::atoi(arg[7]), accumulate = std::atoi(arg[8]);
  const size_t b = size_of(dtype), g = size_of(out);
  std::srand(1);
  auto uniform = [] { return (std::rand() + 0.5) / (RAND_MAX + 1.0); };

  // kind 0: all alike; 1: one token in half of the rows; 2: one token; 3:
  // none; 4: a third is no token; 5: token r about as often as 1 / r
  std::vector<int64_t> token(n);
  for (int64_t& t : token) {
    t = (int64_t)(uniform() * vocab);
    if (kind == 1 && uniform() < 0.5) t = vocab / 2;
    if (kind == 2) t = vocab - 1;
    if (kind == 3) t = -1;
    if (kind == 4 && uniform() < 0.33) t = uniform() < 0.5 ? vocab : -1 - (int64_t)(uniform() * 1e6);
    if (kind == 5) t = uniform() < 0.1 ? -1 : std::min<int64_t>(vocab, (int64_t)std::exp(uniform() * std::log(vocab + 1.))) - 1;
  }
  char* tokens = on_cpu::guarded(n * token_bytes);
  for (int64_t i = 0; i < n; ++i) {
    if (token_bytes == 4) {
      const int32_t t = (int32_t)token[i];
      std::memcpy(tokens + 4 * i, &t, 4);
    } else {
      std::memcpy(tokens + 8 * i, &token[i], 8);
    }
  }
  char* dy = on_cpu::guarded(n * hidden * b);
  for (int64_t i = 0; i < n * hidden; ++i) put(dy, dtype, i, (std::rand() % 129 - 64) / 64.);
  char* grad = on_cpu::guarded(vocab * hidden * g);
  for (int64_t i = 0; i < vocab * hidden; ++i) put(grad, out, i, accumulate ? i % 5 : 7777.);
  const EmbeddingGradLayout l = embedding_grad_layout(n, hidden, dtype);
  char* ws = on_cpu::guarded(l.total);
  for (size_t i = 0; i < l.total; ++i) ws[i] = (char)(0x91 + i % 111);

  EmbeddingGradArgs a{dy, n, hidden, vocab, hidden, tokens, token_bytes, 0.5f, grad, out, accumulate, ws};
  launch_embedding_grad(dtype, a, nullptr);

  // the list: tokens by their workgroup (the low bits), then by themselves,
  // then rows in order
  std::vector<int64_t> rows;
  for (int64_t i = 0; i < n; ++i)
    if (token[i] >= 0 && token[i] < vocab) rows.push_back(i);
  const int shift = group_shift(vocab);
  const int64_t mask = (int64_t(1) << shift) - 1;
  std::stable_sort(rows.begin(), rows.end(), [&](int64_t x, int64_t y) {
    const int64_t s = token[x], t = token[y];
    return (s & mask) != (t & mask) ? (s & mask) < (t & mask) : s < t;
  });
  const int32_t* listed = reinterpret_cast<int32_t*>(ws + l.rows);
  const int32_t* named = reinterpret_cast<int32_t*>(ws + l.tokens);
  if (*reinterpret_cast<int32_t*>(ws + l.count) != (int64_t)rows.size()) on_cpu::stop("a wrong number of listed rows");
  for (size_t p = 0; p < rows.size(); ++p)
    if (listed[p] != rows[p] || named[p] != token[rows[p]]) on_cpu::stop("a wrong place of the list");

  // 64ths and quarters of whole numbers: fp32 sums of up to 2^17 rows are
  // exact, and what is stored is rounded once (added to: from fp32)
  std::vector<double> sum(vocab * hidden, 0.0);
  for (int64_t r : rows)
    for (int c = 0; c < hidden; ++c) sum[token[r] * hidden + c] += value(dy, dtype, r * hidden + c);
  const double half = out == 0 ? 0.0 : half_step(out);
  for (int64_t i = 0; i < vocab * hidden; ++i) {
    const double want = 0.5 * sum[i] + (accumulate ? (double)(i % 5) : 0.0);
    if (!(std::abs(value(grad, out, i) - want) <= std::abs(want) * half)) on_cpu::stop("a wrong sum");
  }
  std::printf("done\n");
}
