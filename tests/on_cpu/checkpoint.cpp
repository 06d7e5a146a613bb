// The 8-bit pack and unpack kernels on the CPU: rows given and taken back,
// and the last pieces of the widest row that a call takes.
#include "checkpoint.inc"

using namespace adasum;

template <typename T>
static void round_trip(int dtype, int64_t rows, int hidden) {
  const int64_t nb = (hidden + 31) / 32;
  T* x = reinterpret_cast<T*>(on_cpu::guarded(rows * hidden * sizeof(T)));
  int8_t* codes = reinterpret_cast<int8_t*>(on_cpu::guarded(rows * hidden));
  uint8_t* scales = reinterpret_cast<uint8_t*>(on_cpu::guarded(rows * nb));
  T* out = reinterpret_cast<T*>(on_cpu::guarded(rows * hidden * sizeof(T)));
  for (int64_t i = 0; i < rows * hidden; ++i) x[i] = (T)(float)(std::rand() % 2001 - 1000);
  PackArgs p{x, rows, hidden, hidden, codes, scales};
  UnpackArgs u{codes, scales, rows, hidden, hidden, out};
  launch_pack(dtype, p, nullptr);
  launch_unpack(dtype, u, nullptr);
  for (int64_t r = 0; r < rows; ++r)
    for (int64_t b = 0; b < nb; ++b) {
      float top = 0.f;
      const int64_t end = std::min<int64_t>(hidden, 32 * b + 32);
      for (int64_t c = 32 * b; c < end; ++c) top = std::max(top, std::abs((float)x[r * hidden + c]));
      for (int64_t c = 32 * b; c < end; ++c)
        if (!(std::abs((float)out[r * hidden + c] - (float)x[r * hidden + c]) <= top / 127.f))
          on_cpu::stop("a value is off by more than half a step");
    }
  std::printf("round trip %d %lld x %d\n", dtype, (long long)rows, hidden);
}

// One row of 2^31 - 1 values: the workgroups of its first and its last pieces.
template <typename T>
static void widest(int dtype) {
  const int hidden = 0x7fffffff;
  const int64_t nb = ((int64_t)hidden + 31) / 32, tail = 5000;
  int8_t* codes = reinterpret_cast<int8_t*>(on_cpu::guarded(hidden));
  uint8_t* scales = reinterpret_cast<uint8_t*>(on_cpu::guarded(nb));
  T* out = reinterpret_cast<T*>(on_cpu::guarded((size_t)hidden * sizeof(T)));
  for (int64_t c = hidden - tail; c < hidden; ++c) codes[c] = (int8_t)(c % 251 - 125);
  for (int64_t b = nb - tail / 32 - 1; b < nb; ++b) scales[b] = (uint8_t)(126 + b % 3);
  UnpackArgs u{codes, scales, 1, hidden, hidden, out};
  on_cpu::wanted = [](unsigned x) { return x == 0 || x + 2 >= gridDim.x; };
  launch_unpack(dtype, u, nullptr);
  on_cpu::wanted = [](unsigned) { return true; };
  for (int64_t c = hidden - 1000; c < hidden; ++c)
    if ((float)out[c] != (float)codes[c] * std::exp2((float)scales[c / 32] - 127.f)) on_cpu::stop("a wrong value");
  std::printf("widest %d\n", dtype);
}

int main() {
  std::setvbuf(stdout, nullptr, _IONBF, 0);
  for (int hidden : {1, 7, 31, 32, 33, 100, 1001}) {
    round_trip<float>(0, 5, hidden);
    round_trip<_Float16>(1, 5, hidden);
    round_trip<__bf16>(2, 5, hidden);
  }
  widest<float>(0);
  widest<__bf16>(2);
  std::printf("done\n");
}
