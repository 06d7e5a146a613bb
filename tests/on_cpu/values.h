// Arrays of a dtype code (0 fp32, 1 fp16, 2 bf16) for the programs here.
#pragma once

#include <hip/hip_runtime.h>

inline size_t size_of(int dtype) { return dtype == 0 ? 4 : 2; }
inline double value(const void* p, int dtype, int64_t i) {
  if (dtype == 0) return static_cast<const float*>(p)[i];
  if (dtype == 1) return (double)(float)static_cast<const _Float16*>(p)[i];
  return (double)(float)static_cast<const __bf16*>(p)[i];
}
inline void put(void* p, int dtype, int64_t i, double v) {
  if (dtype == 0)
    static_cast<float*>(p)[i] = (float)v;
  else if (dtype == 1)
    static_cast<_Float16*>(p)[i] = (_Float16)(float)v;
  else
    static_cast<__bf16*>(p)[i] = (__bf16)(float)v;
}
inline double half_step(int dtype) { return std::exp2(dtype == 0 ? -24 : dtype == 1 ? -11 : -8); }

// Guarded rows, `stride` apart, of whole numbers / 64 in [-1, 1]; the gaps
// hold NaN.
inline char* rows_of(int64_t rows, int64_t width, int64_t stride, int dtype) {
  const int64_t n = (rows - 1) * stride + width;
  char* p = on_cpu::guarded(n * size_of(dtype));
  for (int64_t i = 0; i < n; ++i)
    put(p, dtype, i, i % stride < width ? (std::rand() % 129 - 64) / 64. : std::nan(""));
  return p;
}
