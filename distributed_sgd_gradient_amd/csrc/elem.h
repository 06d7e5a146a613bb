// elem.h - element types, vector access and wave reductions of the layer
// operators' kernels (embedding, layer norm, 8-bit activations, linear
// gradients).  Device code only.
//
// A vector is 16 bytes: 8 values of a 16-bit type or 4 of fp32.  Rows may
// start at any multiple of the element size (an odd width, a gradient segment
// in the middle of a flat buffer), so every vector access is declared with
// the element's alignment only.  Global memory on gfx950 takes 16-byte
// accesses at any address, so the aligned and the unaligned case are the same
// instruction and need no second code path.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace adasum {
namespace elem {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));

template <typename V, int A>
struct __attribute__((packed, aligned(A))) Unaligned {
  V v;
};

template <typename V, int A>
__device__ __forceinline__ V load_at(const void* p) {
  return static_cast<const Unaligned<V, A>*>(p)->v;
}
template <typename V, int A>
__device__ __forceinline__ void store_at(void* p, V v) {
  static_cast<Unaligned<V, A>*>(p)->v = v;
}

template <typename T>
struct Type;
template <>
struct Type<float> {
  static constexpr int kVec = 4;
};
template <>
struct Type<_Float16> {
  static constexpr int kVec = 8;
};
template <>
struct Type<__bf16> {
  static constexpr int kVec = 8;
};

// 16 bytes of T, widened.  bf16 is the upper half of an fp32: shifts and
// masks instead of conversions.
template <typename T>
__device__ __forceinline__ void widen(v4u raw, float (&v)[Type<T>::kVec]) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 4) {
      v[i] = __builtin_bit_cast(float, w[i]);
    } else if constexpr (__is_same(T, __bf16)) {
      v[2 * i] = __builtin_bit_cast(float, w[i] << 16);
      v[2 * i + 1] = __builtin_bit_cast(float, w[i] & 0xffff0000u);
    } else {
      v[2 * i] = (float)__builtin_bit_cast(_Float16, (uint16_t)(w[i] & 0xffffu));
      v[2 * i + 1] = (float)__builtin_bit_cast(_Float16, (uint16_t)(w[i] >> 16));
    }
  }
}

// The raw 16 bytes of the kVec elements at p, of which the first `valid` are
// inside the row (fewer at a row's end, none past it): the others read as
// zeros and are not touched in memory.
template <typename T>
__device__ __forceinline__ v4u load_raw(const T* p, int valid) {
  constexpr int N = Type<T>::kVec;
  v4u raw = {0u, 0u, 0u, 0u};
  if (valid >= N) {
    raw = load_at<v4u, sizeof(T)>(p);
  } else if (valid > 0) {
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (i < valid) {
        if constexpr (sizeof(T) == 4)
          w[i] = __builtin_bit_cast(uint32_t, p[i]);
        else
          w[i / 2] |= (uint32_t)__builtin_bit_cast(uint16_t, p[i]) << (16 * (i & 1));
      }
    }
    raw = v4u{w[0], w[1], w[2], w[3]};
  }
  return raw;
}

// kVec values rounded to T (to nearest even) and stored at p, the first
// `valid` of them.
template <typename T>
__device__ __forceinline__ void store_vec(T* p, const float (&v)[Type<T>::kVec], int valid) {
  constexpr int N = Type<T>::kVec;
  if (valid >= N) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4)
        w[i] = __builtin_bit_cast(uint32_t, v[i]);
      else
        w[i] = (uint32_t)__builtin_bit_cast(uint16_t, (T)v[2 * i]) |
               ((uint32_t)__builtin_bit_cast(uint16_t, (T)v[2 * i + 1]) << 16);
    }
    store_at<v4u, sizeof(T)>(p, v4u{w[0], w[1], w[2], w[3]});
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < valid) p[i] = (T)v[i];
  }
}

// N values (a multiple of T's vector) at p, widened; the first `valid` lie in
// the row.
template <typename T, int N>
__device__ __forceinline__ void load_row(const T* p, int valid, float (&v)[N]) {
  constexpr int K = Type<T>::kVec;
  static_assert(N % K == 0, "whole vectors");
#pragma unroll
  for (int j = 0; j < N / K; ++j) {
    float t[K];
    widen<T>(load_raw(p + j * K, valid - j * K), t);
#pragma unroll
    for (int i = 0; i < K; ++i) v[j * K + i] = t[i];
  }
}
template <typename T, int N>
__device__ __forceinline__ void store_row(T* p, const float (&v)[N], int valid) {
  constexpr int K = Type<T>::kVec;
  static_assert(N % K == 0, "whole vectors");
#pragma unroll
  for (int j = 0; j < N / K; ++j) {
    float t[K];
#pragma unroll
    for (int i = 0; i < K; ++i) t[i] = v[j * K + i];
    store_vec(p + j * K, t, valid - j * K);
  }
}

// A parameter or gradient array whose dtype code (0 fp32, 1 fp16, 2 bf16) is
// known at run time only: for what is read or written once per workgroup.
__device__ __forceinline__ float load_any(const void* p, int dtype, int64_t i) {
  if (dtype == 0) return static_cast<const float*>(p)[i];
  if (dtype == 1) return (float)static_cast<const _Float16*>(p)[i];
  return (float)static_cast<const __bf16*>(p)[i];
}

// fp64 to fp32 with round-to-odd: rounding the result once more to a 16-bit
// type then gives the correctly rounded value of x.
__device__ __forceinline__ float round_to_odd(double x) {
  float f = (float)x;
  const double back = (double)f;
  if (back != x && x == x) {
    uint32_t u = __builtin_bit_cast(uint32_t, f);
    if (fabs(back) > fabs(x)) u -= 1;
    f = __builtin_bit_cast(float, u | 1u);
  }
  return f;
}
__device__ __forceinline__ void store_any(void* p, int dtype, int64_t i, double x) {
  if (dtype == 0)
    static_cast<float*>(p)[i] = (float)x;
  else if (dtype == 1)
    static_cast<_Float16*>(p)[i] = (_Float16)round_to_odd(x);
  else
    static_cast<__bf16*>(p)[i] = (__bf16)round_to_odd(x);
}

// x of lane (l ^ 1), (l ^ 2), (l ^ 7), (l ^ 15) of each 16 lanes: register
// moves inside the vector unit, no LDS.
template <int kCtrl>
__device__ __forceinline__ uint32_t dpp(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, kCtrl, 0xf, 0xf, true);
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kHalfMirror = 0x141, kMirror = 0x140;
template <int kCtrl>
__device__ __forceinline__ float dpp(float x) {
  return __builtin_bit_cast(float, dpp<kCtrl>(__builtin_bit_cast(uint32_t, x)));
}

__device__ __forceinline__ float lane_value(float x, int lane) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), lane));
}

// The sum over 16 neighbouring lanes or over the wave's 64, in a fixed order,
// the same in every lane.
__device__ __forceinline__ float sum16(float x) {
  x += dpp<kXor1>(x);
  x += dpp<kXor2>(x);
  x += dpp<kHalfMirror>(x);
  return x + dpp<kMirror>(x);
}
__device__ __forceinline__ float wave_sum(float x) {
  x = sum16(x);
  return (lane_value(x, 0) + lane_value(x, 16)) + (lane_value(x, 32) + lane_value(x, 48));
}

// ---------------------------------------------------------------- 8-bit blocks
//
// 32 consecutive values of a row share one power of two 2^e, stored as the
// byte e + 127; a value is code * 2^e with a signed 8-bit code.  e is the
// least exponent with 127 * 2^e >= the block's largest magnitude, so no code
// is clipped, and a code is off by at most half a step: 2^(e-1), 1/127 of
// the block's largest magnitude.  Scaling by a power of two is exact, so
// the only rounding is that of the code.  Byte 255 marks a block that held an
// infinity or NaN: all of it reads back as NaN.

// The scale byte of a block from the bits of its largest magnitude (fp32
// bits without the sign: they order like the values, infinities and NaN
// last).  Adding 0x1ffff carries into the exponent exactly when the
// significand is over 127/64.  `top` bounds the byte so that 127 * 2^e stays
// finite in the type that was packed (the codes of a block above it clip at
// 127, off by less than the half step of the next exponent).
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax, uint32_t top) {
  if (amax >= 0x7f800000u) return 255u;
  const int b = (int)((amax + 0x1ffffu) >> 23) - 6;
  return b < 0 ? 0u : (uint32_t)b < top ? (uint32_t)b : top;
}
// 2^(byte - 127); NaN for 255.
__device__ __forceinline__ float scale_value(uint32_t byte) {
  const uint32_t bits = byte == 0u ? 0x00400000u : byte == 255u ? 0x7fc00000u : byte << 23;
  return __builtin_bit_cast(float, bits);
}
// 2^(127 - byte): what a block's values are multiplied by; 0 for 255, whose
// codes are all zero (see code_of).
__device__ __forceinline__ float scale_inverse(uint32_t byte) {
  return byte == 255u ? 0.f : __builtin_bit_cast(float, (254u - byte) << 23);
}
// x * inv rounded to nearest even and clipped to [-127, 127], as the low byte
// of the result: adding 1.5 * 2^23 leaves the rounded integer in the low
// bits.  NaN (an infinity or NaN times 0) gives 0 through the integer clip.
__device__ __forceinline__ uint32_t code_of(float x, float inv) {
  const float magic = 12582912.f;
  const float f = __builtin_fmaf(x, inv, magic);
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_fmed3f(f, magic - 127.f, magic + 127.f)) & 0xffu;
}

// The four codes of a word, widened.
__device__ __forceinline__ void widen_codes(uint32_t w, float (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = (float)(int8_t)(w >> (8 * i));
}

// N codes (a multiple of 4) at p, the first `valid` of them inside the row.
template <int N>
__device__ __forceinline__ void load_codes(const int8_t* p, int valid, uint32_t (&w)[N / 4]) {
  if (valid >= N) {
    if constexpr (N == 4) {
      w[0] = load_at<uint32_t, 1>(p);
    } else {
      static_assert(N == 8, "4 or 8 codes");
      const v2u r = load_at<v2u, 1>(p);
      w[0] = r.x;
      w[1] = r.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) w[i] = 0u;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < valid) w[i / 4] |= (uint32_t)(uint8_t)p[i] << (8 * (i & 3));
  }
}
template <int N>
__device__ __forceinline__ void store_codes(int8_t* p, const uint32_t (&w)[N / 4], int valid) {
  if (valid >= N) {
    if constexpr (N == 4)
      store_at<uint32_t, 1>(p, w[0]);
    else
      store_at<v2u, 1>(p, v2u{w[0], w[1]});
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < valid) p[i] = (int8_t)(w[i / 4] >> (8 * (i & 3)));
  }
}

// Packs the N = kVec values of each lane, the lanes of a block being 32 / N
// neighbours (values outside the row are zeros); stores the codes, and the
// block's first lane its scale byte.
template <int N>
__device__ __forceinline__ void pack_vec(const float (&v)[N], int valid, uint32_t top, int lane, int8_t* codes,
                                         uint8_t* scale) {
  uint32_t amax = 0u;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t a = __builtin_bit_cast(uint32_t, v[i]) & 0x7fffffffu;
    amax = a > amax ? a : amax;
  }
  uint32_t o = dpp<kXor1>(amax);
  amax = o > amax ? o : amax;
  o = dpp<kXor2>(amax);
  amax = o > amax ? o : amax;
  if constexpr (N == 4) {  // 8 lanes to a block: the other four
    o = dpp<kHalfMirror>(amax);
    amax = o > amax ? o : amax;
  }
  const uint32_t byte = scale_byte(amax, top);
  const float inv = scale_inverse(byte);
  uint32_t w[N / 4];
#pragma unroll
  for (int j = 0; j < N / 4; ++j) {
    w[j] = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[j] |= code_of(v[4 * j + i], inv) << (8 * i);
  }
  if (byte == 255u) {
#pragma unroll
    for (int j = 0; j < N / 4; ++j) w[j] = 0u;
  }
  if (valid > 0) {
    store_codes<N>(codes, w, valid);
    if ((lane & (32 / N - 1)) == 0) *scale = (uint8_t)byte;
  }
}

}  // namespace elem
}  // namespace adasum
