// checkpoint.hip - activations kept in 8 bits for the backward pass, and read
// back.  The format (32 values of a row share a power of two) and its
// rounding are described in elem.h.
//
// Both kernels move each byte once and are bound by HBM.  A lane's piece is
// 16 bytes of the wider side; the pieces of a row are padded to whole blocks,
// so that a block's lanes are always neighbours, and pieces are dealt to the
// lanes across row ends, so that narrow rows fill the waves too.  16384 x 4096
// bf16, mostly resident in the memory-side cache: packing 41 us, reading back
// 31 (5.0 and 6.6 TB/s; a copy of 2 GB reaches 4.8, one of 128 MB 8.6).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "elem.h"
#include "layer_ops.h"

namespace adasum {
namespace {

using namespace elem;

constexpr int kPieces = 4;  // pieces a lane has in flight

template <typename T>
__global__ __launch_bounds__(256) void pack_kernel(PackArgs a, int nblk, uint32_t top) {
  constexpr int VEC = Type<T>::kVec;
  constexpr int PER = kScaleBlock / VEC;  // pieces of a block
  const uint32_t per_row = (uint32_t)nblk * PER;
  const int64_t total = a.rows * per_row;
  for (int64_t first = (int64_t)blockIdx.x * 256 * kPieces; first < total;
       first += (int64_t)gridDim.x * 256 * kPieces) {
    const int64_t row0 = first / per_row;
    const uint32_t p0 = (uint32_t)(first - row0 * per_row);
    v4u raw[kPieces];
    int64_t row[kPieces];
    int col[kPieces], valid[kPieces];
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      const uint32_t k = p0 + u * 256 + threadIdx.x;
      const uint32_t q = k / per_row;
      row[u] = row0 + q;
      col[u] = (int)(k - q * per_row) * VEC;
      valid[u] = row[u] < a.rows ? a.hidden - col[u] : 0;
      raw[u] = load_raw(static_cast<const T*>(a.x) + row[u] * a.stride + col[u], valid[u]);
    }
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      float v[VEC];
      widen<T>(raw[u], v);
      pack_vec<VEC>(v, valid[u], top, (int)threadIdx.x, a.codes + row[u] * a.hidden + col[u],
                    a.scales + row[u] * nblk + col[u] / kScaleBlock);
    }
  }
}

template <typename T>
__global__ __launch_bounds__(256) void unpack_kernel(UnpackArgs a, int nblk) {
  constexpr int VEC = Type<T>::kVec;
  const uint32_t per_row = ((uint32_t)a.hidden + VEC - 1) / VEC;  // a.hidden may be 2^31 - 1
  const int64_t total = a.rows * per_row;
  for (int64_t first = (int64_t)blockIdx.x * 256 * kPieces; first < total;
       first += (int64_t)gridDim.x * 256 * kPieces) {
    const int64_t row0 = first / per_row;
    const uint32_t p0 = (uint32_t)(first - row0 * per_row);
    uint32_t w[kPieces][VEC / 4], byte[kPieces];
    int64_t row[kPieces];
    int col[kPieces], valid[kPieces];
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      const uint32_t k = p0 + u * 256 + threadIdx.x;
      const uint32_t q = k / per_row;
      row[u] = row0 + q;
      col[u] = (int)(k - q * per_row) * VEC;
      valid[u] = row[u] < a.rows ? a.hidden - col[u] : 0;
      load_codes<VEC>(a.codes + row[u] * a.hidden + col[u], valid[u], w[u]);
      byte[u] = valid[u] > 0 ? a.scales[row[u] * nblk + col[u] / kScaleBlock] : 127u;
    }
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      const float s = scale_value(byte[u]);
      float v[VEC];
#pragma unroll
      for (int j = 0; j < VEC / 4; ++j) {
        float t[4];
        widen_codes(w[u][j], t);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[4 * j + i] = t[i] * s;
      }
      store_vec(static_cast<T*>(a.out) + row[u] * a.stride + col[u], v, valid[u]);
    }
  }
}

unsigned piece_blocks(int64_t pieces) {
  return (unsigned)std::min<int64_t>(ceil_div(pieces, 256 * kPieces), int64_t(1) << 20);
}

}  // namespace

hipError_t launch_pack(int dtype, const PackArgs& a, hipStream_t st) {
  const int nblk = (int)ceil_div(a.hidden, kScaleBlock);
  const int64_t blocks32 = a.rows * nblk;
  // the largest exponent whose 127 steps are finite: 2^121 in fp32 and bf16,
  // 2^9 in fp16
  if (dtype == 0)
    pack_kernel<float><<<piece_blocks(blocks32 * 8), 256, 0, st>>>(a, nblk, 248u);
  else if (dtype == 1)
    pack_kernel<_Float16><<<piece_blocks(blocks32 * 4), 256, 0, st>>>(a, nblk, 136u);
  else
    pack_kernel<__bf16><<<piece_blocks(blocks32 * 4), 256, 0, st>>>(a, nblk, 248u);
  return hipGetLastError();
}

hipError_t launch_unpack(int dtype, const UnpackArgs& a, hipStream_t st) {
  const int nblk = (int)ceil_div(a.hidden, kScaleBlock);
  if (dtype == 0)
    unpack_kernel<float><<<piece_blocks(a.rows * ceil_div(a.hidden, 4)), 256, 0, st>>>(a, nblk);
  else if (dtype == 1)
    unpack_kernel<_Float16><<<piece_blocks(a.rows * ceil_div(a.hidden, 8)), 256, 0, st>>>(a, nblk);
  else
    unpack_kernel<__bf16><<<piece_blocks(a.rows * ceil_div(a.hidden, 8)), 256, 0, st>>>(a, nblk);
  return hipGetLastError();
}

}  // namespace adasum
