// relative_bias.hip - a learned bias of attention scores by the distance
// between query and key, and its table's gradient.
//
//   forward    out[n][h][i][j] = scores[n][h][i][j] + table[bucket(d)][h],
//              d = j - i - offset
//   gradient   dtable[b][h] = sum over n, i, j with bucket(d) = b of
//              dscores[n][h][i][j]
//
// A head's bias depends on d alone.  The forward pass puts the line of all d of
// its tile in LDS once, and every row of the tile and of the batch is a piece of
// it.  The gradient first sums along the diagonals of the score matrices: a lane
// owns a vector of neighbouring diagonals and walks down the rows, its column
// moving on by one each row, so the sums stay in registers (loads need no
// alignment on gfx950, and the lanes of a wave read neighbouring vectors).
// Buckets are runs of diagonals, summed by a second kernel.  Both are bound by
// HBM: 32 x 16 x 512 x 512 bf16, forward 99 us (537 MB, 5.4 TB/s), gradient 63 + 7
// us (268 MB, 4.3 TB/s).  16 lanes a row instead of 64 in the gradient: 103 us
// against 71 in all; rows of a tile in units of 64: 3 x 12 x 127 x 131 fp32 12 us
// against 7 with 16 (an eighth of the workgroups).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <vector>

#include "elem.h"
#include "layer_ops.h"

namespace adasum {
namespace {

using namespace elem;

constexpr int kTileRows = 16, kTileCols = 1024;  // of the forward pass
constexpr int kPieces = 4;                       // pieces a lane has in flight
constexpr int kGradUnit = 16, kGradAhead = 8;   // rows of a unit, rows in flight
// A bucket of more sums of diagonals than this is joined in pieces, by two
// launches: 64 x 16 x 1 x 4096 bf16 takes 18 us a call (one workgroup a bucket 42),
// 1 x 16 x 1 x 2^20 122 (6263).  Below it the second launch costs more
// than it saves: 32 x 16 x 512 x 512, 12288 sums, 70 us against 74.
constexpr int64_t kJoinValues = 16384, kPieceValues = 4096;

// The bucket of distance n on its side: the last border at or below n.
__device__ __forceinline__ int bucket_of(const BiasBuckets& k, uint32_t n) {
  int lo = 0, hi = k.side;  // border[lo] <= n < border[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (k.border[mid] <= n)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// The table's row for distance d = key - query.
__device__ __forceinline__ int bucket_at(const BiasBuckets& k, int64_t d) {
  const int64_t n = k.both ? (d < 0 ? -d : d) : (d < 0 ? -d : 0);
  const int b = bucket_of(k, (uint32_t)min<int64_t>(n, 0x7fffffff));
  return k.both && d > 0 ? b + k.side : b;
}

// A step of nine words for eight values keeps the lanes' pieces of the line in
// different banks.
__device__ __forceinline__ int line_at(int k) { return k + (k >> 3); }

template <typename T, bool ADD>
__global__ __launch_bounds__(256) void bias_kernel(BiasArgs a, BiasLayout l) {
  constexpr int VEC = Type<T>::kVec;
  __shared__ float line[(kTileRows + kTileCols) * 9 / 8 + 1];
  uint32_t block = blockIdx.x;
  const int64_t col_tile = block % l.col_tiles;
  block /= l.col_tiles;
  const int64_t row_tile = block % l.row_tiles;
  block /= l.row_tiles;
  const int64_t head = block % a.heads, part = block / a.heads;
  const int64_t i0 = row_tile * kTileRows, j0 = col_tile * kTileCols;
  const int rows = (int)min<int64_t>(kTileRows, a.queries - i0), cols = (int)min<int64_t>(kTileCols, a.keys - j0);
  // line[k] is the bias at key - query = first + k
  const int64_t first = j0 - (i0 + rows - 1) - a.offset, last = first + rows + cols - 2;
  // all of them in a side's last bucket, as most are of long rows: no search
  const int64_t far = a.buckets.far;
  const bool before = last <= -far, behind = a.buckets.both && first >= far;
  const int all = before ? a.buckets.side - 1 : behind ? 2 * a.buckets.side - 1 : -1;
  for (int k = threadIdx.x; k < rows + cols - 1; k += 256) {
    const int b = all >= 0 ? all : bucket_at(a.buckets, first + k);
    line[line_at(k)] = load_any(a.table, a.table_dtype, (int64_t)b * a.table_stride + head);
  }
  __syncthreads();
  const int64_t n_begin = part * l.part_batch, n_end = min(a.batch, n_begin + l.part_batch);
  const uint32_t per_row = (uint32_t)(cols + VEC - 1) / VEC, per_batch = per_row * rows;
  // below 2^30: bias_layout leaves a workgroup 1 / 2048 of 2^40 elements at most
  const uint32_t total = (uint32_t)(n_end - n_begin) * per_batch;
  const T* scores = static_cast<const T*>(a.scores);
  T* out = static_cast<T*>(a.out);
  for (uint32_t p0 = 0; p0 < total; p0 += 256 * kPieces) {
    v4u raw[kPieces];
    int64_t row[kPieces];
    int col[kPieces], at[kPieces], valid[kPieces];
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      const uint32_t p = p0 + u * 256 + threadIdx.x, n = p / per_batch, q = p - n * per_batch, r = q / per_row;
      col[u] = (int)(q - r * per_row) * VEC;
      row[u] = ((n_begin + n) * a.heads + head) * a.queries + i0 + r;
      at[u] = rows - 1 - (int)r + col[u];
      valid[u] = p < total ? cols - col[u] : 0;
      if constexpr (ADD) raw[u] = load_raw(scores + row[u] * a.scores_stride + j0 + col[u], valid[u]);
    }
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      float v[VEC];
      if constexpr (ADD) widen<T>(raw[u], v);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float b = e < valid[u] ? line[line_at(at[u] + e)] : 0.f;
        v[e] = ADD ? v[e] + b : b;
      }
      store_vec(out + row[u] * a.out_stride + j0 + col[u], v, valid[u]);
    }
  }
}

// Sums along diagonals.  Diagonal D = j - i + queries - 1; LPD lanes own VEC
// diagonals each, and the workgroup's groups of lanes take units of kGradUnit
// rows of a sequence in turn.
template <typename T, int LPD>
__global__ __launch_bounds__(256) void bias_grad_kernel(BiasGradArgs a, BiasGradLayout l) {
  constexpr int VEC = Type<T>::kVec, GROUPS = 256 / LPD;
  const int lane = threadIdx.x & (LPD - 1), group = threadIdx.x / LPD;
  uint32_t block = blockIdx.x;
  const uint32_t tile = block % l.tiles;
  block /= l.tiles;
  const uint32_t head = block % (uint32_t)a.heads, split = block / (uint32_t)a.heads;
  const int queries = (int)a.queries, keys = (int)a.keys;  // together at most 2^30
  const int tile_shift = (int)(tile * LPD * VEC) - (queries - 1);
  const int shift = tile_shift + lane * VEC;  // column of the lane's first diagonal in row 0
  const T* base = static_cast<const T*>(a.dscores);
  const int64_t all_rows = a.batch * a.heads * queries;
  const uint32_t row_units = (uint32_t)(queries + kGradUnit - 1) / kGradUnit, units = (uint32_t)a.batch * row_units;
  // A vector that reaches over its row's ends reads its neighbours in memory,
  // whose values are dropped.  There are none before the first row and behind
  // the last, which are taken value by value, like rows narrower than a vector.
  const bool narrow = keys < VEC;
  float acc[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) acc[e] = 0.f;
  for (uint32_t unit = split * GROUPS + group; unit < units; unit += (uint32_t)l.splits * GROUPS) {
    const uint32_t n = unit / row_units;
    const int begin = (int)(unit - n * row_units) * kGradUnit, end = min(queries, begin + kGradUnit);
    // rows in which any of the tile's diagonals has a column
    int lo = max(begin, -(tile_shift + LPD * VEC - 1)), hi = min(end, keys - tile_shift);
    const int64_t row0 = ((int64_t)n * a.heads + head) * queries;
    auto one_row = [&](int i) {
      const T* p = base + (row0 + i) * a.stride;
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if ((uint32_t)(shift + i + e) < (uint32_t)keys) acc[e] += (float)p[shift + i + e];
    };
    if (lo >= hi) continue;
    if (narrow) {
      for (int i = lo; i < hi; ++i) one_row(i);
      continue;
    }
    if (row0 + lo == 0) one_row(lo++);
    if (lo < hi && row0 + hi == all_rows) one_row(--hi);
    for (int i0 = lo; i0 < hi; i0 += kGradAhead) {
      v4u raw[kGradAhead];
      const T* p = base + (row0 + i0) * a.stride;
#pragma unroll
      for (int u = 0; u < kGradAhead; ++u) {
        // no branch: all loads are on their way at once.  A lane without a
        // column in this row reads the row's first vector.
        const int j = shift + i0 + u;
        const int64_t row = i0 + u < hi ? u * a.stride : 0;
        const bool inside = (uint32_t)(j + VEC - 1) < (uint32_t)(keys + VEC - 1) && i0 + u < hi;
        raw[u] = load_at<v4u, sizeof(T)>(p + row + (inside ? j : 0));
      }
#pragma unroll
      for (int u = 0; u < kGradAhead; ++u) {
        const int j = shift + i0 + u;
        float v[VEC];
        widen<T>(raw[u], v);
        if (!((uint32_t)j <= (uint32_t)(keys - VEC) && i0 + u < hi)) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) v[e] = (uint32_t)(j + e) < (uint32_t)keys && i0 + u < hi ? v[e] : 0.f;
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[e] += v[e];
      }
    }
  }
  // the groups' sums, added in their order in fp64 and rounded once
  __shared__ float part[256 * VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) part[e * 256 + threadIdx.x] = acc[e];
  __syncthreads();
  if (group == 0) {
    const int diagonals = queries + keys - 1, d0 = (int)(tile * LPD + lane) * VEC;
    float* out = a.partials + ((int64_t)split * a.heads + head) * diagonals;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      double s = 0.0;
#pragma unroll
      for (int g = 0; g < GROUPS; ++g) s += (double)part[e * 256 + g * LPD + lane];
      if (d0 + e < diagonals) out[d0 + e] = (float)s;
    }
  }
}

// The diagonals of bucket b, first to last (none: first > last).
__host__ __device__ inline void diagonals_of(const BiasGradArgs& a, int b, int64_t* first, int64_t* last) {
  const BiasBuckets& k = a.buckets;
  const bool ahead = k.both && b >= k.side;  // keys behind the query
  const int s = ahead ? b - k.side : b;
  const int64_t beyond = int64_t(1) << 40;
  const int64_t near = k.border[s], far = s + 1 < k.side ? (int64_t)k.border[s + 1] : beyond;  // near <= n < far
  // as key - query, both ends included
  int64_t lo, hi;
  if (ahead) {
    lo = near > 1 ? near : 1;
    hi = far - 1;
  } else {
    lo = -(far - 1);
    hi = !k.both && s == 0 ? beyond : -near;
  }
  const int64_t zero = a.queries - 1 + a.offset, end = a.queries + a.keys - 2;
  *first = lo + zero > 0 ? lo + zero : 0;
  *last = hi + zero < end ? hi + zero : end;
}

// A lane's share of a head's diagonals lo to hi of every split: the workgroup
// takes 256 / G diagonals of G splits at a time, a lane eight of these at once,
// of V splits G apart.  What lies past the last is read at the last.
template <int G, int V>
__device__ __forceinline__ double lane_sum(const float* from, int64_t pitch, int splits, int64_t lo, int64_t hi) {
  constexpr int U = 8 / V, WIDTH = 256 / G;
  double t = 0.0;
  for (int64_t d = lo + threadIdx.x % WIDTH; d <= hi; d += U * WIDTH)
    for (int first = threadIdx.x / WIDTH; first < splits; first += G * V) {
      float v[U][V];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int w = 0; w < V; ++w) v[u][w] = from[min(first + G * w, splits - 1) * pitch + min(d + WIDTH * u, hi)];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int w = 0; w < V; ++w)
          t += d + WIDTH * u <= hi && first + G * w < splits ? (double)v[u][w] : 0.0;
    }
  return t;
}

// The sum in fp64 by a workgroup in a fixed order; the result in lane 0.
__device__ __forceinline__ double sum_diagonals(const BiasGradArgs& a, int splits, int64_t head, int64_t lo,
                                                int64_t hi) {
  __shared__ double sums[256];
  const int64_t diagonals = a.queries + a.keys - 1, pitch = a.heads * diagonals;
  const float* from = a.partials + head * diagonals;
  sums[threadIdx.x] = splits < 4    ? lane_sum<1, 1>(from, pitch, splits, lo, hi)
                      : splits <= 8   ? lane_sum<4, 2>(from, pitch, splits, lo, hi)
                      : splits <= 16  ? lane_sum<4, 4>(from, pitch, splits, lo, hi)
                                      : lane_sum<4, 8>(from, pitch, splits, lo, hi);
  __syncthreads();
  for (int w = 128; w > 0; w /= 2) {
    if ((int)threadIdx.x < w) sums[threadIdx.x] += sums[threadIdx.x + w];
    __syncthreads();
  }
  return sums[0];
}

__device__ __forceinline__ void store_bucket(const BiasGradArgs& a, int64_t b, int64_t head, double sum) {
  const int64_t i = b * a.heads + head;
  store_any(a.dtable, a.grad_dtype, i, a.accumulate ? sum + (double)load_any(a.dtable, a.grad_dtype, i) : sum);
}

// dtable[b][h], a workgroup each.
__global__ __launch_bounds__(256) void bias_join_kernel(BiasGradArgs a, int splits) {
  const int64_t head = blockIdx.x % (uint32_t)a.heads;
  const int b = blockIdx.x / (uint32_t)a.heads;
  int64_t lo, hi;
  diagonals_of(a, b, &lo, &hi);
  const double sum = sum_diagonals(a, splits, head, lo, hi);
  if (threadIdx.x == 0) store_bucket(a, b, head, sum);
}

// The first piece of every bucket, and behind the last bucket how many there are.
struct Pieces {
  uint32_t first[kMaxBuckets + 1];
};

// A piece's sum, a workgroup each.
__global__ __launch_bounds__(256) void bias_piece_kernel(BiasGradArgs a, Pieces k, int splits, int64_t length,
                                                         double* out) {
  __shared__ int which;
  const int64_t head = blockIdx.x % (uint32_t)a.heads;
  const uint32_t piece = blockIdx.x / (uint32_t)a.heads;
  const int t = threadIdx.x;
  if (t < a.buckets_total && k.first[t] <= piece && piece < k.first[t + 1]) which = t;
  __syncthreads();
  const int b = which;
  int64_t lo, hi;
  diagonals_of(a, b, &lo, &hi);
  lo += (piece - k.first[b]) * length;
  const double sum = sum_diagonals(a, splits, head, lo, min(hi, lo + length - 1));
  if (t == 0) out[(int64_t)piece * a.heads + head] = sum;
}

// dtable[b][h] from its pieces' sums, a wave each.
__global__ __launch_bounds__(256) void bias_pieces_kernel(BiasGradArgs a, Pieces k, const double* sums) {
  const int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (i >= a.buckets_total * a.heads) return;
  const int64_t b = i / a.heads, head = i - b * a.heads;
  const uint32_t end = k.first[b + 1];
  double t = 0.0;
  for (uint32_t p = k.first[b] + (threadIdx.x & 63); p < end; p += 64) t += sums[(int64_t)p * a.heads + head];
  t = wave_sum(t);
  if ((threadIdx.x & 63) == 0) store_bucket(a, b, head, t);
}

// Whole numbers of any size, for borders that are powers.
typedef std::vector<uint32_t> Whole;
void times(Whole* w, uint32_t f) {
  uint64_t carry = 0;
  for (uint32_t& x : *w) {
    carry += (uint64_t)x * f;
    x = (uint32_t)carry;
    carry >>= 32;
  }
  if (carry) w->push_back((uint32_t)carry);
}
Whole product(uint32_t x, int times_x, uint32_t y, int times_y) {
  Whole w{1u};
  for (int i = 0; i < times_x; ++i) times(&w, x);
  for (int i = 0; i < times_y; ++i) times(&w, y);
  return w;
}
bool at_least(const Whole& a, const Whole& b) {
  if (a.size() != b.size()) return a.size() > b.size();
  for (size_t i = a.size(); i-- > 0;)
    if (a[i] != b[i]) return a[i] > b[i];
  return true;
}

}  // namespace

// border[k] is the least n with (n / e)^(m - e) >= (reach / e)^(k - e), decided
// in whole numbers where the quotient of logarithms cannot.
BiasBuckets bias_buckets(int buckets, int64_t reach, bool both) {
  BiasBuckets t{};
  t.both = both;
  t.side = both ? buckets / 2 : buckets;
  const int m = t.side, e = m / 2;
  for (int k = 0; k < m; ++k) {
    if (k <= e) {
      t.border[k] = (uint32_t)k;
      continue;
    }
    const double x = e * std::pow((double)reach / e, (double)(k - e) / (m - e)), near = std::nearbyint(x);
    uint32_t n = (uint32_t)std::ceil(x);
    if (std::fabs(x - near) <= 1e-9 * x) {
      n = (uint32_t)near;
      if (!at_least(product(n, m - e, (uint32_t)e, k - e), product((uint32_t)reach, k - e, (uint32_t)e, m - e))) ++n;
    }
    t.border[k] = n;
  }
  t.far = t.border[m - 1];
  return t;
}

BiasLayout bias_layout(int64_t batch, int64_t heads, int64_t queries, int64_t keys) {
  BiasLayout l{};
  l.row_tiles = ceil_div(queries, kTileRows);
  l.col_tiles = ceil_div(keys, kTileCols);
  const int64_t tiles = l.row_tiles * l.col_tiles * heads;
  // a workgroup keeps its line for as many sequences as leave 2048 workgroups
  const int64_t parts = std::min(batch, std::max<int64_t>(1, ceil_div(2048, tiles)));
  l.part_batch = ceil_div(batch, parts);
  l.blocks = tiles * ceil_div(batch, l.part_batch);
  return l;
}

hipError_t launch_bias(int dtype, const BiasArgs& a, hipStream_t st) {
  const BiasLayout l = bias_layout(a.batch, a.heads, a.queries, a.keys);
  return with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    if (a.scores)
      bias_kernel<T, true><<<(unsigned)l.blocks, 256, 0, st>>>(a, l);
    else
      bias_kernel<T, false><<<(unsigned)l.blocks, 256, 0, st>>>(a, l);
    return hipGetLastError();
  });
}

BiasGradLayout bias_grad_layout(int64_t batch, int64_t heads, int64_t queries, int64_t keys, int dtype) {
  BiasGradLayout l{};
  const int vec = dtype == 0 ? 4 : 8;
  const int64_t diagonals = queries + keys - 1;
  l.lanes = diagonals <= 32 * vec ? 16 : 64;
  l.tiles = ceil_div(diagonals, l.lanes * vec);
  const int64_t units = batch * ceil_div(queries, kGradUnit), groups = 256 / l.lanes;
  // four workgroups a CU, each group with a unit at least; and no more than 4096
  // rows in one fp32 sum
  const int64_t fill = ceil_div(4 * kCUs, l.tiles * heads), most = ceil_div(units, groups);
  l.splits = std::max<int64_t>({1, std::min(fill, most), ceil_div(units, groups * (4096 / kGradUnit))});
  l.blocks = l.splits * heads * l.tiles;
  l.bytes = (size_t)l.splits * heads * diagonals * sizeof(float);
  if (l.splits * diagonals > kJoinValues) {
    l.piece = std::max<int64_t>(64, kPieceValues / l.splits);
    l.piece_blocks = (kMaxBuckets + diagonals / l.piece) * heads;
    l.sums = (l.bytes + 7) / 8 * 8;
    l.bytes = l.sums + (size_t)l.piece_blocks * sizeof(double);
  }
  return l;
}

hipError_t launch_bias_grad(int dtype, const BiasGradArgs& a, hipStream_t st) {
  const BiasGradLayout l = bias_grad_layout(a.batch, a.heads, a.queries, a.keys, dtype);
  const hipError_t e = with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    if (l.lanes == 16)
      bias_grad_kernel<T, 16><<<(unsigned)l.blocks, 256, 0, st>>>(a, l);
    else
      bias_grad_kernel<T, 64><<<(unsigned)l.blocks, 256, 0, st>>>(a, l);
    return hipGetLastError();
  });
  if (e != hipSuccess) return e;
  Pieces k{};
  int64_t longest = 0;
  for (int b = 0; b < a.buckets_total; ++b) {
    int64_t lo, hi;
    diagonals_of(a, b, &lo, &hi);
    const int64_t length = std::max<int64_t>(hi - lo + 1, 0);
    longest = std::max(longest, length);
    if (l.piece > 0) k.first[b + 1] = k.first[b] + (uint32_t)ceil_div(length, l.piece);
  }
  if (longest * l.splits <= kJoinValues) {
    bias_join_kernel<<<(unsigned)(a.buckets_total * a.heads), 256, 0, st>>>(a, (int)l.splits);
  } else {
    double* sums = reinterpret_cast<double*>(reinterpret_cast<char*>(a.partials) + l.sums);
    const unsigned blocks = (unsigned)(k.first[a.buckets_total] * a.heads);
    bias_piece_kernel<<<blocks, 256, 0, st>>>(a, k, (int)l.splits, l.piece, sums);
    bias_pieces_kernel<<<(unsigned)ceil_div(a.buckets_total * a.heads, 4), 256, 0, st>>>(a, k, sums);
  }
  return hipGetLastError();
}

}  // namespace adasum
