// embedding.hip - rows of a table by token, and the table's gradient.
//
//   forward   y[i] = scale * table[t_i]
//   backward  grad[t] = scale * (sum of dy[i] over the rows i with t_i = t),
//             every row of grad written (or, accumulating, the named ones
//             added to)
//
// A token outside [0, vocab) is no token: zeros forward, nothing backward.
//
// The gradient is a sum by token without atomics, in three launches:
//   group   lists the rows of every token, in row order, the tokens dealt to
//           the workgroups by their low bits; also clears the rows of grad
//           that no token names
//   sum     walks the grouped list in pieces of equal length, so that a
//           frequent token is summed by many workgroups; a token whose rows
//           lie inside one piece is written at once, the sums of the others
//           are left for
//   join    adds them in the order of the list, in fp64.
// Every sum has a fixed order, so the result is bitwise reproducible.
//
// Measured.  Lookup of 65536 rows of 1024 in bf16: 39 us, bound by HBM (134 MB
// written; 12500 different rows of the table, 26 MB, read 2.4 times over by
// XCDs with an L2 each: 5.0 TB/s).  Gradient of the same 65536 rows, a
// tenth without token, into 30522 x 1024 fp32: group 27 us, sum 48 (3.8 TB/s of
// rows in no order), join 6; two tables' worth of bytes, 246 MB, would take 51
// at the rate of a large copy.  Grouping is bound by its scan, which every
// workgroup makes of all tokens, and by the workgroup of the most frequent
// token.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "elem.h"
#include "layer_ops.h"

namespace adasum {
namespace {

using namespace elem;

// ---------------------------------------------------------------- forward

constexpr int kLookups = 4;  // pieces of 16 bytes of the table a lane has in flight

template <typename T, typename O, typename TOK>
__global__ __launch_bounds__(256) void embedding_kernel(EmbeddingArgs a) {
  constexpr int VEC = Type<T>::kVec;
  constexpr int N = VEC > Type<O>::kVec ? VEC : Type<O>::kVec;  // values per piece
  const uint32_t per_row = (uint32_t)((a.hidden + N - 1) / N);
  const int64_t total = a.n * per_row;
  const TOK* tokens = static_cast<const TOK*>(a.tokens);
  for (int64_t first = (int64_t)blockIdx.x * 256 * kLookups; first < total;
       first += (int64_t)gridDim.x * 256 * kLookups) {
    const int64_t row0 = first / per_row;
    const uint32_t p0 = (uint32_t)(first - row0 * per_row);
    int64_t row[kLookups], tok[kLookups];
    int col[kLookups], valid[kLookups];
#pragma unroll
    for (int u = 0; u < kLookups; ++u) {
      const uint32_t k = p0 + u * 256 + threadIdx.x;
      const uint32_t q = k / per_row;
      row[u] = row0 + q;
      col[u] = (int)(k - q * per_row) * N;
      valid[u] = row[u] < a.n ? a.hidden - col[u] : 0;
      tok[u] = valid[u] > 0 ? (int64_t)tokens[row[u]] : -1;
    }
    float v[kLookups][N];
#pragma unroll
    for (int u = 0; u < kLookups; ++u) {
      const bool there = tok[u] >= 0 && tok[u] < a.vocab;
      load_row<T, N>(static_cast<const T*>(a.table) + (there ? tok[u] : 0) * a.table_stride + col[u],
                     there ? valid[u] : 0, v[u]);
    }
#pragma unroll
    for (int u = 0; u < kLookups; ++u) {
      const bool there = tok[u] >= 0 && tok[u] < a.vocab;
#pragma unroll
      for (int i = 0; i < N; ++i) v[u][i] = there ? v[u][i] * a.scale : 0.f;
      store_row<O, N>(static_cast<O*>(a.out) + row[u] * a.out_stride + col[u], v[u], valid[u]);
    }
  }
}

// ---------------------------------------------------------------- group

constexpr int kGroupWaves = 16;
constexpr int kGroupKeys = 512;  // most tokens a workgroup of the grouping kernel owns (32 KB of counts)
constexpr int kNotes = 512;      // owned rows that a wave of the grouping kernel notes
constexpr int kCrowd = 64;       // owned rows of a step above which the first one's token is counted at once
constexpr int kGroupBatch = 4;   // steps of 256 tokens whose loads a wave has in flight

// Four consecutive places of the list from i on: for each the token's low
// bits (those in `mask`), or mask + 1 where it is no token or past n; and the
// token itself.
template <typename TOK>
__device__ __forceinline__ void load_tokens(const TOK* tokens, int64_t i, int64_t n, uint32_t vocab, uint32_t mask,
                                            uint32_t (&low)[4], uint32_t (&t)[4]) {
  uint32_t high[4] = {0u, 0u, 0u, 0u};  // of a token of 64 bits
  if (i + 4 <= n) {
    if constexpr (sizeof(TOK) == 4) {
      const v4u r = load_at<v4u, 4>(tokens + i);
      t[0] = r.x; t[1] = r.y; t[2] = r.z; t[3] = r.w;
    } else {
      const v4u r = load_at<v4u, 8>(tokens + i), s = load_at<v4u, 8>(tokens + i + 2);
      t[0] = r.x; t[1] = r.z; t[2] = s.x; t[3] = s.z;
      high[0] = r.y; high[1] = r.w; high[2] = s.y; high[3] = s.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) t[j] = ~0u;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i + j < n) {
        const int64_t x = (int64_t)tokens[i + j];
        t[j] = x >= 0 && x < (int64_t)vocab ? (uint32_t)x : ~0u;
      }
  }
  // a negative token has a sign bit in its low or its high word, and vocab is
  // far below 2^31
#pragma unroll
  for (int j = 0; j < 4; ++j) low[j] = t[j] < vocab && high[j] == 0u ? t[j] & mask : mask + 1u;
}

struct GroupArgs {
  const void* tokens;
  int64_t n, vocab;
  int shift;          // log2 of the number of workgroups
  int keys;           // tokens per workgroup
  int32_t* rows;      // grouped: row index
  int32_t* grouped;   // grouped: token
  int32_t* count;     // [1]: how many rows have a token
  char* grad;         // cleared where no token names the row; NULL: nothing is cleared
  int64_t row_bytes;
};

__device__ __forceinline__ int lanes_below(uint64_t mask) {
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
}

// Workgroup g owns the tokens t with t mod G = g (dealing them by their low
// bits spreads the frequent ones, which many vocabularies put first).  Its 16
// waves each scan a sixteenth of the list.  The scan counts, per wave, the
// rows of every owned token, and the rows of the tokens of lower workgroups:
// their number is where this workgroup's part of the grouped list begins, so
// the workgroups need nothing from each other.  It also notes the owned rows
// it meets, in order, in LDS.  A wave's position for a token starts where the
// counts of the waves before it end, so the rows of a token stay in order
// when the notes are written out.  A wave that met more rows than its notes
// hold (a token of many rows) scans its part again instead.
template <typename TOK>
__global__ __launch_bounds__(1024) void group_kernel(GroupArgs a) {
  extern __shared__ int32_t counts[];  // [16][keys]: counts, then positions
  __shared__ int32_t lower[kGroupWaves], scan[kGroupWaves];
  __shared__ int32_t totals[kGroupKeys];
  __shared__ uint32_t note_row[kGroupWaves][kNotes];
  __shared__ uint16_t note_key[kGroupWaves][kNotes];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const uint32_t G = 1u << a.shift, g = blockIdx.x;
  const int keys = a.keys;
  const TOK* tokens = static_cast<const TOK*>(a.tokens);
  for (int i = tid; i < kGroupWaves * keys; i += 1024) counts[i] = 0;
  __syncthreads();

  const int64_t steps = (a.n + 1024 * 4 - 1) / (1024 * 4);  // of 256 tokens, per wave
  const int64_t begin = wave * steps * 256;
  const uint32_t mask = G - 1, vocab = (uint32_t)a.vocab;
  int32_t* mine = counts + wave * keys;
  auto fetch = [&](int64_t s, uint32_t (&low)[kGroupBatch][4], uint32_t (&t)[kGroupBatch][4])
                   __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < kGroupBatch; ++u)
      load_tokens(tokens, s + u < steps ? begin + (s + u) * 256 + lane * 4 : a.n, a.n, vocab, mask, low[u], t[u]);
  };

  int less = 0, noted = 0;  // of the wave
  for (int64_t s = 0; s < steps; s += kGroupBatch) {
    uint32_t low[kGroupBatch][4], t[kGroupBatch][4];
    fetch(s, low, t);
#pragma unroll
    for (int u = 0; u < kGroupBatch; ++u) {
      uint64_t met[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        less += __popcll(__ballot(low[u][j] < g));
        met[j] = __ballot(low[u][j] == g);
      }
      if ((met[0] | met[1] | met[2] | met[3]) == 0) continue;
      // Where many rows are owned, most of them have one frequent token: the
      // first one's rows are counted with one addition, where LDS would make
      // them one by one.  131072 rows of one token: 183 us for this kernel
      // without, 67 with; about 45 rows a step: 76 us, and 88 if counted so
      // from eight rows on, hence the bound.
      const int owned = __popcll(met[0]) + __popcll(met[1]) + __popcll(met[2]) + __popcll(met[3]);
      if (owned > kCrowd) {
        uint32_t pick = t[u][3] >> a.shift;
#pragma unroll
        for (int j = 2; j >= 0; --j)
          if ((met[j] >> lane) & 1u) pick = t[u][j] >> a.shift;
        const uint32_t now = (uint32_t)__builtin_amdgcn_readlane(
            (int)pick, __builtin_ctzll(met[0] | met[1] | met[2] | met[3]));
        int sum = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const bool own = low[u][j] == g, same = t[u][j] >> a.shift == now;
          sum += __popcll(__ballot(own && same));
          if (own && !same) atomicAdd(&mine[t[u][j] >> a.shift], 1);
        }
        if (lane == 0) atomicAdd(&mine[now], sum);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (low[u][j] == g) atomicAdd(&mine[t[u][j] >> a.shift], 1);
      }
      // the places of this step's owned rows among the notes: by lane, then
      // by place in the lane
      int at = noted;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        at += lanes_below(met[j]);
        noted += __popcll(met[j]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (low[u][j] == g) {
          if (at < kNotes) {
            note_row[wave][at] = (uint32_t)(begin + (s + u) * 256 + lane * 4 + j);
            note_key[wave][at] = (uint16_t)(t[u][j] >> a.shift);
          }
          ++at;
        }
    }
  }
  if (lane == 0) lower[wave] = less;
  __syncthreads();

  // positions: the tokens in the order of their keys, each token's rows wave
  // by wave (at most one key a thread)
  int32_t total = 0;
  if (tid < keys) {
#pragma unroll
    for (int w = 0; w < kGroupWaves; ++w) total += counts[w * keys + tid];
    totals[tid] = total;
  }
  int32_t before = total;
  for (int o = 1; o < 64; o <<= 1) {
    const int32_t up = __shfl_up(before, o);
    if (lane >= o) before += up;
  }
  if (lane == 63) scan[wave] = before;
  __syncthreads();
  int32_t base = 0, own = 0;
  for (int w = 0; w < kGroupWaves; ++w) {
    base += lower[w];
    own += scan[w];
    if (w < wave) before += scan[w];
  }
  if (g == G - 1 && tid == 0) *a.count = base + own;
  if (tid < keys) {
    int32_t c[kGroupWaves];
#pragma unroll
    for (int w = 0; w < kGroupWaves; ++w) c[w] = counts[w * keys + tid];
    int32_t at = base + before - total;
#pragma unroll
    for (int w = 0; w < kGroupWaves; ++w) {
      counts[w * keys + tid] = at;
      at += c[w];
    }
  }
  // the gradient rows of owned tokens that the list does not hold
  if (a.grad) {
    for (int k = wave; k < keys; k += kGroupWaves) {
      const int64_t t = ((int64_t)k << a.shift) + g;
      if (t >= a.vocab || totals[k] != 0) continue;
      char* row = a.grad + t * a.row_bytes;
      const int64_t whole = a.row_bytes & ~int64_t(15);
      for (int64_t i = lane * 16; i < whole; i += 1024) store_at<v4u, 1>(row + i, v4u{0u, 0u, 0u, 0u});
      for (int64_t i = whole + lane * 2; i < a.row_bytes; i += 128) *reinterpret_cast<uint16_t*>(row + i) = 0;
    }
  }
  __syncthreads();

  // One key of a group of up to 64 x P rows after another: `want` says which
  // of a lane's P rows are in the group; their places are by lane, then by
  // place in the lane.
  auto write = [&](auto parts, uint64_t (&want)[decltype(parts)::value], const uint32_t (&key)[decltype(parts)::value],
                   const uint32_t (&row)[decltype(parts)::value]) __attribute__((always_inline)) {
    constexpr int P = decltype(parts)::value;
    for (int turn = 0; turn < 64 * P; ++turn) {
      uint64_t left = 0;
#pragma unroll
      for (int j = 0; j < P; ++j) left |= want[j];
      if (left == 0) break;
      uint32_t pick = key[P - 1];
#pragma unroll
      for (int j = P - 2; j >= 0; --j)
        if ((want[j] >> lane) & 1u) pick = key[j];
      const uint32_t now = (uint32_t)__builtin_amdgcn_readlane((int)pick, __builtin_ctzll(left));
      uint64_t eq[P];
      int below = 0, sum = 0;
#pragma unroll
      for (int j = 0; j < P; ++j) {
        eq[j] = __ballot(key[j] == now) & want[j];
        want[j] &= ~eq[j];
        below += lanes_below(eq[j]);
        sum += __popcll(eq[j]);
      }
      int pos = mine[now] + below;
      bool fours = false;  // all of a lane's rows or none: their places follow each other
      if constexpr (P == 4) fours = eq[0] == eq[1] && eq[0] == eq[2] && eq[0] == eq[3];
      if (fours) {
        if (((eq[0] >> lane) & 1u) && pos >= 0 && pos + 4 <= a.n) {
          const uint32_t token = (now << a.shift) + g;
          store_at<v4u, 4>(a.rows + pos, v4u{row[0], row[1 % P], row[2 % P], row[3 % P]});
          store_at<v4u, 4>(a.grouped + pos, v4u{token, token, token, token});
        }
      } else {
#pragma unroll
        for (int j = 0; j < P; ++j)
          if ((eq[j] >> lane) & 1u) {
            if (pos >= 0 && pos < a.n) {
              a.rows[pos] = (int32_t)row[j];
              a.grouped[pos] = (int32_t)((now << a.shift) + g);
            }
            ++pos;
          }
      }
      // the wave's own counter: every lane has read it before lane 0 moves it
      // on (the wave runs in step and its LDS operations stay in order); the
      // fences keep the compiler from holding it in a register
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      if (lane == 0) mine[now] += sum;
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    }
  };
  if (noted <= kNotes) {
    for (int i = 0; i < noted; i += 64) {
      const int at = i + lane < noted ? i + lane : i;
      const uint32_t key[1] = {note_key[wave][at]}, row[1] = {note_row[wave][at]};
      uint64_t want[1] = {__ballot(i + lane < noted)};
      write(std::integral_constant<int, 1>(), want, key, row);
    }
    return;
  }
  for (int64_t s = 0; s < steps; s += kGroupBatch) {
    uint32_t low[kGroupBatch][4], t[kGroupBatch][4];
    fetch(s, low, t);
#pragma unroll
    for (int u = 0; u < kGroupBatch; ++u) {
      uint64_t want[4];
      uint32_t key[4], row[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        want[j] = __ballot(low[u][j] == g);
        key[j] = t[u][j] >> a.shift;
        row[j] = (uint32_t)(begin + (s + u) * 256 + lane * 4 + j);
      }
      write(std::integral_constant<int, 4>(), want, key, row);
    }
  }
}

// ---------------------------------------------------------------- sum

struct RunArgs {
  const void* dy;
  int64_t n, dy_stride, vocab;
  int hidden, span, lanes_shift, tiles;
  const int32_t* rows;
  const int32_t* grouped;
  const int32_t* count;
  float scale;
  void* grad;
  int accumulate;
  float* head;  // [workgroup][tiles * 64 * VEC]: the first run's sum where it began before the workgroup
  float* tail;  // the last run's sum where it began in the workgroup and goes on after it
  int64_t pitch;
};

// The grouped list as the summing kernels read it.  The bounds are a guard, not
// part of the sum: versions of these kernels without them failed twice on the
// GPU (a silent stop, an illegal access), no reading of the sources and no run
// of them on the CPU showed why, and the list is the only thing read back that
// becomes an address.  A wrong list, from that cause or from a caller that
// changes the tokens during the call, would show as wrong sums and not as a
// fault: an index out of range counts as row 0 or token 0.  So the tests
// compare the list at every position, on the CPU and on the GPU.
__device__ __forceinline__ int64_t listed_rows(const RunArgs& a) {
  const int64_t m = *a.count;
  return m < 0 ? 0 : m < a.n ? m : a.n;
}
__device__ __forceinline__ int32_t listed_token(const RunArgs& a, int64_t p) {
  const int32_t t = a.grouped[p];
  return t >= 0 && t < a.vocab ? t : 0;
}
__device__ __forceinline__ int32_t listed_row(const RunArgs& a, int64_t p) {
  const int32_t r = a.rows[p];
  return r >= 0 && r < a.n ? r : 0;
}

constexpr int kSumThreads = 512;
constexpr int kSumSpots = 2048;  // grouped positions of a workgroup at most
constexpr int kSumBatch = 8;     // rows a lane has in flight

// A lane's N columns of a row.  The last lane of a row whose width is no
// multiple of N takes the row's last N columns instead, so that every load
// and store is a whole vector without a branch: it sums the first `shift` of
// them like the lane before it, to the same bits, and both store them.  Only
// where a stored value depends on the one it replaces (adding to the
// gradient) does it leave those out, since the lane before may be in another
// workgroup.  A width below N is loaded value by value, the last one again in
// place of those past it.
template <typename T, int N, bool NARROW>
struct Columns {
  v4u raw[N / Type<T>::kVec];
  __device__ __forceinline__ void load(const T* p, int hidden) {
    constexpr int K = Type<T>::kVec;
    if constexpr (NARROW) {
#pragma unroll
      for (int j = 0; j < N / K; ++j) {
        uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int i = 0; i < K; ++i) {
          const T x = p[min(j * K + i, hidden - 1)];
          if constexpr (sizeof(T) == 4)
            w[i] = __builtin_bit_cast(uint32_t, x);
          else
            w[i / 2] |= (uint32_t)__builtin_bit_cast(uint16_t, x) << (16 * (i & 1));
        }
        raw[j] = v4u{w[0], w[1], w[2], w[3]};
      }
    } else {
#pragma unroll
      for (int j = 0; j < N / K; ++j) raw[j] = load_at<v4u, sizeof(T)>(p + j * K);
    }
  }
  __device__ __forceinline__ void values(float (&v)[N]) const {
    constexpr int K = Type<T>::kVec;
#pragma unroll
    for (int j = 0; j < N / K; ++j) {
      float t[K];
      widen<T>(raw[j], t);
#pragma unroll
      for (int i = 0; i < K; ++i) v[j * K + i] = t[i];
    }
  }
};
template <typename O, int N, bool NARROW>
__device__ __forceinline__ void store_columns(O* p, const float (&v)[N], int hidden) {
  if constexpr (NARROW) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < hidden) p[i] = (O)v[i];
  } else {
    store_row<O, N>(p, v, N);
  }
}

// A workgroup's `units` row groups of 2^lanes_shift lanes each walk `span`
// consecutive grouped positions, one column vector a lane.  A run (the
// positions of one token) belongs to the row group it begins in.  A row group
// adds its part of a run begun before it into LDS (`heads`); the run's owner
// collects these parts in order.  At the workgroup's ends the same is done
// through memory by the join kernel.
template <typename T, typename O, bool NARROW, bool ADD>
__global__ __launch_bounds__(kSumThreads) void sum_runs_kernel(RunArgs a) {
  constexpr int VEC = Type<T>::kVec;
  constexpr int N = VEC > Type<O>::kVec ? VEC : Type<O>::kVec;
  __shared__ int32_t tok[kSumSpots + 2];  // tok[1 + i]: position i; tok[0], tok[spots + 1]: the neighbours
  __shared__ int32_t row[kSumSpots];
  __shared__ float heads[kSumThreads][N];
  const int tid = threadIdx.x;
  // the tiles of a row next to each other: they are read at about one time
  const int64_t block = blockIdx.x / a.tiles;
  const int tile = (int)(blockIdx.x - block * a.tiles);
  const int lanes = 1 << a.lanes_shift, units = kSumThreads >> a.lanes_shift;
  const int unit = tid >> a.lanes_shift, lane = tid & (lanes - 1);
  const int spots = units * a.span;
  const int64_t first = (int64_t)block * spots;
  const int64_t m = listed_rows(a);
  if (first >= m) return;
  const int here = (int)(m - first < spots ? m - first : spots);
  for (int i = tid; i < spots + 2; i += kSumThreads) {
    const int64_t p = first + i - 1;
    tok[i] = p >= 0 && p < m ? listed_token(a, p) : -1;
  }
  for (int i = tid; i < here; i += kSumThreads) row[i] = listed_row(a, first + i);
  __syncthreads();

  const int want = (int)(tile * lanes + lane) * N;
  const bool any = want < a.hidden;  // the other lanes repeat the last columns and store nothing
  const int col = NARROW ? 0 : min(want, a.hidden - N), shift = want - col;
  const T* dy = static_cast<const T*>(a.dy) + col;
  O* grad = static_cast<O*>(a.grad) + col;
  const int p0 = unit * a.span;
  const int num = here - p0 < a.span ? (here - p0 > 0 ? here - p0 : 0) : a.span;

  float acc[N];
#pragma unroll
  for (int i = 0; i < N; ++i) acc[i] = 0.f;
  auto write = [&](int t) {
    if (!any) return;
    O* p = grad + (int64_t)t * a.hidden;
    float v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = acc[i] * a.scale;
    if constexpr (ADD) {
      Columns<O, N, NARROW> now;
      now.load(p, a.hidden);
      float old[N];
      now.values(old);
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += old[i];
    }
    if (ADD && !NARROW && shift > 0) {
#pragma unroll
      for (int i = 1; i < N; ++i)
        if (i >= shift) p[i] = (O)v[i];
    } else {
      store_columns<O, N, NARROW>(p, v, a.hidden);
    }
  };
  int token = num > 0 ? tok[1 + p0] : -1;
  bool ours = num > 0 && tok[p0] != token;  // this run begins in this row group
  bool head = false;                        // heads[tid] holds the end of a run begun before
  // Positions past the last read the last row again and are dropped.
  for (int i0 = 0; i0 < num; i0 += kSumBatch) {
    Columns<T, N, NARROW> batch[kSumBatch];
#pragma unroll
    for (int u = 0; u < kSumBatch; ++u)
      batch[u].load(dy + (int64_t)row[p0 + min(i0 + u, num - 1)] * a.dy_stride, a.hidden);
#pragma unroll
    for (int u = 0; u < kSumBatch; ++u) {
      if (i0 + u >= num) continue;
      const int t = tok[1 + p0 + i0 + u];
      if (t != token) {
        if (ours) {
          write(token);
        } else {
          head = true;
#pragma unroll
          for (int i = 0; i < N; ++i) heads[tid][i] = acc[i];
        }
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] = 0.f;
        token = t;
        ours = true;
      }
      float v[N];
      batch[u].values(v);
#pragma unroll
      for (int i = 0; i < N; ++i) acc[i] += v[i];
    }
  }
  if (num > 0 && !ours) {
    // the whole row group lies in a run begun before it
    head = true;
#pragma unroll
    for (int i = 0; i < N; ++i) heads[tid][i] = acc[i];
  }
  __syncthreads();
  if (num == 0) return;
  // collect the parts of later row groups: of this row group's last run, and
  // in row group 0 also of a run begun before the workgroup
  const int64_t spot = (int64_t)block * a.pitch + col;
  auto collect = [&](float (&sum)[N], int t) {
    for (int u = unit + 1; u < units; ++u) {
      if (u * a.span >= here || tok[1 + u * a.span] != t) break;
#pragma unroll
      for (int i = 0; i < N; ++i) sum[i] += heads[u * lanes + lane][i];
      // the run ends inside row group u unless its last position has the token
      if (tok[min((u + 1) * a.span, here)] != t) return false;
    }
    return true;  // not seen to end inside the workgroup's positions
  };
  if (unit == 0 && head) {
    const int t = tok[1];
    float sum[N];
#pragma unroll
    for (int i = 0; i < N; ++i) sum[i] = heads[tid][i];
    if (tok[min(a.span, here)] == t) (void)collect(sum, t);
    if (any) store_columns<float, N, NARROW>(a.head + spot, sum, a.hidden);
  }
  if (ours) {
    const bool on = collect(acc, token) && tok[here + 1] == token;
    if (!on)
      write(token);
    else if (any)
      store_columns<float, N, NARROW>(a.tail + spot, acc, a.hidden);
  }
}

// ---------------------------------------------------------------- join

// A run that begins in workgroup b's positions and goes on after them: its
// tail and the heads of the workgroups it reaches, in order, one column a
// thread.
__global__ __launch_bounds__(256) void join_runs_kernel(RunArgs a, int spots, int grad_dtype) {
  const int64_t m = listed_rows(a);
  const int64_t first = (int64_t)blockIdx.x * spots, next = first + spots;
  if (next >= m) return;
  const int32_t t = listed_token(a, next - 1);
  if (listed_token(a, next) != t) return;
  // the run's owner is this workgroup unless all its positions belong to a
  // run begun before it
  if (first > 0 && listed_token(a, first) == t && listed_token(a, first - 1) == t) return;
  // workgroups whose first position has the token, found 64 at a time
  int reach = 0;
  const int blocks = (int)((m + spots - 1) / spots);
  for (int b0 = (int)blockIdx.x + 1; b0 < blocks; b0 += 64) {
    const int b = b0 + (int)(threadIdx.x & 63);
    const uint64_t off = ~__ballot(b < blocks && listed_token(a, (int64_t)b * spots) == t);
    reach += off != 0 ? __builtin_ctzll(off) : 64;
    if (off != 0) break;
  }
  const int64_t col = (int64_t)blockIdx.y * 256 + threadIdx.x;
  if (col >= a.hidden) return;
  double s = (double)a.tail[blockIdx.x * a.pitch + col];
  const float* head = a.head + ((int64_t)blockIdx.x + 1) * a.pitch + col;
#pragma unroll 16
  for (int b = 0; b < reach; ++b) s += (double)head[b * a.pitch];
  s *= (double)a.scale;
  const int64_t i = (int64_t)t * a.hidden + col;
  store_any(a.grad, grad_dtype, i, a.accumulate ? s + (double)load_any(a.grad, grad_dtype, i) : s);
}

size_t align256(size_t b) { return (b + 255) & ~size_t(255); }

int group_shift(int64_t vocab) {
  // one workgroup per CU, more where a workgroup would own too many tokens,
  // fewer where there are fewer tokens
  int shift = 8;
  while (shift > 0 && (int64_t(1) << (shift - 1)) >= vocab) --shift;
  while (ceil_div(vocab, int64_t(1) << shift) > kGroupKeys) ++shift;
  return shift;
}

}  // namespace

hipError_t launch_embedding(int table_dtype, int out_dtype, const EmbeddingArgs& a, hipStream_t st) {
  return with_dtype(table_dtype, [&](auto t) {
    return with_dtype(out_dtype, [&](auto o) {
      using T = decltype(t);
      using O = decltype(o);
      constexpr int N = Type<T>::kVec > Type<O>::kVec ? Type<T>::kVec : Type<O>::kVec;
      const int64_t pieces = a.n * ceil_div(a.hidden, N);
      const unsigned blocks = (unsigned)std::min<int64_t>(ceil_div(pieces, 256 * kLookups), int64_t(1) << 20);
      if (a.token_bytes == 4)
        embedding_kernel<T, O, int32_t><<<blocks, 256, 0, st>>>(a);
      else
        embedding_kernel<T, O, int64_t><<<blocks, 256, 0, st>>>(a);
      return hipGetLastError();
    });
  });
}

EmbeddingGradLayout embedding_grad_layout(int64_t n, int hidden, int dtype) {
  EmbeddingGradLayout l{};
  // 8 columns a lane where either side is 16 bits wide; the layout does not
  // depend on the gradient's type, so it takes the narrower vector
  const int vec = dtype == 0 ? 4 : 8;
  l.lanes = 1;
  while (l.lanes < 64 && l.lanes * vec < hidden) l.lanes *= 2;
  l.units = kSumThreads / l.lanes;
  l.tiles = (int)ceil_div(hidden, (int64_t)l.lanes * vec);
  // long spans leave less to join, short ones fill the GPU: the longest of 8
  // to 32 positions with two workgroups per CU (65536 rows of 1024: 48 us with
  // 32; asking for four or eight per CU changed nothing beyond noise)
  l.span = 32;
  while (l.span > 8 && ceil_div(n, (int64_t)l.units * l.span) * l.tiles < 2 * kCUs) l.span /= 2;
  while (l.span > 1 && l.units * l.span > kSumSpots) l.span /= 2;
  l.blocks = ceil_div(n, (int64_t)l.units * l.span);
  const size_t pitch = (size_t)l.tiles * l.lanes * 8;
  size_t at = 0;
  l.rows = at;
  at += align256((size_t)n * 4);
  l.tokens = at;
  at += align256((size_t)n * 4);
  l.count = at;
  at += 256;
  l.head = at;
  at += align256((size_t)l.blocks * pitch * 4);
  l.tail = at;
  at += align256((size_t)l.blocks * pitch * 4);
  l.total = at;
  return l;
}

hipError_t launch_embedding_grad(int dtype, const EmbeddingGradArgs& a, hipStream_t st) {
  const EmbeddingGradLayout l = embedding_grad_layout(a.n, a.hidden, dtype);
  const int grad_size = a.grad_dtype == 0 ? 4 : 2;
  GroupArgs g{};
  g.tokens = a.tokens;
  g.n = a.n;
  g.vocab = a.vocab;
  g.shift = group_shift(a.vocab);
  g.keys = (int)ceil_div(a.vocab, int64_t(1) << g.shift);
  g.rows = reinterpret_cast<int32_t*>(a.ws + l.rows);
  g.grouped = reinterpret_cast<int32_t*>(a.ws + l.tokens);
  g.count = reinterpret_cast<int32_t*>(a.ws + l.count);
  g.grad = a.accumulate ? nullptr : static_cast<char*>(a.grad);
  g.row_bytes = (int64_t)a.hidden * grad_size;
  const size_t lds = (size_t)kGroupWaves * g.keys * sizeof(int32_t);
  const unsigned groups = 1u << g.shift;
  if (a.token_bytes == 4)
    group_kernel<int32_t><<<groups, 1024, lds, st>>>(g);
  else
    group_kernel<int64_t><<<groups, 1024, lds, st>>>(g);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.n == 0) return e;

  RunArgs s{};
  s.dy = a.dy;
  s.n = a.n;
  s.dy_stride = a.dy_stride;
  s.vocab = a.vocab;
  s.hidden = a.hidden;
  s.span = l.span;
  while ((1 << s.lanes_shift) < l.lanes) ++s.lanes_shift;
  s.rows = g.rows;
  s.grouped = g.grouped;
  s.count = g.count;
  s.scale = a.scale;
  s.grad = a.grad;
  s.accumulate = a.accumulate;
  s.head = reinterpret_cast<float*>(a.ws + l.head);
  s.tail = reinterpret_cast<float*>(a.ws + l.tail);
  s.pitch = (int64_t)l.tiles * l.lanes * 8;
  e = with_dtype(dtype, [&](auto t) {
    return with_dtype(a.grad_dtype, [&](auto o) {
      using T = decltype(t);
      using O = decltype(o);
      constexpr int N = Type<T>::kVec > Type<O>::kVec ? Type<T>::kVec : Type<O>::kVec;
      const unsigned tiles = (unsigned)ceil_div(a.hidden, (int64_t)l.lanes * N);
      RunArgs b = s;
      b.tiles = (int)tiles;
      const unsigned grid = (unsigned)(l.blocks * tiles);
      if (a.hidden < N && a.accumulate)
        sum_runs_kernel<T, O, true, true><<<grid, kSumThreads, 0, st>>>(b);
      else if (a.hidden < N)
        sum_runs_kernel<T, O, true, false><<<grid, kSumThreads, 0, st>>>(b);
      else if (a.accumulate)
        sum_runs_kernel<T, O, false, true><<<grid, kSumThreads, 0, st>>>(b);
      else
        sum_runs_kernel<T, O, false, false><<<grid, kSumThreads, 0, st>>>(b);
      return hipGetLastError();
    });
  });
  if (e != hipSuccess) return e;
  if (l.blocks > 1) {
    join_runs_kernel<<<dim3((unsigned)(l.blocks - 1), (unsigned)ceil_div(a.hidden, 256)), 256, 0, st>>>(
        s, l.units * l.span, a.grad_dtype);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace adasum
