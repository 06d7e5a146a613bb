// The kernels' sources on the CPU: what they use of HIP, one fiber per lane.
//
// A workgroup's lanes run one after another up to their next meeting point: a
// barrier of the workgroup, or an operation of the wave (ballot, lane
// exchange).  Waves are taken in random order, LDS starts as garbage, and a
// meeting that not all lanes of a wave (or of a workgroup) come to ends the
// program, unless it allows a wave's lanes to divide: then those furthest back
// in the code go on first.  Every shared array is thread_local here, and nothing else of the
// program may be: that is how a new workgroup finds them to overwrite.
#pragma once

#include <elf.h>
#include <link.h>
#include <sys/mman.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <functional>
#include <type_traits>
#include <vector>

#define __global__
#define __device__
#define __host__
#define __forceinline__ inline __attribute__((always_inline))
#define __launch_bounds__(...)
#define __shared__ thread_local

struct dim3 {
  unsigned x, y, z;
  dim3(unsigned x_ = 1, unsigned y_ = 1, unsigned z_ = 1) : x(x_), y(y_), z(z_) {}
};
typedef int hipError_t;
typedef void* hipStream_t;
constexpr hipError_t hipSuccess = 0;
inline hipError_t hipGetLastError() { return hipSuccess; }
using std::max;
using std::min;

inline dim3 threadIdx, blockIdx, gridDim, blockDim;

namespace on_cpu {

[[noreturn]] inline void stop(const char* what) {
  std::printf("%s at workgroup %u, %u\n", what, blockIdx.x, blockIdx.y);
  std::fflush(stdout);
  std::exit(3);
}

enum State { kRun, kBarrier, kBallot, kExchange, kOrder, kDone };
struct Lane {
  void* sp;
  State state;
  uint64_t in, from, out;
  const void* site;  // where in the code it waits
};
inline std::vector<Lane> lanes;
inline std::vector<char*> stacks;
inline unsigned current;
inline void* scheduler;
inline const std::function<void()>* body;
inline bool may_divide = false;
constexpr size_t kStack = 1 << 16;

// Saves what a call must keep, and goes on with the other stack.
extern "C" void on_cpu_switch(void** save, void* to);
asm(R"(
  .text
  .globl on_cpu_switch
  .type on_cpu_switch, @function
on_cpu_switch:
  push %rbp
  push %rbx
  push %r12
  push %r13
  push %r14
  push %r15
  mov %rsp, (%rdi)
  mov %rsi, %rsp
  pop %r15
  pop %r14
  pop %r13
  pop %r12
  pop %rbx
  pop %rbp
  ret
)");

__attribute__((noinline)) inline void wait(State s) {
  lanes[current].state = s;
  lanes[current].site = __builtin_return_address(0);
  on_cpu_switch(&lanes[current].sp, scheduler);
}
inline void lane_main() {
  (*body)();
  wait(kDone);
  std::abort();
}
inline void start(unsigned i) {
  void** top = reinterpret_cast<void**>(stacks[i] + kStack);
  *--top = nullptr;  // the return address of lane_main; rsp is then as after a call
  *--top = reinterpret_cast<void*>(&lane_main);
  for (int r = 0; r < 6; ++r) *--top = nullptr;
  lanes[i] = Lane{top, kRun, 0, 0, 0, nullptr};
}

// Every shared array of the program overwritten.
inline void spoil_lds() {
  dl_iterate_phdr(
      [](dl_phdr_info* info, size_t, void*) {
        for (int i = 0; i < info->dlpi_phnum; ++i)
          if (info->dlpi_phdr[i].p_type == PT_TLS && info->dlpi_tls_data) {
            uint32_t* w = static_cast<uint32_t*>(info->dlpi_tls_data);
            for (size_t k = 0; k < info->dlpi_phdr[i].p_memsz / 4; ++k) w[k] = 0x7f1a2b3cu + (uint32_t)k;
          }
        return 1;  // the first one is the program itself
      },
      nullptr);
}

inline void run_wave(unsigned w) {
  unsigned meet[kDone + 1] = {};
  Lane* const wave = &lanes[w * 64];
  for (unsigned l = 0; l < 64; ++l) {
    if (wave[l].state == kRun) {
      current = w * 64 + l;
      threadIdx.x = current;
      on_cpu_switch(&scheduler, wave[l].sp);
    }
    ++meet[wave[l].state];
  }
  const unsigned in_wave = meet[kBallot] + meet[kExchange] + meet[kOrder];
  if (in_wave == 0) return;  // all at a barrier or done
  const void* site = nullptr;
  for (unsigned l = 0; l < 64; ++l)
    if (wave[l].state != kBarrier && wave[l].state != kDone &&
        (site == nullptr || std::less<const void*>()(wave[l].site, site)))
      site = wave[l].site;
  bool meets[64];
  unsigned together = 0;
  for (unsigned l = 0; l < 64; ++l) {
    meets[l] = wave[l].state != kBarrier && wave[l].state != kDone && wave[l].site == site;
    together += meets[l];
  }
  if (!may_divide && meet[kBarrier]) stop("a wave is divided between a barrier and an operation of its own");
  if (!may_divide && together != in_wave) stop("a wave meets at two operations");
  uint64_t mask = 0;
  for (unsigned l = 0; l < 64; ++l)
    if (meets[l] && wave[l].state == kBallot && wave[l].in) mask |= uint64_t(1) << l;
  for (unsigned l = 0; l < 64; ++l) {
    if (!meets[l]) continue;
    if (wave[l].state == kBallot) wave[l].out = mask;
    if (wave[l].state == kExchange) {
      if (!meets[wave[l].from]) stop("a value of a lane that is not there");
      wave[l].out = wave[wave[l].from].in;
    }
  }
  for (unsigned l = 0; l < 64; ++l)
    if (meets[l]) wave[l].state = kRun;
}

inline void run_workgroup(unsigned threads) {
  spoil_lds();
  lanes.resize(threads);
  while (stacks.size() < threads) stacks.push_back(static_cast<char*>(std::aligned_alloc(64, kStack)));
  for (unsigned i = 0; i < threads; ++i) start(i);
  for (;;) {
    const unsigned waves = threads / 64, first = std::rand() % waves;
    for (unsigned k = 0; k < waves; ++k) {
      const unsigned w = (first + k * 7) % waves;  // 7 divides no number of waves in use
      if (std::rand() % 3) run_wave(w);
    }
    unsigned barrier = 0, done = 0;
    for (const Lane& l : lanes) {
      barrier += l.state == kBarrier;
      done += l.state == kDone;
    }
    if (done == threads) return;
    if (barrier + done != threads) continue;
    if (done) stop("a barrier that some lanes do not come to");
    for (Lane& l : lanes) l.state = kRun;
  }
}

// Workgroups to run of a launch: all, unless the program limits them.
inline std::function<bool(unsigned)> wanted = [](unsigned) { return true; };

template <typename... P>
auto launch(void (*kernel)(P...), dim3 grid, unsigned threads, size_t, hipStream_t) {
  return [=](std::common_type_t<P>... args) {
    const std::function<void()> f = [&] { kernel(args...); };
    body = &f;
    gridDim = grid;
    blockDim = dim3(threads);
    for (unsigned y = 0; y < grid.y; ++y)
      for (unsigned x = 0; x < grid.x; ++x) {
        if (!wanted(x)) continue;
        blockIdx = dim3(x, y);
        run_workgroup(threads);
      }
  };
}

// Memory whose last byte is followed, and whose first page is preceded, by a
// page that must not be touched.
inline char* guarded(size_t bytes) {
  const size_t page = 4096, whole = (bytes + page - 1) / page * page;
  char* p = static_cast<char*>(
      mmap(nullptr, whole + 2 * page, PROT_NONE, MAP_PRIVATE | MAP_ANONYMOUS | MAP_NORESERVE, -1, 0));
  if (p == MAP_FAILED || mprotect(p + page, whole, PROT_READ | PROT_WRITE)) stop("no memory");
  return p + page + whole - bytes;
}

__forceinline__ uint32_t exchange(uint32_t v, unsigned lane) {
  Lane& l = lanes[current];
  l.in = v;
  l.from = lane;
  wait(kExchange);
  return (uint32_t)lanes[current].out;
}
inline unsigned lane_id() { return current & 63; }

// f(from): what the lane makes of the wave's values of v, from(l) being lane
// l's.  No lane goes on before all have read.
template <typename V, typename F>
__forceinline__ auto together(const V& v, F f) {
  Lane& l = lanes[current];
  l.in = reinterpret_cast<uint64_t>(&v);
  const unsigned wave = current & ~63u;
  wait(kOrder);
  auto out = f([wave](unsigned i) -> const V& {
    if (lanes[wave + i].state == kDone) stop("a value of a lane that is not there");
    return *reinterpret_cast<const V*>(lanes[wave + i].in);
  });
  wait(kOrder);
  return out;
}

}  // namespace on_cpu

__forceinline__ void __syncthreads() { on_cpu::wait(on_cpu::kBarrier); }
__forceinline__ uint64_t __ballot(int p) {
  on_cpu::lanes[on_cpu::current].in = p != 0;
  on_cpu::wait(on_cpu::kBallot);
  return on_cpu::lanes[on_cpu::current].out;
}
__forceinline__ int __shfl_up(int v, unsigned by) {
  const unsigned l = on_cpu::lane_id();
  return (int)on_cpu::exchange((uint32_t)v, l >= by ? l - by : l);
}
__forceinline__ float __shfl_xor(float v, unsigned by) {
  return __builtin_bit_cast(float, on_cpu::exchange(__builtin_bit_cast(uint32_t, v), on_cpu::lane_id() ^ by));
}
__forceinline__ double __shfl_xor(double v, unsigned by) {
  const uint64_t w = __builtin_bit_cast(uint64_t, v);
  const unsigned from = on_cpu::lane_id() ^ by;
  const uint64_t low = on_cpu::exchange((uint32_t)w, from), high = on_cpu::exchange((uint32_t)(w >> 32), from);
  return __builtin_bit_cast(double, high << 32 | low);
}
inline int __popcll(uint64_t x) { return __builtin_popcountll(x); }
inline int32_t atomicAdd(int32_t* p, int32_t v) {
  const int32_t old = *p;
  *p += v;
  return old;
}
inline int on_cpu_mbcnt(uint64_t mask, int add) {
  return add + __builtin_popcountll(mask & ((uint64_t(1) << on_cpu::lane_id()) - 1));
}
__forceinline__ int on_cpu_dpp(int v, int ctrl) {
  const unsigned l = on_cpu::lane_id();
  unsigned from = 0;
  if (ctrl < 0x100)  // of each four lanes
    from = (l & ~3u) | ((ctrl >> (2 * (l & 3))) & 3);
  else if (ctrl == 0x140)  // of each 16, turned round
    from = l ^ 15;
  else if (ctrl == 0x141)  // of each 8
    from = l ^ 7;
  else
    on_cpu::stop("an unknown lane pattern");
  return (int)on_cpu::exchange((uint32_t)v, from);
}
#define __builtin_amdgcn_readfirstlane(x) (x)
#define __builtin_amdgcn_readlane(v, lane) ((int)on_cpu::exchange((uint32_t)(v), (unsigned)(lane)))
#define __builtin_amdgcn_mbcnt_lo(m, add) on_cpu_mbcnt((uint32_t)(m), add)
#define __builtin_amdgcn_mbcnt_hi(m, add) on_cpu_mbcnt((uint64_t)(m) << 32, add)
#define __builtin_amdgcn_fence(order, scope) on_cpu::wait(on_cpu::kOrder)
#define __builtin_amdgcn_wave_barrier() on_cpu::wait(on_cpu::kOrder)
#define __builtin_amdgcn_update_dpp(old, v, ctrl, rows, banks, bound) on_cpu_dpp(v, ctrl)
#define __builtin_amdgcn_fmed3f(a, b, c) std::min(std::max(a, b), c)
#define __builtin_amdgcn_rsqf(x) (1.f / std::sqrt(x))
#define __builtin_amdgcn_sched_barrier(mask) ((void)0)

inline uint32_t on_cpu_perm(uint32_t hi, uint32_t lo, uint32_t select) {
  const uint64_t both = (uint64_t)hi << 32 | lo;
  uint32_t r = 0;
  for (int i = 0; i < 4; ++i) r |= (uint32_t)(both >> (8 * ((select >> (8 * i)) & 7)) & 0xff) << (8 * i);
  return r;
}
#define __builtin_amdgcn_perm(hi, lo, select) on_cpu_perm(hi, lo, select)

// Lane i of 16 names four values of row i / 4 and gets value i of the four
// rows: the four that lane 4 r + i / 4 names hold row r's.
template <typename P>
__forceinline__ auto on_cpu_read_turned(P p) {
  typedef short v4s __attribute__((ext_vector_type(4)));
  const v4s mine = *p;
  return on_cpu::together(mine, [](auto from) {
    const unsigned l = on_cpu::lane_id(), i = l & 15;
    v4s r;
    for (unsigned k = 0; k < 4; ++k) r[k] = from((l & ~15u) + 4 * k + i / 4)[i & 3];
    return r;
  });
}
#define __builtin_amdgcn_ds_read_tr16_b64_v4i16(p) on_cpu_read_turned(p)

// A lane of a 16 x 16 x 32 product holds terms 8 (l / 16) .. of row or column
// l % 16, and of the sums rows 4 (l / 16) .. of column l % 16.
template <typename V, typename C>
__forceinline__ C on_cpu_multiply(V a, V b, C c) {
  struct Both {
    V a, b;
  } mine{a, b};
  return on_cpu::together(mine, [&](auto from) {
    const unsigned l = on_cpu::lane_id();
    C r = c;
    for (unsigned q = 0; q < 4; ++q) {
      float sum = 0.f;
      for (unsigned k = 0; k < 32; ++k)
        sum += (float)from(k / 8 * 16 + l / 16 * 4 + q).a[k % 8] * (float)from(k / 8 * 16 + l % 16).b[k % 8];
      r[q] += sum;
    }
    return r;
  });
}
#define __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, x, y, z) on_cpu_multiply(a, b, c)
#define __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, x, y, z) on_cpu_multiply(a, b, c)

// A wave's 64 pieces of 16 bytes from anywhere to consecutive places in LDS.
template <typename G, typename L>
__forceinline__ void on_cpu_load_lds(G from, L to) {
  std::memcpy((char*)to + 16 * on_cpu::lane_id(), (const char*)from, 16);
}
#define __builtin_amdgcn_global_load_lds(from, to, bytes, offset, aux) on_cpu_load_lds(from, to)
#define __builtin_amdgcn_s_waitcnt(counts) ((void)0)
#define __builtin_amdgcn_s_barrier() on_cpu::wait(on_cpu::kBarrier)

// A lane of a 16 x 16 x 4 product in fp64 holds term l / 16 of row or column
// l % 16, and of the sums rows 4 r + l / 16 of column l % 16.
template <typename C>
__forceinline__ C on_cpu_multiply64(double a, double b, C c) {
  struct Both {
    double a, b;
  } mine{a, b};
  return on_cpu::together(mine, [&](auto from) {
    const unsigned l = on_cpu::lane_id();
    C r = c;
    for (unsigned q = 0; q < 4; ++q)
      for (unsigned k = 0; k < 4; ++k) r[q] += from(k * 16 + 4 * q + l / 16).a * from(k * 16 + l % 16).b;
    return r;
  });
}
#define __builtin_amdgcn_mfma_f64_16x16x4f64(a, b, c, x, y, z) on_cpu_multiply64(a, b, c)
