// The kernels' sources on the CPU: what they use of HIP, one fiber per lane.
//
// A workgroup's lanes run one after another up to their next meeting point: a
// barrier of the workgroup, or an operation of the wave (ballot, lane
// exchange).  Waves are taken in random order, LDS starts as garbage, and a
// meeting that not all lanes of a wave (or of a workgroup) come to ends the
// program.  Every shared array is thread_local here, and nothing else of the
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
};
inline std::vector<Lane> lanes;
inline std::vector<char*> stacks;
inline unsigned current;
inline void* scheduler;
inline const std::function<void()>* body;
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

inline void wait(State s) {
  lanes[current].state = s;
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
  lanes[i] = Lane{top, kRun, 0, 0, 0};
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
  unsigned live = 0, meet[kDone + 1] = {};
  for (unsigned i = w * 64; i < w * 64 + 64; ++i) {
    if (lanes[i].state == kRun) {
      current = i;
      threadIdx.x = i;
      on_cpu_switch(&scheduler, lanes[i].sp);
    }
    ++meet[lanes[i].state];
    live += lanes[i].state != kDone;
  }
  const unsigned in_wave = meet[kBallot] + meet[kExchange] + meet[kOrder];
  if (in_wave == 0) return;  // all at a barrier or done
  if (meet[kBarrier]) stop("a wave is divided between a barrier and an operation of its own");
  if (std::max({meet[kBallot], meet[kExchange], meet[kOrder]}) != in_wave) stop("a wave meets at two operations");
  uint64_t mask = 0;
  for (unsigned l = 0; l < 64; ++l)
    if (lanes[w * 64 + l].state == kBallot && lanes[w * 64 + l].in) mask |= uint64_t(1) << l;
  for (unsigned l = 0; l < 64; ++l) {
    Lane& x = lanes[w * 64 + l];
    if (x.state == kBallot) x.out = mask;
    if (x.state == kExchange) {
      const Lane& y = lanes[w * 64 + x.from];
      if (y.state != kExchange) stop("a value of a lane that is not there");
      x.out = y.in;
    }
  }
  for (unsigned l = 0; l < 64; ++l)
    if (lanes[w * 64 + l].state != kDone) lanes[w * 64 + l].state = kRun;
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

inline uint32_t exchange(uint32_t v, unsigned lane) {
  Lane& l = lanes[current];
  l.in = v;
  l.from = lane;
  wait(kExchange);
  return (uint32_t)lanes[current].out;
}
inline unsigned lane_id() { return current & 63; }

}  // namespace on_cpu

inline void __syncthreads() { on_cpu::wait(on_cpu::kBarrier); }
inline uint64_t __ballot(int p) {
  on_cpu::lanes[on_cpu::current].in = p != 0;
  on_cpu::wait(on_cpu::kBallot);
  return on_cpu::lanes[on_cpu::current].out;
}
inline int __shfl_up(int v, unsigned by) {
  const unsigned l = on_cpu::lane_id();
  return (int)on_cpu::exchange((uint32_t)v, l >= by ? l - by : l);
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
inline int on_cpu_dpp(int v, int ctrl) {
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
