// cuda_on_host.h -- runs a kernel's source on the host, one block at a time, under a chosen schedule.
//
// Every thread of a block is a fiber.  A fiber runs until it meets a barrier or a warp's exchange,
// so between two of them a warp may be as far ahead of the others as CUDA allows: the schedule
// names which warp, and which lane of it, goes first.  A kernel whose result depends on the
// schedule lacks a barrier.
//
// Loads.  __ldg is for what does not change while a kernel lives, and a kernel launched as a
// programmatic dependent may live from before the launches in front of it: it may return what memory
// held then.  So loads by __ldg from watched buffers, which those launches write, are counted
// (early_loads).
#pragma once
#include <ucontext.h>

#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <functional>
#include <memory>
#include <numeric>
#include <vector>

using std::max;
using std::min;

struct Dim3 {
  unsigned x = 1, y = 1, z = 1;
};

namespace host {

constexpr int kWarp = 32;
enum State { kReady, kBlockBarrier, kWarpExchange, kDone };

struct Fiber {
  ucontext_t ctx;
  std::unique_ptr<char[]> stack;
  Dim3 tid;
  State state = kDone;
  long long in = 0, out = 0;  // a warp's exchange: what the lane gives, what it gets
  std::function<void(std::vector<Fiber*>&)> exchange;
};

struct Machine {
  ucontext_t scheduler;
  std::vector<Fiber> fibers;
  Fiber* now = nullptr;
  Dim3 block_idx, block_dim, grid_dim;
  std::function<void()> kernel;
  std::vector<std::pair<const char*, const char*>> watched;
  long long early_loads = 0;
  const char *changing = nullptr, *changing_end = nullptr, *changed = nullptr;  // see change()
  unsigned changing_loads = 0;
};
inline Machine& machine() {
  static Machine m;
  return m;
}

inline void wait_as(State s) {
  Machine& m = machine();
  m.now->state = s;
  swapcontext(&m.now->ctx, &m.scheduler);
}

// The lanes of a warp meet; `f` sets every lane's `out` from their `in`s.
inline long long exchange(long long in, std::function<void(std::vector<Fiber*>&)> f) {
  Fiber* me = machine().now;
  me->in = in;
  me->exchange = std::move(f);
  wait_as(kWarpExchange);
  return me->out;
}

inline void entry() {
  machine().kernel();
  machine().now->state = kDone;
  swapcontext(&machine().now->ctx, &machine().scheduler);
}

// A schedule: 0 warps and lanes ascending, 1 descending, else a random order of both by this seed.
inline std::vector<int> order(int n, unsigned schedule, unsigned salt) {
  std::vector<int> v(n);
  std::iota(v.begin(), v.end(), 0);
  if (schedule == 1) std::reverse(v.begin(), v.end());
  if (schedule > 1) {
    unsigned long long x = schedule * 0x9e3779b97f4a7c15ull + salt;
    for (int i = n - 1; i > 0; --i) {
      x = x * 6364136223846793005ull + 1442695040888963407ull;
      std::swap(v[i], v[(x >> 33) % (i + 1)]);
    }
  }
  return v;
}

// Runs one block.  Threads in [absent, present) do not exist (for loops too long to run on all).
inline void run_block(Dim3 grid, Dim3 idx, int threads, unsigned schedule, std::function<void()> kernel, int absent = 0,
                      int present = 0) {
  Machine& m = machine();
  m.block_idx = idx;
  m.grid_dim = grid;
  m.block_dim = Dim3{(unsigned)threads, 1, 1};
  m.kernel = std::move(kernel);
  if ((int)m.fibers.size() < threads) m.fibers.resize(threads);
  for (int t = 0; t < threads; ++t) {
    Fiber& f = m.fibers[t];
    f.tid = Dim3{(unsigned)t, 0, 0};
    f.state = kDone;
    if (t >= absent && t < present) continue;
    constexpr size_t kStack = 64 << 10;
    if (!f.stack) f.stack.reset(new char[kStack]);
    getcontext(&f.ctx);
    f.ctx.uc_stack.ss_sp = f.stack.get();
    f.ctx.uc_stack.ss_size = kStack;
    f.ctx.uc_link = nullptr;
    makecontext(&f.ctx, entry, 0);
    f.state = kReady;
  }
  const int warps = (threads + kWarp - 1) / kWarp;
  for (unsigned turn = 0;; ++turn) {
    bool ran = false, alive = false;
    for (int w : order(warps, schedule, turn)) {
      for (;;) {  // as far as this warp can go
        bool here = false;
        for (int l : order(min(kWarp, threads - w * kWarp), schedule, turn + 77)) {
          Fiber& f = m.fibers[w * kWarp + l];
          if (f.state != kReady) continue;
          m.now = &f;
          swapcontext(&m.scheduler, &f.ctx);
          here = ran = true;
        }
        std::vector<Fiber*> meet;
        bool others = false;
        for (int l = 0; l < kWarp && w * kWarp + l < threads; ++l) {
          Fiber& f = m.fibers[w * kWarp + l];
          if (f.state == kWarpExchange) meet.push_back(&f);
          else if (f.state != kDone) others = true;
        }
        if (!meet.empty()) {
          if (others) {
            std::fprintf(stderr, "a warp's lanes wait at different places\n");
            std::abort();
          }
          auto f = meet[0]->exchange;
          f(meet);
          for (Fiber* x : meet) x->state = kReady;
          here = true;
        }
        if (!here) break;
      }
    }
    for (int t = 0; t < threads; ++t) alive |= m.fibers[t].state != kDone;
    if (!alive) return;
    if (!ran) {
      for (int t = 0; t < threads; ++t)
        if (m.fibers[t].state == kBlockBarrier) m.fibers[t].state = kReady;
    }
  }
}

inline void watch(const void* p, size_t bytes) {
  machine().watched.emplace_back(static_cast<const char*>(p), static_cast<const char*>(p) + bytes);
}
// Loads by __ldg from these bytes return, every other time, what is at `other`: a buffer that is rewritten meanwhile.
inline void change(const void* p, size_t bytes, const void* other) {
  machine().changing = static_cast<const char*>(p);
  machine().changing_end = machine().changing + bytes;
  machine().changed = static_cast<const char*>(other);
}
inline void forget() {
  machine().watched.clear();
  machine().early_loads = 0;
  machine().changing = machine().changing_end = nullptr;
}

}  // namespace host

#define __global__
#define __device__
#define __forceinline__ inline
#define __launch_bounds__(...)
#define __shared__ static
#define threadIdx (host::machine().now->tid)
#define blockIdx (host::machine().block_idx)
#define blockDim (host::machine().block_dim)
#define gridDim (host::machine().grid_dim)

inline void __syncthreads() { host::wait_as(host::kBlockBarrier); }
inline void __threadfence_block() {}
inline int __popc(unsigned v) { return __builtin_popcount(v); }

template <typename T>
T __ldcg(const T* p) {
  return *p;
}
template <typename T>
T __ldg(const T* p) {
  const char* at = reinterpret_cast<const char*>(p);
  for (auto& b : host::machine().watched) host::machine().early_loads += at >= b.first && at < b.second;
  host::Machine& m = host::machine();
  if (at >= m.changing && at < m.changing_end && (m.changing_loads++ & 1))
    return *reinterpret_cast<const T*>(m.changed + (at - m.changing));
  return *p;
}
inline int atomicMin(int* p, int v) {
  const int old = *p;
  *p = min(old, v);
  return old;
}

inline long long __shfl_up_sync(unsigned, long long v, int delta) {
  return host::exchange(v, [delta](std::vector<host::Fiber*>& x) {
    for (size_t i = 0; i < x.size(); ++i) x[i]->out = (int)i >= delta ? x[i - delta]->in : x[i]->in;
  });
}
inline int __reduce_min_sync(unsigned, int v) {
  return (int)host::exchange(v, [](std::vector<host::Fiber*>& x) {
    long long least = x[0]->in;
    for (auto* f : x) least = min(least, f->in);
    for (auto* f : x) f->out = least;
  });
}
inline unsigned __ballot_sync(unsigned, bool v) {
  return (unsigned)host::exchange(v, [](std::vector<host::Fiber*>& x) {
    long long bits = 0;
    for (auto* f : x) bits |= (long long)(f->in != 0) << (f->tid.x % host::kWarp);
    for (auto* f : x) f->out = bits;
  });
}
