// The kernels of the shared-prefix tables on the host (cuda_on_host.h).  KERNELS is their source with the
// includes and the PTX taken out.
#include <signal.h>
#include <sys/mman.h>
#include <unistd.h>

#include "cuda_on_host.h"
#include KERNELS

using namespace mla;

namespace {

// n ints, all of which lie in the same 64 MB of memory, with nothing mapped for 8 GB on either side.
int32_t* far_ints(size_t n) {
  constexpr size_t kChunk = 64 << 20, kNothing = 9ull << 30;
  const size_t bytes = (n * 4 + kChunk - 1) / kChunk * kChunk;
  char* at = static_cast<char*>(
      mmap(nullptr, bytes + 2 * kNothing, PROT_NONE, MAP_PRIVATE | MAP_ANONYMOUS | MAP_NORESERVE, -1, 0));
  const int fd = memfd_create("ints", 0);
  if (at == MAP_FAILED || fd < 0 || ftruncate(fd, kChunk) != 0) std::exit(4);
  for (size_t o = 0; o < bytes; o += kChunk)
    if (mmap(at + kNothing + o, kChunk, PROT_READ | PROT_WRITE, MAP_SHARED | MAP_FIXED, fd, 0) == MAP_FAILED) std::exit(4);
  return reinterpret_cast<int32_t*>(at + kNothing);
}

}  // namespace

extern "C" {

// The launches of a table by its rows, as launch_shared_tables orders them; `later` (or null): the lengths
// as they are from the second launch on, or for every other load of a single one.  Returns 0, without the lists, if an offset could lead out of them.
int tables_run(SharedTableParams* p, int small, unsigned schedule, const int32_t* later) {
  const size_t n = p->batch;
  host::forget();
  for (const int32_t* list : {(const int32_t*)p->group_indptr, (const int32_t*)p->prefix_indptr, (const int32_t*)p->kv_indptr})
    host::watch(list, (n + 1) * 4);
  const auto ascend = [p, n] {
    for (const int32_t* list : {(const int32_t*)p->prefix_indptr, (const int32_t*)p->kv_indptr})
      for (size_t i = 0; i <= n; ++i)
        if (list[i] < (i > 0 ? list[i - 1] : 0)) return 0;
    return 1;
  };
  if (small) {
    if (later) host::change(p->seq_lens, n * 4, later);
    host::run_block({1, 1, 1}, {0, 0, 0}, kScanThreads, schedule, [p] { small_tables_kernel(*p); });
    return ascend();
  }
  const unsigned rows = n > 0 ? (unsigned)n : 1;
  for (unsigned i : host::order(rows, schedule, 1))
    host::run_block({rows, 1, 1}, {i, 0, 0}, kThreads, schedule, [p] { common_pages_kernel(*p); });
  if (later) p->seq_lens = later;
  host::run_block({1, 1, 1}, {0, 0, 0}, kScanThreads, schedule, [p] { groups_kernel(*p); });
  if (!ascend()) return 0;
  for (unsigned i : host::order(rows, schedule, 2))
    for (unsigned y = 0; y < (unsigned)kFillBlocks; ++y)
      host::run_block({rows, (unsigned)kFillBlocks, 1}, {i, y, 0}, kThreads, schedule, [p] { lists_kernel(*p); });
  return 1;
}

// Lists and rows of 2^31 - 1 entries, by the first and the last warp of the last block.  Exits with 3 on an
// access outside of them.
int tables_far(int what) {
  signal(SIGSEGV, [](int) { _exit(3); });
  constexpr int kMost = 0x7fffffff;
  int32_t table[2] = {0, 0}, lens[2] = {kMost, kMost}, groups[3] = {0, 2, 2}, prefix[3] = {0, kMost, kMost}, own[3] = {0, 0, 0};
  SharedTableParams p{table, lens, 2, 1, kMost, 1, groups, prefix, nullptr, own, nullptr, 0, 0};
  const auto two_warps = [&](std::function<void()> kernel, unsigned x, unsigned y) {
    host::run_block({2, (unsigned)kFillBlocks, 1}, {x, y, 0}, kThreads, 0, std::move(kernel), 32, kThreads - 32);
  };
  if (what == 0) {  // two rows of a page that both have in full: their prefix
    p.prefix_indices = far_ints(kMost);
    p.prefix_capacity = kMost;
    two_warps([&] { lists_kernel(p); }, 0, kFillBlocks - 1);
    return p.prefix_indices[kMost - 1] == kMost - 1;
  }
  if (what == 1) {  // a row's own keys
    p.batch = 1;
    groups[1] = 1;
    prefix[1] = 0;
    own[1] = kMost;
    p.kv_indices = far_ints(kMost);
    p.capacity = kMost;
    two_warps([&] { lists_kernel(p); }, 0, kFillBlocks - 1);
    return p.kv_indices[kMost - 1] == kMost - 1;
  }
  p.page_size = 1;  // rows of as many pages
  p.max_blocks = kMost;
  p.block_table = far_ints(2 * (size_t)kMost);
  two_warps([&] { common_pages_kernel(p); }, 1, 0);
  return 1;
}

long long tables_early_loads() { return host::machine().early_loads; }

}
