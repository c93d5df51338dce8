// The kernels of the shared-prefix tables on the host (cuda_on_host.h).  KERNELS is their source with the
// includes and the PTX taken out.
#include "cuda_on_host.h"
#include KERNELS

using namespace mla;

extern "C" {

// The launches of a table by its rows, as launch_shared_tables orders them; `later` (or null): the lengths
// as they are from the second launch on.  Returns 0, without the lists, if an offset could lead out of them.
int tables_run(SharedTableParams* p, int small, unsigned schedule, const int32_t* later) {
  const size_t n = p->batch;
  host::forget();
  for (const int32_t* list : {(const int32_t*)p->group_indptr, (const int32_t*)p->prefix_indptr, (const int32_t*)p->kv_indptr})
    host::watch(list, (n + 1) * 4);
  if (small) {
    host::run_block({1, 1, 1}, {0, 0, 0}, kScanThreads, schedule, [p] { small_tables_kernel(*p); });
    return 1;
  }
  const unsigned rows = n > 0 ? (unsigned)n : 1;
  for (unsigned i : host::order(rows, schedule, 1))
    host::run_block({rows, 1, 1}, {i, 0, 0}, kThreads, schedule, [p] { common_pages_kernel(*p); });
  if (later) p->seq_lens = later;
  host::run_block({1, 1, 1}, {0, 0, 0}, kScanThreads, schedule, [p] { groups_kernel(*p); });
  for (const int32_t* list : {(const int32_t*)p->prefix_indptr, (const int32_t*)p->kv_indptr})
    for (size_t i = 0; i <= n; ++i)
      if (list[i] < (i > 0 ? list[i - 1] : 0)) return 0;
  for (unsigned i : host::order(rows, schedule, 2))
    for (unsigned y = 0; y < (unsigned)kFillBlocks; ++y)
      host::run_block({rows, (unsigned)kFillBlocks, 1}, {i, y, 0}, kThreads, schedule, [p] { lists_kernel(*p); });
  return 1;
}

long long tables_early_loads() { return host::machine().early_loads; }

}
