// Plan of kv_attn_paged: which kernels a batch needs and how many runs each gets.
#include <algorithm>
#include <cmath>

#include "launch.h"

namespace kva {

bool attn_paged_supports(int Dk, int Dv) {
  return (Dk == 64 && Dv == 64) || (Dk == 128 && Dv == 128) || (Dk == 192 && Dv == 128);
}

cudaError_t launch_attn_paged(const PagedArgs& args, int Dk, int Dv, kva_dtype dtype, const int32_t* lengths,
                              const int32_t* start, cudaStream_t s, unsigned* n_launches) {
  const int G = args.Hq / args.Hkv;
  int64_t steps = 0, units = 0;
  for (int b = 0; b < args.B; ++b) {
    const int64_t rows = (int64_t)(start[b + 1] - start[b]) * G;
    if (rows == 0) continue;
    const int64_t n = (rows + PAGED_ROWS - 1) / PAGED_ROWS * args.Hkv;
    units += n;
    steps += n * std::max(1, (lengths[b] + 127) / 128);
  }
  PagedArgs a = args;
  a.rows_lo = 0;
  a.rows_hi = INT32_MAX;
  // as many runs as the GPU holds at once, and not so many that joining a unit's parts costs more than its steps
  const int64_t most = std::min<int64_t>(PAGED_SMS * 3, (int64_t)(2.0 * std::sqrt((double)steps * (double)units)));
  const int runs = (int)std::max<int64_t>(1, std::min(most, steps));
  (void)Dv;
  const cudaError_t e = launch_attn_paged_simt(a, Dk, dtype, runs, s);
  if (e == cudaSuccess) *n_launches = 1;
  return e;
}

}  // namespace kva
