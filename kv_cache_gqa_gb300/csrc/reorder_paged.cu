// Beams over a paged cache follow their parents (kv_cache_reorder_paged).
//
// A CTA belongs to one beam.  Its first warp, a lane per beam of the group, finds out what becomes of every
// partly filled last page: the first beam that carries it on keeps it, the others copy its filled rows into their
// spare pages, and a page that no beam carries on becomes the spare of one that used its own.  Every CTA of the
// group comes to the same answer.  Then the CTA's warps copy their share of the beam's rows of all layers and
// KV heads: fill * row bytes a head, contiguous in source and destination.
//
// Bound: HBM, 2 bytes moved per byte copied (32 x 8 beams of 16-slot pages, every layer, 213 MB: 34.5 us, 6.2 TB/s); a few beams:
// latency, three dependent loads before the copy (4 beams: 3.8 us).  CTAs of one beam repeat its search, which costs
// less than a launch of its own would.
// The reference has no beams.
#include <algorithm>

#include "common.cuh"
#include "launch.h"

namespace kva {

namespace {

constexpr int THREADS = 256, WARPS = THREADS / 32;

// What becomes of one beam: its parent's number (-1: none), slots, and the copy of its last page.
struct Fate {
  int parent, len, src, dst, fill;
};

__global__ void __launch_bounds__(THREADS)
reorder_paged_kernel(const __grid_constant__ ReorderPagedArgs a) {
  __shared__ Fate s_fate;
  const int row = blockIdx.x, b = row / a.K, k = row - b * a.K;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int page = 1 << a.page_shift;
  griddep_wait();                               // inputs of this launch are complete from here on
  griddep_launch_dependents();
  if (warp == 0) {
    const bool on = lane < a.K;
    const int64_t at = (int64_t)b * a.K + lane, slots = a.table_stride << a.page_shift;
    const int parent = on ? a.parent[at] : -1;
    const int spare = on ? a.spare[at] : -1;
    const int own_len = on ? (int)min((int64_t)max(a.lengths[at], 0), slots) : 0;
    const bool own_partly = (own_len & (page - 1)) != 0;
    const int own_tail = own_partly ? a.table[at * a.table_stride + (own_len >> a.page_shift)] : -1;
    const bool valid = parent >= 0 && parent < a.K;
    const int len_p = __shfl_sync(FULL_MASK, own_len, parent & 31), tail = __shfl_sync(FULL_MASK, own_tail, parent & 31);
    const int len = valid ? len_p : 0;
    const bool partly = (len & (page - 1)) != 0;
    bool copy = false, kept = false, twice = false;
    for (int i = 0; i < a.K; ++i) {
      const int tail_i = __shfl_sync(FULL_MASK, tail, i), own_i = __shfl_sync(FULL_MASK, own_tail, i);
      const bool partly_i = __shfl_sync(FULL_MASK, (int)partly, i), own_partly_i = __shfl_sync(FULL_MASK, (int)own_partly, i);
      copy |= i < lane && partly && partly_i && tail_i == tail;
      kept |= partly_i && tail_i == own_tail;
      twice |= i < lane && own_partly_i && own_i == own_tail;
    }
    const unsigned copies = __ballot_sync(FULL_MASK, copy), frees = __ballot_sync(FULL_MASK, own_partly && !kept && !twice);
    // the n-th freed page goes to the n-th beam that copies
    const int nth = __popc(copies & ((1u << lane) - 1u));
    int from = -1, n = 0;
    for (unsigned f = frees; f != 0; f &= f - 1, ++n)
      if (n == nth) from = __ffs(f) - 1;
    const int freed = __shfl_sync(FULL_MASK, own_tail, from & 31);
    if (lane == k) {
      // a copy without a page to copy from or to: the beam loses its slots
      const bool lost = copy && ((unsigned)spare >= (unsigned)a.n_pages || (unsigned)tail >= (unsigned)a.n_pages);
      s_fate.parent = valid && !lost ? parent : -1;
      s_fate.len = len;
      s_fate.src = tail;
      s_fate.dst = spare;
      s_fate.fill = copy && !lost ? len & (page - 1) : 0;
      if (blockIdx.y == 0) {
        a.lengths_out[row] = lost ? -1 : len;
        a.spare_out[row] = copy && !lost ? (from < 0 ? -1 : freed) : spare;
      }
    }
  }
  __syncthreads();
  const Fate f = s_fate;
  if (f.parent < 0) return;
  // the table: the CTAs of a beam share it
  const int used = (int)(((int64_t)f.len + page - 1) >> a.page_shift);
  const int32_t* from = a.table + ((int64_t)b * a.K + f.parent) * a.table_stride;
  int32_t* to = a.table_out + (int64_t)row * a.table_stride;
  for (int i = blockIdx.y * THREADS + tid; i < used; i += gridDim.y * THREADS)
    to[i] = f.fill > 0 && i == used - 1 ? f.dst : from[i];
  if (f.fill == 0) return;
  // segments (layer, K or V, head), a warp each
  const int segments = a.layers * 2 * a.Hkv;
  for (int sg = blockIdx.y * WARPS + warp; sg < segments; sg += gridDim.y * WARPS) {
    const int g = sg % a.Hkv, v = sg / a.Hkv % 2, layer = sg / a.Hkv / 2;
    const int bytes = v ? a.row_v : a.row_k;
    const int64_t ps = v ? a.page_stride_v : a.page_stride;
    char* pool = static_cast<char*>(v ? a.v : a.k) + layer * (v ? a.layer_stride_v : a.layer_stride) +
                 ((int64_t)g << a.page_shift) * bytes;
    const uint4* src = reinterpret_cast<const uint4*>(pool + f.src * ps);
    uint4* dst = reinterpret_cast<uint4*>(pool + f.dst * ps);
    const int n = f.fill * bytes / 16;
    constexpr int U = 8;
    for (int i = lane; i < n; i += 32 * U) {
      uint4 x[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i + 32 * u < n) x[u] = src[i + 32 * u];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i + 32 * u < n) dst[i + 32 * u] = x[u];
    }
  }
}

constexpr int SMS = 152;          // grids are sized for the whole GPU

}  // namespace

cudaError_t launch_reorder_paged(const ReorderPagedArgs& a, cudaStream_t s) {
  const int64_t rows = (int64_t)a.B * a.K, most = ((int64_t)a.layers * 2 * a.Hkv + WARPS - 1) / WARPS;
  // about eight CTAs an SM, at most a segment a warp
  const int64_t parts = std::max<int64_t>(1, std::min<int64_t>(most, (8 * SMS + rows - 1) / rows));
  return launch_pdl(reorder_paged_kernel, dim3((unsigned)rows, (unsigned)std::min<int64_t>(parts, 65535)), dim3(THREADS), 0, s, a);
}

}  // namespace kva
