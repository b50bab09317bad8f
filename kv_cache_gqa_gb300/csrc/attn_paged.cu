// Plan of kv_attn_paged: which kernels a batch needs and how many runs each gets.
#include <algorithm>
#include <cmath>
#include <mutex>

#include "launch.h"

namespace kva {

namespace {

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

// Steps and units of the sequences of lo < T * G <= hi rows, in tiles of `tile` rows and steps of `keys` slots.
struct Load {
  int64_t steps = 0, units = 0;
};
Load load_of(const PagedArgs& a, const int32_t* lengths, const int32_t* start, int64_t lo, int64_t hi, int tile, int keys) {
  const int G = a.Hq / a.Hkv;
  Load w;
  for (int b = 0; b < a.B; ++b) {
    const int64_t rows = (int64_t)(start[b + 1] - start[b]) * G;
    if (rows <= lo || rows > hi) continue;
    const int64_t n = (rows + tile - 1) / tile * a.Hkv;
    w.units += n;
    w.steps += n * std::max(1, (lengths[b] + keys - 1) / keys);
  }
  return w;
}

// As many runs as the GPU holds at once, and not so many that joining a unit's parts costs more than its steps: `worth` is the
// square root of a step's time over a part's, doubled (one sequence of 768 slots in float32: 2 gives 18.9 us, 4 14.6).  A whole number of
// runs a unit, where there are four of them or more: units of equal length (one sequence's heads) then begin with a run each
// (one sequence of 768 slots: 13.0 us, so 10.5).
int runs_of(const Load& w, int slots, double worth = 2.0) {
  const int64_t most = std::min<int64_t>(slots, (int64_t)(worth * std::sqrt((double)w.steps * (double)w.units)));
  const int64_t runs = std::max<int64_t>(1, std::min(most, w.steps));
  return (int)(runs >= 4 * w.units ? runs / w.units * w.units : runs);
}

}  // namespace

bool attn_paged_supports(int Dk, int Dv) {
  return (Dk == 64 && Dv == 64) || (Dk == 128 && Dv == 128) || (Dk == 192 && Dv == 128);
}

// A bf16 pool as (width, slot of a page, KV head, page): boxes of [rows x 64 columns] with 128-byte swizzle.
cudaError_t paged_pool_map(CUtensorMap* map, const void* base, const PagedArgs& a, int width, int64_t page_stride, int rows) {
  const EncodeTiledFn fn = encode_fn();
  if (!fn) return cudaErrorNotSupported;
  const cuuint64_t page = 1u << a.page_shift;
  const cuuint64_t dims[4] = {(cuuint64_t)width, page, (cuuint64_t)a.Hkv, (cuuint64_t)a.n_pages};
  const cuuint64_t strides[3] = {(cuuint64_t)width * 2, page * width * 2, (cuuint64_t)page_stride * 2};
  const cuuint32_t box[4] = {64, (cuuint32_t)rows, 1, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// The queries as (width, head, token): boxes of [tokens x heads x 64 columns], rows in (token, head) order.
cudaError_t paged_query_map(CUtensorMap* map, const PagedArgs& a, int width, int heads, int tokens) {
  const EncodeTiledFn fn = encode_fn();
  if (!fn) return cudaErrorNotSupported;
  const cuuint64_t dims[4] = {(cuuint64_t)width, (cuuint64_t)a.Hq, (cuuint64_t)a.T, 1};
  const cuuint64_t row = (cuuint64_t)width * 2;
  const cuuint64_t strides[3] = {row, row * a.Hq, row * a.Hq * a.T};
  const cuuint32_t box[4] = {64, (cuuint32_t)heads, (cuuint32_t)tokens, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(a.q), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// float32 caches: CUDA cores.  bf16 caches: mma.sync tiles of 16 rows for sequences of up to 16 rows a KV head (all of them with
// the same bits, however many rows the batch's others have), and for all of
// them where the output is float32 (the only form that holds its weights and sums to 24 bits); tcgen05 for the others.
cudaError_t launch_attn_paged(const PagedArgs& args, int Dk, int Dv, kva_dtype dtype, const int32_t* lengths,
                              const int32_t* start, cudaStream_t s, unsigned* n_launches) {
  PagedArgs a = args;
  const int G = a.Hq / a.Hkv;
  cudaError_t e = cudaSuccess;
  a.rows_lo = 0;
  a.rows_hi = INT32_MAX;
  if (dtype == KVA_F32) {
    int rows = 0;
    for (int b = 0; b < a.B; ++b) rows = std::max(rows, std::min(start[b + 1] - start[b], PAGED_ROWS) * G);
    const Load w = load_of(a, lengths, start, 0, INT32_MAX, PAGED_ROWS, 128);
    e = launch_attn_paged_simt(a, Dk, rows, runs_of(w, PAGED_SMS * (Dk == 64 ? 2 : 1), 4.0), s);
    if (e == cudaSuccess) ++*n_launches;
    return e;
  }
  if (a.out_bf16) a.rows_hi = PAGED_ROWS;
  int rows = 0;                                  // the most rows of a sequence in the class
  Load more;
  for (int b = 0; b < a.B; ++b) {
    const int T = start[b + 1] - start[b];
    if ((int64_t)T * G <= a.rows_hi) rows = std::max(rows, T * G);
    else attn_paged_chunk_load(T, lengths[b], G, &more.steps, &more.units);
  }
  if (rows > 0) {
    const Load w = load_of(a, lengths, start, 0, a.rows_hi, PAGED_ROWS, 64);
    e = launch_attn_paged_step(a, Dk, rows, runs_of(w, PAGED_SMS * 2), s);
    if (e != cudaSuccess) return e;
    ++*n_launches;
  }
  if (more.units > 0) {
    more.steps *= a.Hkv;
    more.units *= a.Hkv;
    a.rows_lo = PAGED_ROWS;
    a.rows_hi = INT32_MAX;
    e = launch_attn_paged_chunk(a, Dk, Dv, runs_of(more, PAGED_SMS), s, n_launches);
  }
  return e;
}

}  // namespace kva
