// Beam search's selection over beams and vocabulary (beam_select).
//
// A CTA takes a slice of one beam's logits.  A lane keeps its own running maximum and sum of exponentials; a warp
// keeps the best n of its logits as sorted 64-bit keys, a lane each (value, then lower id first), against whose
// last one a batch of 16 values a lane is checked by its maximum alone.  A batch with many better values (the first
// one) is sorted in lane maxima at a time, one with few inserts them one by one.  The CTA joins its warps' lists and
// sums and writes them; the last CTA of a group joins the slices: a warp per beam, then the best n of the beams'
// sorted lists, a lane per beam, by totals in 64 bits (beams that are nearly even keep their order).
// A beam that is done, or whose score is -infinity, is not read.
//
// Sums are float32 per lane and slice, 64 bits where they are joined.  Which lane takes an element depends on its index
// alone, so equal rows give equal totals.  x - m is exact or nearly so where its exponential counts, which
// x * log2 e - m * log2 e is not.
//
// The runtime's own options (HunyuanOCR v1.5 ncnn port, section 3.6) stop at top_k; it has no beams.
#include <algorithm>

#include "common.cuh"
#include "launch.h"

namespace kva {

namespace {

constexpr int THREADS = 256, WARPS = THREADS / 32;
constexpr int PER = 16;                          // values of a lane in a batch
constexpr int BATCH = THREADS * PER;             // of a CTA
constexpr float LOW = -3.402823466e38f;          // a maximum of nothing (finite: no infinity minus infinity)

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

using Key = unsigned long long;
__device__ __forceinline__ Key key_of(float v, int id) { return argmax_key(v, (uint32_t)id); }
__device__ __forceinline__ float key_value(Key k) { return float_from_order_bits((uint32_t)(k >> 32)); }
__device__ __forceinline__ int key_id(Key k) { return (int)(0xffffffffu - (uint32_t)k); }
__device__ __forceinline__ Key key_max(Key a, Key b) { return a > b ? a : b; }
__device__ __forceinline__ Key key_min(Key a, Key b) { return a < b ? a : b; }

// A warp's keys, descending from lane 0.
__device__ __forceinline__ Key sort_down(Key k, int lane) {
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
    for (int o = size >> 1; o > 0; o >>= 1) {
      const Key other = __shfl_xor_sync(FULL_MASK, k, o);
      const bool first = (lane & o) == 0, down = (lane & size) == 0;
      k = first == down ? key_max(k, other) : key_min(k, other);
    }
  return k;
}
// The best 32 of two descending lists.
__device__ __forceinline__ Key join(Key list, Key more, int lane) {
  Key k = key_max(list, __shfl_sync(FULL_MASK, more, 31 - lane));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const Key other = __shfl_xor_sync(FULL_MASK, k, o);
    k = (lane & o) == 0 ? key_max(k, other) : key_min(k, other);
  }
  return k;
}
__device__ __forceinline__ Key insert(Key list, Key k, int lane) {      // k: the same in all lanes
  const int at = __popc(__ballot_sync(FULL_MASK, list > k));
  const Key up = __shfl_up_sync(FULL_MASK, list, 1);
  return lane < at ? list : (lane == at ? k : up);
}

// 16 values from index i on of a row of V values (-infinity past its end).
template <typename T>
__device__ __forceinline__ void load_values(const T* row, int i, int V, bool aligned, float (&x)[PER]) {
  if (aligned && i + PER <= V) {
#pragma unroll
    for (int e = 0; e < PER; e += 8) {
      float y[8];
      load8(row + i + e, y);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[e + j] = y[j];
    }
  } else {
#pragma unroll
    for (int e = 0; e < PER; ++e) x[e] = i + e < V ? load1(row + i + e) : -INFINITY;
  }
}

template <typename T>
__global__ void __launch_bounds__(THREADS)
beam_select_kernel(const __grid_constant__ BeamArgs a) {
  __shared__ Key s_list[WARPS][32];
  __shared__ float s_m[WARPS], s_s[WARPS];
  __shared__ int s_last;
  __shared__ double s_base[BEAM_MAX], s_top[BEAM_MAX];   // score - log sum of a beam (NaN: it offers nothing), its maximum
  __shared__ Key s_best[BEAM_MAX][33];
  const int row = blockIdx.y, split = blockIdx.x, b = row / a.K;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, n = a.n;
  griddep_wait();                               // inputs of this launch are complete from here on
  griddep_launch_dependents();
  const float score = a.scores[row];
  const bool done = a.finished != nullptr && a.finished[row] != 0;
  if (!done && score > -INFINITY) {
    const T* z = reinterpret_cast<const T*>(a.logits) + (int64_t)row * a.row_stride;
    const bool aligned = (reinterpret_cast<uintptr_t>(z) & 15u) == 0;
    const int batches = (a.V + BATCH - 1) / BATCH;
    const int b0 = (int)((int64_t)batches * split / gridDim.x), b1 = (int)((int64_t)batches * (split + 1) / gridDim.x);
    float m = LOW, s = 0.f;
    Key list = 0, last = 0;                        // last: the list's n-th (0: not full)
    float thr = -INFINITY;                         // its value
    auto renew = [&]() {
      last = __shfl_sync(FULL_MASK, list, n - 1);
      thr = last ? key_value(last) : -INFINITY;
    };
    for (int bt = b0; bt < b1; ++bt) {
      float x[PER];
      const int i0 = bt * BATCH + tid * PER;
      load_values(z, i0, a.V, aligned, x);
      float top = x[0];
#pragma unroll
      for (int e = 1; e < PER; ++e) top = fmaxf(top, x[e]);
      if (top > m) { s *= ex2((m - top) * LOG2E); m = top; }
#pragma unroll
      for (int e = 0; e < PER; ++e) s += ex2((x[e] - m) * LOG2E);
      // a warp's ids grow from batch to batch: a later value equal to the n-th is not better
      unsigned better = __ballot_sync(FULL_MASK, top > thr);
      if (better == 0) continue;
      if (__popc(better) > 4) {
        // lane maxima, sorted, until none of what is left is better than the list's n-th
        Key left = ~0ull;                          // keys below this one are not taken yet
        for (;;) {
          Key k = 0;
#pragma unroll
          for (int e = 0; e < PER; ++e) {
            const Key c = key_of(x[e], i0 + e);
            if (x[e] >= thr && x[e] > -INFINITY && c > last && c < left && c > k) k = c;
          }
          if (__ballot_sync(FULL_MASK, k != 0) == 0) break;
          left = k != 0 ? k : left;
          list = join(list, sort_down(k, lane), lane);
          renew();
        }
      } else {
        for (; better; better &= better - 1) {
          const int src = __ffs(better) - 1;
#pragma unroll
          for (int e = 0; e < PER; ++e) {
            const float v = __shfl_sync(FULL_MASK, x[e], src);
            const Key k = key_of(v, bt * BATCH + (tid - lane + src) * PER + e);
            if (v >= thr && k > last && v > -INFINITY) {
              list = insert(list, k, lane);
              renew();
            }
          }
        }
      }
    }
    // the warp's sums, then the CTA's
    float M = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(FULL_MASK, M, o));
    s *= ex2((m - M) * LOG2E);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(FULL_MASK, s, o);
    if (lane == 0) { s_m[warp] = M; s_s[warp] = s; }
    s_list[warp][lane] = lane < n ? list : 0;
    __syncthreads();
    if (warp == 0) {
      Key k = s_list[0][lane];
      for (int w = 1; w < WARPS; ++w) k = join(k, s_list[w][lane], lane);
      const int64_t part = (int64_t)row * gridDim.x + split;
      if (lane < n) a.part_key[part * n + lane] = k;
      if (lane == 0) {
        float CM = LOW, S = 0.f;
        for (int w = 0; w < WARPS; ++w) CM = fmaxf(CM, s_m[w]);
        for (int w = 0; w < WARPS; ++w) S = fmaf(s_s[w], ex2((s_m[w] - CM) * LOG2E), S);
        a.part_stat[2 * part] = CM;
        a.part_stat[2 * part + 1] = S;
      }
    }
  }
  // the group's last CTA joins
  __threadfence();
  __syncthreads();
  if (tid == 0) s_last = atomicAdd(a.counters + b, 1u) == gridDim.x * a.K - 1u;
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  for (int k = warp; k < a.K; k += WARPS) {
    const int r = b * a.K + k;
    const float sc = a.scores[r];
    const bool is_done = a.finished != nullptr && a.finished[r] != 0;
    Key list = 0;
    double base = NAN, top = 0.0;
    if (is_done) {
      base = (double)sc;
      if (lane == 0) list = key_of(0.f, a.end_id);
    } else if (sc > -INFINITY) {
      const int64_t part = (int64_t)r * gridDim.x;
      float M = LOW;
      for (int i = lane; i < (int)gridDim.x; i += 32) M = fmaxf(M, __ldcg(a.part_stat + 2 * (part + i)));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(FULL_MASK, M, o));
      double S = 0.0;
      for (int i = lane; i < (int)gridDim.x; i += 32) {
        const float2 st = __ldcg(reinterpret_cast<const float2*>(a.part_stat) + part + i);
        S += (double)st.y * exp((double)st.x - (double)M);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) S += __shfl_xor_sync(FULL_MASK, S, o);
      const bool good = S > 0.0 && S < 1e300;      // not a row of -infinity, nor one with NaN or +infinity
      if (good) {
        base = (double)sc - log(S);
        top = (double)M;
        Key thr = 0;
        for (int j = 0; j < n; ++j) {              // all slices' best, then their second best, ...
          bool any = false;
          for (int i0 = 0; i0 < (int)gridDim.x; i0 += 32) {
            Key c = i0 + lane < (int)gridDim.x ? __ldcg(a.part_key + (part + i0 + lane) * n + j) : 0;
            if (c <= thr) c = 0;
            unsigned better = __ballot_sync(FULL_MASK, c != 0);
            any |= better != 0;
            if (__popc(better) > 4) {
              list = join(list, sort_down(c, lane), lane);
            } else {
              for (; better; better &= better - 1) list = insert(list, __shfl_sync(FULL_MASK, c, __ffs(better) - 1), lane);
            }
            thr = __shfl_sync(FULL_MASK, list, n - 1);
          }
          if (!any) break;
        }
      }
    }
    s_best[k][lane] = lane < n ? list : 0;
    if (lane == 0) { s_base[k] = base; s_top[k] = top; }
  }
  __syncthreads();
  if (warp != 0) return;
  // a lane per beam with its list's head; n times the best of them, the lower beam among equals
  int at = 0;
  const bool beam = lane < a.K;
  const double base = beam ? s_base[lane] : NAN, top = beam ? s_top[lane] : 0.0;   // done: a value of 0, less 0
  for (int j = 0; j < n; ++j) {
    const Key head = beam && at < 32 ? s_best[lane][at] : 0;
    double total = -INFINITY;
    if (head != 0 && base == base) total = ((double)key_value(head) - top) + base;   // the difference first: both may be huge
    double best = total;
    int who = lane;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const double t = __shfl_xor_sync(FULL_MASK, best, o);
      const int w = __shfl_xor_sync(FULL_MASK, who, o);
      if (t > best || (t == best && w < who)) { best = t; who = w; }
    }
    const int id = __shfl_sync(FULL_MASK, key_id(head), who);
    if (lane == who) ++at;
    if (lane == 0) {
      const bool none = !(best > -INFINITY);
      const int64_t o = (int64_t)b * n + j;
      a.out_beam[o] = none ? -1 : who;
      a.out_token[o] = none ? -1 : id;
      a.out_score[o] = none ? -INFINITY : (float)best;
    }
  }
  if (lane == 0) a.counters[b] = 0u;
}

constexpr int SMS = 152;          // grids are sized for the whole GPU

}  // namespace

// Slices of a row: about four CTAs an SM over all rows, a batch each at least.
int beam_splits(int rows, int V) {
  const int batches = (V + BATCH - 1) / BATCH;
  return std::max(1, std::min(batches, (4 * SMS + rows - 1) / rows));
}
int beam_parts_bound(int rows) { return 4 * SMS + rows; }

cudaError_t launch_beam_select(const BeamArgs& a, kva_dtype dtype, cudaStream_t s) {
  const dim3 grid(a.splits, a.B * a.K);
  if (dtype == KVA_BF16) return launch_pdl(beam_select_kernel<bf16_t>, grid, dim3(THREADS), 0, s, a);
  return launch_pdl(beam_select_kernel<float>, grid, dim3(THREADS), 0, s, a);
}

}  // namespace kva
