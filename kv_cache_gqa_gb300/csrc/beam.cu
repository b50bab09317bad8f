// Beam search's selection over beams and vocabulary (beam_select).
//
// A CTA takes a slice of one beam's logits in batches of 64 bytes a thread, the next batch on its way.  A thread keeps its own
// maximum, its sum of exponentials, the best of its batch maxima and the second best.  At the slice's end a warp sorts its threads'
// maxima; the n-th of them, the largest over the warps, is a bound that at least n values of the slice reach and few others do.  The
// threads that reach it read the one batch again that holds their maximum (all of theirs where the second best reaches it, too), and
// the values at or above the bound are sorted: about n to 3 n of them.  Where they do not fit a list of 1024 (rows of equal or
// sorted values), warps keep sorted lists over the whole slice instead.  The last CTA of a group joins the slices: a warp per
// beam, then a thread per offer, which counts the offers of the other beams before its own (binary searches), by totals in 64 bits
// (beams that are nearly even keep their order).
// A beam that is done, or whose score is no finite number, is not read.
//
// Sums are float32 per thread and slice, with what their additions round away where slices are joined.  Which thread takes an element
// depends on its index alone, so equal rows give equal totals.  exp(x - m) is 2^((x - m) log2 e), the difference first: it is exact for
// values near m whatever the size of both, so masked tokens at -1e10 or -1e30 are numbers like others (m log2 e, rounded before x log2 e
// is taken from it, would be off by more than float32's exponents hold).  Slices hand over (maximum, sum).  Totals are 64-bit: the value
// less the row's maximum, plus the score less the sum's logarithm (64-bit arithmetic is slow here: a logarithm takes 1.2 us).
//
// Bound: 32 x 8 beams over 151643 bf16 values by the slices' ends (30 us; 78 MB, 60% of them read, are 7 us of HBM, and the pass's
// instructions about 5; 1024 CTAs on 608 places spend 7 us each beside reading, in sorts and barriers); one sequence's 4 beams over
// 151936 float32 values by latency (12.7 us: a slice's pass, its sort, the join).
//
// The runtime's own options (HunyuanOCR v1.5 ncnn port, section 3.6) stop at top_k; it has no beams.
#include <algorithm>

#include "common.cuh"
#include "launch.h"

namespace kva {

namespace {

constexpr int THREADS = 256, WARPS = THREADS / 32;
constexpr int PER = 16;                          // values that a thread works on at a time
constexpr float LOW = -3.402823466e38f;          // a maximum of nothing (finite: no infinity minus infinity)

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
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

// 64 bytes of a row as they lie in memory (-infinity past its end), taken as GROUPS times 16 floats.
template <typename T> struct Batch {
  static constexpr int GROUPS = 4 / sizeof(T), WIDE = PER * GROUPS, WORDS = 16;     // WIDE: values
  uint32_t r[WORDS];
  // shift: the bytes of the row's start past a multiple of 16 (uniform over the CTA)
  __device__ __forceinline__ void load(const T* row, int i, int V, int shift) {
    if (shift == 0 && i + WIDE <= V) {
#pragma unroll
      for (int e = 0; e < WORDS / 4; ++e) {
        const uint4 w = __ldg(reinterpret_cast<const uint4*>(row + i) + e);
        r[4 * e] = w.x; r[4 * e + 1] = w.y; r[4 * e + 2] = w.z; r[4 * e + 3] = w.w;
      }
    } else if (shift != 0 && i > 0 && i + WIDE + 16 / (int)sizeof(T) <= V) {
      // the aligned words around them, moved down by `shift` bytes
      uint32_t w[WORDS + 4];
      const uint4* at = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(row + i) - shift);
#pragma unroll
      for (int e = 0; e < WORDS / 4 + 1; ++e) {
        const uint4 x = __ldg(at + e);
        w[4 * e] = x.x; w[4 * e + 1] = x.y; w[4 * e + 2] = x.z; w[4 * e + 3] = x.w;
      }
      if (shift & 8) {
#pragma unroll
        for (int e = 0; e < WORDS + 2; ++e) w[e] = w[e + 2];
      }
      if (shift & 4) {
#pragma unroll
        for (int e = 0; e < WORDS + 1; ++e) w[e] = w[e + 1];
      }
#pragma unroll
      for (int e = 0; e < WORDS; ++e) r[e] = sizeof(T) == 2 ? __funnelshift_r(w[e], w[e + 1], (shift & 2) * 8) : w[e];
    } else {                                       // the row's ends
#pragma unroll
      for (int e = 0; e < WORDS; ++e) {
        if constexpr (sizeof(T) == 2) {
          const uint32_t lo = i + 2 * e < V ? row[i + 2 * e].bits : 0xff80u, hi = i + 2 * e + 1 < V ? row[i + 2 * e + 1].bits : 0xff80u;
          r[e] = lo | hi << 16;
        } else {
          r[e] = i + e < V ? __float_as_uint(row[i + e]) : 0xff800000u;
        }
      }
    }
  }
  __device__ __forceinline__ void values(int g, float (&x)[PER]) const {
#pragma unroll
    for (int e = 0; e < WORDS / GROUPS; ++e) {
      const uint32_t w = r[g * (WORDS / GROUPS) + e];
      if constexpr (sizeof(T) == 2) { x[2 * e] = bf16_lo(w); x[2 * e + 1] = bf16_hi(w); }
      else x[e] = __uint_as_float(w);
    }
  }
};

// The best keys among a warp's values x of ids first + lane * PER + e into its list; last: the list's n-th (0: not full).
__device__ __forceinline__ void warp_best(const float (&x)[PER], int i0, int n, int lane, Key& list, Key& last) {
  Key left = ~0ull;                              // keys below this one are not taken yet
  for (;;) {
    Key k = 0;
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      const Key c = key_of(x[e], i0 + e);
      if (x[e] > -INFINITY && c > last && c < left && c > k) k = c;
    }
    const unsigned more = __ballot_sync(FULL_MASK, k != 0);
    if (more == 0) return;
    left = k != 0 ? k : left;
    if (__popc(more) > 4) {
      list = join(list, sort_down(k, lane), lane);
    } else {
      for (unsigned b = more; b; b &= b - 1) list = insert(list, __shfl_sync(FULL_MASK, k, __ffs(b) - 1), lane);
    }
    last = __shfl_sync(FULL_MASK, list, n - 1);
  }
}

constexpr int LIST = 1024;                       // candidates of a slice that are sorted at once

template <typename T>
__global__ void __launch_bounds__(THREADS, 4)
beam_select_kernel(const __grid_constant__ BeamArgs a) {
  __shared__ Key s_cand[LIST];
  __shared__ Key s_list[WARPS][32];
  __shared__ float s_m[WARPS], s_s[WARPS], s_bound[WARPS];
  __shared__ int s_count, s_last;
  __shared__ Key s_best[BEAM_MAX][33];             // a beam's offers
  __shared__ Key s_total[BEAM_MAX][33];            // and their totals, ordered as whole numbers (0: no offer)
  const int row = blockIdx.y, split = blockIdx.x, b = row / a.K;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, n = a.n;
  griddep_wait();                               // inputs of this launch are complete from here on
  griddep_launch_dependents();
  const float score = a.scores[row];
  const bool done = a.finished != nullptr && a.finished[row] != 0;
  if (!done && fabsf(score) < INFINITY) {
    const T* z = reinterpret_cast<const T*>(a.logits) + (int64_t)row * a.row_stride;
    const int shift = (int)(reinterpret_cast<uintptr_t>(z) & 15u);
    using Part = Batch<T>;
    constexpr int BATCH = THREADS * Part::WIDE;
    const int batches = (a.V + BATCH - 1) / BATCH;
    const int b0 = (int)((int64_t)batches * split / gridDim.x), b1 = (int)((int64_t)batches * (split + 1) / gridDim.x);
    if (tid == 0) s_count = 0;
    float m = LOW, s = 0.f;                        // the maximum, and the sum of exp(x - m)
    float best = -INFINITY, second = -INFINITY;    // of the batches' maxima
    int best_at = b0;
    Part next;
    if (b0 < b1) next.load(z, b0 * BATCH + tid * Part::WIDE, a.V, shift);
    for (int bt = b0; bt < b1; ++bt) {
      const Part now = next;
      if (bt + 1 < b1) next.load(z, (bt + 1) * BATCH + tid * Part::WIDE, a.V, shift);
      float high = -INFINITY;
#pragma unroll
      for (int g = 0; g < Part::GROUPS; ++g) {
        float x[PER];
        now.values(g, x);
        float top = fmaxf(x[0], x[1]);
#pragma unroll
        for (int e = 2; e < PER; e += 2) top = fmax3(top, x[e], x[e + 1]);
        high = fmaxf(high, top);
        if (top > m) {
          s *= ex2((m - top) * LOG2E);
          m = top;
        }
        const uint64_t l2 = pack_f32x2(LOG2E, LOG2E), m2 = pack_f32x2(-m, -m);
        uint64_t sum = 0ull;
#pragma unroll
        for (int e = 0; e < PER; e += 2) {
          const uint64_t t = mul_f32x2(add_f32x2(pack_f32x2(x[e], x[e + 1]), m2), l2);
          sum = add_f32x2(sum, pack_f32x2(ex2(f32x2_lo(t)), ex2(f32x2_hi(t))));
        }
        s += f32x2_lo(sum) + f32x2_hi(sum);
      }
      if (high > best) { second = best; best = high; best_at = bt; }
      else second = fmaxf(second, high);
    }
    // the warp's sums, and its n-th best maximum of a thread
    float M = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(FULL_MASK, M, o));
    s *= ex2((m - M) * LOG2E);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(FULL_MASK, s, o);
    float ordered = best;
#pragma unroll
    for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
      for (int o = size >> 1; o > 0; o >>= 1) {
        const float other = __shfl_xor_sync(FULL_MASK, ordered, o);
        ordered = ((lane & o) == 0) == ((lane & size) == 0) ? fmaxf(ordered, other) : fminf(ordered, other);
      }
    ordered = __shfl_sync(FULL_MASK, ordered, n - 1);
    if (lane == 0) { s_m[warp] = M; s_s[warp] = s; s_bound[warp] = ordered; }
    __syncthreads();
    float bound = s_bound[0];
#pragma unroll
    for (int w = 1; w < WARPS; ++w) bound = fmaxf(bound, s_bound[w]);
    // the values that reach it
    if (best >= bound && best > -INFINITY) {
      const bool all = second >= bound && second > -INFINITY;
      for (int bt = all ? b0 : best_at; bt < (all ? b1 : best_at + 1); ++bt) {
        const int i0 = bt * BATCH + tid * Part::WIDE;
        next.load(z, i0, a.V, shift);
        uint32_t hits = 0u;
#pragma unroll
        for (int g = 0; g < Part::GROUPS; ++g) {
          float x[PER];
          next.values(g, x);
#pragma unroll
          for (int e = 0; e < PER; ++e) hits |= (x[e] >= bound && x[e] > -INFINITY ? 1u : 0u) << (g * PER + e);
        }
        for (; hits; hits &= hits - 1) {
          const int id = i0 + __ffs(hits) - 1, at = atomicAdd(&s_count, 1);
          if (at < LIST) s_cand[at] = key_of(load1(z + id), id);
        }
      }
    }
    __syncthreads();
    const int count = s_count;
    Key list = 0, last = 0;
    if (count <= LIST) {
      for (int i = warp * 32; i < count; i += THREADS) {
        const Key k = i + lane < count ? s_cand[i + lane] : 0;
        list = join(list, sort_down(k, lane), lane);
      }
    } else {
      for (int bt = b0; bt < b1; ++bt) {
        const int i0 = bt * BATCH + tid * Part::WIDE;
        next.load(z, i0, a.V, shift);
#pragma unroll 1
        for (int g = 0; g < Part::GROUPS; ++g) {
          float x[PER];
          if (g == 0) next.values(0, x);
          else next.values(Part::GROUPS - 1, x);
          warp_best(x, i0 + g * PER, n, lane, list, last);
        }
      }
    }
    s_list[warp][lane] = lane < n ? list : 0;
    __syncthreads();
    if (warp == 0) {
      const int lists = count <= LIST ? min(WARPS, (count + 31) / 32) : WARPS;
      Key k = s_list[0][lane];
      for (int w = 1; w < lists; ++w) k = join(k, s_list[w][lane], lane);
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
    Key list = 0, last = 0;
    double base = NAN;                               // an offer's total is (value - top) + base
    float top = 0.f;
    const bool finite = fabsf(sc) < INFINITY;        // else it offers nothing
    if (finite && is_done) {
      base = (double)sc;
      if (lane == 0) list = key_of(0.f, a.end_id);
    } else if (finite) {
      const int64_t part = (int64_t)r * gridDim.x;
      const int keys = (int)gridDim.x * n;
      constexpr int KPL = 12;                        // keys of a lane at a time
      Key ahead[KPL];
      auto fetch = [&](int i0) {
#pragma unroll
        for (int u = 0; u < KPL; ++u) {
          const int i = i0 + u * 32 + lane;
          ahead[u] = i < keys ? __ldcg(a.part_key + part * n + i) : 0;
        }
      };
      fetch(0);
      float M = -INFINITY;                           // the row's maximum
      bool odd = false;
      for (int i = lane; i < (int)gridDim.x; i += 32) {
        const float2 st = __ldcg(reinterpret_cast<const float2*>(a.part_stat) + part + i);
        odd |= !(st.y < INFINITY);
        if (st.y > 0.f) M = fmaxf(M, st.x);          // a slice of -infinity alone has the sum 0
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(FULL_MASK, M, o));
      float S = 0.f, rest = 0.f;                     // a sum and what its additions rounded away
      auto add = [&](float y, float more) {
        const float t = S + y, u = t - S;
        rest += (S - (t - u)) + (y - u) + more;
        S = t;
      };
      for (int i = lane; i < (int)gridDim.x; i += 32) {
        const float2 st = __ldcg(reinterpret_cast<const float2*>(a.part_stat) + part + i);
        if (st.y > 0.f) add(st.y * ex2((st.x - M) * LOG2E), 0.f);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) add(__shfl_xor_sync(FULL_MASK, S, o), __shfl_xor_sync(FULL_MASK, rest, o));
      odd = __any_sync(FULL_MASK, odd);
      if (!odd && S > 0.f) {                         // neither a row of -infinity, nor one with NaN or +infinity
        base = (double)sc - log((double)S + (double)rest);
        top = M;
        for (int i0 = 0; i0 < keys; i0 += 32 * KPL) {
          if (i0 > 0) fetch(i0);
          Key left = ~0ull;                          // keys below this one are not taken yet
          for (;;) {
            Key best = 0;
#pragma unroll
            for (int u = 0; u < KPL; ++u)
              if (ahead[u] > last && ahead[u] < left && ahead[u] > best) best = ahead[u];
            const unsigned more = __ballot_sync(FULL_MASK, best != 0);
            if (more == 0) break;
            left = best != 0 ? best : left;
            if (__popc(more) > 4) {
              list = join(list, sort_down(best, lane), lane);
            } else {
              for (unsigned x = more; x; x &= x - 1) list = insert(list, __shfl_sync(FULL_MASK, best, __ffs(x) - 1), lane);
            }
            last = __shfl_sync(FULL_MASK, list, n - 1);
          }
        }
      }
    }
    if (lane >= n) list = 0;
    Key total = 0;
    if (list != 0 && base == base) {
      const double v = ((double)key_value(list) - (double)top) + base;       // the difference first: both may be huge
      const unsigned long long bits = (unsigned long long)__double_as_longlong(v + 0.0);
      if (v > -INFINITY) total = bits >> 63 ? ~bits : bits | (1ull << 63);
    }
    s_best[k][lane] = list;
    s_total[k][lane] = total;
  }
  __syncthreads();
  // a thread per offer: its place is the number of offers before it
  int offers = 0;
  for (int k = 0; k < a.K; ++k) {                   // how many there are, by binary search for the first 0
    int lo = 0, hi = n;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (s_total[k][mid] != 0) lo = mid + 1; else hi = mid;
    }
    offers += lo;
  }
  for (int i = tid; i < a.K * n; i += THREADS) {
    const int k = i / n, j = i - k * n;
    const Key total = s_total[k][j];
    if (total == 0) continue;
    int place = j;
    for (int q = 0; q < a.K && place < n; ++q) {
      if (q == k) continue;
      int lo = 0, hi = n;                           // offers of beam q before this one: larger, or equal and of a lower beam
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        const Key t = s_total[q][mid];
        if (t > total || (t == total && q < k)) lo = mid + 1; else hi = mid;
      }
      place += lo;
    }
    if (place >= n) continue;
    const int64_t o = (int64_t)b * n + place;
    a.out_beam[o] = k;
    a.out_token[o] = key_id(s_best[k][j]);
    const unsigned long long bits = total >> 63 ? total & ~(1ull << 63) : ~total;
    a.out_score[o] = (float)__longlong_as_double((long long)bits);
  }
  if (tid >= offers && tid < n) {
    const int64_t o = (int64_t)b * n + tid;
    a.out_beam[o] = -1;
    a.out_token[o] = -1;
    a.out_score[o] = -INFINITY;
  }
  if (tid == 0) a.counters[b] = 0u;
}

constexpr int SMS = 152;          // grids are sized for the whole GPU

}  // namespace

// Slices of a row: about six CTAs an SM over all rows, a batch of float32 values each at least.  A CTA spends about 7 us beside reading,
// which others' reading should cover: 32 x 8 beams, 40% of them done, took 41 / 33.5 / 34 / 38.5 us with 3 / 6 / 8 / 12.
int beam_splits(int rows, int V) {
  const int batches = (V + THREADS * PER - 1) / (THREADS * PER);
  return std::max(1, std::min(batches, (6 * SMS + rows - 1) / rows));
}
int beam_parts_bound(int rows) { return 6 * SMS + rows; }

cudaError_t launch_beam_select(const BeamArgs& a, kva_dtype dtype, cudaStream_t s) {
  const dim3 grid(a.splits, a.B * a.K);
  if (dtype == KVA_BF16) return launch_pdl(beam_select_kernel<bf16_t>, grid, dim3(THREADS), 0, s, a);
  return launch_pdl(beam_select_kernel<float>, grid, dim3(THREADS), 0, s, a);
}

}  // namespace kva
