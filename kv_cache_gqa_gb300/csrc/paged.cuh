// What the kernels over a paged cache share: a sequence's numbers, the cut of all work into equal
// runs, and the join of a CTA's warps and of the CTAs that share a unit.
#pragma once

#include "common.cuh"
#include "launch.h"

namespace kva {
namespace paged {

// A reference maximum below every score (finite: differences of two of them are 0, not NaN).
constexpr float M_NONE = -3.402823466e38f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A pair of bf16 numbers, its NaNs and infinities as zeros.
__device__ __forceinline__ uint32_t finite_pair(uint32_t w) {
  if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
  if ((w & 0x7f800000u) == 0x7f800000u) w &= 0xffffu;
  return w;
}
// Notes in `seen` (0 at first) whether one of a pair is NaN or infinite: an exponent of ones carries into bit 15 or 31.
__device__ __forceinline__ void see_pair(uint32_t& seen, uint32_t w) { seen |= (w & 0x7f807f80u) + 0x00800080u; }
__device__ __forceinline__ bool saw_odd(uint32_t seen) { return (seen & 0x80008000u) != 0u; }

// A whole warp waits for the phase of this parity, up to WAIT_LIMIT_NS; false if it gave up.  With a hint the hardware suspends
// the warp for up to so many nanoseconds and wakes it when the phase ends.  Without, it looks again every few hundred cycles,
// and the issue slots that takes were the softmax warps' (a 2048-token chunk behind 30000 slots: 821 us, with the hint 680).
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  constexpr uint32_t HINT_NS = 1000000;
  uint64_t t0 = 0;
  for (;;) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n"
        " mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2, %3;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity), "r"(HINT_NS) : "memory");
    if (__all_sync(FULL_MASK, ok != 0)) return true;
    const uint64_t now = global_timer_ns();
    if (t0 == 0) t0 = now;
    if (__any_sync(FULL_MASK, now - t0 > WAIT_LIMIT_NS)) {
      atomicAdd(&g_wait_timeouts, 1u);
      return false;
    }
  }
}

// New tokens [t0, t0 + T) of sequence b and its L slots, forced into the buffers' bounds: a device copy that
// disagrees with its host mirror gives other results, but no access outside.
struct Seq {
  int t0, T, L;
};
__device__ __forceinline__ Seq sequence(const PagedArgs& a, int b) {
  Seq s;
  s.t0 = min(max(a.start[b], 0), a.T);
  s.T = max(min(a.start[b + 1], a.T) - s.t0, 0);
  s.L = (int)min((int64_t)max(a.lengths[b], 0), a.slots);
  return s;
}

// Units of a class of sequences: (sequence, KV head, tile of R query rows), rows being (token, query head of
// the group) with the heads fastest; a unit's work is its key steps of KEYS slots (one at least: rows that
// see nothing still get their zeros).  All steps, in the order (sequence, head, tile, step), are cut
// into equal runs, one for each CTA; CTAs beyond the number of steps have none (no run is empty).
struct Cut {
  int R, KEYS, G, lo, hi;                         // sequences of lo < T * G <= hi rows
  __device__ __forceinline__ int tiles(const Seq& s) const {
    const int64_t rows = (int64_t)s.T * G;
    return rows > lo && rows <= hi ? (int)((rows + R - 1) / R) : 0;
  }
  // slots that tile rt's last row sees (its other rows see no more)
  __device__ __forceinline__ int visible(const Seq& s, int rt) const {
    const int last = (int)((min((int64_t)s.T * G, (int64_t)(rt + 1) * R) - 1) / G);
    return min(max(s.L - s.T + last + 1, 0), s.L);
  }
  __device__ __forceinline__ int steps(const Seq& s, int rt) const { return max(1, (visible(s, rt) + KEYS - 1) / KEYS); }
  __device__ __forceinline__ int64_t head_steps(const Seq& s) const {
    const int n = tiles(s);
    int64_t sum = 0;
    for (int rt = 0; rt < n; ++rt) sum += steps(s, rt);
    return sum;
  }
};

// The place in the order of all steps: the unit and the global number of its first step.
struct Place {
  int b, g, rt, n_tiles, n_steps;
  int64_t at;
  Seq s;
  template <typename C>
  __device__ __forceinline__ void next(const PagedArgs& a, const C& c) {
    at += n_steps;
    if (++rt == n_tiles) {
      rt = 0;
      if (++g == a.Hkv) {
        g = 0;
        do {
          if (++b >= a.B) return;
          s = sequence(a, b);
          n_tiles = c.tiles(s);
        } while (n_tiles == 0);
      }
    }
    n_steps = c.steps(s, rt);
  }
};

// Quotients of numbers that mostly fit 32 bits (a division of 64 takes some hundred cycles).
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {
  return (a | b) >> 32 == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// All steps, their runs, and this CTA's run [x0, x1).
struct Run {
  int64_t total, x0, x1;
  int runs;
  __device__ __forceinline__ int64_t start_of(int c) const { return divide(total * c, runs); }
  __device__ __forceinline__ int of(int64_t x) const { return (int)divide((x + 1) * runs - 1, total); }
};

// This CTA's run and the place of its first step (none: x0 = x1).  Whole CTA; scratch: THREADS / 32 + 4 words.
template <int THREADS, typename C>
__device__ __forceinline__ Run first_place(const PagedArgs& a, const C& c, int64_t* scratch, Place* p) {
  constexpr int W = THREADS / 32;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // sum of all sequences, kept per thread for a batch of up to THREADS of them
  __shared__ Seq s_seq;
  int64_t mine = 0, first = 0;
  Seq kept{};
  for (int b = tid; b < a.B; b += THREADS) {
    const Seq seq = sequence(a, b);
    const int64_t n = c.head_steps(seq) * a.Hkv;
    if (b == tid) { first = n; kept = seq; }
    mine += n;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(FULL_MASK, mine, o);
  if (lane == 0) scratch[warp] = mine;
  __syncthreads();
  int64_t total = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) total += scratch[w];
  Run run;
  run.total = total;
  run.runs = (int)min((int64_t)gridDim.x, total);
  run.x0 = run.x1 = 0;
  if ((int)blockIdx.x < run.runs) {
    run.x0 = run.start_of(blockIdx.x);
    run.x1 = run.start_of(blockIdx.x + 1);
  }
  p->at = 0;
  p->b = a.B;
  if (run.x0 >= run.x1) return run;               // uniform over the CTA
  const int64_t x0 = run.x0;
  // the sequence that holds step x0: prefix sums, THREADS sequences at a time
  int64_t base = 0;
  for (int b0 = 0; b0 < a.B; b0 += THREADS) {
    const int b = b0 + tid;
    if (b0 > 0) {
      first = 0;
      if (b < a.B) {
        kept = sequence(a, b);
        first = c.head_steps(kept) * a.Hkv;
      }
    }
    const int64_t n = first;
    int64_t upto = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(FULL_MASK, upto, o);
      if (lane >= o) upto += v;
    }
    __syncthreads();
    if (lane == 31) scratch[warp] = upto;
    __syncthreads();
    int64_t before = base, all = base;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      if (w < warp) before += scratch[w];
      all += scratch[w];
    }
    const int64_t lo = before + upto - n;
    if (b < a.B && x0 >= lo && x0 < lo + n) { scratch[W] = lo; scratch[W + 1] = b; s_seq = kept; }
    base = all;
    if (x0 < all) break;                          // uniform
  }
  __syncthreads();
  p->b = (int)scratch[W + 1];
  p->s = s_seq;
  p->n_tiles = c.tiles(p->s);
  const int64_t head = c.head_steps(p->s), in = x0 - scratch[W];
  p->g = (int)divide(in, head);
  int64_t rest = in - p->g * head;
  p->rt = 0;
  p->n_steps = c.steps(p->s, 0);
  while (rest >= p->n_steps) {
    rest -= p->n_steps;
    p->n_steps = c.steps(p->s, ++p->rt);
  }
  p->at = x0 - rest;
  return run;
}

__device__ __forceinline__ void store_out(const PagedArgs& a, int64_t row, int d, float v) {
  if (a.out_bf16) reinterpret_cast<uint16_t*>(a.out)[row + d] = (uint16_t)f32_to_bf16_rne(v);
  else reinterpret_cast<float*>(a.out)[row + d] = v;
}

// The end of a unit (or of a run's part of it): warps' (max, sum, O) of R rows in shared memory, sm = [W][R] max,
// [W][R] sum, [W][R][DV] O.  A CTA that holds the whole unit writes the rows; else it writes a part, and the
// last CTA of the unit to come joins the parts, in order.  Whole CTA; [st0, st1): the CTA's steps of the unit.
template <int R, int DV, int W, int SCRATCH>
__device__ __forceinline__ void finish_unit(const PagedArgs& a, const Cut& cut, const Place& p, const Run& run, int st0,
                                            int st1, float* sm) {
  constexpr int THREADS = W * 32, EPT = R * DV / THREADS;
  static_assert(R * DV % THREADS == 0, "outputs per thread");
  __shared__ float s_M[R], s_L[R];
  __shared__ int s_last;
  const int tid = threadIdx.x, G = cut.G;
  float* sm_m = sm;
  float* sm_l = sm + W * R;
  const float* sm_o = sm + 2 * W * R;
  __syncthreads();
  if (tid < R) {
    float M = M_NONE, L = 0.f, nan = 0.f;
    for (int w = 0; w < W; ++w) M = fmaxf(M, sm_m[w * R + tid]);
    for (int w = 0; w < W; ++w) {
      const float x = ex2(sm_m[w * R + tid] - M);
      L = fmaf(x, sm_l[w * R + tid], L);
      nan += sm_m[w * R + tid] * 0.f;
      sm_m[w * R + tid] = x;                      // the warp's weight
    }
    s_M[tid] = M;
    s_L[tid] = nan == 0.f ? L : NAN;              // a reference of NaN or infinity: no result
  }
  __syncthreads();
  const int64_t rows = (int64_t)p.s.T * G;
  const int here = (int)min((int64_t)R, rows - (int64_t)p.rt * R);
  const bool whole = st0 == 0 && st1 == p.n_steps;
  const int mine = (blockIdx.x * 2 + (run.x0 >= p.at ? 0 : 1)) * R;     // [0]: the unit that the run begins in, [1]: its last
  auto row_at = [&](int r) {
    const int row = p.rt * R + r;
    return ((int64_t)(p.s.t0 + row / G) * a.Hq + p.g * G + row % G) * DV;
  };
#pragma unroll
  for (int e = 0; e < EPT; ++e) {
    const int idx = tid + e * THREADS, r = idx / DV, d = idx % DV;
    if (r >= here) continue;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) v = fmaf(sm_m[w * R + r], sm_o[(w * R + r) * DV + d], v);
    if (whole) {
      store_out(a, row_at(r), d, s_L[r] == 0.f ? 0.f : v / s_L[r]);
    } else {
      a.part_acc[(int64_t)(mine + r) * DV + d] = v;
      if (d == 0) { a.part_ml[2 * (mine + r)] = s_M[r]; a.part_ml[2 * (mine + r) + 1] = s_L[r]; }
    }
  }
  if (whole) return;
  const int c0 = run.of(p.at), c1 = run.of(p.at + p.n_steps - 1);
  __syncthreads();                                // the CTA's part is written; thread 0's fences cover all of it
  unsigned* counter = a.counters + c0;            // only the last unit of a run goes on into the next one
  if (tid == 0) {
    __threadfence();
    s_last = atomicAdd(counter, 1u) == (unsigned)(c1 - c0);
    __threadfence();
  }
  __syncthreads();
  if (!s_last) return;
  const int first = (c0 * 2 + (run.start_of(c0) >= p.at ? 0 : 1)) * R;   // the others' parts are their [0]
  auto part = [&](int c) { return c == c0 ? first : 2 * R * c; };
  constexpr int BLOCK = SCRATCH / (R * 8) < 512 ? SCRATCH / (R * 8) : 512;    // parts whose (maximum, sum) fit
  float2* ml = reinterpret_cast<float2*>(sm);     // [R][BLOCK]; the maxima become weights
  __shared__ float s_alpha[R];
  float acc[EPT];
#pragma unroll
  for (int e = 0; e < EPT; ++e) acc[e] = 0.f;
  if (tid < R) { s_M[tid] = M_NONE; s_L[tid] = 0.f; }
  for (int cb = c0; cb <= c1; cb += BLOCK) {      // one pass, unless the unit has very many parts
    const int n = min(BLOCK, c1 + 1 - cb);
    constexpr int U = EPT <= 8 ? 4 : 2;           // parts on their way, the first ones before the weights are known
    float v[U][EPT];
    auto fetch = [&](int c) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float* src = a.part_acc + (int64_t)part(cb + c + u) * DV;
#pragma unroll
        for (int e = 0; e < EPT; ++e)
          v[u][e] = c + u < n && (tid + e * THREADS) / DV < here ? __ldcg(src + tid + e * THREADS) : 0.f;
      }
    };
    fetch(0);
    __syncthreads();
    for (int i = tid; i < R * n; i += THREADS) {
      const int c = i / R, r = i % R;
      ml[r * BLOCK + c] = r < here ? __ldcg(reinterpret_cast<const float2*>(a.part_ml) + part(cb + c) + r) : make_float2(M_NONE, 0.f);
    }
    __syncthreads();
    const int lane = tid & 31;
    for (int r = tid >> 5; r < R; r += W) {       // weights against the maximum so far
      const float before = s_M[r];
      float M = before, den = 0.f;
      for (int c = lane; c < n; c += 32) M = fmaxf(M, ml[r * BLOCK + c].x);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(FULL_MASK, M, o));
      for (int c = lane; c < n; c += 32) {
        const float w = ex2(ml[r * BLOCK + c].x - M);
        den = fmaf(w, ml[r * BLOCK + c].y, den);
        ml[r * BLOCK + c].x = w;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(FULL_MASK, den, o);
      __syncwarp();
      if (lane == 0) {
        s_alpha[r] = ex2(before - M);
        s_L[r] = fmaf(s_L[r], s_alpha[r], den);
        s_M[r] = M;
      }
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < EPT; ++e) acc[e] *= s_alpha[(tid + e * THREADS) / DV];
    for (int c = 0; c < n; c += U) {
      if (c > 0) fetch(c);
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 0; e < EPT; ++e)
          if (c + u < n) acc[e] = fmaf(ml[(tid + e * THREADS) / DV * BLOCK + c + u].x, v[u][e], acc[e]);
    }
  }
#pragma unroll
  for (int e = 0; e < EPT; ++e) {
    const int idx = tid + e * THREADS, r = idx / DV, d = idx % DV;
    if (r < here) store_out(a, row_at(r), d, s_L[r] == 0.f ? 0.f : acc[e] / s_L[r]);
  }
  if (tid == 0) *counter = 0u;
}

}  // namespace paged
}  // namespace kva
