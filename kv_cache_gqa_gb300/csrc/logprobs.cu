// Log probabilities over the vocabulary (lmhead_logprobs): a streaming form for any table, and the
// merge that ends every form.
//
// Streaming form: grid (vocabulary split p, block of 8 batch rows).  The 8 warps of a CTA dot 4
// table rows each with the 8 hidden rows (staged in shared memory) and leave 32 x 8 logits in
// shared memory; then warp b owns batch row b and lane r the r-th logit.  A lane keeps, over the
// rows that pass it, the running maximum m, s = sum exp(z - m), u = sum exp(z - m) (z - m) and a
// sorted list of its TK best (logit, id) keys; the warp joins its lanes at the end and writes one
// partial per (split, batch row).
//
// Merge (one CTA per batch row): joins the splits' (m, s, u) in a fixed order and their lists, then
// scores the given token and the TK candidates again: the lists hold TK > top_k candidates by
// float32 (or two-bf16-halves) logits, whose rounding may exchange neighbours, while the second
// scoring carries each product and sum with its rounding error (compensated dot product: Ogita,
// Rump and Oishi, "Accurate sum and dot product"), about twice float32 precision, and orders them.
// entropy = log s - u / s and lse = m + log s need no cancellation against m.
//
// Method: the lm_head over the whole tied table and the pick of tokens after the final RMSNorm
// (Youtu-VL-4B ncnn port, step 6 and "decoding and sampling").
#include <algorithm>

#include "common.cuh"
#include "launch.h"

namespace kva {

namespace {

constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;
constexpr int BG = 8;                         // batch rows per CTA (one per warp)
constexpr int ROWS = 32;                      // vocabulary rows per step (one per lane)
constexpr int MERGE_THREADS = 128;
constexpr int MERGE_WARPS = MERGE_THREADS / 32;

using u64 = unsigned long long;

// Sorted list of the TK best keys (larger key = larger logit, then lower id).
template <int TK>
__device__ __forceinline__ void list_insert(u64 (&L)[TK], u64 key) {
  if (key <= L[TK - 1]) return;
#pragma unroll
  for (int i = TK - 1; i > 0; --i) L[i] = key > L[i - 1] ? L[i - 1] : (key > L[i] ? key : L[i]);
  L[0] = key > L[0] ? key : L[0];
}
// The TK best of the warp's 32 lists, into out[] (lane 0 writes).
template <int TK>
__device__ __forceinline__ void warp_merge(u64 (&L)[TK], u64* out) {
  const int lane = threadIdx.x & 31;
  for (int r = 0; r < TK; ++r) {
    u64 best = L[0];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const u64 other = __shfl_xor_sync(FULL_MASK, best, o);
      best = other > best ? other : best;
    }
    if (lane == 0) out[r] = best;
    if (best != 0ull && L[0] == best) {       // keys are unique: one lane pops
#pragma unroll
      for (int i = 0; i < TK - 1; ++i) L[i] = L[i + 1];
      L[TK - 1] = 0ull;
    }
  }
}

// Softmax statistics of a set of logits: maximum, sum exp(z - m), sum exp(z - m)(z - m).
struct Stat { float m, s, u; };
__device__ __forceinline__ void stat_add(Stat& a, float z) {
  if (z > a.m) {
    const float d = a.m - z;                  // -inf on the first logit, whose sums are 0
    const float e = __expf(d);
    a.u = a.s == 0.f ? 0.f : e * fmaf(a.s, d, a.u);
    a.s = fmaf(a.s, e, 1.f);
    a.m = z;
  } else {
    const float d = z - a.m, e = __expf(d);
    a.s += e;
    if (e > 0.f) a.u = fmaf(e, d, a.u);
  }
}
__device__ __forceinline__ Stat stat_join(const Stat& a, const Stat& b) {
  const float m = fmaxf(a.m, b.m);
  Stat r{m, 0.f, 0.f};
  if (a.s != 0.f) { const float d = a.m - m, e = __expf(d); r.s += a.s * e; r.u += e * fmaf(a.s, d, a.u); }
  if (b.s != 0.f) { const float d = b.m - m, e = __expf(d); r.s += b.s * e; r.u += e * fmaf(b.s, d, b.u); }
  return r;
}
__device__ __forceinline__ Stat stat_warp(Stat a) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const Stat b{__shfl_xor_sync(FULL_MASK, a.m, o), __shfl_xor_sync(FULL_MASK, a.s, o), __shfl_xor_sync(FULL_MASK, a.u, o)};
    a = stat_join(a, b);
  }
  return a;
}

// One CTA per row: the final RMSNorm in float32.
__global__ void __launch_bounds__(THREADS)
logprob_norm_kernel(const __grid_constant__ LogprobArgs a) {
  __shared__ float s_part[WARPS];
  const int b = blockIdx.x, tid = threadIdx.x;
  griddep_wait();
  griddep_launch_dependents();
  const int64_t row = (int64_t)b * a.H;
  auto at = [&](int k) {
    return a.h_dtype == KVA_BF16 ? load1(reinterpret_cast<const bf16_t*>(a.h) + row + k)
                                 : reinterpret_cast<const float*>(a.h)[row + k];
  };
  float ss = 0.f;
  for (int k = tid; k < a.H; k += THREADS) { const float x = at(k); ss = fmaf(x, x, ss); }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(FULL_MASK, ss, o);
  if ((tid & 31) == 0) s_part[tid >> 5] = ss;
  __syncthreads();
  float tot = 0.f;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) tot += s_part[w];
  const float r = 1.0f / sqrtf(tot / (float)a.H + a.eps);
  for (int k = tid; k < a.H; k += THREADS) a.hn[row + k] = at(k) * r * a.norm_w[k];
}

// The row that the table meets: normalised (float32), or h itself.
__device__ __forceinline__ float hidden_at(const LogprobArgs& a, int64_t i) {
  if (a.norm_w) return a.hn[i];
  return a.h_dtype == KVA_BF16 ? load1(reinterpret_cast<const bf16_t*>(a.h) + i) : reinterpret_cast<const float*>(a.h)[i];
}

template <typename WT, int TK>
__global__ void __launch_bounds__(THREADS)
logprob_stream_kernel(const __grid_constant__ LogprobArgs a) {
  extern __shared__ __align__(16) float sh[];   // [nb][H]
  __shared__ float s_z[BG][ROWS + 1];
  __shared__ u64 s_list[WARPS][TK > 0 ? TK : 1];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b0 = blockIdx.y * BG, nb = min(BG, a.B - b0), H = a.H;
  griddep_wait();
  griddep_launch_dependents();
  for (int i = tid; i < nb * H; i += THREADS) sh[i] = hidden_at(a, (int64_t)b0 * H + i);
  __syncthreads();

  Stat st{-INFINITY, 0.f, 0.f};
  u64 L[TK > 0 ? TK : 1];
#pragma unroll
  for (int i = 0; i < (TK > 0 ? TK : 1); ++i) L[i] = 0ull;
  const int n_steps = (a.V + ROWS - 1) / ROWS;
  for (int step = blockIdx.x; step < n_steps; step += a.splits) {
    for (int r = 0; r < ROWS / WARPS; ++r) {
      const int rr = warp * (ROWS / WARPS) + r, v = step * ROWS + rr;
      float part[BG];
#pragma unroll
      for (int b = 0; b < BG; ++b) part[b] = 0.f;
      if (v < a.V) {                            // warp-uniform
        const WT* wrow = reinterpret_cast<const WT*>(a.W) + (int64_t)v * H;
        for (int c = lane * 8; c < H; c += 256) {
          float x[8];
          load8(wrow + c, x);
#pragma unroll
          for (int b = 0; b < BG; ++b)
            if (b < nb) {
              const float4 p = *reinterpret_cast<const float4*>(sh + b * H + c);
              const float4 q = *reinterpret_cast<const float4*>(sh + b * H + c + 4);
              part[b] = fmaf(x[0], p.x, part[b]); part[b] = fmaf(x[1], p.y, part[b]);
              part[b] = fmaf(x[2], p.z, part[b]); part[b] = fmaf(x[3], p.w, part[b]);
              part[b] = fmaf(x[4], q.x, part[b]); part[b] = fmaf(x[5], q.y, part[b]);
              part[b] = fmaf(x[6], q.z, part[b]); part[b] = fmaf(x[7], q.w, part[b]);
            }
        }
      }
#pragma unroll
      for (int b = 0; b < BG; ++b) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) part[b] += __shfl_xor_sync(FULL_MASK, part[b], o);
        if (lane == 0) s_z[b][rr] = part[b];
      }
    }
    __syncthreads();
    const int v = step * ROWS + lane;
    if (v < a.V && warp < nb) {
      const float z = s_z[warp][lane];
      stat_add(st, z);
      if constexpr (TK > 0) list_insert<TK>(L, argmax_key(z, (uint32_t)v));
    }
    __syncthreads();
  }
  if (warp >= nb) return;
  st = stat_warp(st);
  const int64_t slot = (int64_t)(b0 + warp) * a.splits + blockIdx.x;
  if (lane == 0) {
    float* p = a.part_stat + slot * 4;
    p[0] = st.m; p[1] = st.s; p[2] = st.u;
  }
  if constexpr (TK > 0) {
    warp_merge<TK>(L, s_list[warp]);
    __syncwarp();
    for (int i = lane; i < TK; i += 32) a.part_key[slot * TK + i] = s_list[warp][i];
  }
}

// s + p with its rounding error added to c.
__device__ __forceinline__ void sum_two(float& s, float& c, float p) {
  const float t = __fadd_rn(s, p), z = __fsub_rn(t, s);
  c = __fadd_rn(c, __fadd_rn(__fsub_rn(s, __fsub_rn(t, z)), __fsub_rn(p, z)));
  s = t;
}
// W[v] . h_b in about twice float32 precision (a warp; every lane gets the result).
template <typename WT>
__device__ __forceinline__ double dot_again(const LogprobArgs& a, int b, int v) {
  const WT* w = reinterpret_cast<const WT*>(a.W) + (int64_t)v * a.H;
  float s = 0.f, c = 0.f;
  for (int k = (threadIdx.x & 31) * 8; k < a.H; k += 256) {
    float x[8];
    load8(w + k, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float y = hidden_at(a, (int64_t)b * a.H + k + i);
      const float p = __fmul_rn(x[i], y);
      c = __fadd_rn(c, __fmaf_rn(x[i], y, -p));
      sum_two(s, c, p);
    }
  }
  double d = (double)s + (double)c;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(FULL_MASK, d, o);
  return d;
}

template <typename WT, int TK>
__global__ void __launch_bounds__(MERGE_THREADS)
logprob_merge_kernel(const __grid_constant__ LogprobArgs a) {
  constexpr int TL = TK > 0 ? TK : 1;
  __shared__ u64 s_w[MERGE_WARPS][TL];
  __shared__ u64 s_top[TL];
  __shared__ double s_val[TL + 1];
  __shared__ Stat s_stat[MERGE_WARPS];
  __shared__ double s_lse;
  __shared__ int s_rank[TL];                            // candidate of each rank, -1: none
  const int b = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  griddep_wait();
  griddep_launch_dependents();
  Stat st{-INFINITY, 0.f, 0.f};
  u64 L[TL];
#pragma unroll
  for (int i = 0; i < TL; ++i) L[i] = 0ull;
  for (int p = tid; p < a.splits; p += MERGE_THREADS) {
    const int64_t slot = (int64_t)b * a.splits + p;
    const float4 q = *reinterpret_cast<const float4*>(a.part_stat + slot * 4);
    st = stat_join(st, Stat{q.x, q.y, q.z});
    if constexpr (TK > 0)
      for (int i = 0; i < TK; ++i) {
        const u64 key = a.part_key[slot * TK + i];
        if (key <= L[TK - 1]) break;                    // lists are sorted
        list_insert<TK>(L, key);
      }
  }
  st = stat_warp(st);
  if (lane == 0) s_stat[warp] = st;
  if constexpr (TK > 0) warp_merge<TK>(L, s_w[warp]);
  __syncthreads();
  if (warp == 0) {
    if constexpr (TK > 0) {
#pragma unroll
      for (int i = 0; i < TK; ++i) L[i] = lane < MERGE_WARPS ? s_w[lane][i] : 0ull;
      warp_merge<TK>(L, s_top);
    }
    Stat all = s_stat[0];
    for (int w = 1; w < MERGE_WARPS; ++w) all = stat_join(all, s_stat[w]);
    if (lane == 0) {
      const double ls = log((double)all.s);
      s_lse = (double)all.m + ls;
      if (a.out_lse) a.out_lse[b] = (float)s_lse;
      if (a.out_entropy) a.out_entropy[b] = (float)(ls - (double)all.u / (double)all.s);
    }
  }
  __syncthreads();
  const int target = a.targets ? a.targets[b] : -1;
  for (int c = warp; c <= TK; c += MERGE_WARPS) {       // candidate TK is the given token
    int v = target;
    if (c < TK) v = s_top[c] ? (int)(0xffffffffu - (uint32_t)(s_top[c] & 0xffffffffull)) : -1;
    const double d = v >= 0 && v < a.V ? dot_again<WT>(a, b, v) : 0.0;
    if (lane == 0) s_val[c] = d;
  }
  if (tid < TL) s_rank[tid] = -1;
  __syncthreads();
  if (tid == 0 && a.targets)
    a.out_logprob[b] = target < 0 ? 0.f : (target < a.V ? (float)(s_val[TK] - s_lse) : __uint_as_float(0x7fc00000u));
  if (tid < TK) {
    const u64 key = s_top[tid];
    const uint32_t id = 0xffffffffu - (uint32_t)(key & 0xffffffffull);
    int rank = 0;
    for (int c = 0; c < TK; ++c) {
      const uint32_t other = 0xffffffffu - (uint32_t)(s_top[c] & 0xffffffffull);
      if (s_top[c] && (s_val[c] > s_val[tid] || (s_val[c] == s_val[tid] && other < id))) ++rank;
    }
    if (key) s_rank[rank] = tid;
  }
  __syncthreads();
  if (tid < a.top_k) {
    const int c = s_rank[tid];
    const int64_t o = (int64_t)b * a.top_k + tid;
    a.top_ids[o] = c < 0 ? -1 : (int32_t)(0xffffffffu - (uint32_t)(s_top[c] & 0xffffffffull));
    if (a.top_logprobs) a.top_logprobs[o] = c < 0 ? __uint_as_float(0x7fc00000u) : (float)(s_val[c] - s_lse);
  }
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// Candidates kept for top_k alternatives: the rest is room for neighbours that rounding exchanges.
int list_len(int top_k) { return top_k == 0 ? 0 : (top_k <= 4 ? 8 : (top_k <= 10 ? 16 : 32)); }

constexpr int CTAS = 152 * 2;
int stream_splits(int B, int V) {
  const int groups = (B + BG - 1) / BG;
  return std::max(1, std::min((V + ROWS - 1) / ROWS, CTAS / std::min(groups, CTAS)));
}

template <typename WT, int TK>
cudaError_t launch_stream(const LogprobArgs& a, cudaStream_t s) {
  const size_t smem = sizeof(float) * (size_t)std::min(BG, a.B) * a.H;
  static DeviceOnce configured;
  if (!configured.done()) {
    cudaError_t e = cudaFuncSetAttribute(logprob_stream_kernel<WT, TK>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)(sizeof(float) * BG * lmhead_max_hidden()));
    if (e != cudaSuccess) return e;
    configured.mark();
  }
  cudaError_t e = launch_pdl(logprob_stream_kernel<WT, TK>, dim3(a.splits, (a.B + BG - 1) / BG), dim3(THREADS), smem, s, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(logprob_merge_kernel<WT, TK>, dim3(a.B), dim3(MERGE_THREADS), 0, s, a);
}

template <typename WT>
cudaError_t launch_w(const LogprobArgs& a, cudaStream_t s) {
  switch (list_len(a.top_k)) {
    case 0: return launch_stream<WT, 0>(a, s);
    case 8: return launch_stream<WT, 8>(a, s);
    case 16: return launch_stream<WT, 16>(a, s);
    default: return launch_stream<WT, 32>(a, s);
  }
}

}  // namespace

// Workspace: [normalised rows, float32][partial statistics][partial lists]
size_t logprob_workspace_bytes(int B, int H, int V, int top_k) {
  const size_t parts = (size_t)B * stream_splits(B, V);
  return up256(sizeof(float) * (size_t)B * H) + up256(parts * 16) + up256(parts * 8 * list_len(top_k));
}

cudaError_t launch_logprobs(LogprobArgs a, kva_dtype w_dtype, void* workspace, cudaStream_t s, unsigned* n_launches) {
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  *n_launches = 2;
  a.splits = stream_splits(a.B, a.V);
  a.hn = reinterpret_cast<float*>(ws);
  ws += up256(sizeof(float) * (size_t)a.B * a.H);
  a.part_stat = reinterpret_cast<float*>(ws);
  a.part_key = reinterpret_cast<u64*>(ws + up256((size_t)a.B * a.splits * 16));
  if (a.norm_w) {
    cudaError_t e = launch_pdl(logprob_norm_kernel, dim3(a.B), dim3(THREADS), 0, s, a);
    if (e != cudaSuccess) return e;
    *n_launches = 3;
  }
  return w_dtype == KVA_BF16 ? launch_w<bf16_t>(a, s) : launch_w<float>(a, s);
}

}  // namespace kva
