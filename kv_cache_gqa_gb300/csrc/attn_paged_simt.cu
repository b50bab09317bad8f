// Attention of new tokens over a paged cache on the CUDA cores (kv_attn_paged).
//
// A unit is 16 query rows (token, head of the group) of one KV head; a step is 128 slots, 32 for each of
// the CTA's four warps, which keep their own running maximum, sum and output and join them at the unit's
// end (paged.cuh).  A lane takes one key's scores against all rows (its K row from global memory, q rows
// broadcast from shared memory), the weights go through shared memory, and then a lane takes DV/32 columns of
// the output for all rows.  The reference maximum moves only when a score exceeds it by 2^8.
//
// Method: one pass over the keys with the running maximum and sum of the softmax; the visible prefix of a
// token as in the decode and verify steps (Youtu-VL-4B ncnn port, step 8; HunyuanOCR v1.5 ncnn port, section
// 3.8).  The reference keeps fixed windows; a cache in pages has no counterpart there.
#include "paged.cuh"

namespace kva {

namespace {

using paged::Cut;
using paged::ex2;
using paged::M_NONE;
using paged::Place;

constexpr int WARPS = 4, THREADS = WARPS * 32, R = 16, KT = 32;
static_assert(R == PAGED_ROWS, "partial results");
constexpr float RESCALE_LOG2 = 8.0f;

template <int N> struct Cols { float v[N]; };
template <typename T, int N>
__device__ __forceinline__ Cols<N> load_cols(const T* p) {
  Cols<N> c;
  if constexpr (sizeof(T) == 4) {
    if constexpr (N == 4) {
      const float4 x = __ldg(reinterpret_cast<const float4*>(p));
      c.v[0] = x.x; c.v[1] = x.y; c.v[2] = x.z; c.v[3] = x.w;
    } else {
      const float2 x = __ldg(reinterpret_cast<const float2*>(p));
      c.v[0] = x.x; c.v[1] = x.y;
    }
  } else {
    if constexpr (N == 4) {
      const uint2 x = __ldg(reinterpret_cast<const uint2*>(p));
      c.v[0] = bf16_lo(x.x); c.v[1] = bf16_hi(x.x); c.v[2] = bf16_lo(x.y); c.v[3] = bf16_hi(x.y);
    } else {
      const uint32_t x = __ldg(reinterpret_cast<const uint32_t*>(p));
      c.v[0] = bf16_lo(x); c.v[1] = bf16_hi(x);
    }
  }
  return c;
}

template <int DK, int DV>
struct Smem {
  static constexpr int Q = R * DK, P = WARPS * KT * R, O = WARPS * R * DV, ML = 2 * WARPS * R;
  static constexpr int BYTES = 4 * (Q + P > ML + O ? Q + P : ML + O);
};

template <typename T, int DK, int DV>
__global__ void __launch_bounds__(THREADS)
attn_paged_simt_kernel(const __grid_constant__ PagedArgs a) {
  constexpr int NC = DV / 32;
  extern __shared__ __align__(16) float sm[];
  __shared__ int64_t scratch[WARPS + 4];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Cut cut{R, KT * WARPS, a.Hq / a.Hkv, a.rows_lo, a.rows_hi};
  const int G = cut.G, page_mask = (1 << a.page_shift) - 1;
  griddep_wait();                               // inputs of this launch are complete from here on
  griddep_launch_dependents();
  Place p;
  const paged::Run run = paged::first_place<THREADS>(a, cut, scratch, &p);
  if (run.x0 >= run.x1) return;
  float* sm_q = sm;
  float* sm_p = sm + R * DK + warp * KT * R;

  for (; p.b < a.B && p.at < run.x1; p.next(a, cut)) {
    const int st0 = (int)max((int64_t)0, run.x0 - p.at), st1 = (int)min((int64_t)p.n_steps, run.x1 - p.at);
    const int64_t rows = (int64_t)p.s.T * G;
    __syncthreads();                            // the unit before is done with the shared memory
    for (int i = tid; i < R * DK; i += THREADS) {
      const int64_t row = (int64_t)p.rt * R + i / DK;
      float x = 0.f;
      if (row < rows)
        x = load1(reinterpret_cast<const T*>(a.q) + ((p.s.t0 + row / G) * a.Hq + p.g * G + row % G) * DK + i % DK) *
            a.scale_log2;
      sm_q[i] = x;
    }
    __syncthreads();
    float m[R], l[R], o[R][NC];
    int lim[R];                                 // slots that row r sees
    int lim_all = 0;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      m[r] = M_NONE;
      l[r] = 0.f;
#pragma unroll
      for (int c = 0; c < NC; ++c) o[r][c] = 0.f;
      const int64_t row = (int64_t)p.rt * R + r;
      lim[r] = row < rows ? min(max(p.s.L - p.s.T + (int)(row / G) + 1, 0), p.s.L) : 0;
      lim_all = max(lim_all, lim[r]);
    }
    const int32_t* pages = a.table + (int64_t)p.b * a.table_stride;
    for (int st = st0; st < st1; ++st) {
      const int ks = (st * WARPS + warp) * KT;
      if (ks >= lim_all) break;
      const int key = ks + lane;
      bool bad = false;
      int64_t at = 0, atv = 0;                  // the key's rows in K and V
      if (key < lim_all) {
        const int page = pages[key >> a.page_shift];
        bad = (unsigned)page >= (unsigned)a.n_pages;
        const int64_t pg = bad ? 0 : page;
        const int in = (p.g << a.page_shift) + (key & page_mask);
        at = pg * a.page_stride + (int64_t)in * DK;
        atv = pg * a.page_stride_v + (int64_t)in * DV;
      }
      float s[R];
#pragma unroll
      for (int r = 0; r < R; ++r) s[r] = 0.f;
      if (key < lim_all) {
        const T* kp = reinterpret_cast<const T*>(a.k) + at;
#pragma unroll 4
        for (int d = 0; d < DK; d += 4) {
          const Cols<4> kk = load_cols<T, 4>(kp + d);
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const float4 qv = *reinterpret_cast<const float4*>(sm_q + r * DK + d);
            s[r] = fmaf(qv.x, kk.v[0], fmaf(qv.y, kk.v[1], fmaf(qv.z, kk.v[2], fmaf(qv.w, kk.v[3], s[r]))));
          }
        }
      }
      bool grow = false;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (bad) s[r] = NAN;
        if (key >= lim[r]) s[r] = -INFINITY;
        grow |= s[r] > m[r] + RESCALE_LOG2;
      }
      if (__any_sync(FULL_MASK, grow)) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
          float mt = s[r];
#pragma unroll
          for (int x = 16; x > 0; x >>= 1) mt = fmaxf(mt, __shfl_xor_sync(FULL_MASK, mt, x));
          mt = fmaxf(mt, m[r]);
          const float alpha = ex2(m[r] - mt);
          m[r] = mt;
          l[r] *= alpha;
#pragma unroll
          for (int c = 0; c < NC; ++c) o[r][c] *= alpha;
        }
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float w = ex2(s[r] - m[r]);
        l[r] += w;
        s[r] = w;
      }
#pragma unroll
      for (int r = 0; r < R; r += 4)
        *reinterpret_cast<float4*>(sm_p + lane * R + r) = make_float4(s[r], s[r + 1], s[r + 2], s[r + 3]);
      __syncwarp();
      const int n = min(KT, lim_all - ks);
#pragma unroll 4
      for (int j = 0; j < n; ++j) {
        const int64_t vj = __shfl_sync(FULL_MASK, atv, j);
        const Cols<NC> vv = load_cols<T, NC>(reinterpret_cast<const T*>(a.v) + vj + lane * NC);
#pragma unroll
        for (int r = 0; r < R; r += 4) {
          const float4 w = *reinterpret_cast<const float4*>(sm_p + j * R + r);
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            o[r][c] = fmaf(w.x, vv.v[c], o[r][c]);
            o[r + 1][c] = fmaf(w.y, vv.v[c], o[r + 1][c]);
            o[r + 2][c] = fmaf(w.z, vv.v[c], o[r + 2][c]);
            o[r + 3][c] = fmaf(w.w, vv.v[c], o[r + 3][c]);
          }
        }
      }
      __syncwarp();
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) l[r] += __shfl_xor_sync(FULL_MASK, l[r], x);
    __syncthreads();
    float* sm_m = sm;
    float* sm_l = sm + WARPS * R;
    float* sm_o = sm + 2 * WARPS * R + warp * R * DV;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (lane == 0) { sm_m[warp * R + r] = m[r]; sm_l[warp * R + r] = l[r]; }
#pragma unroll
      for (int c = 0; c < NC; ++c) sm_o[r * DV + lane * NC + c] = o[r][c];
    }
    paged::finish_unit<R, DV, WARPS, Smem<DK, DV>::BYTES>(a, cut, p, run, st0, st1, sm);
  }
}

template <typename T, int DK, int DV>
cudaError_t launch_t(const PagedArgs& a, int runs, cudaStream_t s) {
  constexpr int smem = Smem<DK, DV>::BYTES;
  static DeviceOnce configured;
  if (!configured.done()) {
    const cudaError_t e = cudaFuncSetAttribute(attn_paged_simt_kernel<T, DK, DV>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    configured.mark();
  }
  return launch_pdl(attn_paged_simt_kernel<T, DK, DV>, dim3(runs), dim3(THREADS), (size_t)smem, s, a);
}

template <typename T>
cudaError_t launch_d(const PagedArgs& a, int Dk, int runs, cudaStream_t s) {
  if (Dk == 64) return launch_t<T, 64, 64>(a, runs, s);
  if (Dk == 128) return launch_t<T, 128, 128>(a, runs, s);
  return launch_t<T, 192, 128>(a, runs, s);
}

}  // namespace

cudaError_t launch_attn_paged_simt(const PagedArgs& a, int Dk, kva_dtype dtype, int runs, cudaStream_t s) {
  return dtype == KVA_F32 ? launch_d<float>(a, Dk, runs, s) : launch_d<bf16_t>(a, Dk, runs, s);
}

}  // namespace kva
