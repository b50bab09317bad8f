// The 4-bit cache's write and read-back: QK-Norm + RoPE + quantisation fused into the cache write
// (kv_cache_append_q4), and the expansion of listed slots into a bf16 or float32 cache
// (kv_cache_expand_q4).  Layout and quantiser: kva_cache_q4 in kv_attn.h.
//
// Append: one CTA per (token t, instance n, row group).  A row of D values belongs to SW lanes of a
// warp (SW = 8, 16 or 32 for rows up to 64, 128 or 256 wide), 8 consecutive values a lane, so the
// 64 values of a quantisation group sit in 8 consecutive lanes: the group's minimum and maximum
// are three shuffles each, a lane's 8 codes are one 32-bit word of the cache, and a group's first
// lane writes its scale and midpoint.  A warp issues the loads of RB row sets before transforming
// any of them.  Norm and rotation are float32, as in the unquantised append; the angles of a token
// are evaluated once per CTA.
//
// Method: the append of the decode step (Youtu-VL-4B ncnn port, step 6) with per-head RMSNorm and
// rotate-half RoPE (Penguin-VL ncnn port, sections 2.1 and 4.2; Youtu-VL-4B ncnn port,
// implementation difficulty 2).  The pages hold their caches in 16 or 32 bits; the 4-bit form has
// no counterpart there.
#include <algorithm>

#include "common.cuh"
#include "launch.h"

namespace kva {

namespace {

constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;
constexpr int RB = 4;            // row sets a warp loads before transforming them
constexpr int MAX_D = 256;

template <int SW>
__device__ __forceinline__ float sub_sum(float v) {
#pragma unroll
  for (int o = SW / 2; o > 0; o >>= 1) v += __shfl_xor_sync(FULL_MASK, v, o);
  return v;
}

// Quantise the 8 values of this lane, whose group of 64 is the lane's aligned set of 8 lanes.
// Returns the code word; *par = (scale, mid) packed for the group's first lane.
__device__ __forceinline__ uint32_t quantise8(const float (&x)[8], uint32_t* par) {
  float lo = x[0], hi = x[0];
  bool odd = false;                                     // a NaN or an infinity (fminf drops NaN)
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    lo = fminf(lo, x[i]); hi = fmaxf(hi, x[i]);
    odd |= !(fabsf(x[i]) <= 3.402823466e38f);
  }
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) {
    lo = fminf(lo, __shfl_xor_sync(FULL_MASK, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(FULL_MASK, hi, o));
  }
  const unsigned any = __ballot_sync(FULL_MASK, odd);
  odd = ((any >> (threadIdx.x & 24)) & 0xffu) != 0;
  // the scale is rounded up, so 15 steps cover the spread; one below bf16's normal range is 0
  float scale = __bfloat162float(__float2bfloat16_ru(__fdiv_rn(hi - lo, 15.0f)));
  if (scale < 1.17549435e-38f) scale = 0.f;
  float mid = __bfloat162float(__float2bfloat16_rn(fmaf(8.0f, scale, lo)));
  if (odd || !(scale <= 3.402823466e38f) || !(fabsf(mid) <= 3.402823466e38f)) scale = mid = __uint_as_float(0x7fc00000u);
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // a quotient, not a product with the inverse: bf16 inputs meet exact half steps, which
    // round to even
    const float q = scale > 0.f ? __fdiv_rn(x[i] - mid, scale) : 0.f;
    const int c = (int)fminf(fmaxf(rintf(q), -8.f), 7.f) + 8;
    w |= (uint32_t)c << (4 * i);
  }
  *par = (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(scale)) |
         ((uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(mid)) << 16);
  return w;
}

template <typename InT, typename QOutT, int SW>
__global__ void __launch_bounds__(THREADS, 3)
append_q4_kernel(const __grid_constant__ AppendQ4Args a) {
  constexpr int RPW = 32 / SW;                          // rows a warp holds at once
  __shared__ float s_cos[MAX_ROPE_FREQ];
  __shared__ float s_sin[MAX_ROPE_FREQ];
  __shared__ __align__(16) float s_row[WARPS][RPW][SW * 8];

  const int t = blockIdx.x, n = blockIdx.y;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int sub = lane / SW, sl = lane % SW;
  const int Dk = a.c.Dk, Dv = a.c.Dv, Hkv = a.c.Hkv;
  const int Hq = a.q ? a.Hq : 0;
  const int ro = a.rot_offset, rw = a.rot_dim, half = rw / 2, quarter = rw / 4;
  const int kind_r = a.rope.kind;
  const int n_rows = Hq + 2 * Hkv;
  const float* qw = a.q_w ? a.q_w + (int64_t)n * a.w_stride : nullptr;
  const float* kw = a.k_w ? a.k_w + (int64_t)n * a.w_stride : nullptr;
  griddep_wait();                               // inputs of this launch are complete from here on
  const int32_t slot = a.slot[(int64_t)n * a.slot_stride + t];
  const int64_t tok = (int64_t)n * a.T + t;
  const int e0 = sl * 8;

  const int stride = WARPS * RPW * gridDim.z;
  const int first = (blockIdx.z * WARPS + warp) * RPW;
  for (int base = first; base < n_rows || base == first;
       base += RB * stride) {
    float xs[RB][8];
#pragma unroll
    for (int k = 0; k < RB; ++k) {
      const int r = base + k * stride + sub;
      const int kind = r < Hq ? 0 : (r < Hq + Hkv ? 1 : 2);
      const int head = kind == 0 ? r : (kind == 1 ? r - Hq : r - Hq - Hkv);
      if (r < n_rows && e0 < (kind == 2 ? Dv : Dk)) {
        if (kind == 0) load8(reinterpret_cast<const InT*>(a.q) + (tok * a.Hq + head) * Dk + e0, xs[k]);
        else if (kind == 1) load8(reinterpret_cast<const InT*>(a.k) + (tok * Hkv + head) * Dk + e0, xs[k]);
        else load8(reinterpret_cast<const InT*>(a.v) + (tok * Hkv + head) * Dv + e0, xs[k]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) xs[k][i] = 0.f;
      }
    }
    if (base == first) {   // first pass: the angles, behind the loads
      if (kind_r != KVA_ROPE_NONE) {
        for (int j = tid; j < half; j += THREADS) {
          const int32_t p = a.pos[(int64_t)n * a.pos_stride + (int64_t)t * a.rope.n_axes + a.rope.axis[j]];
          rope_cos_sin(p, a.rope.inv_hi[j], a.rope.inv_lo[j], a.rope.inv[j], &s_cos[j], &s_sin[j]);
        }
      }
      __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < RB; ++k) {
      if (base + k * stride >= n_rows) break;           // warp-uniform
      const int r = base + k * stride + sub;
      const int kind = r < Hq ? 0 : (r < Hq + Hkv ? 1 : 2);
      const int head = kind == 0 ? r : (kind == 1 ? r - Hq : r - Hq - Hkv);
      const bool on = r < n_rows && e0 < (kind == 2 ? Dv : Dk);
      const bool qk = kind <= 1;
      float (&x)[8] = xs[k];
      const float* w = kind == 0 ? qw : kw;
      auto apply_norm = [&]() {                         // every lane takes part in the shuffles
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss += x[i] * x[i];
        ss = sub_sum<SW>(ss);
        if (qk && on && w != nullptr) {
          float wv[8];
          load8(w + e0, wv);
          const float rinv = 1.0f / sqrtf(ss / (float)Dk + a.eps);
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = x[i] * rinv * wv[i];
        }
      };
      if (qw != nullptr && !a.after_rope) apply_norm();
      if (kind_r != KVA_ROPE_NONE) {
        float* rowbuf = s_row[warp][sub];
        if (qk) store8(rowbuf + e0, x);
        __syncwarp();
        if (qk && on) {
          float y[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int dd = e0 + i - ro;                 // index inside the rotated range
            y[i] = x[i];
            if (dd >= 0 && dd < rw) {
              const float* xr = rowbuf + ro;
              if (kind_r == KVA_ROPE_INTERLEAVED) {
                const int j = dd < half ? dd : dd - half;
                const float ev = xr[2 * j], od = xr[2 * j + 1];
                y[i] = dd < half ? ev * s_cos[j] - od * s_sin[j] : od * s_cos[j] + ev * s_sin[j];
              } else if (kind_r == KVA_ROPE_2D) {
                const int b = dd / half, e2 = dd - b * half;
                const bool low = e2 < quarter;
                const int j = b * quarter + (low ? e2 : e2 - quarter);
                const float pv = xr[low ? dd + quarter : dd - quarter];
                y[i] = x[i] * s_cos[j] + (low ? -pv : pv) * s_sin[j];
              } else {                                  // 1D and sections: rotate-half over the range
                const bool low = dd < half;
                const int j = low ? dd : dd - half;
                const float pv = xr[low ? dd + half : dd - half];
                y[i] = x[i] * s_cos[j] + (low ? -pv : pv) * s_sin[j];
              }
            }
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = y[i];
        }
        __syncwarp();                                   // buffer reads done before the next row
      }
      if (qw != nullptr && a.after_rope) apply_norm();

      uint32_t par;
      const uint32_t word = quantise8(x, &par);         // q rows too: the shuffles need every lane
      if (!on) continue;
      if (kind == 0) {
        store8(reinterpret_cast<QOutT*>(a.q_out) + (tok * a.Hq + head) * Dk + e0, x);
      } else if (slot >= 0 && slot < a.c.capacity) {
        const int D = kind == 1 ? Dk : Dv, G = D / Q4_GROUP;
        const int64_t row = (int64_t)n * a.c.inst_rows + (int64_t)head * a.c.capacity + slot;
        uint32_t* codes = (kind == 1 ? a.c.k : a.c.v) + row * (D / 8);
        codes[(sl & 7) * G + (sl >> 3)] = word;
        if ((sl & 7) == 0) (kind == 1 ? a.c.ks : a.c.vs)[row * G + (sl >> 3)] = par;
      }
    }
  }
  // a long append must not have its SMs taken by a waiting persistent kernel
  griddep_launch_dependents();
}

// One thread per word of 8 codes; consecutive threads take consecutive words of a row.
template <typename OutT>
__global__ void __launch_bounds__(THREADS)
expand_q4_kernel(const __grid_constant__ ExpandQ4Args a) {
  const int wk = a.c.Dk / 8, wv = a.c.Dv / 8;
  const int per = wk + wv;                              // words of a slot, K then V
  griddep_wait();
  const int n = blockIdx.z, g = blockIdx.y;
  const int64_t total = (int64_t)a.T * per;
  for (int64_t i = (int64_t)blockIdx.x * THREADS + threadIdx.x; i < total; i += (int64_t)gridDim.x * THREADS) {
    const int t = (int)(i / per);
    int w = (int)(i - (int64_t)t * per);
    const bool is_k = w < wk;
    if (!is_k) w -= wk;
    const int32_t slot = a.slot[(int64_t)n * a.slot_stride + t];
    if (slot < 0 || slot >= a.c.capacity) continue;
    const int D = is_k ? a.c.Dk : a.c.Dv, G = D / Q4_GROUP;
    const int64_t row = (int64_t)n * a.c.inst_rows + (int64_t)g * a.c.capacity + slot;
    const uint32_t code = (is_k ? a.c.k : a.c.v)[row * (D / 8) + w];
    const int grp = w % G, first = Q4_GROUP * grp + 8 * (w / G);
    const uint32_t par = (is_k ? a.c.ks : a.c.vs)[row * G + grp];
    const float scale = bf16_lo(par), mid = bf16_hi(par);
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = fmaf(scale, (float)((int)((code >> (4 * e)) & 15u) - 8), mid);
    OutT* dst = reinterpret_cast<OutT*>(is_k ? a.dk : a.dv) + (int64_t)n * (is_k ? a.d_stride : a.d_stride_v) +
                ((int64_t)g * a.d_capacity + a.d_first + t) * D + first;
    store8(dst, y);
  }
  griddep_launch_dependents();
}

int num_sms_q4() {
  static int n = 0;
  if (n == 0) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        n <= 0)
      n = 152;
  }
  return n;
}

template <typename InT, typename QOutT>
cudaError_t launch_w(const AppendQ4Args& a, cudaStream_t s) {
  const int D = std::max(a.c.Dk, a.c.Dv);
  const int rows = (a.q ? a.Hq : 0) + 2 * a.c.Hkv, rpw = D <= 64 ? 4 : (D <= 128 ? 2 : 1);
  // row groups per token: about two CTAs per SM, at most one row set per warp
  const int64_t tokens = (int64_t)a.T * a.N;
  const int most = (rows + WARPS * rpw - 1) / (WARPS * rpw);
  const int groups = (int)std::max<int64_t>(1, std::min<int64_t>(most, 2 * num_sms_q4() / tokens));
  const dim3 grid(a.T, a.N, std::min(groups, 65535));
  if (D <= 64) return launch_pdl(append_q4_kernel<InT, QOutT, 8>, grid, dim3(THREADS), 0, s, a);
  if (D <= 128) return launch_pdl(append_q4_kernel<InT, QOutT, 16>, grid, dim3(THREADS), 0, s, a);
  return launch_pdl(append_q4_kernel<InT, QOutT, 32>, grid, dim3(THREADS), 0, s, a);
}

}  // namespace

cudaError_t launch_append_q4(const AppendQ4Args& a, kva_dtype in_dtype, kva_dtype q_out_dtype, cudaStream_t s) {
  if (a.c.Dk > MAX_D || a.c.Dv > MAX_D || a.rot_dim / 2 > MAX_ROPE_FREQ || a.N > 65535) return cudaErrorInvalidValue;
  if (in_dtype == KVA_BF16)
    return q_out_dtype == KVA_BF16 ? launch_w<bf16_t, bf16_t>(a, s) : launch_w<bf16_t, float>(a, s);
  return q_out_dtype == KVA_BF16 ? launch_w<float, bf16_t>(a, s) : launch_w<float, float>(a, s);
}

cudaError_t launch_expand_q4(const ExpandQ4Args& a, kva_dtype dst_dtype, cudaStream_t s) {
  const int64_t total = (int64_t)a.T * (a.c.Dk / 8 + a.c.Dv / 8);
  // enough CTAs for the whole GPU, each with a few words per thread
  const int64_t want = (total + THREADS - 1) / THREADS;
  const int64_t cap = std::max<int64_t>(1, (int64_t)num_sms_q4() * 16 / std::max(1, a.N * a.c.Hkv));
  const dim3 grid((unsigned)std::max<int64_t>(1, std::min(want, std::max(cap, want / 8))), a.c.Hkv, a.N);
  if (dst_dtype == KVA_BF16) return launch_pdl(expand_q4_kernel<bf16_t>, grid, dim3(THREADS), 0, s, a);
  return launch_pdl(expand_q4_kernel<float>, grid, dim3(THREADS), 0, s, a);
}

}  // namespace kva
