// Attention of new tokens over a 4-bit cache (kv_attn_decode_q4): one warp per query row.  A lane
// scores one key of a 32-key tile, then the lanes turn to the value dims.
#include <algorithm>

#include "common.cuh"
#include "launch.h"

namespace kva {

namespace {

__device__ __forceinline__ float code_value(uint32_t w, int i, uint32_t par) {
  return fmaf(bf16_lo(par), (float)((int)((w >> (4 * i)) & 15u) - 8), bf16_hi(par));
}

template <typename QT, int DK, int DV>
__global__ void __launch_bounds__(32)
decode_q4_kernel(const __grid_constant__ DecodeQ4Args a) {
  constexpr int GK = DK / Q4_GROUP, GV = DV / Q4_GROUP, WK = DK / 8, WV = DV / 8, PER = DV / 32;
  __shared__ float s_q[DK];
  const int h = blockIdx.x, t = blockIdx.y, b = blockIdx.z, lane = threadIdx.x;
  const int g = h / (a.Hq / a.c.Hkv);
  griddep_wait();
  const int64_t qrow = ((int64_t)b * a.T + t) * a.Hq + h;
  for (int i = lane; i < DK; i += 32) s_q[i] = load1(reinterpret_cast<const QT*>(a.q) + qrow * DK + i) * a.scale_log2;
  __syncwarp();
  const int L = min(max(a.lengths[b], 0), a.c.capacity) - a.T + t + 1;      // visible slots
  const int64_t row0 = (int64_t)b * a.c.inst_rows + (int64_t)g * a.c.capacity;
  float m = -INFINITY, l = 0.f, o[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) o[i] = 0.f;
  for (int k0 = 0; k0 < L; k0 += 32) {
    float x = -INFINITY;
    if (k0 + lane < L) {
      x = 0.f;
      const int64_t row = row0 + k0 + lane;
      for (int w = 0; w < WK; ++w) {
        const uint32_t code = a.c.k[row * WK + w], par = a.c.ks[row * GK + w % GK];
        for (int i = 0; i < 8; ++i) x = fmaf(s_q[64 * (w % GK) + 8 * (w / GK) + i], code_value(code, i, par), x);
      }
    }
    float mt = x;
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) mt = fmaxf(mt, __shfl_xor_sync(FULL_MASK, mt, s));
    mt = fmaxf(mt, m);
    const float p = exp2f(x - mt), alpha = exp2f(m - mt);
    m = mt;
    l = l * alpha + p;
#pragma unroll
    for (int i = 0; i < PER; ++i) o[i] *= alpha;
    for (int j = 0; j < 32 && k0 + j < L; ++j) {
      const float pj = __shfl_sync(FULL_MASK, p, j);
      const int64_t row = row0 + k0 + j;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int d = lane + 32 * i, gr = d / 64, w = (d % 64 / 8) * GV + gr;
        o[i] = fmaf(pj, code_value(a.c.v[row * WV + w], d & 7, a.c.vs[row * GV + gr]), o[i]);
      }
    }
  }
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) l += __shfl_xor_sync(FULL_MASK, l, s);
#pragma unroll
  for (int i = 0; i < PER; ++i) a.out[qrow * DV + lane + 32 * i] = L > 0 ? o[i] / l : 0.f;
}

template <int DK, int DV>
cudaError_t launch_d(const DecodeQ4Args& a, kva_dtype q_dtype, cudaStream_t s) {
  const dim3 grid(a.Hq, a.T, a.B);
  if (q_dtype == KVA_BF16) return launch_pdl(decode_q4_kernel<bf16_t, DK, DV>, grid, dim3(32), 0, s, a);
  return launch_pdl(decode_q4_kernel<float, DK, DV>, grid, dim3(32), 0, s, a);
}

}  // namespace

bool decode_q4_supports(int Dk, int Dv) {
  return (Dk == 64 && Dv == 64) || (Dk == 128 && Dv == 128) || (Dk == 192 && Dv == 128);
}

int decode_q4_row_tile(int rows) { return rows <= 4 ? 4 : (rows <= 8 ? 8 : 16); }

int decode_q4_plan_chunk(const int32_t*, int, int, int max_len, int) { return max_len; }

cudaError_t launch_decode_q4(const DecodeQ4Args& a, kva_dtype q_dtype, cudaStream_t s) {
  if (a.c.Dk == 64) return launch_d<64, 64>(a, q_dtype, s);
  if (a.c.Dk == 128) return launch_d<128, 128>(a, q_dtype, s);
  return launch_d<192, 128>(a, q_dtype, s);
}

}  // namespace kva
