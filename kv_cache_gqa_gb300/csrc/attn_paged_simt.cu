// Attention of new tokens over a paged cache on the CUDA cores (kv_attn_paged).
//
// A unit is ROWS (8 or 16) query rows (token, head of the group) of one KV head; a step is 128 slots, 32 for each of
// the CTA's four warps, which keep their own running maximum, sum and output and join them at the unit's
// end (paged.cuh).  Each lane has the K row and the V row of its slot copied into the warp's shared memory (one bulk copy
// each, whatever page the slot is in); K of the next 32 slots is on its way during the weights' product, V during the
// scores.  A lane takes one key's scores against all rows (q rows broadcast from shared memory), the weights go
// through shared memory, and then a lane takes DV/32 columns of the output for all rows.  The reference maximum moves only
// when a score exceeds it by 2^8.
//
// Bound: long chunks by shared-memory reads (each key's q values, 16 rows of them, beside 64 multiply-adds per 4 dims): 512
// tokens behind 1536 slots at 16/8 heads of 128 take 370 us (20 TFLOP/s; lanes that read K and V from global
// memory themselves took 530), 2000 from the first one 1108.  Small batches by latency: one 768-slot sequence 14.6 us (34 so), seven
// ragged sequences 21.6 us (25 so).  64 single tokens over 500 to 4000 slots: 353 us, 3.6 TB/s, a tile of K and V at a time on its way.
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

constexpr int WARPS = 4, THREADS = WARPS * 32, KT = 32;
constexpr float RESCALE_LOG2 = 8.0f;

template <int DK, int DV, int ROWS>
struct Smem {
  static constexpr int LDK = DK + 4;              // floats of a K row: lanes that read a row each meet different banks
  static constexpr int K = KT * LDK, V = KT * DV; // of a warp
  static constexpr int TILES = WARPS * (K + V);
  static constexpr int Q = ROWS * DK, P = WARPS * KT * ROWS, ML = 2 * WARPS * ROWS, O = WARPS * ROWS * DV;
  static constexpr int REST = 4 * (Q + P > ML + O ? Q + P : ML + O);       // the join reuses q and the weights
  static constexpr int BYTES = 4 * TILES + REST;
};

template <int DK, int DV, int ROWS>
__global__ void __launch_bounds__(THREADS)
attn_paged_simt_kernel(const __grid_constant__ PagedArgs a) {
  using S = Smem<DK, DV, ROWS>;
  constexpr int NC = DV / 32, R = ROWS;
  extern __shared__ __align__(16) float smem[];
  __shared__ int64_t scratch[WARPS + 4];
  __shared__ uint64_t s_bar[WARPS][2];            // a warp's K and V have landed
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  float* tile_k = smem + warp * (S::K + S::V);
  float* tile_v = tile_k + S::K;
  float* sm = smem + S::TILES;
  float* sm_q = sm;
  float* sm_p = sm + S::Q + warp * KT * R;
  uint64_t* bar = s_bar[warp];
  if (lane == 0) {
    mbar_init(&bar[0], 1);
    mbar_init(&bar[1], 1);
    fence_mbar_init();
  }
  const Cut cut{R, KT * WARPS, a.Hq / a.Hkv, a.rows_lo, a.rows_hi};
  const int G = cut.G, page_mask = (1 << a.page_shift) - 1;
  griddep_wait();                               // inputs of this launch are complete from here on
  griddep_launch_dependents();
  Place p;
  const paged::Run run = paged::first_place<THREADS>(a, cut, scratch, &p);
  if (run.x0 >= run.x1) return;
  uint32_t phase = 0;
  bool ok = true;                               // no wait of this warp has given up

  for (; p.b < a.B && p.at < run.x1; p.next(a, cut)) {
    const int st0 = (int)max((int64_t)0, run.x0 - p.at), st1 = (int)min((int64_t)p.n_steps, run.x1 - p.at);
    const int rows = p.s.T * G;                 // the call's rows fit 32 bits
    const int lim_all = cut.visible(p.s, p.rt); // slots that the tile's last row sees
    const int32_t* pages = a.table + (int64_t)p.b * a.table_stride;
    const int first = (st0 * WARPS + warp) * KT;                  // first key of this warp's first tile
    const int n_mine = !ok ? 0 : max(0, min(st1 - st0, (lim_all - first + KT * WARPS - 1) / (KT * WARPS)));
    // this lane's slot of tile u: its rows in K and V, -1 for none; a page outside the pool makes its scores NaN
    int64_t at_k = -1, at_v = -1;
    bool bad = false;
    auto look_up = [&](int u) {
      const int key = first + u * (KT * WARPS) + lane;
      at_k = at_v = -1;
      bad = false;
      if (u >= n_mine || key >= lim_all) return;
      const int page = pages[key >> a.page_shift];
      bad = (unsigned)page >= (unsigned)a.n_pages;
      const int64_t pg = bad ? 0 : page;
      const int in = (p.g << a.page_shift) + (key & page_mask);
      at_k = pg * a.page_stride + (int64_t)in * DK;
      at_v = pg * a.page_stride_v + (int64_t)in * DV;
    };
    auto copy_k = [&]() {                       // whole warp
      const int n = __popc(__ballot_sync(FULL_MASK, at_k >= 0));
      if (lane == 0) mbar_arrive_expect_tx(&bar[0], n * DK * 4);
      __syncwarp();
      if (at_k >= 0) bulk_g2s(tile_k + lane * S::LDK, reinterpret_cast<const float*>(a.k) + at_k, DK * 4, &bar[0]);
    };
    auto copy_v = [&]() {
      const int n = __popc(__ballot_sync(FULL_MASK, at_v >= 0));
      if (lane == 0) mbar_arrive_expect_tx(&bar[1], n * DV * 4);
      __syncwarp();
      if (at_v >= 0) bulk_g2s(tile_v + lane * DV, reinterpret_cast<const float*>(a.v) + at_v, DV * 4, &bar[1]);
    };
    look_up(0);
    if (n_mine > 0) { copy_k(); copy_v(); }
    __syncthreads();                            // the unit before is done with q's place
    for (int i = tid; i < R * DK / 4; i += THREADS) {
      const int row = p.rt * R + i / (DK / 4);
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (row < rows) {
        x = __ldg(reinterpret_cast<const float4*>(reinterpret_cast<const float*>(a.q) +
                                                  ((int64_t)(p.s.t0 + row / G) * a.Hq + p.g * G + row % G) * DK) + i % (DK / 4));
        x.x *= a.scale_log2; x.y *= a.scale_log2; x.z *= a.scale_log2; x.w *= a.scale_log2;
      }
      reinterpret_cast<float4*>(sm_q)[i] = x;
    }
    __syncthreads();
    float m[R], l[R], o[R][NC];
    int lim[R];                                 // slots that row r sees
#pragma unroll
    for (int r = 0; r < R; ++r) {
      m[r] = M_NONE;
      l[r] = 0.f;
#pragma unroll
      for (int c = 0; c < NC; ++c) o[r][c] = 0.f;
      const int row = p.rt * R + r;
      lim[r] = row < rows ? min(max(p.s.L - p.s.T + row / G + 1, 0), p.s.L) : 0;
    }
    for (int u = 0; u < n_mine; ++u) {
      const int ks = first + u * (KT * WARPS), key = ks + lane;
      const bool wrong = bad;                   // of this tile's slot
      if (!paged::warp_wait(&bar[0], phase)) {
        ok = false;                             // gave up: the copy of V lands first (bounded)
        (void)paged::warp_wait(&bar[1], phase);
        break;
      }
      float s[R];
#pragma unroll
      for (int r = 0; r < R; ++r) s[r] = 0.f;
#pragma unroll 4
      for (int d = 0; d < DK; d += 4) {
        const float4 kk = *reinterpret_cast<const float4*>(tile_k + lane * S::LDK + d);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float4 qv = *reinterpret_cast<const float4*>(sm_q + r * DK + d);
          s[r] = fmaf(qv.x, kk.x, fmaf(qv.y, kk.y, fmaf(qv.z, kk.z, fmaf(qv.w, kk.w, s[r]))));
        }
      }
      __syncwarp();                             // K is read
      if (u + 1 < n_mine) {
        look_up(u + 1);
        copy_k();
      }
      bool grow = false;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (wrong) s[r] = NAN;
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
      if (!paged::warp_wait(&bar[1], phase)) {
        ok = false;                             // gave up: the next copy of K lands first (bounded)
        if (u + 1 < n_mine) (void)paged::warp_wait(&bar[0], phase ^ 1);
        break;
      }
      const int n = min(KT, lim_all - ks);
      auto value = [&](int j, float (&vv)[NC]) {
        if constexpr (NC == 4) {
          const float4 x = *reinterpret_cast<const float4*>(tile_v + j * DV + lane * 4);
          vv[0] = x.x; vv[1] = x.y; vv[2] = x.z; vv[3] = x.w;
        } else {
          const float2 x = *reinterpret_cast<const float2*>(tile_v + j * DV + lane * 2);
          vv[0] = x.x; vv[1] = x.y;
        }
      };
      const int common = max(0, min(n, lim[0] - ks));        // keys that all rows see (the first row sees the fewest)
#pragma unroll 8
      for (int j = 0; j < common; ++j) {
        float vv[NC];
        value(j, vv);
#pragma unroll
        for (int r = 0; r < R; r += 4) {
          const float4 w = *reinterpret_cast<const float4*>(sm_p + j * R + r);
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            o[r][c] = fmaf(w.x, vv[c], o[r][c]);
            o[r + 1][c] = fmaf(w.y, vv[c], o[r + 1][c]);
            o[r + 2][c] = fmaf(w.z, vv[c], o[r + 2][c]);
            o[r + 3][c] = fmaf(w.w, vv[c], o[r + 3][c]);
          }
        }
      }
      // The others, one less than the tile has tokens, meet only the rows that see them: a weight of 0 would make NaN of a NaN.
#pragma unroll 1
      for (int j = common; j < n; ++j) {
        float vv[NC];
        value(j, vv);
#pragma unroll
        for (int r = 0; r < R; ++r)
          if (ks + j < lim[r]) {
            const float w = sm_p[j * R + r];
#pragma unroll
            for (int c = 0; c < NC; ++c) o[r][c] = fmaf(w, vv[c], o[r][c]);
          }
      }
      __syncwarp();                             // V and the weights are read
      if (u + 1 < n_mine) copy_v();
      phase ^= 1;
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
      if (lane == 0) { sm_m[warp * R + r] = m[r]; sm_l[warp * R + r] = ok ? l[r] : NAN; }
#pragma unroll
      for (int c = 0; c < NC; ++c) sm_o[r * DV + lane * NC + c] = o[r][c];
    }
    paged::finish_unit<R, DV, WARPS, S::REST>(a, cut, p, run, st0, st1, sm);
  }
}

template <int DK, int DV, int ROWS>
cudaError_t launch_t(const PagedArgs& a, int runs, cudaStream_t s) {
  constexpr int smem = Smem<DK, DV, ROWS>::BYTES;
  static DeviceOnce configured;
  if (!configured.done()) {
    const cudaError_t e = cudaFuncSetAttribute(attn_paged_simt_kernel<DK, DV, ROWS>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    configured.mark();
  }
  return launch_pdl(attn_paged_simt_kernel<DK, DV, ROWS>, dim3(runs), dim3(THREADS), (size_t)smem, s, a);
}

template <int DK, int DV>
cudaError_t launch_d(const PagedArgs& a, int rows, int runs, cudaStream_t s) {
  return rows <= 8 ? launch_t<DK, DV, 8>(a, runs, s) : launch_t<DK, DV, 16>(a, runs, s);
}

}  // namespace

cudaError_t launch_attn_paged_simt(const PagedArgs& a, int Dk, int rows, int runs, cudaStream_t s) {
  if (Dk == 64) return launch_d<64, 64>(a, rows, runs, s);
  if (Dk == 128) return launch_d<128, 128>(a, rows, runs, s);
  return launch_d<192, 128>(a, rows, runs, s);
}

}  // namespace kva
