// Attention over a paged bf16 cache in tiles of up to 16 query rows (kv_attn_paged): single tokens and short draft blocks (up
// to 16 rows (token, head of the group) a KV head), and chunks of any length where the output is float32.
//
// A unit is a row tile of a (sequence, KV head), a step 64 slots: 16 for each of the CTA's four warps, which are independent until
// the unit's end.  A warp streams its 16-key tiles through a ring of NS shared-memory stages: lane 0 issues TMA copies,
// [16 keys x 64 dims] boxes with 128-byte swizzle, whose page the warp has looked up 32 tiles ahead (a page
// holds whole tiles), and ldmatrix reads them without bank conflicts.  Per tile mma.sync m16n8k16 forms S = q K^T,
// the softmax keeps a reference maximum that moves only when a score exceeds it by 2^8, and P V follows with P
// taken from the score registers.  All units' steps are cut into equal runs (paged.cuh), so ragged batches leave no CTA behind.
//
// Weights meet V as two bf16 parts, 16 bits: a bf16 output's own rounding then outweighs theirs, and a sequence keeps them whoever
// shares its launch.  With at most 8 rows (ROWS = 8) the tile's other 8 rows hold the second part, at no cost.  EXACT (a float32
// output) adds a third part, 24 bits, and keeps the tensor core's sums to one tile, joined by float32 additions: it cuts sums
// off towards zero, which over a long run would show (7e-6).
//
// Bound: many long sequences by HBM (64 of 1k to 32k slots at 16/8 heads of 128, 4.7 GB: 673 us, 7.0 TB/s; 64 of 500 to 4000, 650 MB:
// 108 us, 6.0 TB/s; 64 blocks of 4 and of 8 tokens over 2048 slots 90 and 96 us; 16 blocks of head dims 192/128 with float32 out, 892 MB:
// 145 us, 6.1 TB/s, its third part and short sums beside the loads); one sequence by latency (768 slots 10.4 us: the plan, a table
// read, one ring's loads, the join of the parts).  Chunks with float32 out read K and V again for every 16 rows: 512 tokens behind 1536
// slots 95 us, 2048 behind 30000 at 32/8 heads 7.0 ms (the tcgen05 form's bf16 out: 0.74).
//
// Method: one pass over the keys with the running maximum and sum of the softmax; GQA by repeat-interleave
// grouping (Penguin-VL ncnn port, section 3), the visible prefix of decode and verify steps (Youtu-VL-4B ncnn
// port, step 8; HunyuanOCR v1.5 ncnn port, section 3.8), bf16 storage with fp32 accumulation (section 3.7 there).
#include "paged.cuh"
#include "tc.cuh"

namespace kva {

namespace {

using paged::Cut;
using paged::ex2;
using paged::finite_pair;
using paged::M_NONE;
using paged::Place;
using paged::saw_odd;
using paged::see_pair;

constexpr int WARPS = 4, THREADS = WARPS * 32;
constexpr int KT = 16;                          // keys of a warp's tile
constexpr int BOX = KT * 128;                   // one [16 keys x 64 dims] swizzled box
constexpr float RESCALE_LOG2 = 8.0f;

template <int DK, int DV, int ROWS>
struct Shape {
  static constexpr int STAGE = (DK + DV) / 64 * BOX;
  static constexpr int NS = DK == 64 ? 6 : (DK == 128 ? 3 : 2);   // about 100 KB a CTA, two CTAs an SM
  static constexpr int RING = NS * STAGE;                          // per warp
  static constexpr int BAR = WARPS * RING;
  static constexpr int SMEM = BAR + WARPS * NS * 8 + 1024;         // + slack to align the base to 1024
  static_assert(4 * (2 * WARPS * ROWS + WARPS * ROWS * DV) <= BAR, "the join reuses the rings");
};

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
// D = A B + D: rows g = lane / 4 (a0, a2) and g + 8 (a1, a3)
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// byte offset of 16-byte chunk `ch` of key row `key` inside a 128-byte-swizzled box
__device__ __forceinline__ uint32_t swz(int key, int ch) { return key * 128 + ((ch ^ (key & 7)) << 4); }

template <int DK, int DV, int ROWS, bool EXACT>
__global__ void __launch_bounds__(THREADS, 2)
attn_paged_step_kernel(const __grid_constant__ PagedArgs a, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV) {
  using S = Shape<DK, DV, ROWS>;
  constexpr int NS = S::NS, KB = DK / 64, VB = DV / 64, NT = DV / 8, H = ROWS / 8;   // H: row sets with rows of their own
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ int64_t scratch[WARPS + 4];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = lane >> 2, t = lane & 3;
  unsigned char* ring = smem + warp * S::RING;
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + S::BAR) + warp * NS;
  if (lane == 0) {
    for (int s = 0; s < NS; ++s) mbar_init(&bar[s], 1);
    fence_mbar_init();
    if (warp == 0) { tc::tma_prefetch_desc(&tmK); tc::tma_prefetch_desc(&tmV); }
  }
  const Cut cut{ROWS, KT * WARPS, a.Hq / a.Hkv, a.rows_lo, a.rows_hi};
  const int G = cut.G, page_mask = (1 << a.page_shift) - 1;
  griddep_wait();                               // inputs of this launch are complete from here on
  griddep_launch_dependents();
  Place p;
  const paged::Run run = paged::first_place<THREADS>(a, cut, scratch, &p);
  if (run.x0 >= run.x1) return;
  int slot = 0;                                 // the ring's next stage and its phase
  uint32_t phase = 0;
  bool ok = true;                               // no wait of this warp has given up

  for (; p.b < a.B && p.at < run.x1; p.next(a, cut)) {
    const int st0 = (int)max((int64_t)0, run.x0 - p.at), st1 = (int)min((int64_t)p.n_steps, run.x1 - p.at);
    const int64_t rows = (int64_t)p.s.T * G - (int64_t)p.rt * ROWS;    // of this tile and the ones behind it
    const int lim_all = cut.visible(p.s, p.rt); // slots that the tile's last row sees
    const int first = (st0 * WARPS + warp) * KT;                  // first key of this warp's first tile
    const int n_mine = !ok ? 0 : max(0, min(st1 - st0, (lim_all - first + KT * WARPS - 1) / (KT * WARPS)));
    const int32_t* pages = a.table + (int64_t)p.b * a.table_stride;
    // pages of tiles u .. u + 31, a lane each
    bool bad = false;
    int ahead = 0;
    auto look_up = [&](int u) {
      const int key = first + (u + lane) * (KT * WARPS);
      ahead = 0;
      if (u + lane < n_mine) {
        ahead = pages[key >> a.page_shift];
        if ((unsigned)ahead >= (unsigned)a.n_pages) { bad = true; ahead = a.n_pages; }   // outside: the copies read zeros
      }
    };
    auto issue = [&](int u, int stage) {        // whole warp; tile u into ring stage `stage`
      if ((u & 31) == 0) look_up(u);
      const int page = __shfl_sync(FULL_MASK, ahead, u & 31);
      if (lane == 0) {
        const int row = (first + u * (KT * WARPS)) & page_mask;
        unsigned char* dst = ring + stage * S::STAGE;
        mbar_arrive_expect_tx(&bar[stage], S::STAGE);
#pragma unroll
        for (int c = 0; c < KB; ++c) tc::tma_load_4d(dst + c * BOX, &tmK, c * 64, row, p.g, page, &bar[stage]);
#pragma unroll
        for (int c = 0; c < VB; ++c) tc::tma_load_4d(dst + (KB + c) * BOX, &tmV, c * 64, row, p.g, page, &bar[stage]);
      }
    };
    auto after = [](int s, int n) { return s + n >= NS ? s + n - NS : s + n; };
    for (int u = 0; u < NS && u < n_mine; ++u) issue(u, after(slot, u));

    // ---- query fragments: row r (and r + 8), k pairs 2t, 2t + 8 of 16-wide slices ----
    uint32_t qa[H][DK / 16][2];
    int lim[H];                                 // slots that row r (+ 8) sees
    int lim_min = lim_all;                      // and what every row sees
#pragma unroll
    for (int h = 0; h < H; ++h) {
      const bool on = r + 8 * h < rows;
      const int row = on ? p.rt * ROWS + r + 8 * h : 0;
      lim[h] = on ? min(max(p.s.L - p.s.T + row / G + 1, 0), p.s.L) : lim_all;
      const uint16_t* q = reinterpret_cast<const uint16_t*>(a.q) +
                          ((int64_t)(p.s.t0 + row / G) * a.Hq + p.g * G + row % G) * DK + 2 * t;
#pragma unroll
      for (int kk = 0; kk < DK / 16; ++kk) {
        qa[h][kk][0] = on ? __ldg(reinterpret_cast<const uint32_t*>(q + 16 * kk)) : 0u;
        qa[h][kk][1] = on ? __ldg(reinterpret_cast<const uint32_t*>(q + 16 * kk + 8)) : 0u;
      }
      lim_min = min(lim_min, lim[h]);
    }
    lim_min = __reduce_min_sync(FULL_MASK, lim_min);

    float o[NT][EXACT && H == 1 ? 2 : 4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < (EXACT && H == 1 ? 2 : 4); ++e) o[n][e] = 0.f;
    float m[H], l[H];
#pragma unroll
    for (int h = 0; h < H; ++h) { m[h] = M_NONE; l[h] = 0.f; }

    for (int u = 0; u < n_mine; ++u) {
      if (!paged::warp_wait(&bar[slot], phase)) {
        ok = false;                             // gave up: the copies still in flight land first (bounded)
        for (int v = u + 1; v < n_mine && v < u + NS; ++v) {
          if (++slot == NS) { slot = 0; phase ^= 1; }
          (void)paged::warp_wait(&bar[slot], phase);
        }
        break;
      }
      unsigned char* stg = ring + slot * S::STAGE;
      const int ks = first + u * (KT * WARPS);
      if (ks + KT > lim_min) {                  // keys that some rows, or none, see: 0 times what they do not see must be 0
        unsigned char* sv = stg + KB * BOX;
        if (lim_min < lim_all) {
          uint32_t seen = 0u;
          for (int i = lane; i < KT * DV / 8; i += 32) {
            const uint4 x = *reinterpret_cast<const uint4*>(sv + i * 16);
            see_pair(seen, x.x); see_pair(seen, x.y); see_pair(seen, x.z); see_pair(seen, x.w);
          }
          if (__builtin_expect(__any_sync(FULL_MASK, saw_odd(seen)), 0)) {
#pragma unroll 1
            for (int j = 0; j < KT; ++j)        // a NaN or infinity: NaN for the rows that see it,
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                const uint32_t x = *reinterpret_cast<const uint32_t*>(sv + (n >> 3) * BOX + swz(j, n & 7) + 4 * t), odd = x ^ finite_pair(x);
#pragma unroll
                for (int h = 0; h < H; ++h) {
                  if ((odd & 0xffffu) && ks + j < lim[h]) o[n][2 * h] = NAN;
                  if ((odd >> 16) && ks + j < lim[h]) o[n][2 * h + 1] = NAN;
                }
              }
            __syncwarp();
#pragma unroll 1
            for (int i = lane; i < KT * DV / 8; i += 32) {           // and 0 for the products
              uint4* x = reinterpret_cast<uint4*>(sv + i * 16);
              const uint4 v = *x;
              *x = make_uint4(finite_pair(v.x), finite_pair(v.y), finite_pair(v.z), finite_pair(v.w));
            }
            fence_proxy_async_smem();           // before the stage's next copies
          }
        }
        const int nk = max(0, lim_all - ks);
        for (int i = lane; i < (KT - nk) * (DV / 8); i += 32) {
          const int key = nk + i / (DV / 8), ch = i % (DV / 8);
          *reinterpret_cast<uint4*>(sv + (ch / 8) * BOX + swz(key, ch % 8)) = make_uint4(0, 0, 0, 0);
        }
        __syncwarp();
      }
      const uint32_t sK = smem_u32(stg), sV = sK + KB * BOX;
      // ---- S: keys 0..7 and 8..15 ----
      float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
      {
        const int mi = lane >> 3, rr = lane & 7, key = rr + 8 * (mi >> 1);
#pragma unroll
        for (int kk = 0; kk < DK / 16; ++kk) {
          uint32_t bf[4];
          ldsm_x4(sK + (kk >> 2) * BOX + swz(key, ((kk & 3) << 1) + (mi & 1)), bf);
          const uint32_t a1 = H == 2 ? qa[H - 1][kk][0] : 0u, a3 = H == 2 ? qa[H - 1][kk][1] : 0u;
          mma16816(s0, qa[0][kk][0], a1, qa[0][kk][1], a3, bf[0], bf[1]);
          mma16816(s1, qa[0][kk][0], a1, qa[0][kk][1], a3, bf[2], bf[3]);
        }
      }
      // ---- softmax of this lane's keys 2t, 2t + 1, 8 + 2t, 9 + 2t ----
      float w[H][4];
      bool grow = false;
#pragma unroll
      for (int h = 0; h < H; ++h) {
        w[h][0] = s0[2 * h] * a.scale_log2; w[h][1] = s0[2 * h + 1] * a.scale_log2;
        w[h][2] = s1[2 * h] * a.scale_log2; w[h][3] = s1[2 * h + 1] * a.scale_log2;
      }
      if (ks + KT > lim_min) {
#pragma unroll
        for (int h = 0; h < H; ++h) {
          const int left = lim[h] - ks - 2 * t;
          if (left <= 0) w[h][0] = -INFINITY;
          if (left <= 1) w[h][1] = -INFINITY;
          if (left <= 8) w[h][2] = -INFINITY;
          if (left <= 9) w[h][3] = -INFINITY;
        }
      }
      float mt[H];
#pragma unroll
      for (int h = 0; h < H; ++h) {
        mt[h] = fmaxf(fmaxf(w[h][0], w[h][1]), fmaxf(w[h][2], w[h][3]));
        grow |= mt[h] > m[h] + RESCALE_LOG2;
      }
      if (__any_sync(FULL_MASK, grow)) {
#pragma unroll
        for (int h = 0; h < H; ++h) {
          mt[h] = fmaxf(mt[h], __shfl_xor_sync(FULL_MASK, mt[h], 1));
          mt[h] = fmaxf(mt[h], __shfl_xor_sync(FULL_MASK, mt[h], 2));
          float alpha = 1.f;                    // uniform over the row's four lanes
          if (mt[h] > m[h] + RESCALE_LOG2) {
            alpha = ex2(m[h] - mt[h]);
            m[h] = mt[h];
          }
          l[h] *= alpha;
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            o[n][2 * h] *= alpha; o[n][2 * h + 1] *= alpha;
            if constexpr (H == 1 && !EXACT) { o[n][2] *= alpha; o[n][3] *= alpha; }
          }
        }
      }
      // ---- weights as bf16 parts ----
      uint32_t hi[H][2], mid[H][2], lo[H][2];
#pragma unroll
      for (int h = 0; h < H; ++h)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float p0 = ex2(w[h][2 * i] - m[h]), p1 = ex2(w[h][2 * i + 1] - m[h]);
          hi[h][i] = pack_bf16x2(p0, p1);
          l[h] += p0 + p1;
          const float r0 = p0 - bf16_lo(hi[h][i]), r1 = p1 - bf16_hi(hi[h][i]);
          mid[h][i] = pack_bf16x2(r0, r1);
          if constexpr (EXACT) lo[h][i] = pack_bf16x2(r0 - bf16_lo(mid[h][i]), r1 - bf16_hi(mid[h][i]));
        }
      // ---- O += P V ----
      {
        const int mi = lane >> 3, rr = lane & 7, key = rr + 8 * (mi & 1);
#pragma unroll
        for (int nd = 0; nd < NT / 2; ++nd) {
          uint32_t bf[4];
          ldsm_x4_t(sV + (nd >> 2) * BOX + swz(key, ((nd & 3) << 1) + (mi >> 1)), bf);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t b0 = bf[2 * j], b1 = bf[2 * j + 1];
            if constexpr (EXACT) {
              float z[4] = {0.f, 0.f, 0.f, 0.f};
              if constexpr (H == 1) {
                mma16816(z, lo[0][0], 0u, lo[0][1], 0u, b0, b1);
                mma16816(z, hi[0][0], mid[0][0], hi[0][1], mid[0][1], b0, b1);
                o[2 * nd + j][0] += z[0] + z[2];
                o[2 * nd + j][1] += z[1] + z[3];
              } else {
                mma16816(z, lo[0][0], lo[H - 1][0], lo[0][1], lo[H - 1][1], b0, b1);
                mma16816(z, mid[0][0], mid[H - 1][0], mid[0][1], mid[H - 1][1], b0, b1);
                mma16816(z, hi[0][0], hi[H - 1][0], hi[0][1], hi[H - 1][1], b0, b1);
#pragma unroll
                for (int e = 0; e < 4; ++e) o[2 * nd + j][e] += z[e];
              }
            } else if constexpr (H == 1) {
              mma16816(o[2 * nd + j], hi[0][0], mid[0][0], hi[0][1], mid[0][1], b0, b1);
            } else {
              mma16816(o[2 * nd + j], mid[0][0], mid[H - 1][0], mid[0][1], mid[H - 1][1], b0, b1);
              mma16816(o[2 * nd + j], hi[0][0], hi[H - 1][0], hi[0][1], hi[H - 1][1], b0, b1);
            }
          }
        }
      }
      __syncwarp();                             // all lanes are done with this stage
      if (u + NS < n_mine) {
        if (lane == 0) fence_proxy_async_smem();   // this stage's generic accesses before the refill
        issue(u + NS, slot);
      }
      if (++slot == NS) { slot = 0; phase ^= 1; }
    }
    bad = __any_sync(FULL_MASK, bad);
#pragma unroll
    for (int h = 0; h < H; ++h) {
      l[h] += __shfl_xor_sync(FULL_MASK, l[h], 1);
      l[h] += __shfl_xor_sync(FULL_MASK, l[h], 2);
      if (bad || !ok) l[h] = NAN;
    }
    // ---- join the warps (the rings are drained) ----
    __syncthreads();
    float* sm = reinterpret_cast<float*>(smem);
    float* sm_o = sm + 2 * WARPS * ROWS + warp * ROWS * DV;
#pragma unroll
    for (int h = 0; h < H; ++h) {
      const int row = r + 8 * h;
      if (t == 0) { sm[warp * ROWS + row] = m[h]; sm[(WARPS + warp) * ROWS + row] = l[h]; }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float x0 = o[n][2 * h], x1 = o[n][2 * h + 1];
        if constexpr (H == 1 && !EXACT) { x0 += o[n][2]; x1 += o[n][3]; }
        *reinterpret_cast<float2*>(sm_o + row * DV + 8 * n + 2 * t) = make_float2(x0, x1);
      }
    }
    paged::finish_unit<ROWS, DV, WARPS, S::BAR>(a, cut, p, run, st0, st1, sm);
    fence_proxy_async_smem();                   // the join's accesses before the next unit's copies
    __syncthreads();
  }
}

template <int DK, int DV, int ROWS, bool EXACT>
cudaError_t launch_t(const PagedArgs& a, const CUtensorMap& mk, const CUtensorMap& mv, int runs, cudaStream_t s) {
  constexpr int smem = Shape<DK, DV, ROWS>::SMEM;
  static DeviceOnce configured;
  if (!configured.done()) {
    const cudaError_t e = cudaFuncSetAttribute(attn_paged_step_kernel<DK, DV, ROWS, EXACT>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    configured.mark();
  }
  return launch_pdl(attn_paged_step_kernel<DK, DV, ROWS, EXACT>, dim3(runs), dim3(THREADS), (size_t)smem, s, a, mk, mv);
}

template <int DK, int DV>
cudaError_t launch_d(const PagedArgs& a, int rows, int runs, cudaStream_t s) {
  CUtensorMap mk, mv;
  cudaError_t e = paged_pool_map(&mk, a.k, a, DK, a.page_stride, KT);
  if (e != cudaSuccess || (e = paged_pool_map(&mv, a.v, a, DV, a.page_stride_v, KT)) != cudaSuccess) return e;
  if (rows <= 8) return a.out_bf16 ? launch_t<DK, DV, 8, false>(a, mk, mv, runs, s) : launch_t<DK, DV, 8, true>(a, mk, mv, runs, s);
  return a.out_bf16 ? launch_t<DK, DV, 16, false>(a, mk, mv, runs, s) : launch_t<DK, DV, 16, true>(a, mk, mv, runs, s);
}

}  // namespace

cudaError_t launch_attn_paged_step(const PagedArgs& a, int Dk, int rows, int runs, cudaStream_t s) {
  if (Dk == 64) return launch_d<64, 64>(a, rows, runs, s);
  if (Dk == 128) return launch_d<128, 128>(a, rows, runs, s);
  return launch_d<192, 128>(a, rows, runs, s);
}

}  // namespace kva
