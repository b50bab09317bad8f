// Attention of new tokens over a 4-bit cache (kv_attn_decode_q4): split-KV, the codes fed to the
// tensor cores as they are.
//
// Work unit = (KV head g and tile of query rows, instance b): a walk over the instance's keys in stages
// of 32.  The query rows of a group are (token i, head j) -> i * G + j, 4, 8 or 16 a unit.  The stages of
// all units, in order, are cut into one equal run per CTA, as many CTAs as the GPU holds at once: a
// CTA ends one unit, takes whole ones and begins the next, so that ragged contexts leave no tail and a
// single long one still fills the GPU.  (Equal chunks of up to 2048 keys, one CTA each: 64 ragged sequences
// 282 us against 278, two contexts of 100k 104 against 80.)  A unit that several CTAs share is joined by the last of them to finish:
// they count themselves at the index of the first one, so that the counters lie in the same words of the workspace whatever
// the call's shape.  The runs follow from the lengths on the device: every CTA sums them itself.
//   A CTA's 4 warps are independent: warp w takes the stages w, w+4, ... of a run through a private ring,
// filled by 1-D bulk copies (a head's codes and scales are contiguous in the cache).  Per 16 keys:
//   S^T = K q^T   keys are the 16 rows of the MMA, query rows its 8 columns.  A 4-bit code u taken
//                 out of a word by one AND is the float16 subnormal u 2^-24 (or u 2^-20 for the odd
//                 nibble), so K needs 5 instructions per 8 codes; q is scaled by a power of two per
//                 row so that its float16 loses nothing: bf16 as it is, float32 as multiples of 2^-11
//                 of the largest element, whose sums stay exact, and what is left, summed apart.
//                 Scale and midpoint of a group enter in float32 after the product:
//                   s = sum_g scale_g (u . q)_g + (mid_g - 8 scale_g) sum(q)_g.
//   softmax       online, against a reference maximum that moves only when a score exceeds it by
//                 more than 2^5, float32
//   O^T += V^T P  value dims are the MMA's rows, keys its K axis.  The weights p * scale_g are two
//                 float16 halves, 22 bits against a power of two that each tile and group takes from its
//                 largest scale (2^9 to 2^10 where p = 1) and that leaves again with the products: a group or
//                 key of large scale takes no bits from the others.  A weight below 2^-3 there loses bits to
//                 float16's 2^-24: with S the tile's largest scale of the group it is off by at most
//                 2^-22 of itself and 2^-34 S; with at most 4 rows the second halves are held 2^11
//                 times, and it is 2^-45 S (the same with more rows took a product more: 144 us instead of 136 on
//                 blocks).  They turn from S^T's layout to the operand layout with movmatrix.  The codes are
//                 centred in the operand, (u - 8) 2^-9 by one multiply-add of halves: else O would be
//                 the small difference of sums of positive codes.  The tensor core cuts a sum off
//                 towards zero: kept in its accumulators, the sums of 64 long sequences came out
//                 7e-6 too small.  So it sums 16 or 32 keys, which float32 additions join (6e-7;
//                 1-2% slower, 6% with 16 rows).
//                 mid enters as sum p mid_g in float32.
// With at most 4 query rows the two halves of the weights (and of q) share the 8 columns.  The
// contraction runs over code positions, so the order of a row's words (kv_attn.h) only decides that
// a lane's codes of K, and of V, are adjacent bytes.
//
// Bound: no single unit.  64 sequences of 1k to 32k tokens run at 4.3 TB/s (282 us; HBM would take 180): 66% of
// the issue slots are used, the logic pipe 57% of the time, the tensor pipe 22%, DRAM 54%.  Of a 16-key tile's about 367 warp
// instructions a warp waits, each time, for a fixed latency (0.9 of an issue), for the pipe it needs (0.9) or for
// its turn (1.2); for memory 0.2.  More warps per SM or more tiles in flight per warp did not change the time.
//
// Method: attention over the valid prefix of the cache (Youtu-VL-4B ncnn port, step 8), GQA grouping
// (Penguin-VL ncnn port, section 3), softmax as max/subtract/exp/sum/divide (Youtu-VL-4B ncnn port,
// implementation difficulty 3); the 4-bit cache has no counterpart on the pages.
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "common.cuh"
#include "launch.h"

namespace kva {

namespace {

constexpr int WARPS = 4;
constexpr int THREADS = WARPS * 32;
constexpr int SK = 32;                          // keys per stage
constexpr int NS = 3;                           // ring stages per warp
constexpr float RESCALE_LOG2 = 5.0f;            // a row's reference max lags its true max by <= 2^5
constexpr float GRID = 100663296.f;              // 1.5 2^26: adding it rounds to a multiple of 8
constexpr float M_NONE = -3.0e38f;              // reference max of a row that has seen no key

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Transpose of an 8 x 8 matrix of 16-bit elements held as one register a lane.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 unpack_f16x2(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2*>(&v)); }
// N consecutive 32-bit words of shared memory at an address that is a multiple of 4 N bytes (of 16 at most; odd N: 4)
template <int N>
__device__ __forceinline__ void load_words(const unsigned char* p, uint32_t (&w)[N]) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const uint4 q = *reinterpret_cast<const uint4*>(p + 4 * i);
      w[i] = q.x; w[i + 1] = q.y; w[i + 2] = q.z; w[i + 3] = q.w;
    }
  } else if constexpr (N % 2 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const uint2 q = *reinterpret_cast<const uint2*>(p + 4 * i);
      w[i] = q.x; w[i + 1] = q.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = *reinterpret_cast<const uint32_t*>(p + 4 * i);
  }
}
__device__ __forceinline__ float pow2(int biased) { return __uint_as_float((uint32_t)biased << 23); }
__device__ __forceinline__ int exponent(float x) { return (int)((__float_as_uint(x) >> 23) & 255u); }

template <int DK, int DV, int MODE, bool SPLITQ>
struct Shape {
  static constexpr int GK = DK / Q4_GROUP, GV = DV / Q4_GROUP;
  static constexpr int NB = MODE == 2 ? 2 : 1;              // 8-column blocks of query rows
  static constexpr int ROWS = MODE == 0 ? 4 : 8 * NB;
  static constexpr int KC = SK * DK / 2, VC = SK * DV / 2, KP = SK * GK * 4, VP = SK * GV * 4;
  static constexpr int STAGE = KC + VC + KP + VP;
  static constexpr int RING = NS * STAGE;
  static constexpr int MERGE = WARPS * ROWS * (DV + 2) * 4;
  static constexpr int QP = MODE != 0 && SPLITQ ? 2 : 1;    // products per K fragment and block
  static constexpr bool QS = MODE == 2;                     // query fragments in shared memory
  static constexpr int QF = QS ? NB * QP * GK * 4 * 256 : 0;
  static constexpr int BAR = (WARPS * RING > MERGE ? WARPS * RING : MERGE) + QF;
  static constexpr int SMEM = BAR + WARPS * NS * 8;
  static constexpr int SUB = MODE == 0 ? 2 : 1;            // 16-key tiles worked on together
  static constexpr int CTAS = MODE == 0 && DK <= 128 ? 4 : 3;   // resident per SM, for the register limit
};

// MODE 0: up to 4 rows, halves side by side in the 8 columns; 1: 8 rows; 2: 16 rows.
// SPLITQ: float32 queries (two halves); else bf16 (exact in one).
template <int DK, int DV, int MODE, bool SPLITQ>
__global__ void __launch_bounds__(THREADS, (Shape<DK, DV, MODE, SPLITQ>::CTAS))
decode_q4_kernel(const __grid_constant__ DecodeQ4Args a) {
  using S = Shape<DK, DV, MODE, SPLITQ>;
  constexpr int GK = S::GK, GV = S::GV, NB = S::NB, ROWS = S::ROWS, QP = S::QP, SUB = S::SUB;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ float s_M[ROWS], s_L[ROWS], s_alpha[ROWS];
  __shared__ int s_last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = lane >> 2, t = lane & 3;
  const int G = a.Hq / a.c.Hkv, n_rows = G * a.T, units = a.c.Hkv * a.RT;
  unsigned char* ring = smem + warp * S::RING;
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + S::BAR) + warp * NS;
  if (lane == 0) {
    for (int s = 0; s < NS; ++s) mbar_init(&bar[s], 1);
    fence_mbar_init();
  }
  __syncwarp();
  griddep_wait();                               // inputs of this launch are complete from here on
  griddep_launch_dependents();

  // ---- this CTA's run: stages [x, x_end) of all units in order (instance, KV head, row tile) ----
  auto length = [&](int i) { return min(max(a.lengths[i], 0), a.c.capacity); };
  auto stages_of = [&](int i) { return (length(i) + SK - 1) / SK; };
  const int c = blockIdx.x;
  for (int i = c; i < a.B; i += gridDim.x)      // instances that see nothing: zeros
    if (length(i) == 0) {
      const int64_t n = (int64_t)a.T * a.Hq * DV;
      for (int64_t k = tid; k < n; k += THREADS) a.out[i * n + k] = 0.f;
    }
  int b, n_cta = 1;
  int64_t total = 1, base = 0, x, x_end;        // base: first stage of instance b
  auto start_of = [&](int cta) { return total * cta / n_cta; };
  auto cta_of = [&](int64_t stage) { return (int)(((stage + 1) * n_cta - 1) / total); };
  if (a.whole) {                                // one unit each
    b = c / units;
    const int stages = stages_of(b);
    if (stages == 0) return;
    x = (int64_t)(c % units) * stages;
    x_end = x + stages;
  } else {
    __shared__ int64_t s_sum[WARPS], s_base;
    __shared__ int s_inst;
    const int per = (a.B + THREADS - 1) / THREADS, i0 = min(a.B, tid * per), i1 = min(a.B, i0 + per);
    int64_t mine = 0;                           // stages of the instances i0 .. i1 - 1, per unit
    for (int i = i0; i < i1; ++i) mine += stages_of(i);
    int64_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(FULL_MASK, upto, o);
      if (lane >= o) upto += v;
    }
    if (lane == 31) s_sum[warp] = upto;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      if (w < warp) upto += s_sum[w];
      total += s_sum[w];
    }
    total *= units;
    n_cta = (int)min((int64_t)gridDim.x, total);   // every run has a stage
    if (c >= n_cta) return;
    x = start_of(c);
    x_end = start_of(c + 1);
    int64_t at = (upto - mine) * units;         // stages before instance i0
    if (at <= x && x < upto * units) {          // one thread's
      int i = i0;
      for (; x >= at + (int64_t)stages_of(i) * units; ++i) at += (int64_t)stages_of(i) * units;
      s_inst = i;
      s_base = at;
    }
    __syncthreads();
    b = s_inst;
    base = s_base;
  }
  const int64_t x0 = x;

  int slot = 0;                                 // ring position of the next stage to use
  uint32_t phase = 0;
  bool ok = true;                               // false: a wait gave up, everything after it is void
  while (x < x_end) {
    const int L = length(b), stages = (L + SK - 1) / SK;
    if (x >= base + (int64_t)stages * units) {    // on to the next instance
      base += (int64_t)stages * units;
      ++b;
      continue;
    }
    const int unit = (int)((x - base) / stages), g = unit / a.RT, rt = unit % a.RT;
    const int64_t unit_at = base + (int64_t)unit * stages;
    const int st0 = (int)(x - unit_at), st1 = (int)min((int64_t)stages, x_end - unit_at);
    x = unit_at + st1;
    const int row_end = min(n_rows, (rt + 1) * ROWS);
    auto out_row = [&](int row) {                 // row of the tile -> its output
      const int rr = rt * ROWS + row;
      return a.out + (((int64_t)b * a.T + rr / G) * a.Hq + g * G + rr % G) * DV;
    };
    const int k1 = min(L, st1 * SK);
    const int n_mine = ok && st1 - st0 > warp ? (st1 - st0 - 1 - warp) / WARPS + 1 : 0;
    const int64_t row0 = (int64_t)b * a.c.inst_rows + (int64_t)g * a.c.capacity;
    const int slot0 = slot;                       // of this run's stage 0
    auto issue = [&](int u) {                     // lane 0: stage u of this warp
      const int ks = (st0 + warp + u * WARPS) * SK;
      const int n = min(SK, (k1 - ks + 3) & ~3);  // whole 16-byte pieces of the scales; capacity is a multiple of 4
      const int at = (slot0 + u) % NS;
      unsigned char* dst = ring + at * S::STAGE;
      uint64_t* bb = &bar[at];
      const int64_t row = row0 + ks;
      mbar_arrive_expect_tx(bb, (uint32_t)n * (DK / 2 + DV / 2 + GK * 4 + GV * 4));
      bulk_g2s(dst, a.c.k + row * (DK / 8), (uint32_t)n * (DK / 2), bb);
      bulk_g2s(dst + S::KC + S::VC, a.c.ks + row * GK, (uint32_t)n * (GK * 4), bb);
      bulk_g2s(dst + S::KC, a.c.v + row * (DV / 8), (uint32_t)n * (DV / 2), bb);
      bulk_g2s(dst + S::KC + S::VC + S::KP, a.c.vs + row * GV, (uint32_t)n * (GV * 4), bb);
    };
    if (lane == 0)
      for (int u = 0; u < NS && u < n_mine; ++u) issue(u);
    __syncwarp();

    // ---- query fragments: column r of block nb, dims 64 gk + 16 t + 0..15 ----
    // word j (8 dims) of group gk gives two MMAs h = 0, 1 with b0 = dims (2h, 2h + 4), b1 = (2h + 1, 2h + 5)
    // (16 rows: in shared memory, written by warp 0)
    uint32_t qf[S::QS ? 1 : NB][QP][GK][2][2][2];
    uint2* s_qf = reinterpret_cast<uint2*>(smem + S::BAR - S::QF) + lane;
    float qs[NB][GK][2], qf_scale[NB][2];         // of the S^T columns 2t, 2t + 1
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int col = MODE == 0 ? (r & 3) : 8 * nb + r;
      const int rr = rt * ROWS + col;
      const bool on = rr < n_rows;
      const int64_t qrow = (((int64_t)b * a.T + (on ? rr / G : 0)) * a.Hq + g * G + (on ? rr % G : 0)) * DK;
      float x[GK][16], big = 0.f, sum[GK];
#pragma unroll
      for (int gk = 0; gk < GK; ++gk) {
        const int64_t o = qrow + 64 * gk + 16 * t;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float y[8];
          if constexpr (SPLITQ) load8(reinterpret_cast<const float*>(a.q) + o + 8 * j, y);
          else load8(reinterpret_cast<const bf16_t*>(a.q) + o + 8 * j, y);
#pragma unroll
          for (int i = 0; i < 8; ++i) x[gk][8 * j + i] = on ? y[i] : 0.f;
        }
        sum[gk] = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) { big = fmaxf(big, fabsf(x[gk][i])); sum[gk] += x[gk][i]; }
        sum[gk] += __shfl_xor_sync(FULL_MASK, sum[gk], 1);
        sum[gk] += __shfl_xor_sync(FULL_MASK, sum[gk], 2);
      }
      big = fmaxf(big, __shfl_xor_sync(FULL_MASK, big, 1));
      big = fmaxf(big, __shfl_xor_sync(FULL_MASK, big, 2));
      // the row's largest element becomes 2^13 .. 2^14
      const int e = min(max(exponent(big), 20), 240);
      const float up = pow2(267 - e), down = pow2(e + 11) * a.scale_log2;   // 2^(13-(e-127)); 2^24 / up
#pragma unroll
      for (int gk = 0; gk < GK; ++gk)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t f[QP][2];
#pragma unroll
            for (int o = 0; o < 2; ++o) {         // the odd nibble counts 16 times the even one
              const int d = 8 * j + 2 * h + o;
              const float by = o ? 0.0625f : 1.f;
              float y0 = x[gk][d] * up, y1 = x[gk][d + 4] * up;
              if constexpr (SPLITQ) {             // first halves: multiples of 8, whose sums the tensor core keeps whole
                const float h0 = (y0 + GRID) - GRID, h1 = (y1 + GRID) - GRID;
                const uint32_t hi = pack_f16x2(h0 * by, h1 * by), lo = pack_f16x2((y0 - h0) * by, (y1 - h1) * by);
                f[0][o] = MODE == 0 && r < 4 ? hi : lo;
                if constexpr (QP == 2) f[1][o] = hi;
              } else {
                f[0][o] = pack_f16x2(y0 * by, y1 * by);
              }
            }
#pragma unroll
            for (int p = 0; p < QP; ++p) {
              if constexpr (S::QS) {
                if (warp == 0) s_qf[32 * ((((nb * QP + p) * GK + gk) * 2 + j) * 2 + h)] = make_uint2(f[p][0], f[p][1]);
              } else {
                qf[nb][p][gk][j][h][0] = f[p][0];
                qf[nb][p][gk][j][h][1] = f[p][1];
              }
            }
          }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int src = 4 * (2 * t + i);          // any lane of column 2t + i
        qf_scale[nb][i] = __shfl_sync(FULL_MASK, down, src);
#pragma unroll
        for (int gk = 0; gk < GK; ++gk)           // in units of the product (2^-24 up)
          qs[nb][gk][i] = __shfl_sync(FULL_MASK, sum[gk] * (up * 5.9604644775390625e-8f), src);
      }
    }

    if constexpr (S::QS) __syncthreads();

    int lim[NB][2];                               // slots that the columns' tokens see
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int col = MODE == 0 ? ((2 * t + i) & 3) : 8 * nb + 2 * t + i;
        lim[nb][i] = min(L - a.T + min(rt * ROWS + col, n_rows - 1) / G + 1, k1);
      }
    const int lim_all = min(L - a.T + (rt * ROWS) / G + 1, k1);   // slots that every column sees

    uint64_t o[NB][GV][4][2];                     // value dims 64 gv + 8 r + i ([1]: + 4), columns 2t, 2t + 1
    float om[NB][GV][2], m[NB][2], thr[NB][2], l[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int gv = 0; gv < GV; ++gv) {
#pragma unroll
        for (int i = 0; i < 4; ++i) o[nb][gv][i][0] = o[nb][gv][i][1] = 0ull;
        om[nb][gv][0] = om[nb][gv][1] = 0.f;
      }
      m[nb][0] = m[nb][1] = M_NONE;               // reference maximum, log2 units
      thr[nb][0] = thr[nb][1] = -INFINITY;        // (m + RESCALE_LOG2) in units of the raw score
      l[nb][0] = l[nb][1] = 0.f;
    }

    // key order inside a 16-key tile: MMA row (and K index) j holds key sigma(j); adjacent rows and
    // every second row alternate between even and odd keys, which spreads the 64-byte rows over the
    // shared-memory banks
    const int kr = r ^ ((r >> 1) & 1);            // sigma(r); rows r + 8: + 8
    const int kv0 = (2 * t) ^ (t & 1), kv1 = (2 * t + 1) ^ (t & 1);
    const int k_at = kr * (DK / 2) + t * (DK / 8), kp_at = S::KC + S::VC + kr * (GK * 4);
    const int v0_at = S::KC + kv0 * (DV / 2) + r * (GV * 4), v1_at = S::KC + kv1 * (DV / 2) + r * (GV * 4);
    const int vp_at = S::KC + S::VC + S::KP + kr * (GV * 4);
    // a factor that the compiler does not know: a shift to the left as a product, on the multiply-add pipe
    // (the logic pipe carries the unpacking)
    uint32_t two16;
    asm volatile("mov.u32 %0, 65536;" : "=r"(two16));
    auto scale_of = [&](uint32_t w) { return __uint_as_float(w * two16); };   // bf16_lo
    // second halves are held 2^11 times: what float16 leaves of a weight is normal as long as the weight is.
    // MODE 0: lanes t >= 2 pass on second halves and take their sums back
    const bool second = MODE == 0 && t >= 2;
    [[maybe_unused]] const uint64_t half_of = second ? pack_f32x2(2048.f, 2048.f) : pack_f32x2(1.f, 1.f);
    [[maybe_unused]] const uint64_t half_less = second ? pack_f32x2(-2048.f, -2048.f) : 0ull;
    const int half_exp = second ? 11 : 0;

    const __half2 times_even = __halves2half2(__ushort_as_half(0x7800), __ushort_as_half(0x7800));   // 2^15
    const __half2 times_odd = __halves2half2(__ushort_as_half(0x6800), __ushort_as_half(0x6800));    // 2^11
    const __half2 centre = __halves2half2(__ushort_as_half(0xa400), __ushort_as_half(0xa400));       // -8 2^-9
    // SUB 16-key tiles of a stage from tile t0 on; kb: their first key.  TAIL: some key is hidden from some
    // column.
    auto tiles = [&](auto tail, const unsigned char* stg, int t0, int kb) {
      constexpr bool TAIL = decltype(tail)::value;
      float s[SUB][NB][4];                        // scores of keys kr (e = 0, 1) and kr + 8 (e = 2, 3); columns 2t, 2t + 1
      uint32_t vp[SUB][2][GV];                    // scales and midpoints of V
      float top[GV];                              // the largest scale of V in these tiles, by group
#pragma unroll
      for (int gv = 0; gv < GV; ++gv) top[gv] = 0.f;
      // ---- S^T: chains of products into the same accumulator interleave ----
      float d[SUB][NB][GK][QP][4];             // the halves of q apart: the first ones' sums stay exact
      uint32_t wk[SUB][2][2 * GK], kp[SUB][2][GK];
#pragma unroll
      for (int q = 0; q < SUB; ++q) {
        const int tt = t0 + q;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int gk = 0; gk < GK; ++gk)
#pragma unroll
            for (int p = 0; p < QP; ++p) d[q][nb][gk][p][0] = d[q][nb][gk][p][1] = d[q][nb][gk][p][2] = d[q][nb][gk][p][3] = 0.f;
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          load_words(stg + k_at + (16 * tt + 8 * hh) * (DK / 2), wk[q][hh]);
          load_words(stg + kp_at + (16 * tt + 8 * hh) * (GK * 4), kp[q][hh]);
          load_words(stg + vp_at + (16 * tt + 8 * hh) * (GV * 4), vp[q][hh]);
        }
      }
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int gk = 0; gk < GK; ++gk)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
              for (int p = 0; p < QP; ++p) {
                uint2 f;
                if constexpr (S::QS) f = s_qf[32 * ((((nb * QP + p) * GK + gk) * 2 + j) * 2 + h)];
                else f = make_uint2(qf[nb][p][gk][j][h][0], qf[nb][p][gk][j][h][1]);
#pragma unroll
                for (int q = 0; q < SUB; ++q) {
                  const uint32_t x = wk[q][0][j * GK + gk] >> (8 * h), y = wk[q][1][j * GK + gk] >> (8 * h);
                  mma16816(d[q][nb][gk][p], x & 0x000f000fu, y & 0x000f000fu, x & 0x00f000f0u, y & 0x00f000f0u, f.x, f.y);
                }
              }
#pragma unroll
      for (int q = 0; q < SUB; ++q) {
        const int k0 = kb + 16 * q;
        // ---- scale and midpoint ----
        float sp[NB][4], sc[NB][4];
#pragma unroll
        for (int hh = 0; hh < 2; ++hh)
#pragma unroll
          for (int gk = 0; gk < GK; ++gk) {
            const float scale = scale_of(kp[q][hh][gk]), off = fmaf(-8.f, scale, bf16_hi(kp[q][hh][gk]));
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const int e = 2 * hh + i;
                const float z = QP == 2 ? d[q][nb][gk][0][e] + d[q][nb][gk][QP - 1][e] : d[q][nb][gk][0][e];
                sp[nb][e] = gk == 0 ? scale * z : fmaf(scale, z, sp[nb][e]);
                sc[nb][e] = gk == 0 ? off * qs[nb][gk][i] : fmaf(off, qs[nb][gk][i], sc[nb][e]);
              }
          }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if constexpr (MODE == 0 && SPLITQ) sp[nb][e] += __shfl_xor_sync(FULL_MASK, sp[nb][e], 2);
            s[q][nb][e] = sp[nb][e] + sc[nb][e];          // times qf_scale: log2 units
            if (TAIL && k0 + kr + 8 * (e >> 1) >= lim[nb][e & 1]) s[q][nb][e] = -INFINITY;
          }
#pragma unroll
        for (int hh = 0; hh < 2; ++hh)
#pragma unroll
          for (int gv = 0; gv < GV; ++gv) {
            if (TAIL && k0 + kr + 8 * hh >= k1) vp[q][hh][gv] = 0u;   // slots past the run may hold anything
            top[gv] = fmaxf(top[gv], fabsf(scale_of(vp[q][hh][gv])));
          }
      }
      // ---- online softmax: move the references when a score outgrows them (rare) ----
      float high[NB][2];
      bool grow = false;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          high[nb][i] = fmaxf(s[0][nb][i], s[0][nb][2 + i]);
#pragma unroll
          for (int q = 1; q < SUB; ++q) high[nb][i] = fmaxf(fmaxf(high[nb][i], s[q][nb][i]), s[q][nb][2 + i]);
          grow |= high[nb][i] > thr[nb][i];
        }
      if (__any_sync(FULL_MASK, grow)) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          float by[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float mt = high[nb][i];
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) mt = fmaxf(mt, __shfl_xor_sync(FULL_MASK, mt, x));
            float alpha = 1.f;
            if (mt > thr[nb][i]) {                        // uniform over the column's lanes
              mt *= qf_scale[nb][i];
              alpha = ex2(m[nb][i] - mt);
              m[nb][i] = mt;
              thr[nb][i] = (mt + RESCALE_LOG2) / qf_scale[nb][i];
              l[nb][i] *= alpha;
            }
#pragma unroll
            for (int gv = 0; gv < GV; ++gv) om[nb][gv][i] *= alpha;
            by[i] = alpha;
          }
          const uint64_t by2 = pack_f32x2(by[0], by[1]);
#pragma unroll
          for (int gv = 0; gv < GV; ++gv)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              o[nb][gv][k][0] = mul_f32x2(o[nb][gv][k][0], by2);
              o[nb][gv][k][1] = mul_f32x2(o[nb][gv][k][1], by2);
            }
        }
      }
      // ---- a power of two for these tiles' weights, by group: p = 1 at the largest scale becomes 2^9 .. 2^10, p = 2^5 2^15 ----
      float vmul[GV], vinv[GV];
#pragma unroll
      for (int gv = 0; gv < GV; ++gv) {
        const int e = min(max(exponent(__uint_as_float(__reduce_max_sync(FULL_MASK, __float_as_uint(top[gv])))) + 1, 14), 251);
        vmul[gv] = pow2(264 - e);
        vinv[gv] = pow2(e - 1 - half_exp);                // 2^9 / vmul: the codes' step is 2^-9
      }
      // ---- weights p * scale of V, per group: operand fragments of keys 2t, 2t + 1 (and + 8), column r ----
      uint32_t bh[SUB][NB][GV][2];
      [[maybe_unused]] uint32_t bl[SUB][NB][GV][2];
#pragma unroll
      for (int q = 0; q < SUB; ++q) {
        float p[NB][4];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            p[nb][e] = ex2(fmaf(s[q][nb][e], qf_scale[nb][e & 1], -m[nb][e & 1]));
            l[nb][e & 1] += p[nb][e];
          }
#pragma unroll
        for (int gv = 0; gv < GV; ++gv)
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const float mul = scale_of(vp[q][hh][gv]) * vmul[gv], mid = bf16_hi(vp[q][hh][gv]);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
              float w[2];
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const float pi = p[nb][2 * hh + i];
                w[i] = pi * mul;
                if constexpr (TAIL) {                     // a hidden key's values may be NaN: no 0 * NaN
                  const bool hidden = s[q][nb][2 * hh + i] == -INFINITY;
                  if (hidden) w[i] = 0.f;
                  om[nb][gv][i] += hidden ? 0.f : pi * mid;
                } else {
                  om[nb][gv][i] = fmaf(pi, mid, om[nb][gv][i]);
                }
              }
              const uint32_t hi = pack_f16x2(w[0], w[1]);
              const float2 f = unpack_f16x2(hi);
              if constexpr (MODE == 0) {                  // lanes t < 2: the first halves; t >= 2: what they leave
                const uint64_t z = fma_f32x2(pack_f32x2(f.x, f.y), half_less, mul_f32x2(pack_f32x2(w[0], w[1]), half_of));
                bh[q][nb][gv][hh] = transpose8x8(pack_f16x2(f32x2_lo(z), f32x2_hi(z)));
              } else {
                bh[q][nb][gv][hh] = transpose8x8(hi);
                bl[q][nb][gv][hh] = transpose8x8(pack_f16x2(w[0] - f.x, w[1] - f.y));
              }
            }
          }
      }
      // ---- O^T += V^T P: the tensor core cuts a sum off towards zero, so its sums stay short ----
      uint32_t wv[SUB][4][GV];
#pragma unroll
      for (int q = 0; q < SUB; ++q)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          load_words(stg + (k & 1 ? v1_at : v0_at) + (16 * (t0 + q) + (k & 2 ? 8 : 0)) * (DV / 2), wv[q][k]);
#pragma unroll
      for (int gv = 0; gv < GV; ++gv) {
        // halves of two keys' words side by side, nibbles 0..3 (x) and 4..7 (y), and with their bytes exchanged
        uint32_t x[SUB][4][2];
#pragma unroll
        for (int q = 0; q < SUB; ++q)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t lo = wv[q][k & 2][gv], hi = wv[q][(k & 2) + 1][gv];
            x[q][k][0] = __byte_perm(lo, hi, k & 1 ? 0x7632 : 0x5410);
            x[q][k][1] = __byte_perm(lo, hi, k & 1 ? 0x6723 : 0x4501);
          }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float z[NB][4];
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) z[nb][0] = z[nb][1] = z[nb][2] = z[nb][3] = 0.f;
#pragma unroll
          for (int q = 0; q < SUB; ++q) {
            // nibble i of each half as the float16 subnormal u 2^-24 or u 2^-20, made (u - 8) 2^-9: the
            // tensor core aligns a subnormal as if it were 2^-14, and the sums would lose as many bits
            auto code = [&](const uint32_t (&v)[2]) {
              const uint32_t w = v[i >> 1] & (i & 1 ? 0x00f000f0u : 0x000f000fu);
              const __half2 c = __hfma2(*reinterpret_cast<const __half2*>(&w), i & 1 ? times_odd : times_even, centre);
              return *reinterpret_cast<const uint32_t*>(&c);
            };
            const uint32_t a0 = code(x[q][0]), a1 = code(x[q][1]), a2 = code(x[q][2]), a3 = code(x[q][3]);
            if constexpr (MODE != 0) {
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) mma16816(z[nb], a0, a1, a2, a3, bl[q][nb][gv][0], bl[q][nb][gv][1]);
            }
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) mma16816(z[nb], a0, a1, a2, a3, bh[q][nb][gv][0], bh[q][nb][gv][1]);
          }
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            o[nb][gv][i][0] = fma_f32x2(pack_f32x2(z[nb][0], z[nb][1]), pack_f32x2(vinv[gv], vinv[gv]), o[nb][gv][i][0]);
            o[nb][gv][i][1] = fma_f32x2(pack_f32x2(z[nb][2], z[nb][3]), pack_f32x2(vinv[gv], vinv[gv]), o[nb][gv][i][1]);
          }
        }
      }
    };

    for (int u = 0; u < n_mine; ++u) {
      if (!__all_sync(FULL_MASK, mbar_wait_bounded(&bar[slot], phase))) {
        ok = false;                               // gave up: the copies still in flight land first (bounded)
        for (int v = u + 1; v < n_mine && v < u + NS; ++v) {
          if (++slot == NS) { slot = 0; phase ^= 1; }
          (void)mbar_wait_bounded(&bar[slot], phase);
        }
        break;
      }
      const unsigned char* stg = ring + slot * S::STAGE;
      const int ks = (st0 + warp + u * WARPS) * SK;
      if (ks + SK <= lim_all) {
#pragma unroll 1                                // unrolled, 16 rows spill (64 blocks of 16 tokens: 151 us, so 139)
        for (int tt = 0; tt < SK / 16; tt += SUB) tiles(std::false_type{}, stg, tt, ks + 16 * tt);
      } else {
#pragma unroll 1
        for (int tt = 0; tt < SK / 16 && ks + 16 * tt < k1; tt += SUB) tiles(std::true_type{}, stg, tt, ks + 16 * tt);
      }
      __syncwarp();                               // all lanes are done with this stage
      if (lane == 0 && u + NS < n_mine) issue(u + NS);
      if (++slot == NS) { slot = 0; phase ^= 1; }
    }

    // ---- merge the warps ----
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) {
          l[nb][i] += __shfl_xor_sync(FULL_MASK, l[nb][i], x);
#pragma unroll
          for (int gv = 0; gv < GV; ++gv) om[nb][gv][i] += __shfl_xor_sync(FULL_MASK, om[nb][gv][i], x);
        }
    __syncthreads();                              // rings drained: reuse them
    float* sm_m = reinterpret_cast<float*>(smem);                 // [WARPS][ROWS]
    float* sm_l = sm_m + WARPS * ROWS;
    float* sm_o = sm_l + WARPS * ROWS;                            // [WARPS][ROWS][DV]
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int row = 8 * nb + 2 * t + i;       // MODE 0: rows 0..3 in lanes t < 2
        if (r == 0 && row < ROWS) {
          sm_m[warp * ROWS + row] = ok ? m[nb][i] : NAN;
          sm_l[warp * ROWS + row] = ok ? l[nb][i] : NAN;
        }
#pragma unroll
        for (int gv = 0; gv < GV; ++gv) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float lo = i ? f32x2_hi(o[nb][gv][k][0]) : f32x2_lo(o[nb][gv][k][0]);
            float hi = i ? f32x2_hi(o[nb][gv][k][1]) : f32x2_lo(o[nb][gv][k][1]);
            if constexpr (MODE == 0) {
              lo += __shfl_xor_sync(FULL_MASK, lo, 2);
              hi += __shfl_xor_sync(FULL_MASK, hi, 2);
            }
            if (row < ROWS) {
              float* dst = sm_o + (warp * ROWS + row) * DV + 64 * gv + 8 * r + k;
              dst[0] = lo + om[nb][gv][i];
              dst[4] = hi + om[nb][gv][i];
            }
          }
        }
      }
    __syncthreads();
    if (tid < ROWS) {
      float M = M_NONE, Ls = 0.f;
      for (int w = 0; w < WARPS; ++w) M = fmaxf(M, sm_m[w * ROWS + tid]);
      for (int w = 0; w < WARPS; ++w) Ls += ex2(sm_m[w * ROWS + tid] - M) * sm_l[w * ROWS + tid];
      s_M[tid] = M; s_L[tid] = Ls;
    }
    __syncthreads();
    const bool whole = st0 == 0 && st1 == stages;
    const int rows_here = row_end - rt * ROWS;
    // parts of shared units: a CTA keeps two, [0] of the unit that its run begins in, [1] of its last one
    const int64_t my_part = ((int64_t)c * 2 + (x0 >= unit_at ? 0 : 1)) * ROWS;
    for (int idx = tid; idx < rows_here * DV; idx += THREADS) {
      const int row = idx / DV, dd = idx % DV;
      float tot = 0.f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) tot += ex2(sm_m[w * ROWS + row] - s_M[row]) * sm_o[(w * ROWS + row) * DV + dd];
      if (whole) {
        out_row(row)[dd] = s_L[row] == 0.f ? 0.f : tot / s_L[row];
      } else {
        const int64_t pi = my_part + row;
        a.part_acc[pi * DV + dd] = tot;
        if (dd == 0) { a.part_ml[2 * pi] = s_M[row]; a.part_ml[2 * pi + 1] = s_L[row]; }
      }
    }
    if (!whole) {
      const int c0 = cta_of(unit_at), c1 = cta_of(unit_at + stages - 1);
      __threadfence();
      __syncthreads();
      unsigned* counter = a.counters + c0;        // only the last unit of a run goes on into the next one
      if (tid == 0) s_last = atomicAdd(counter, 1u) == (unsigned)(c1 - c0);
      __syncthreads();
      if (s_last) {                               // the unit's last part: join them in order
        __threadfence();
        constexpr int EPT = ROWS * DV / THREADS;              // outputs per thread
        constexpr int BLOCK = (S::BAR - S::QF) / (ROWS * 8) < 256 ? (S::BAR - S::QF) / (ROWS * 8) : 256;   // parts at a time
        float2* s_ml = reinterpret_cast<float2*>(smem);       // [ROWS][BLOCK] (max, sum); then (weight, -)
        const int first = c0 * 2 + (start_of(c0) >= unit_at ? 0 : 1);   // the others' parts are their [0]
        auto part = [&](int cc) { return (int64_t)(cc == c0 ? first : 2 * cc) * ROWS; };
        float acc[EPT];
#pragma unroll
        for (int e = 0; e < EPT; ++e) acc[e] = 0.f;
        if (tid < ROWS) { s_M[tid] = M_NONE; s_L[tid] = 0.f; }
        for (int cb = c0; cb <= c1; cb += BLOCK) {            // one pass, unless the unit has very many parts
          const int n = min(BLOCK, c1 + 1 - cb);
          __syncthreads();
          for (int i = tid; i < ROWS * n; i += THREADS) {
            const int cc = i / ROWS, row = i - cc * ROWS;
            s_ml[row * BLOCK + cc] = row < rows_here ? __ldcg(reinterpret_cast<const float2*>(a.part_ml) + part(cb + cc) + row)
                                                     : make_float2(M_NONE, 0.f);
          }
          __syncthreads();
          for (int row = warp; row < ROWS; row += WARPS) {    // weights against the maximum so far
            float M = s_M[row], den = 0.f;
            const float before = M;
            for (int cc = lane; cc < n; cc += 32) M = fmaxf(M, s_ml[row * BLOCK + cc].x);
#pragma unroll
            for (int x = 16; x > 0; x >>= 1) M = fmaxf(M, __shfl_xor_sync(FULL_MASK, M, x));
            for (int cc = lane; cc < n; cc += 32) {
              const float2 ml = s_ml[row * BLOCK + cc];
              const float w = ex2(ml.x - M);
              den = fmaf(w, ml.y, den);
              s_ml[row * BLOCK + cc].x = w;
            }
#pragma unroll
            for (int x = 16; x > 0; x >>= 1) den += __shfl_xor_sync(FULL_MASK, den, x);
            __syncwarp();
            if (lane == 0) {
              const float alpha = ex2(before - M);
              s_L[row] = fmaf(s_L[row], alpha, den);
              s_M[row] = M;
              s_alpha[row] = alpha;
            }
          }
          __syncthreads();
#pragma unroll
          for (int e = 0; e < EPT; ++e) acc[e] *= s_alpha[(tid + e * THREADS) / DV];
          for (int cc = 0; cc < n; ++cc) {
            const float* src = a.part_acc + part(cb + cc) * DV;
            float v[EPT];
#pragma unroll
            for (int e = 0; e < EPT; ++e)
              v[e] = (tid + e * THREADS) / DV < rows_here ? __ldcg(src + tid + e * THREADS) : 0.f;
#pragma unroll
            for (int e = 0; e < EPT; ++e) acc[e] = fmaf(s_ml[(tid + e * THREADS) / DV * BLOCK + cc].x, v[e], acc[e]);
          }
        }
#pragma unroll
        for (int e = 0; e < EPT; ++e) {
          const int row = (tid + e * THREADS) / DV, dd = (tid + e * THREADS) % DV;
          if (row < rows_here) out_row(row)[dd] = s_L[row] == 0.f ? 0.f : acc[e] / s_L[row];
        }
        if (tid == 0) *counter = 0u;
      }
    }
    fence_proxy_async_smem();                     // the merge's writes before the next run's copies
    __syncthreads();
  }
}

template <int DK, int DV, int MODE, bool SPLITQ>
cudaError_t launch_m(const DecodeQ4Args& a, cudaStream_t s) {
  constexpr int smem = Shape<DK, DV, MODE, SPLITQ>::SMEM;
  static DeviceOnce configured;
  if (!configured.done()) {
    cudaError_t e = cudaFuncSetAttribute(decode_q4_kernel<DK, DV, MODE, SPLITQ>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    configured.mark();
  }
  return launch_pdl(decode_q4_kernel<DK, DV, MODE, SPLITQ>, dim3(a.ctas), dim3(THREADS), smem, s, a);
}

template <int DK, int DV>
cudaError_t launch_d(const DecodeQ4Args& a, kva_dtype q_dtype, cudaStream_t s) {
  const bool split = q_dtype == KVA_F32;
  switch (decode_q4_row_tile(a.Hq / a.c.Hkv * a.T)) {
    case 4: return split ? launch_m<DK, DV, 0, true>(a, s) : launch_m<DK, DV, 0, false>(a, s);
    case 8: return split ? launch_m<DK, DV, 1, true>(a, s) : launch_m<DK, DV, 1, false>(a, s);
    default: return split ? launch_m<DK, DV, 2, true>(a, s) : launch_m<DK, DV, 2, false>(a, s);
  }
}

}  // namespace

bool decode_q4_supports(int Dk, int Dv) {
  return (Dk == 64 && Dv == 64) || (Dk == 128 && Dv == 128) || (Dk == 192 && Dv == 128);
}

// Query rows of a unit.  16 in one rather than 8 in two: 139 against 159 us on blocks of 32 rows a KV head.
int decode_q4_row_tile(int rows) { return rows <= 4 ? 4 : (rows <= 8 ? 8 : 16); }

// CTAs for `stages` stages of 32 keys in `units` units of at most `longest` stages.  Many units, none of them
// long against what a CTA would get: one CTA each, in the order that the GPU takes them, and nothing to
// join (61 sequences x 16 units of about 62 stages: 139 us against 146 in equal runs).  Else equal runs: as many as
// the GPU holds at once, each with a stage per warp, and not so many that joining a unit's parts
// (about 40 ns each, one CTA) costs more than its stages take (about 150 ns each, spread over the parts).
// The stage per warp is counted over all units: short contexts give a CTA several units, one after another (64
// sequences of 1 to 64 keys x 8 heads 18 us, a block of 16 tokens of one sequence of 30 keys 39 us; one of 768 keys 9).
int decode_q4_ctas(int Dk, int rows, int64_t stages, int64_t units, int64_t longest, int64_t all_units, int* whole) {
  const int per_sm = rows <= 4 && Dk <= 128 ? 4 : (rows <= 8 || Dk <= 128 ? 3 : 2);
  const int64_t slots = DECODE_Q4_SMS * per_sm;
  *whole = stages >= 2 * slots * longest && stages > 0 && all_units <= (1 << 24);
  if (*whole) return (int)all_units;
  const int64_t most = std::min<int64_t>(slots, (int64_t)(2.0 * std::sqrt((double)stages * (double)units)));
  return (int)std::max<int64_t>(1, std::min<int64_t>(most, stages / WARPS));
}

cudaError_t launch_decode_q4(const DecodeQ4Args& a, kva_dtype q_dtype, cudaStream_t s) {
  if (a.c.Dk == 64) return launch_d<64, 64>(a, q_dtype, s);
  if (a.c.Dk == 128) return launch_d<128, 128>(a, q_dtype, s);
  return launch_d<192, 128>(a, q_dtype, s);
}

}  // namespace kva
