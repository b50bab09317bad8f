// Log probabilities over the vocabulary (lmhead_logprobs): a tcgen05 form for bf16 tables, a
// streaming form for the others, and the merge that ends both.
//
// Bound: HBM for up to 128 rows or so (151936 x 1024, one row: 52 us, 88% of the copy rate, 61 us with the
// kernels around it; 64 rows 72 us, where the two halves keep the tensor pipe 61% busy), then the L2 feed of
// the products (1999 bf16 rows: 390 us of 480, tensor pipe 74%).
//
// tcgen05 form (H a multiple of 64): D[128 batch rows x N vocabulary rows] = h W^T with the batch on the
// TMEM lanes, so that an epilogue thread owns a batch row and every sum over the vocabulary is a sum
// along its own columns.  A float32 (or normalised) row is two bf16 halves, h = hi + lo (about 17
// significant bits): two products into the same accumulator; a bf16 row is one.  Persistent CTAs
// walk vocabulary tiles for one block of 128 rows: warp 0 loads (TMA, 128-byte swizzle, a ring of
// 64-wide K chunks), warp 1 issues the MMAs into one of two accumulators, warps 2-9 read the other one
// (a thread: one row, half of the columns) and keep, per row, the maximum, the two sums and a list of
// candidates.  With fewer than 128 rows only those are loaded: the MMA reads whatever follows them in
// shared memory into lanes that nobody reads.  Up to 8 row blocks run side by side, so that a table tile is read from HBM once per 8.
//
// Streaming form: grid (vocabulary split, block of NB = 1, 2, 4 or 8 batch rows).  A warp takes 4 table rows at
// a time and loads the next 256 columns of them before it multiplies the current ones with the NB hidden
// rows, which lie in shared memory in the lanes' order (two products an instruction).  The lanes' 4 NB sums
// are reduced by halving, which leaves one logit (table row, batch row) in a lane or a few: it keeps the
// maximum, the two sums and a list of the logits that it meets, and the CTA joins its lanes at the end.
//
// A kernel before either form norms the rows (and splits them into halves): in the streaming kernel and the
// merge themselves, without that launch, 5 rows of 520 took 14.7 us instead of 13.1.
//
// Merge (one CTA per batch row): joins the splits' (m, s, u) in a fixed order and their lists, then
// scores the given token and the TK candidates again: the lists hold TK > top_k candidates by
// float32 (or two-bf16-halves) logits, whose rounding may exchange neighbours, while the second
// scoring carries each product and sum with its rounding error (compensated dot product: Ogita,
// Rump and Oishi, "Accurate sum and dot product"), about twice float32 precision, and orders them.  The
// other logits of the tcgen05 form enter the sums with 16 to 17 bits of a float32 or normalised row: a third bf16
// part, which float32 would need, is half as many products again.
// entropy = log s - u / s and lse = m + log s need no cancellation against m.  The candidates' terms
// of s and u are exchanged for those of the second scoring: the tensor core drops a little of every
// sum that it adds to (6e-6 of a logit at H = 4096), and the largest logits lose and weigh most.
//
// Method: the lm_head over the whole tied table and the pick of tokens after the final RMSNorm
// (Youtu-VL-4B ncnn port, step 6 and "decoding and sampling").
#include <algorithm>

#include <mutex>

#include "launch.h"
#include "tc.cuh"

namespace kva {

namespace {

constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;
// Most threads of a merge CTA: at least one per split, and (lists of up to 16) a warp per candidate; no more
// than the lists' registers allow.
__host__ __device__ constexpr int merge_max(int TK) { return TK <= 24 ? 512 : 320; }

using u64 = unsigned long long;

// Sorted list of the TK best keys (larger key = larger logit, then lower id).
template <int TK>
__device__ __forceinline__ void list_insert(u64 (&L)[TK], u64 key) {
  if (key <= L[TK - 1]) return;
#pragma unroll
  for (int i = TK - 1; i > 0; --i) L[i] = key > L[i - 1] ? L[i - 1] : (key > L[i] ? key : L[i]);
  L[0] = key > L[0] ? key : L[0];
}
// The TK best of the warp's 32 lists, into out[] (lane 0 writes).  The maximum of the list heads is
// found in two 32-bit steps, logit bits and then ids.
template <int TK>
__device__ __forceinline__ void warp_merge(u64 (&L)[TK], u64* out) {
  const int lane = threadIdx.x & 31;
  for (int r = 0; r < TK; ++r) {
    const uint32_t hi = (uint32_t)(L[0] >> 32), top = __reduce_max_sync(FULL_MASK, hi);
    const uint32_t id = __reduce_max_sync(FULL_MASK, hi == top ? (uint32_t)L[0] : 0u);
    const u64 best = ((u64)top << 32) | id;
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
// The union of the warp's 32 sets, in every lane.
__device__ __forceinline__ Stat stat_warp(Stat a) {
  float m = a.m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL_MASK, m, o));
  if (a.s != 0.f) {                           // an empty set has m = -inf
    const float d = a.m - m, e = __expf(d);
    a.u = e * fmaf(a.s, d, a.u);
    a.s *= e;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a.s += __shfl_xor_sync(FULL_MASK, a.s, o);
    a.u += __shfl_xor_sync(FULL_MASK, a.u, o);
  }
  a.m = m;
  return a;
}

// One CTA per row: the final RMSNorm in float32 (norm_w given) and the two bf16 halves (hb given).
__global__ void __launch_bounds__(THREADS)
logprob_prep_kernel(const __grid_constant__ LogprobArgs a) {
  __shared__ float s_part[WARPS];
  const int b = blockIdx.x, tid = threadIdx.x;
  griddep_wait();
  griddep_launch_dependents();
  const int64_t row = (int64_t)b * a.H;
  constexpr int MAX_PER = 4096 / THREADS / 4;             // pieces of 4 a thread holds (H <= 4096)
  float x[MAX_PER][4], w[MAX_PER][4];
  float ss = 0.f;
#pragma unroll
  for (int j = 0; j < MAX_PER; ++j) {
    const int k = 4 * (tid + j * THREADS);
    if (k >= a.H) continue;
    if (a.h_dtype == KVA_BF16) {
      const uint2 u = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(a.h) + row + k);
      x[j][0] = bf16_lo(u.x); x[j][1] = bf16_hi(u.x); x[j][2] = bf16_lo(u.y); x[j][3] = bf16_hi(u.y);
    } else {
      const float4 u = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(a.h) + row + k);
      x[j][0] = u.x; x[j][1] = u.y; x[j][2] = u.z; x[j][3] = u.w;
    }
    if (a.norm_w) {
      const float4 u = *reinterpret_cast<const float4*>(a.norm_w + k);
      w[j][0] = u.x; w[j][1] = u.y; w[j][2] = u.z; w[j][3] = u.w;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) ss = fmaf(x[j][i], x[j][i], ss);
  }
  float r = 1.f;
  if (a.norm_w) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(FULL_MASK, ss, o);
    if ((tid & 31) == 0) s_part[tid >> 5] = ss;
    __syncthreads();
    float tot = 0.f;
#pragma unroll
    for (int v = 0; v < WARPS; ++v) tot += s_part[v];
    r = 1.0f / sqrtf(tot / (float)a.H + a.eps);
  }
#pragma unroll
  for (int j = 0; j < MAX_PER; ++j) {
    const int k = 4 * (tid + j * THREADS);
    if (k >= a.H) continue;
    if (a.norm_w) {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[j][i] = x[j][i] * r * w[j][i];
      *reinterpret_cast<float4*>(a.hn + row + k) = make_float4(x[j][0], x[j][1], x[j][2], x[j][3]);
    }
    if (a.hb) {
      const uint32_t h01 = pack_bf16x2(x[j][0], x[j][1]), h23 = pack_bf16x2(x[j][2], x[j][3]);
      *reinterpret_cast<uint2*>(a.hb + row + k) = make_uint2(h01, h23);
      *reinterpret_cast<uint2*>(a.hb + (int64_t)a.B * a.H + row + k) =
          make_uint2(pack_bf16x2(x[j][0] - bf16_lo(h01), x[j][1] - bf16_hi(h01)),
                     pack_bf16x2(x[j][2] - bf16_lo(h23), x[j][3] - bf16_hi(h23)));
    }
  }
}

// The row that the table meets: normalised (float32), or h itself.
__device__ __forceinline__ float hidden_at(const LogprobArgs& a, int64_t i) {
  if (a.norm_w) return a.hn[i];
  return a.h_dtype == KVA_BF16 ? load1(reinterpret_cast<const bf16_t*>(a.h) + i) : reinterpret_cast<const float*>(a.h)[i];
}

// Sorted list of a row's TK best logits; larger first, equal ones in the order of insertion.
template <int TK>
struct TopList {
  float v[TK];
  int id[TK];                                 // -1: none yet
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < TK; ++i) { v[i] = -INFINITY; id[i] = -1; }
  }
  // x takes its place and moves the rest down: v[i] becomes the middle one of v[i - 1], v[i] and x
  __device__ __forceinline__ void insert(float x, int token) {
    bool above[TK];                           // x goes before entry i
#pragma unroll
    for (int i = 0; i < TK; ++i) above[i] = x > v[i];
#pragma unroll
    for (int i = TK - 1; i > 0; --i) {
      id[i] = above[i - 1] ? id[i - 1] : (above[i] ? token : id[i]);
      v[i] = fminf(v[i - 1], fmaxf(v[i], x));
    }
    id[0] = above[0] ? token : id[0];
    v[0] = fmaxf(v[0], x);
  }
  __device__ __forceinline__ u64 key(int i) const { return id[i] < 0 ? 0ull : argmax_key(v[i], (uint32_t)id[i]); }
};

// Sum over the warp of N values a lane (N a power of two up to 32): by halving, so that lane l ends with the
// sum of value l / (32 / N).
template <int N>
__device__ __forceinline__ float reduce_spread(float (&v)[N]) {
  const int lane = threadIdx.x & 31;
  int o = 16;
#pragma unroll
  for (int n = N; n > 1; n /= 2, o /= 2) {
    const bool upper = lane & o;
#pragma unroll
    for (int i = 0; i < n / 2; ++i) {
      const float keep = upper ? v[i + n / 2] : v[i], send = upper ? v[i] : v[i + n / 2];
      v[i] = keep + __shfl_xor_sync(FULL_MASK, send, o);
    }
  }
  for (; o > 0; o /= 2) v[0] += __shfl_xor_sync(FULL_MASK, v[0], o);
  return v[0];
}

constexpr int R = 4;                          // table rows at a time of a warp
// CTAs per SM: two where 128 registers hold the sums (4 x 1024 columns of a 32000-row float32 table: 48 us with
// the flush of L2, 52 with one CTA of 8 table rows a warp).
__host__ __device__ constexpr int stream_ctas(int nb, int tk) { return nb <= 4 && tk <= 16 ? 2 : 1; }

template <typename WT, int NB, int TK>
__global__ void __launch_bounds__(THREADS, stream_ctas(NB, TK))
logprob_stream_kernel(const __grid_constant__ LogprobArgs a) {
  constexpr int N = R * NB, SHARE = 32 / N;             // lanes that hold one logit
  constexpr int LISTS = R * WARPS;                      // of a batch row, one per lane of the warp that joins them
  static_assert(LISTS == 32, "a list per lane");
  extern __shared__ __align__(16) unsigned char smem[];
  float* s_h = reinterpret_cast<float*>(smem);          // [NB][columns / 256][2][32 lanes][4]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b0 = blockIdx.y * NB, nb = min(NB, a.B - b0), H = a.H, chunks = (H + 255) / 256;
  griddep_wait();
  griddep_launch_dependents();

  const int groups = (a.V + R - 1) / R, step = gridDim.x * WARPS;
  const WT* table = reinterpret_cast<const WT*>(a.W) + 8 * lane;
  Raw8<WT> raw[R];
  auto load = [&](int g, int c) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (256 * c + 8 * lane < H) raw[r].load(table + (int64_t)min(g * R + r, a.V - 1) * H + 256 * c);
      else raw[r].zero();
    }
  };
  int g = blockIdx.x * WARPS + warp;
  if (g < groups) load(g, 0);
  // column k = 256 c + 8 l + 4 h + e of a batch row at [c][h][l][e]; columns past H are zeros
  for (int i = tid; i < NB * chunks * 256; i += THREADS) {
    const int b = i / (chunks * 256), k = i - b * chunks * 256;
    const float x = b < nb && k < H ? hidden_at(a, (int64_t)(b0 + b) * H + k) : 0.f;
    s_h[b * chunks * 256 + (k & ~255) + ((k >> 2) & 1) * 128 + ((k >> 3) & 31) * 4 + (k & 3)] = x;
  }
  __syncthreads();

  const int value = lane / SHARE, my_r = value / NB, my_b = value % NB;
  const bool counts = lane % SHARE == 0 && my_b < nb;
  Stat st{-INFINITY, 0.f, 0.f};
  TopList<TK> list;
  list.clear();
  for (; g < groups; g += step) {
    uint64_t acc[R][NB];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int b = 0; b < NB; ++b) acc[r][b] = 0ull;
    for (int c = 0; c < chunks; ++c) {
      uint64_t x[R][4];
#pragma unroll
      for (int r = 0; r < R; ++r) raw[r].pairs(x[r]);
      if (c + 1 < chunks) load(g, c + 1);
      else if (g + step < groups) load(g + step, 0);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        if (b >= nb) break;                             // warp-uniform
        const ulonglong2* h = reinterpret_cast<const ulonglong2*>(s_h + (b * chunks + c) * 256) + lane;
        const ulonglong2 lo = h[0], hi = h[32];
#pragma unroll
        for (int r = 0; r < R; ++r) {
          acc[r][b] = fma_f32x2(x[r][0], lo.x, acc[r][b]);
          acc[r][b] = fma_f32x2(x[r][1], lo.y, acc[r][b]);
          acc[r][b] = fma_f32x2(x[r][2], hi.x, acc[r][b]);
          acc[r][b] = fma_f32x2(x[r][3], hi.y, acc[r][b]);
        }
      }
    }
    float v[N];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int b = 0; b < NB; ++b) v[r * NB + b] = f32x2_lo(acc[r][b]) + f32x2_hi(acc[r][b]);
    const float z = reduce_spread<N>(v);
    const int id = g * R + my_r;
    if (counts && id < a.V) {
      stat_add(st, z);
      if (z > list.v[TK - 1]) list.insert(z, id);
    }
  }
  // join the CTA's lanes: the lists of batch row b, R a warp, through shared memory
  __syncthreads();
  u64* s_key = reinterpret_cast<u64*>(smem);            // [NB][LISTS][TK]
  float4* s_stat = reinterpret_cast<float4*>(s_key + NB * LISTS * TK);   // [NB][LISTS]
  if (lane % SHARE == 0) {
    const int at = my_b * LISTS + warp * R + my_r;
#pragma unroll
    for (int i = 0; i < TK; ++i) s_key[at * TK + i] = list.key(i);
    s_stat[at] = make_float4(st.m, st.s, st.u, 0.f);
  }
  __syncthreads();
  for (int b = warp; b < nb; b += WARPS) {
    u64 L[TK];
#pragma unroll
    for (int i = 0; i < TK; ++i) L[i] = s_key[(b * LISTS + lane) * TK + i];
    const float4 q = s_stat[b * LISTS + lane];
    const Stat all = stat_warp(Stat{q.x, q.y, q.z});
    const int64_t slot = (int64_t)(b0 + b) * a.splits + blockIdx.x;
    __shared__ u64 s_out[WARPS][TK];
    warp_merge<TK>(L, s_out[warp]);
    __syncwarp();
    if (lane == 0) *reinterpret_cast<float4*>(a.part_stat + slot * 4) = make_float4(all.m, all.s, all.u, 0.f);
    for (int i = lane; i < TK; i += 32) a.part_key[slot * TK + i] = s_out[warp][i];
    __syncwarp();
  }
}

// ---------------------------------------------------------------------------------
// tcgen05 form
// ---------------------------------------------------------------------------------
constexpr int EPI_WARPS = 8;                  // two per TMEM lane quarter, each with half of a tile's columns
constexpr int TC_THREADS = 64 + 32 * EPI_WARPS;
constexpr int KCH = 64;                       // K elements per chunk (one 128-byte swizzle row)
constexpr int MROWS = 128;                    // batch rows per block (TMEM lanes)
constexpr int MAX_N = 256;                    // vocabulary rows per tile
constexpr int MAX_STAGES = 8;
constexpr int Z_LD = 17;                      // padded row of the candidate buffer: 16 logits a thread
constexpr int Z_BYTES = 32 * EPI_WARPS * Z_LD * 4;
constexpr int TC_FIXED = 1024 + Z_BYTES;      // alignment slack, candidate buffer

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

struct TcPlan {
  int N;                                      // vocabulary rows per tile
  int blocks, group, passes;                  // row blocks; side by side; one after the other
  int splits;                                 // CTAs that share a row block's vocabulary
  int parts, a_rows, stages;                  // bf16 parts of h, rows loaded per part, ring depth
};

template <int TK>
__global__ void __launch_bounds__(TC_THREADS, 1)
logprob_tc_kernel(const __grid_constant__ LogprobArgs a, const __grid_constant__ TcPlan p,
                  const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmH) {
  constexpr uint64_t DESC = tc::desc_template(16, 1024, tc::SWIZZLE_128B);
  constexpr uint32_t TMEM_COLS = 2 * MAX_N;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t full[MAX_STAGES], empty[MAX_STAGES], acc_full[2], acc_empty[2], drain;
  __shared__ uint32_t s_taddr;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int w_bytes = p.N * 128, a_bytes = p.a_rows * 128;
  const int stage = w_bytes + p.parts * a_bytes;
  // the MMA reads MROWS rows of h whatever a_rows: past the last stage's rows it meets this buffer
  static_assert(Z_BYTES >= MROWS * 128, "operand reads stay inside shared memory");
  float* s_z = reinterpret_cast<float*>(sm + p.stages * stage);
  const int rb0 = blockIdx.x % p.group, split = blockIdx.x / p.group;
  const int n_tiles = (a.V + p.N - 1) / p.N, kchunks = a.H / KCH;
  const int tiles = split < n_tiles ? (n_tiles - 1 - split) / p.splits + 1 : 0;
  const int my_passes = rb0 < p.blocks ? (p.blocks - 1 - rb0) / p.group + 1 : 0;
  const int items = tiles * my_passes;        // (pass, tile) in order

  if (warp == 1) tc::tmem_alloc(&s_taddr, TMEM_COLS);
  if (tid == 0) {
    for (int s = 0; s < p.stages; ++s) { mbar_init(&full[s], 1); mbar_init(&empty[s], 1); }
    for (int i = 0; i < 2; ++i) { mbar_init(&acc_full[i], 1); mbar_init(&acc_empty[i], EPI_WARPS); }
    mbar_init(&drain, 1);
    fence_mbar_init();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = s_taddr;
  griddep_wait();
  griddep_launch_dependents();

  // Ring positions advance by counting: a division by a run-time ring depth or tile count costs the one
  // issuing thread about 60 ns, several of them a chunk cost more than the chunk's products.
  if (warp == 0) {
    if (lane == 0) {
      tc::tma_prefetch_desc(&tmW);
      tc::tma_prefetch_desc(&tmH);
      int s = 0, it = 0;
      uint32_t phase = 1;                     // of empty[s]: the first round finds it free
      bool ok = true;
      for (int ps = 0, rb = rb0; ps < my_passes && ok; ++ps, rb += p.group)
        for (int tl = 0, tile = split; tl < tiles && ok; ++tl, tile += p.splits)
          for (int c = 0; c < kchunks; ++c, ++it) {
            if (it >= p.stages && !mbar_wait_bounded(&empty[s], phase)) { ok = false; break; }
            uint8_t* dst = sm + s * stage;
            mbar_arrive_expect_tx(&full[s], (uint32_t)stage);
            tc::tma_load_4d(dst, &tmW, c * KCH, tile * p.N, 0, 0, &full[s]);
            for (int h = 0; h < p.parts; ++h)
              tc::tma_load_4d(dst + w_bytes + h * a_bytes, &tmH, c * KCH, rb * MROWS, h, 0, &full[s]);
            if (++s == p.stages) { s = 0; phase ^= 1; }
          }
      if (!ok) {                              // gave up: the copies in flight land first (bounded)
        for (int j = max(0, it - p.stages); j < it; ++j) (void)mbar_wait_bounded(&full[j % p.stages], (j / p.stages) & 1);
      }
    }
  } else if (warp == 1) {
    const uint32_t idesc = tc::idesc_bf16(MROWS, p.N, 0, 0);
    int s = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int item = 0; item < items && ok; ++item) {
      const int ab = item & 1;
      if (item >= 2) ok = __all_sync(FULL_MASK, mbar_wait_bounded(&acc_empty[ab], ((item >> 1) + 1) & 1));
      tc::fence_after_sync();
      for (int c = 0; c < kchunks && ok; ++c) {
        ok = __all_sync(FULL_MASK, mbar_wait_bounded(&full[s], phase));
        if (!ok) break;
        tc::fence_after_sync();
        const uint32_t w_addr = smem_u32(sm + s * stage), h_addr = w_addr + w_bytes;
        for (int h = 0; h < p.parts; ++h)
          tc::mma_ss_x4_elect(tmem + ab * MAX_N, tc::desc_at(DESC, h_addr + h * a_bytes), tc::desc_at(DESC, w_addr), idesc,
                              c > 0 || h > 0);
        tc::mma_commit_elect(&empty[s]);
        if (++s == p.stages) { s = 0; phase ^= 1; }
      }
      if (ok) tc::mma_commit_elect(&acc_full[ab]);
    }
    if (!ok) {                                // gave up: the products in flight end first (bounded)
      tc::mma_commit_elect(&drain);
      (void)mbar_wait_bounded(&drain, 0);
    }
  } else {
    const int q = warp & 3, row = q * 32 + lane;          // TMEM lane = row of the block
    const int side = (warp - 2) >> 2, cols = p.N / 2;     // the warp's half of the columns
    float* zrow = s_z + (tid - 64) * Z_LD;
    Stat st{-INFINITY, 0.f, 0.f};
    TopList<TK> list;
    list.clear();
    bool ok = true;
    int tile = split, rb = rb0;
    for (int item = 0; item < items; ++item) {
      const int ab = item & 1, b = rb * MROWS + row;
      if (!__all_sync(FULL_MASK, mbar_wait_bounded(&acc_full[ab], (item >> 1) & 1))) { ok = false; break; }
      tc::fence_after_sync();
      const uint32_t base = tmem + ((uint32_t)(q * 32) << 16) + ab * MAX_N + side * cols;
      // 32 columns z of the tile: they begin at vocabulary row v0
      auto piece = [&](uint32_t (&z)[32], int v0) {
        const int nv = a.V - v0;
        if (nv <= 0) return;
        if (nv < 32) {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (j >= nv) z[j] = __float_as_uint(-1e30f);  // adds nothing to the sums
        }
        float top = __uint_as_float(z[0]);
#pragma unroll
        for (int j = 1; j < 31; j += 2) top = fmaxf(fmaxf(top, __uint_as_float(z[j])), __uint_as_float(z[j + 1]));
        top = fmaxf(top, __uint_as_float(z[31]));
        if (top > st.m) {
          const float d = st.m - top, e = __expf(d);      // -inf on the first piece, whose sums are 0
          st.u = st.s == 0.f ? 0.f : e * fmaf(st.s, d, st.u);
          st.s *= e;
          st.m = top;
        }
        const uint64_t minus_m = pack_f32x2(-st.m, -st.m), log2e = pack_f32x2(LOG2E, LOG2E);
        uint64_t s2 = 0ull, u2 = 0ull;                         // pairs of zeros
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
          const uint64_t d = add_f32x2(((uint64_t)z[j + 1] << 32) | z[j], minus_m), t = mul_f32x2(d, log2e);
          const uint64_t e = pack_f32x2(ex2(f32x2_lo(t)), ex2(f32x2_hi(t)));
          s2 = add_f32x2(s2, e);
          u2 = fma_f32x2(e, d, u2);
        }
        st.s += f32x2_lo(s2) + f32x2_hi(s2);
        st.u += f32x2_lo(u2) + f32x2_hi(u2);
        if (top > list.v[TK - 1] && b < a.B) {
#pragma unroll
          for (int j0 = 0; j0 < 32; j0 += 16) {
            uint32_t cand = 0;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              zrow[j] = __uint_as_float(z[j0 + j]);
              if (__uint_as_float(z[j0 + j]) > list.v[TK - 1]) cand |= 1u << j;
            }
            if (nv < j0 + 16) cand &= nv > j0 ? (1u << (nv - j0)) - 1 : 0u;
            while (cand) {                                // ids ascend: an equal logit keeps the lower id
              const int j = __ffs(cand) - 1;
              cand &= cand - 1;
              list.insert(zrow[j], v0 + j0 + j);
            }
          }
        }
      };
      if (rb * MROWS + q * 32 < a.B) {                    // a warp with rows (warp-uniform)
        // the next 32 columns are on their way while these are worked on
        uint32_t z0[32], z1[32];
        const int first = tile * p.N + side * cols;
        tc::tmem_ld32(base, z0);
        for (int c0 = 0;; c0 += 64) {
          tc::tmem_wait_ld();
          if (c0 + 32 < cols) tc::tmem_ld32(base + c0 + 32, z1);
          piece(z0, first + c0);
          if (c0 + 32 >= cols) break;
          tc::tmem_wait_ld();
          if (c0 + 64 < cols) tc::tmem_ld32(base + c0 + 64, z0);
          piece(z1, first + c0 + 32);
          if (c0 + 64 >= cols) break;
        }
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[ab]);
      tile += p.splits;
      if (tile >= n_tiles) {                              // the row block's vocabulary is done
        if (b < a.B) {
          const int64_t slot = (int64_t)b * a.splits + 2 * split + side;
          *reinterpret_cast<float4*>(a.part_stat + slot * 4) = make_float4(st.m, st.s, st.u, 0.f);
#pragma unroll
          for (int i = 0; i < TK; ++i) a.part_key[slot * TK + i] = list.key(i);
        }
        tile = split;
        rb += p.group;
        st = Stat{-INFINITY, 0.f, 0.f};
        list.clear();
      }
    }
    if (!ok) {                                            // gave up: the rows of every pass are void (the merge sees NaN)
      for (int ps = 0; ps < my_passes; ++ps) {
        const int b = (rb0 + ps * p.group) * MROWS + row;
        if (b >= a.B) continue;
        const int64_t slot = (int64_t)b * a.splits + 2 * split + side;
        a.part_stat[slot * 4] = a.part_stat[slot * 4 + 1] = a.part_stat[slot * 4 + 2] = __uint_as_float(0x7fc00000u);
        for (int i = 0; i < TK; ++i) a.part_key[slot * TK + i] = 0ull;
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 1) tc::tmem_dealloc(tmem, TMEM_COLS);
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_fn_lp() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(f);
  });
  return fn;
}

// bf16 map [parts, rows, H], box [box_rows x 64]; rows past the end read as zeros.
cudaError_t make_map(CUtensorMap* m, const void* base, int H, int rows, int parts, int box_rows) {
  EncodeTiledFn fn = encode_fn_lp();
  if (!fn) return cudaErrorNotSupported;
  const cuuint64_t dims[4] = {(cuuint64_t)H, (cuuint64_t)rows, (cuuint64_t)parts, 1};
  const cuuint64_t strides[3] = {(cuuint64_t)H * 2, (cuuint64_t)H * 2 * rows, (cuuint64_t)H * 2 * rows * parts};
  const cuuint32_t box[4] = {KCH, (cuuint32_t)box_rows, 1, 1};
  const cuuint32_t es[4] = {1, 1, 1, 1};
  const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, es,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// s + p with its rounding error added to c.
__device__ __forceinline__ void sum_two(float& s, float& c, float p) {
  const float t = __fadd_rn(s, p), z = __fsub_rn(t, s);
  c = __fadd_rn(c, __fadd_rn(__fsub_rn(s, __fsub_rn(t, z)), __fsub_rn(p, z)));
  s = t;
}
// W[v] . h in about twice float32 precision, as a pair (hi, lo) in every lane of the warp; h in shared
// memory.  (The GPU has few float64 units: one row's sums in float64 took longer than its lists.)
template <typename WT>
__device__ __forceinline__ float2 dot_again(const LogprobArgs& a, const float* h, int v) {
  const WT* w = reinterpret_cast<const WT*>(a.W) + (int64_t)v * a.H;
  float s = 0.f, c = 0.f;
  constexpr int AHEAD = 4;                                // 8-element pieces loaded before any is used
#pragma unroll 1
  for (int k0 = (threadIdx.x & 31) * 8; k0 < a.H; k0 += 256 * AHEAD) {
    float x[AHEAD][8];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j)
      if (k0 + 256 * j < a.H) load8(w + k0 + 256 * j, x[j]);
#pragma unroll
    for (int j = 0; j < AHEAD; ++j)
      if (k0 + 256 * j < a.H) {
        const float4 y0 = *reinterpret_cast<const float4*>(h + k0 + 256 * j), y1 = *reinterpret_cast<const float4*>(h + k0 + 256 * j + 4);
        const float y[8] = {y0.x, y0.y, y0.z, y0.w, y1.x, y1.y, y1.z, y1.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float p = __fmul_rn(x[j][i], y[i]);
          c = __fadd_rn(c, __fmaf_rn(x[j][i], y[i], -p));
          sum_two(s, c, p);
        }
      }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float s2 = __shfl_xor_sync(FULL_MASK, s, o), c2 = __shfl_xor_sync(FULL_MASK, c, o);
    const float lo = fminf(s, s2);
    s = fmaxf(s, s2);                                     // both lanes of a pair add in one order
    c = __fadd_rn(c, c2);
    sum_two(s, c, lo);
  }
  const float hi = __fadd_rn(s, c);                       // |c| is far below |s|, or the sum is small: exact enough
  return make_float2(hi, __fadd_rn(__fsub_rn(s, hi), c));
}

template <typename WT, int TK>
__global__ void __launch_bounds__(merge_max(TK))
logprob_merge_kernel(const __grid_constant__ LogprobArgs a) {
  static_assert(TK <= 32, "one lane per candidate");
  extern __shared__ __align__(16) float s_h[];          // [H]
  __shared__ u64 s_w[merge_max(TK) / 32][TK];
  __shared__ u64 s_top[TK];
  __shared__ float2 s_val[TK + 1];                      // logits scored again; [TK]: the given token's
  __shared__ Stat s_stat[merge_max(TK) / 32];
  __shared__ int s_rank[TK];                            // candidate of each rank, -1: none
  const int b = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, warps = blockDim.x >> 5;
  griddep_wait();
  griddep_launch_dependents();
  const int target = a.targets ? a.targets[b] : -1;
  for (int k = tid; k < a.H; k += blockDim.x) s_h[k] = hidden_at(a, (int64_t)b * a.H + k);
  Stat st{-INFINITY, 0.f, 0.f};
  u64 L[TK];
#pragma unroll
  for (int i = 0; i < TK; ++i) L[i] = 0ull;
  __syncthreads();
  auto score = [&](int c, int v) {                      // the logit of token v (< 0: none) for entry c
    const float2 d = v >= 0 && v < a.V ? dot_again<WT>(a, s_h, v) : make_float2(0.f, 0.f);
    if (lane == 0) s_val[c] = d;
  };
  const bool idle = (warps - 1) * 32 >= a.splits;       // a last warp without splits takes the given token now
  if (idle && warp == warps - 1) score(TK, target);
  if (tid < a.splits) {                                 // one split per thread: its list is sorted
    const int64_t slot = (int64_t)b * a.splits + tid;
    const float4 q = *reinterpret_cast<const float4*>(a.part_stat + slot * 4);
    st = Stat{q.x, q.y, q.z};
    const ulonglong2* keys = reinterpret_cast<const ulonglong2*>(a.part_key + slot * TK);
#pragma unroll
    for (int i = 0; i < TK / 2; ++i) {
      const ulonglong2 two = keys[i];
      L[2 * i] = two.x; L[2 * i + 1] = two.y;
    }
  }
  // lists and statistics: within the warps, then (second round) those of the warps in warp 0
#pragma unroll 1
  for (int round = 0; round < 2; ++round) {
    if (round == 1) {
      if (warp == 0) {
#pragma unroll
        for (int i = 0; i < TK; ++i) L[i] = lane < warps ? s_w[lane][i] : 0ull;
        st = lane < warps ? s_stat[lane] : Stat{-INFINITY, 0.f, 0.f};
      }
    }
    if (round == 0 || warp == 0) {
      if (round == 1 || warp * 32 < a.splits) {
        st = stat_warp(st);
        warp_merge<TK>(L, round == 0 ? s_w[warp] : s_top);
      } else if (lane < TK) {                           // a warp without splits
        s_w[warp][lane] = 0ull;
      }
      if (round == 0 && lane == 0) s_stat[warp] = st;
    }
    __syncthreads();
  }
  auto id_of = [&](int c) { return (int)(0xffffffffu - (uint32_t)(s_top[c] & 0xffffffffull)); };
#pragma unroll 1
  for (int c = warp; c < (idle ? TK : TK + 1); c += warps) score(c, c == TK ? target : (s_top[c] ? id_of(c) : -1));
  if (tid < TK) s_rank[tid] = -1;
  __syncthreads();
  if (warp == 0) {
    // the candidates carry most of the sums: exchange their logits y for the ones scored again,
    // x = y + d with a small d, so exp(x) - exp(y) = exp(y) (d + d^2 / 2)
    float ds = 0.f, du = 0.f;
    if (lane < TK && s_top[lane]) {
      const float z = float_from_order_bits((uint32_t)(s_top[lane] >> 32)), y = z - st.m;
      const float2 x = s_val[lane];
      const float d = (x.x - z) + x.y, g = fmaf(0.5f * d, d, d), e = __expf(y);
      ds = e * g;
      du = e * fmaf(g, y + d, d);
      int rank = 0;
#pragma unroll 4
      for (int c = 0; c < TK; ++c) {
        const float2 o = s_val[c];
        const u64 key = s_top[c];
        const bool above = o.x > x.x || (o.x == x.x && (o.y > x.y || (o.y == x.y && (uint32_t)key > (uint32_t)s_top[lane])));
        rank += key != 0ull && above;
      }
      s_rank[rank] = lane;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      ds += __shfl_xor_sync(FULL_MASK, ds, o);
      du += __shfl_xor_sync(FULL_MASK, du, o);
    }
    const float sum = st.s + ds, ls = logf(sum);
    // a sum of NaN: a wait gave up and part of the vocabulary is missing, or a logit is NaN or +infinity.  No id
    // is the best then.
    const bool lost = sum != sum;
    __syncwarp();
    auto logprob = [&](float2 z) { return ((z.x - st.m) + z.y) - ls; };
    if (lane == 0) {
      if (a.out_lse) a.out_lse[b] = st.m + ls;
      if (a.out_entropy) a.out_entropy[b] = ls - (st.u + du) / sum;
      if (a.targets)
        a.out_logprob[b] = target < 0 ? 0.f : (target < a.V ? logprob(s_val[TK]) : __uint_as_float(0x7fc00000u));
    }
    if (lane < a.top_k) {
      const int c = lost ? -1 : s_rank[lane];
      const int64_t o = (int64_t)b * a.top_k + lane;
      a.top_ids[o] = c < 0 ? -1 : id_of(c);
      if (a.top_logprobs) a.top_logprobs[o] = c < 0 ? __uint_as_float(0x7fc00000u) : logprob(s_val[c]);
    }
  }
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// Candidates kept for top_k alternatives: the rest is room for neighbours that rounding exchanges.  (20
// alternatives with lists of 24 instead of 32: 64 rows of 151936 153 to 118 us, 10 rows of 1325 46 to 34 us.)
int list_len(int top_k) { return top_k <= 5 ? 8 : (top_k <= 8 ? 12 : (top_k <= 12 ? 16 : (top_k <= 20 ? 24 : 32))); }

constexpr int SMS = 152;                      // grids are sized for the whole GPU; fewer SMs only take longer
// Streaming form: batch rows of a CTA (1, 2, 4 or 8) and the vocabulary splits.
int stream_rows(int B) { return B >= 5 ? 8 : (B >= 3 ? 4 : B); }
int stream_splits(int B, int V, int tk) {
  const int nb = stream_rows(B), blocks = (B + nb - 1) / nb;
  const int ctas = SMS * stream_ctas(nb, tk);
  return std::max(1, std::min((V + R * WARPS - 1) / (R * WARPS), ctas / std::min(blocks, ctas)));
}

bool tc_supports(int H) { return H % KCH == 0; }

// At most 8 row blocks side by side.  The tile width is the one whose rounds of tiles cost least, a tile
// costing its columns and a fixed part worth about 32 of them.
TcPlan tc_plan(int B, int V, int parts) {
  TcPlan p{};
  p.blocks = (B + MROWS - 1) / MROWS;
  p.passes = (p.blocks + 7) / 8;
  p.group = (p.blocks + p.passes - 1) / p.passes;
  const int most = SMS / p.group;
  int64_t best = 0;
  for (int N = MAX_N; N >= 64; N /= 2) {
    const int tiles = (V + N - 1) / N;
    const int64_t cost = (int64_t)((tiles + most - 1) / most) * (N + 32);
    if (best == 0 || cost < best) { best = cost; p.N = N; p.splits = std::min(tiles, most); }
  }
  p.parts = parts;
  p.a_rows = std::min(MROWS, (B + 7) / 8 * 8);
  const int stage = p.N * 128 + parts * p.a_rows * 128;
  p.stages = std::min(MAX_STAGES, (232448 - 2048 - TC_FIXED) / stage);
  return p;
}

// One thread per split; a warp for each candidate scored again while the rows do not fill the GPU, else 4.
template <typename WT, int TK>
cudaError_t launch_merge(const LogprobArgs& a, cudaStream_t s) {
  const int threads = std::max((a.splits + 31) / 32 * 32, a.B <= SMS ? std::min(32 * TK, merge_max(TK)) : 128);
  return launch_pdl(logprob_merge_kernel<WT, TK>, dim3(a.B), dim3(threads), sizeof(float) * a.H, s, a);
}

template <int TK>
cudaError_t launch_tc(const LogprobArgs& a, const TcPlan& p, cudaStream_t s) {
  constexpr int smem = 232448 - 2048;         // everything but the static barriers: one CTA per SM
  static DeviceOnce configured;
  if (!configured.done()) {
    cudaError_t e = cudaFuncSetAttribute(logprob_tc_kernel<TK>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    configured.mark();
  }
  CUtensorMap mw, mh;
  cudaError_t e = make_map(&mw, a.W, a.H, a.V, 1, p.N);
  if (e != cudaSuccess) return e;
  if ((e = make_map(&mh, p.parts == 2 ? (const void*)a.hb : a.h, a.H, a.B, p.parts, p.a_rows)) != cudaSuccess) return e;
  if ((e = launch_pdl(logprob_tc_kernel<TK>, dim3(p.group * p.splits), dim3(TC_THREADS), smem, s, a, p, mw, mh)) != cudaSuccess)
    return e;
  return launch_merge<bf16_t, TK>(a, s);
}

template <typename WT, int NB, int TK>
cudaError_t launch_stream_n(const LogprobArgs& a, cudaStream_t s) {
  constexpr int join = NB * R * WARPS * (TK * 8 + 16);
  const int smem = std::max(join, (int)(sizeof(float) * NB * ((a.H + 255) / 256 * 256)));
  static DeviceOnce configured;
  if (!configured.done()) {
    cudaError_t e = cudaFuncSetAttribute(logprob_stream_kernel<WT, NB, TK>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         std::max(join, (int)sizeof(float) * NB * lmhead_max_hidden()));
    if (e != cudaSuccess) return e;
    configured.mark();
  }
  const cudaError_t e = launch_pdl(logprob_stream_kernel<WT, NB, TK>, dim3(a.splits, (a.B + NB - 1) / NB), dim3(THREADS),
                                   (size_t)smem, s, a);
  return e != cudaSuccess ? e : launch_merge<WT, TK>(a, s);
}
template <typename WT, int TK>
cudaError_t launch_stream(const LogprobArgs& a, cudaStream_t s) {
  switch (stream_rows(a.B)) {
    case 1: return launch_stream_n<WT, 1, TK>(a, s);
    case 2: return launch_stream_n<WT, 2, TK>(a, s);
    case 4: return launch_stream_n<WT, 4, TK>(a, s);
    default: return launch_stream_n<WT, 8, TK>(a, s);
  }
}

template <int TK>
cudaError_t launch_k(const LogprobArgs& a, kva_dtype w_dtype, const TcPlan* p, cudaStream_t s) {
  if (p) return launch_tc<TK>(a, *p, s);
  return w_dtype == KVA_BF16 ? launch_stream<bf16_t, TK>(a, s) : launch_stream<float, TK>(a, s);
}

}  // namespace

// Workspace: [normalised rows, float32][bf16 halves][partial statistics][partial lists]
static size_t parts_bytes(int B, int H, int V, int tk) {
  int splits = stream_splits(B, V, tk);
  if (tc_supports(H)) splits = std::max(splits, 2 * tc_plan(B, V, 2).splits);
  const size_t parts = (size_t)B * splits;
  return up256(parts * 16) + up256(parts * 8 * tk);
}
size_t logprob_workspace_bytes(int B, int H, int V, int top_k) {
  return 2 * up256(sizeof(float) * (size_t)B * H) + parts_bytes(B, H, V, list_len(top_k));
}
// Enough for this call and for those of fewer rows or alternatives, which may split the vocabulary more: between
// multiples of 8 rows the blocks of either form, and with them the splits, stay the same.
size_t logprob_workspace_bound(int B, int H, int V, int top_k) {
  size_t most = 0;
  for (int tk : {8, 12, 16, 24, 32})
    if (tk <= list_len(top_k))
      for (int b = B; b > 0; b = b <= 8 ? b - 1 : (b - 1) / 8 * 8) most = std::max(most, parts_bytes(b, H, V, tk));
  return 2 * up256(sizeof(float) * (size_t)B * H) + most;
}

cudaError_t launch_logprobs(LogprobArgs a, kva_dtype w_dtype, void* workspace, cudaStream_t s, unsigned* n_launches) {
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  const bool tc = w_dtype == KVA_BF16 && tc_supports(a.H) && encode_fn_lp() != nullptr;
  const bool split = a.h_dtype == KVA_F32 || a.norm_w;    // rows that need two bf16 halves
  TcPlan p{};
  if (tc) p = tc_plan(a.B, a.V, split ? 2 : 1);
  a.splits = tc ? 2 * p.splits : stream_splits(a.B, a.V, list_len(a.top_k));   // two column halves a CTA
  a.hn = reinterpret_cast<float*>(ws);
  ws += up256(sizeof(float) * (size_t)a.B * a.H);
  a.hb = tc && split ? reinterpret_cast<uint16_t*>(ws) : nullptr;
  ws += up256(sizeof(float) * (size_t)a.B * a.H);
  a.part_stat = reinterpret_cast<float*>(ws);
  a.part_key = reinterpret_cast<u64*>(ws + up256((size_t)a.B * a.splits * 16));
  *n_launches = 2;
  if (a.norm_w || a.hb) {
    cudaError_t e = launch_pdl(logprob_prep_kernel, dim3(a.B), dim3(THREADS), 0, s, a);
    if (e != cudaSuccess) return e;
    *n_launches = 3;
  }
  switch (list_len(a.top_k)) {
    case 8: return launch_k<8>(a, w_dtype, tc ? &p : nullptr, s);
    case 12: return launch_k<12>(a, w_dtype, tc ? &p : nullptr, s);
    case 16: return launch_k<16>(a, w_dtype, tc ? &p : nullptr, s);
    case 24: return launch_k<24>(a, w_dtype, tc ? &p : nullptr, s);
    default: return launch_k<32>(a, w_dtype, tc ? &p : nullptr, s);
  }
}

}  // namespace kva
