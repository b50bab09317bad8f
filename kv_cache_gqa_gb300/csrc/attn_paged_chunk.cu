// Attention of chunks of new tokens over a paged bf16 cache on tcgen05 (kv_attn_paged, bf16 output): more than 16
// query rows (token, head of the group) a KV head.
//
// A row tile is tpt = 128 / G tokens with all G heads of the group: up to 128 rows on the M side of the products, so a K/V
// tile is read once for the whole group whatever G is.  A unit is two neighbouring row tiles of one (sequence,
// KV head): the two slots of a CTA, which share every 128-key tile.  A last row tile without a neighbour takes both slots
// alone ("halves"): they alternate over its key tiles and are joined at the end.  A step is one tile for each slot.
// All units' steps are cut into equal runs, one CTA an SM each (paged.cuh); a unit that several runs share leaves
// unnormalised parts, which a second kernel joins.
//
// Twelve warps:
//   0-3, 4-7  softmax of slots 0 and 1, a row a thread: scores from tensor memory, the row's limit, a lazily moved reference
//             maximum (O is rescaled when a score exceeds it by 2^8), P = exp2(S - m) written back over S as bf16.
//   8, 10     TMA of Q and K, and of V.  A key tile is a box for each page it touches; the warp holds the next page ids a lane
//             each.  Slots of a tile at or beyond L are zeroed in V (they may hold anything, and 0 * NaN is NaN), and so are NaNs and
//             infinities in slots that only some rows of the unit see; the rows that do see them get their NaN at the end.
//   9, 11     issue the products of slots 0 and 1 from converged warps (one elected lane): O += P V for a tile, in two halves as
//             the softmax hands them over, then S of the slot's next tile into the same columns.  One warp for both slots was busy
//             all the time with its waits, descriptors and commits (4100 cycles a step; the products take 2048).
// P meets V in bf16, 8 bits: a second part would make three products a tile out of two, on the pipe that bounds long chunks, and its
// columns' writing and waiting would come on top.  A row's error against 64 bits is 2.3e-3 so, where the bf16 output's own rounding
// is 1.7e-3; the row's sum takes the weights before their rounding, in float32.
// Tensor memory: S of slot s at columns [128 s, 128 s + 128), O at [256 + 128 s, ..).  Every wait is bounded; one that
// gives up ends the CTA's work, and its rows become NaN.
//
// Bound: long prefixes by the tensor pipe and the hand-over from softmax to products (2048 tokens behind 29987 at 32/8 heads: 760 us,
// 1.37 PFLOP/s); prompts from their first token (4096 at 16/8 heads: 109 us) and short chunks (300 behind 4000: 41 us) also by the
// parts that units cut by the runs leave, and their join.  The cleaning of V costs the last two 2 to 4% and long prefixes nothing.
//
// Method: the flash-style form of MNN llm_demo walkthrough, section 5.1, over the visible prefix of each token (Youtu-VL-4B
// ncnn port, steps 7 and 8); bf16 storage with fp32 accumulation (HunyuanOCR v1.5 ncnn port, section 3.7).
#include <algorithm>

#include "paged.cuh"
#include "tc.cuh"

namespace kva {

namespace {

using paged::ex2;
using paged::finite_pair;
using paged::M_NONE;
using paged::Place;
using paged::Run;
using paged::saw_odd;
using paged::see_pair;
using paged::Seq;

constexpr int BM = 128, BN = 128;          // query rows of a slot, keys of a tile
constexpr int SOFTMAX_WARPS = 8;
constexpr int K_WARP = 8, MMA_WARP = 9, V_WARP = 10;   // and MMA_WARP + 2 for slot 1
constexpr int THREADS = 384;
// Registers: 168 a thread at launch; the control warpgroup gives up 48, which the two softmax warpgroups take.
constexpr int REGS_LAUNCH = 168, REGS_SOFTMAX = 192, REGS_CONTROL = 120;
static_assert(2 * REGS_SOFTMAX + REGS_CONTROL <= 3 * REGS_LAUNCH, "register split exceeds the launch total");
static_assert(REGS_LAUNCH * THREADS <= 65536, "launch registers");
constexpr int SUB = BM * 128;              // one [128 rows x 64 bf16] swizzled box column
constexpr int ST_BYTES = 32 * 32;          // a warp's staging tile: 32 rows x 16 bf16
constexpr uint32_t TMEM_COLS = 512;
constexpr float RESCALE_LOG2 = 8.0f;

template <int D, int DV>
struct Layout {
  static constexpr int NSUB = D / 64, NSUBV = DV / 64;
  static constexpr int NK = D == 192 ? 1 : 2, NV = 2;      // stages of the K and of the V ring
  static constexpr int Q_OFF = 0;                          // [2 slots][NSUB]
  static constexpr int K_OFF = Q_OFF + 2 * NSUB * SUB;     // [NK][NSUB]
  static constexpr int V_OFF = K_OFF + NK * NSUB * SUB;    // [NV][NSUBV]
  static constexpr int ST_OFF = V_OFF + NV * NSUBV * SUB;  // [softmax warp]
  static constexpr int ML_OFF = ST_OFF + SOFTMAX_WARPS * ST_BYTES;   // slot 1's (maximum, sum) of halves units
  static constexpr int BAR_OFF = ML_OFF + BM * 8;
  static constexpr int SMEM = BAR_OFF + 256 + 1024;        // + slack to align the base to 1024
  static_assert(SMEM + 1536 <= 232448, "shared memory per CTA, with the static part");
};

constexpr uint64_t DESC_KMAJ = tc::desc_template(16, 1024, tc::SWIZZLE_128B);
constexpr uint64_t DESC_VMN = tc::desc_template(SUB, 1024, tc::SWIZZLE_128B);

// Units of sequences of lo < T * G <= hi rows (see paged::Cut).
struct CutPairs {
  int G, tpt, lo, hi;
  __device__ __forceinline__ int row_tiles(const Seq& s) const { return (s.T + tpt - 1) / tpt; }
  __device__ __forceinline__ int tiles(const Seq& s) const {
    const int64_t rows = (int64_t)s.T * G;
    return rows > lo && rows <= hi ? (row_tiles(s) + 1) / 2 : 0;
  }
  __device__ __forceinline__ int visible(const Seq& s, int rt) const {
    return min(max(s.L - s.T + min(s.T, (rt + 1) * tpt), 0), s.L);
  }
  __device__ __forceinline__ int key_tiles(const Seq& s, int rt) const { return (visible(s, rt) + BN - 1) / BN; }
  // slots that all rows of unit z see
  __device__ __forceinline__ int common(const Seq& s, int z) const { return min(max(s.L - s.T + 2 * z * tpt + 1, 0), s.L); }
  __device__ __forceinline__ bool halves(const Seq& s, int z) const { return 2 * z + 1 >= row_tiles(s); }
  __device__ __forceinline__ int steps(const Seq& s, int z) const {
    return halves(s, z) ? max(1, (key_tiles(s, 2 * z) + 1) / 2) : max(1, key_tiles(s, 2 * z + 1));
  }
  __device__ __forceinline__ int64_t head_steps(const Seq& s) const {
    const int n = tiles(s);
    int64_t sum = 0;
    for (int z = 0; z < n; ++z) sum += steps(s, z);
    return sum;
  }
};

// A run's part of a unit: key tiles j0 .. j0 + n - 1 in order, ring entries one each.  Both slots take every tile (slot 0 the
// first c[0] of them), or, in halves, the even ones are slot 0's and the odd ones slot 1's; slot s takes c[s] tiles.
struct Piece {
  int st0, st1, j0, n, c[2];
  bool halves, whole;
  int tail;                                  // entry of the tile that holds L (its slots from L on are zeroed in V), or -1
  int clean;                                 // first entry with slots that not all rows see (V is cleaned there and in those behind it)
  __device__ __forceinline__ int entry(int s, int k) const { return halves ? 2 * k + s : k; }
};
__device__ __forceinline__ Piece piece_of(const CutPairs& cut, const Place& p, const Run& run) {
  Piece q;
  q.st0 = (int)max((int64_t)0, run.x0 - p.at);
  q.st1 = (int)min((int64_t)p.n_steps, run.x1 - p.at);
  q.whole = q.st0 == 0 && q.st1 == p.n_steps;
  q.halves = cut.halves(p.s, p.rt);
  if (q.halves) {
    q.j0 = 2 * q.st0;
    q.n = min(2 * q.st1, max(1, cut.key_tiles(p.s, 2 * p.rt))) - q.j0;
    q.c[0] = (q.n + 1) / 2;
    q.c[1] = q.n / 2;
  } else {
    q.j0 = q.st0;
    q.n = q.st1 - q.st0;
    q.c[0] = max(0, min(cut.key_tiles(p.s, 2 * p.rt) - q.st0, q.n));
    q.c[1] = q.n;
  }
  const int at = p.s.L / BN - q.j0;
  q.tail = p.s.L % BN != 0 && at >= 0 && at < q.n ? at : -1;
  q.clean = max(0, min(cut.common(p.s, p.rt) / BN - q.j0, q.n));
  return q;
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
      :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
         "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// Four products P V over adjacent 16-key slices: A from tensor memory (8 columns a slice), B 16 rows (2048 bytes) apart.
__device__ __forceinline__ void mma_ts_x4_elect(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                                uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, q;\n elect.sync _|q, 0xffffffff;\n setp.ne.b32 p, %9, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %10, p;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%3], %4, %10, 1;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%5], %6, %10, 1;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%7], %8, %10, 1;\n}\n"
      :: "r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(a_tmem + 8), "l"(b_desc + 128), "r"(a_tmem + 16), "l"(b_desc + 256),
         "r"(a_tmem + 24), "l"(b_desc + 384), "r"(accumulate), "r"(idesc) : "memory");
}
__device__ __forceinline__ uint64_t f2(float a, float b) { return pack_f32x2(a, b); }
__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// Phase `count` of a barrier, by all lanes; the vote keeps the warp converged for what follows.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, int count) { return paged::warp_wait(bar, (uint32_t)(count & 1)); }

// Pages that hold n slots.
__device__ __forceinline__ int pages_of(const PagedArgs& a, int n) { return (n + (1 << a.page_shift) - 1) >> a.page_shift; }

// A ring's copies of the pages of key tiles j0, j0 + 1, ..: ids of 32 pages at a time, a lane each.
struct Pages {
  const int32_t* row;                       // the sequence's page table
  int last, base;                           // pages below `last` hold slots below L; the 32 ids from page `base` on
  int id;
  bool bad;                                 // an id of them is outside the pool
  __device__ __forceinline__ void load(const PagedArgs& a, int from, int lane) {
    base = from;
    id = a.n_pages;                         // beyond L, or outside the pool: copies read zeros
    bad = false;
    if (from + lane < last) {
      const int x = row[from + lane];
      bad = (unsigned)x >= (unsigned)a.n_pages;
      if (!bad) id = x;
    }
    bad = __any_sync(FULL_MASK, bad);
  }
  // the ids of key tile j's pages
  __device__ __forceinline__ void need(const PagedArgs& a, int j, int lane) {
    const int n = a.page_shift < 7 ? 128 >> a.page_shift : 1, page = (j * BN) >> a.page_shift;
    if (page + n > base + 32) load(a, page, lane);
  }
};
// Copies key tile j of KV head g into `dst` ([NS columns][128 rows x 128 bytes]).  Whole warp.
template <int NS>
__device__ __forceinline__ void load_tile(const PagedArgs& a, const CUtensorMap* map, Pages& pg, int j, int g, uint8_t* dst,
                                          uint64_t* bar, int lane) {
  const int shift = a.page_shift, n = shift < 7 ? 128 >> shift : 1, page = (j * BN) >> shift;   // pages of a tile, the first one
  pg.need(a, j, lane);
  if (lane == 0) mbar_arrive_expect_tx(bar, NS * SUB);
  __syncwarp();
  const int id = __shfl_sync(FULL_MASK, pg.id, (page - pg.base + (lane & (n - 1))) & 31);
  if (lane < n) {
    const int row = shift < 7 ? 0 : (j * BN) & ((1 << shift) - 1);
    uint8_t* at = dst + ((lane << shift) & 127) * 128;
#pragma unroll
    for (int c = 0; c < NS; ++c) tc::tma_load_4d(at + c * SUB, map, c * 64, row, g, id, bar);
  }
  __syncwarp();
}

// A warp's way through its run, in shared memory (its registers are taken): the unit and its piece.
struct Walk {
  Place p;
  Piece q;
  int more;
};
__device__ __forceinline__ bool enter(Walk& w, const PagedArgs& a, const CutPairs& cut, const Run& run, bool first, int lane) {
  __syncwarp();
  if (lane == 0) {
    if (!first) w.p.next(a, cut);
    w.more = w.p.b < a.B && w.p.at < run.x1;
    if (w.more) w.q = piece_of(cut, w.p, run);
  }
  __syncwarp();
  return w.more != 0;
}

// What is left to do to the row of this thread when something was wrong.  gave_up: a wait did, and the rows from the walk's piece on
// become NaN.  Else the cleaning of V took NaNs or infinities, which make NaN of their columns in the rows that see them: all pieces
// of the CTA's run again.  Whole warp.  Out of line, and one function: a second call in the kernel costs the softmax registers.
template <int DV>
__device__ __noinline__ void mend_rows(Walk& w, const Place& begin, const PagedArgs& a, const CutPairs& cut, const Run& run, int s, int t,
                                       bool gave_up) {
  constexpr int PER = DV / 32;              // columns of a lane
  const int lane = t & 31;
  __syncwarp();
  if (!gave_up && lane == 0) {
    w.p = begin;
    w.more = begin.b < a.B && begin.at < run.x1;
    if (w.more) w.q = piece_of(cut, begin, run);
  }
  __syncwarp();
  for (bool more = w.more != 0; more; more = enter(w, a, cut, run, false, lane)) {
    const Place& p = w.p;
    if (w.q.halves && s == 1) continue;     // slot 0 writes both slots' halves
    const int token = (2 * p.rt + s) * cut.tpt + t / cut.G;
    const bool row_ok = t < cut.tpt * cut.G && token < p.s.T;
    const int64_t part = (int64_t)(blockIdx.x * 2 + (run.x0 >= p.at ? 0 : 1)) * 2 + s;
    uint16_t* out = reinterpret_cast<uint16_t*>(a.out) + ((int64_t)(p.s.t0 + token) * a.Hq + p.g * cut.G + t % cut.G) * DV;
    if (gave_up) {
      if (!w.q.whole) reinterpret_cast<float2*>(a.part_ml)[part * BM + t] = make_float2(M_NONE, NAN);   // whoever joins it finds NaN
      for (int d = 0; row_ok && d < DV; ++d) out[d] = 0x7fc0;
      continue;
    }
    const int lim = row_ok ? min(max(p.s.L - p.s.T + token + 1, 0), p.s.L) : 0;
    const int from = max(cut.common(p.s, p.rt), w.q.j0 * BN);
    const int to = min((w.q.j0 + (w.q.halves ? w.q.n : w.q.c[s])) * BN, lim), last = __reduce_max_sync(FULL_MASK, to);
    for (int key = from; key < last; ++key) {
      const int page = a.table[(int64_t)p.b * a.table_stride + (key >> a.page_shift)];
      if ((unsigned)page >= (unsigned)a.n_pages) continue;
      const uint16_t* v = reinterpret_cast<const uint16_t*>(a.v) + page * a.page_stride_v +
                          (int64_t)((p.g << a.page_shift) + (key & ((1 << a.page_shift) - 1))) * DV + lane * PER;
      uint32_t odd = 0u;                    // this lane's columns
#pragma unroll
      for (int e = 0; e < PER; ++e) odd |= ((v[e] & 0x7f80u) == 0x7f80u ? 1u : 0u) << e;
      for (unsigned hits = __ballot_sync(FULL_MASK, odd != 0u); hits; hits &= hits - 1) {
        const int h = __ffs(hits) - 1;
        for (uint32_t bits = __shfl_sync(FULL_MASK, odd, h); bits; bits &= bits - 1) {
          const int d = h * PER + __ffs(bits) - 1;
          if (key >= to) continue;
          if (w.q.whole) out[d] = 0x7fc0;
          else a.part_acc[((part * (DV / 4) + d / 4) * BM + t) * 4 + d % 4] = NAN;
        }
      }
    }
  }
}

template <int D, int DV>
__global__ void __launch_bounds__(THREADS, 1)
attn_paged_chunk_kernel(const __grid_constant__ PagedArgs a, const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmQ) {
  using LY = Layout<D, DV>;
  constexpr int NSUB = LY::NSUB, NSUBV = LY::NSUBV, NK = LY::NK, NV = LY::NV;
  constexpr uint32_t IDESC_S = tc::idesc_bf16(BM, BN, 0, 0);
  constexpr uint32_t IDESC_PV = tc::idesc_bf16(BM, DV, 0, 1);

  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + LY::BAR_OFF);
  uint64_t* k_full = bars + 0;     // [NK] K tile landed
  uint64_t* k_free = bars + 2;     // [NK] both slots are through with it
  uint64_t* v_full = bars + 4;     // [NV]
  uint64_t* v_free = bars + 6;     // [NV]
  uint64_t* s_full = bars + 8;     // [slot] S ready
  uint64_t* p_half = bars + 10;    // [slot] P of the tile's first 64 keys written by the slot's 4 warps
  uint64_t* p_full = bars + 12;    // [slot] and of the other 64
  uint64_t* o_full = bars + 14;    // [slot] the piece's last P V done
  uint64_t* o_free = bars + 16;    // [slot] O copied out (by 4 warps)
  uint64_t* q_full = bars + 18;    // the piece's Q landed
  uint64_t* q_free = bars + 19;    // both slots' last Q K^T of the piece done
  uint64_t* v_clean = bars + 20;   // [NV] a tile with slots that not all rows see has its V cleaned
  uint64_t* ml_full = bars + 22;   // slot 1's maxima and sums of a halves piece published (4 warps)
  uint64_t* ml_free = bars + 23;   // and read by slot 0 (4 warps)
  uint64_t* turn = bars + 24;      // [slot] the slot's products of a round have been issued
  uint32_t* s_taddr = reinterpret_cast<uint32_t*>(bars + 26);
  volatile int* s_abort = reinterpret_cast<volatile int*>(bars + 27);
  volatile uint32_t* s_bad = reinterpret_cast<volatile uint32_t*>(bars + 28);   // pieces (modulo 32) with a page id outside the pool
  volatile int* s_odd = reinterpret_cast<volatile int*>(bars + 29);             // the cleaning of V took something, now or before
  __shared__ int64_t scratch[THREADS / 32 + 4];
  __shared__ Run run;
  __shared__ Walk walks[THREADS / 32];
  __shared__ Place run_begin;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.Hq / a.Hkv;
  const CutPairs cut{G, BM / G, a.rows_lo, a.rows_hi};
  if (warp == MMA_WARP) tc::tmem_alloc(s_taddr, TMEM_COLS);
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_full[i], 1); mbar_init(&k_free[i], 2); mbar_init(&v_full[i], 1); mbar_init(&v_free[i], 2);
      mbar_init(&s_full[i], 1); mbar_init(&p_half[i], SOFTMAX_WARPS / 2); mbar_init(&p_full[i], SOFTMAX_WARPS / 2);
      mbar_init(&o_full[i], 1); mbar_init(&o_free[i], SOFTMAX_WARPS / 2); mbar_init(&v_clean[i], 1);
      mbar_init(&turn[i], 1);
    }
    mbar_init(q_full, 1); mbar_init(q_free, 2);
    mbar_init(ml_full, SOFTMAX_WARPS / 2); mbar_init(ml_free, SOFTMAX_WARPS / 2);
    *s_abort = 0;
    *s_bad = 0u;
    *s_odd = 0;
    fence_mbar_init();
  }
  if (warp == K_WARP && lane == 0) { tc::tma_prefetch_desc(&tmK); tc::tma_prefetch_desc(&tmV); tc::tma_prefetch_desc(&tmQ); }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *s_taddr;
  griddep_wait();                               // inputs of this launch are complete from here on
  griddep_launch_dependents();
  Walk& walk = walks[warp];
  {
    Place first;
    const Run mine = paged::first_place<THREADS>(a, cut, scratch, &first);
    if (lane == 0) walk.p = first;
    if (tid == 0) {
      run = mine;
      run_begin = first;
      a.joins[blockIdx.x].last = -1;
    }
  }
  __syncthreads();
  const Place& p = walk.p;
  const Piece& pc = walk.q;

  if (warp >= SOFTMAX_WARPS) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(REGS_CONTROL));
    bool ok = true;
    int it = 0;                                 // ring entries of earlier pieces
    int np = 0;                                 // pieces so far
    if (warp == K_WARP) {
      // ------------------------------------------------------------ Q and K copies
      for (bool first = true; ok && enter(walk, a, cut, run, first, lane); first = false) {
        if (np > 0 && !warp_wait(q_free, np - 1)) { ok = false; break; }
        if (lane == 0) {
          const int slots = pc.halves ? 1 : 2;
          mbar_arrive_expect_tx(q_full, slots * NSUB * (cut.tpt * G * 128));
          for (int s = 0; s < slots; ++s)
#pragma unroll
            for (int c = 0; c < NSUB; ++c)
              tc::tma_load_4d(sm + LY::Q_OFF + (s * NSUB + c) * SUB, &tmQ, c * 64, p.g * G,
                              p.s.t0 + (2 * p.rt + s) * cut.tpt, 0, q_full);
        }
        ++np;
        __syncwarp();
        bool bad = false;
        Pages pg{a.table + (int64_t)p.b * a.table_stride, pages_of(a, p.s.L), -64, 0, false};
        for (int i = 0; i < pc.n; ++i, ++it) {
          const int st = it % NK;
          if (it >= NK && !warp_wait(&k_free[st], it / NK - 1)) { ok = false; break; }
          pg.need(a, pc.j0 + i, lane);
          bad |= pg.bad;
          if (lane == 0 && i == pc.n - 1)       // before its last tile; this warp is at most a few pieces ahead of the softmax
            *s_bad = (*s_bad & ~(1u << ((np + 15) & 31))) | ((bad ? 1u : 0u) << ((np - 1) & 31));
          load_tile<NSUB>(a, &tmK, pg, pc.j0 + i, p.g, sm + LY::K_OFF + st * NSUB * SUB, &k_full[st], lane);
        }
        if (*s_abort) ok = false;
      }
      if (!ok) *s_abort = 1;
      // the copies that this warp issued have normally landed long ago; never leave one in flight
      for (int e = max(0, it - NK); e < it; ++e) (void)warp_wait(&k_full[e % NK], e / NK);
      if (np > 0 && !ok) (void)warp_wait(q_full, np - 1);
    } else if (warp == V_WARP) {
      // ------------------------------------------------------------ V copies
      for (bool first = true; ok && enter(walk, a, cut, run, first, lane); first = false) {
        Pages pg{a.table + (int64_t)p.b * a.table_stride, pages_of(a, p.s.L), -64, 0, false};
        for (int i = 0; i < pc.n; ++i, ++it) {
          const int st = it % NV;
          if (it >= NV && !warp_wait(&v_free[st], it / NV - 1)) { ok = false; break; }
          uint8_t* dst = sm + LY::V_OFF + st * NSUBV * SUB;
          load_tile<NSUBV>(a, &tmV, pg, pc.j0 + i, p.g, dst, &v_full[st], lane);
          if (i >= pc.clean) {
            if (!warp_wait(&v_full[st], it / NV)) { ok = false; ++it; break; }
            constexpr int W = 8 * NSUBV;        // 16-byte pieces of a row: a lane takes the same one of every 32 / W-th row
            const int to = i == pc.tail ? p.s.L % BN : BN, from = min(max(cut.common(p.s, p.rt) - (pc.j0 + i) * BN, 0), to);
            uint8_t* at = dst + (lane % W >> 3) * SUB + (lane & 7) * 16;
            uint32_t seen = 0u;
#pragma unroll 2                                // what runs once a unit pays for its instructions' way here: 8 took longer
            for (int r = from + lane / W; r < to; r += 32 / W) {
              const uint4 v = *reinterpret_cast<const uint4*>(at + r * 128);
              see_pair(seen, v.x); see_pair(seen, v.y); see_pair(seen, v.z); see_pair(seen, v.w);
            }
#pragma unroll 1
            for (int r = to + lane / W; r < BN; r += 32 / W) *reinterpret_cast<uint4*>(at + r * 128) = make_uint4(0, 0, 0, 0);
            const bool odd = __any_sync(FULL_MASK, saw_odd(seen));
            if (odd)
#pragma unroll 1
              for (int r = from + lane / W; r < to; r += 32 / W) {
                uint4* x = reinterpret_cast<uint4*>(at + r * 128);
                const uint4 v = *x;
                *x = make_uint4(finite_pair(v.x), finite_pair(v.y), finite_pair(v.z), finite_pair(v.w));
              }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              if (odd) *s_odd = 1;
              mbar_arrive(&v_clean[st]);
            }
          }
        }
        if (*s_abort) ok = false;
      }
      if (!ok) *s_abort = 1;
      for (int e = max(0, it - NV); e < it; ++e) (void)warp_wait(&v_full[e % NV], e / NV);
    } else {
      // ------------------------------------------------------------ products of slot s
      const int s = warp == MMA_WARP ? 0 : 1;
      const uint64_t q_desc = tc::desc_at(DESC_KMAJ, smem_u32(sm + LY::Q_OFF));
      const uint64_t k_desc = tc::desc_at(DESC_KMAJ, smem_u32(sm + LY::K_OFF));
      const uint64_t v_desc = tc::desc_at(DESC_VMN, smem_u32(sm + LY::V_OFF));
      // descriptor start addresses advance by constant offsets (addresses stay below 2^18)
      constexpr uint64_t BOX = (uint64_t)SUB >> 4;
      static_assert(NV == 2, "cleaned tiles are counted by two stages");
      int cleaned[2] = {0, 0};                  // tiles of a V stage so far
      int tiles = 0, used = 0;                  // the slot's tiles, and pieces with any, so far
      int rounds = 0;                           // turns taken so far
      for (bool first = true; ok && enter(walk, a, cut, run, first, lane); first = false, ++np) {
        const int c = pc.c[s];
        int kc = it, vc = it;                   // the next K and V entries to see: every entry is seen, in order, by both warps
        auto pass_k = [&](int e) {              // entries before e are the other slot's alone
          for (; kc < e && ok; ++kc) {
            ok = warp_wait(&k_full[kc % NK], kc / NK);
            if (ok && lane == 0) mbar_arrive(&k_free[kc % NK]);
          }
        };
        auto pass_v = [&](int e) {
          for (; vc < e && ok; ++vc) {
            ok = warp_wait(&v_full[vc % NV], vc / NV);
            if (ok && lane == 0) mbar_arrive(&v_free[vc % NV]);
          }
        };
        auto my_turn = [&]() { return s == 1 ? warp_wait(&turn[0], rounds) : (rounds == 0 || warp_wait(&turn[1], rounds - 1)); };
        auto pass_turn = [&]() {
          if (lane == 0) mbar_arrive(&turn[s]);
          ++rounds;
        };
        auto issue_s = [&](int k) {             // S of the slot's k-th tile
          const int e = it + pc.entry(s, k), st = e % NK;
          const uint64_t qd = q_desc + (uint64_t)(pc.halves ? 0 : s) * NSUB * BOX;
          const uint64_t kd = k_desc + (uint64_t)st * NSUB * BOX;
#pragma unroll
          for (int h = 0; h < NSUB; ++h)
            tc::mma_ss_x4_elect(tmem + s * BN, qd + h * BOX, kd + h * BOX, IDESC_S, h > 0);
          pass_turn();
          tc::mma_commit_elect(&s_full[s]);     // P V of the tile before is done then, too
          tc::mma_commit_elect(&k_free[st]);
          if (k == c - 1) tc::mma_commit_elect(q_free);
          kc = e + 1;
        };
        auto wait_k = [&](int k) {
          const int e = it + pc.entry(s, k);
          pass_k(e);
          ok = ok && warp_wait(&k_full[e % NK], e / NK);
        };
        // The slots take turns, slot 0 first: the tensor core runs one slot's products whole while the other's softmax runs.  Without,
        // both slots' products went through it interleaved and ended together, and both softmaxes then had it idle.
        ok = warp_wait(q_full, np);
        if (c > 0) {
          wait_k(0);
          tc::fence_after_sync();
          ok = ok && my_turn();
          if (ok) issue_s(0);
        } else {
          ok = ok && my_turn();
          if (ok && lane == 0) mbar_arrive(q_free);
          pass_turn();
        }
        const int both = max(pc.c[0], pc.c[1]);
        for (int k = 0; k < both && ok; ++k) {
          if (k >= c) {
            ok = my_turn();
            pass_turn();
            continue;
          }
          const int e = it + pc.entry(s, k), st = e % NV;
          // what is not waiting for the softmax comes first (with one K stage the next K waits for the other slot's S)
          if (NK > 1 && k + 1 < c) wait_k(k + 1);
          pass_v(e);
          ok = ok && warp_wait(&v_full[st], e / NV);
          if (e - it >= pc.clean) ok = ok && warp_wait(&v_clean[st], cleaned[st] + ((e - it - pc.clean) >> 1));
          // the first P V of a piece overwrites O: the one before must have been read
          if (k == 0 && used > 0) ok = ok && warp_wait(&o_free[s], used - 1);
          if (!ok) break;
          const uint64_t vd = v_desc + (uint64_t)st * NSUBV * BOX;
          if (!warp_wait(&p_half[s], tiles + k)) { ok = false; break; }
          if (!my_turn()) { ok = false; break; }
          tc::fence_after_sync();
          mma_ts_x4_elect(tmem + 256 + s * 128, tmem + s * BN, vd, IDESC_PV, k > 0);
          if (!warp_wait(&p_full[s], tiles + k)) { ok = false; break; }
          tc::fence_after_sync();
          mma_ts_x4_elect(tmem + 256 + s * 128, tmem + s * BN + 32, vd + 512, IDESC_PV, 1);
          tc::mma_commit_elect(&v_free[st]);
          vc = e + 1;
          if (NK == 1 && k + 1 < c) {
            wait_k(k + 1);
            tc::fence_after_sync();
            if (!ok) break;
          }
          if (k + 1 < c) {
            issue_s(k + 1);
          } else {
            pass_turn();
            tc::mma_commit_elect(&o_full[s]);
          }
        }
        it += pc.n;
        pass_k(it);
        pass_v(it);
        const int first_clean = (it - pc.n + pc.clean) & 1, clean = pc.n - pc.clean;
        cleaned[0] += (clean + 1 - first_clean) >> 1;
        cleaned[1] += (clean + first_clean) >> 1;
        tiles += c;
        used += c > 0;
        if (*s_abort) ok = false;
      }
      if (!ok) *s_abort = 1;
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(REGS_SOFTMAX));
    // ------------------------------------------------------------ softmax
    const int s = warp >> 2, quarter = warp & 3, t = quarter * 32 + lane;   // slot, lane quarter, row = TMEM lane
    const uint32_t lane_base = tmem + ((uint32_t)(quarter * 32) << 16);
    const uint32_t s_col = s * BN, o_col = 256 + s * 128;
    uint8_t* stage = sm + LY::ST_OFF + warp * ST_BYTES;
    float2* ml = reinterpret_cast<float2*>(sm + LY::ML_OFF);
    const bool in_tile = t < cut.tpt * G;
    bool ok = true;
    int tiles = 0, used = 0, shared = 0;        // this slot's tiles, pieces with any, halves pieces so far
    int pieces = 0;
    for (bool begin = true; ok && enter(walk, a, cut, run, begin, lane); begin = false) {
      const int rt = pc.halves ? 2 * p.rt : 2 * p.rt + s;
      const int token = rt * cut.tpt + t / G;
      const bool row_ok = in_tile && token < p.s.T;
      const int lim = row_ok ? min(max(p.s.L - p.s.T + token + 1, 0), p.s.L) : 0;   // slots that the row sees
      const int c = pc.c[s];
      float m = M_NONE, l = 0.f;
      float x[128];
      for (int k = 0; k < c; ++k) {
        const int kk = tiles + k;
        const int hi = lim - (pc.j0 + pc.entry(s, k)) * BN;             // the row's visible columns: [0, hi)
        if (!warp_wait(&s_full[s], kk)) { ok = false; break; }
        tc::fence_after_sync();
        const int hi_max = __reduce_max_sync(FULL_MASK, hi);           // 32-column chunks beyond it get P = 0
        {
          uint32_t r0[32], r1[32], r2[32], r3[32];
          tc::tmem_ld32(lane_base + s_col, r0);
          tc::tmem_ld32(lane_base + s_col + 32, r1);
          tc::tmem_ld32(lane_base + s_col + 64, r2);
          tc::tmem_ld32(lane_base + s_col + 96, r3);
          tc::tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            x[e] = __uint_as_float(r0[e]); x[32 + e] = __uint_as_float(r1[e]);
            x[64 + e] = __uint_as_float(r2[e]); x[96 + e] = __uint_as_float(r3[e]);
          }
        }
        if (hi < BN) {
#pragma unroll
          for (int e = 0; e < BN; ++e)
            if (e >= hi) x[e] = -INFINITY;
        }
        float mq[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int e = 0; e < BN; e += 8)
#pragma unroll
          for (int q = 0; q < 4; ++q) mq[q] = fmax3(mq[q], x[e + 2 * q], x[e + 2 * q + 1]);
        const float m_tile = fmaxf(fmax3(mq[0], mq[1], mq[2]), mq[3]) * a.scale_log2;   // -infinity: sees nothing here
        const bool first = m == M_NONE;                                 // O holds nothing of this row yet
        const bool grow = !first && m_tile > m + RESCALE_LOG2;
        if (first) m = fmaxf(m, m_tile);
        if (__any_sync(FULL_MASK, grow)) {
          // rescale those rows of O, which holds the P V before (the whole warp takes part; others by 1)
          const float alpha = grow ? ex2(m - m_tile) : 1.0f;
#pragma unroll
          for (int q = 0; q < DV / 16; ++q) {
            uint32_t rr[16];
            tmem_ld16(lane_base + o_col + q * 16, rr);
            tc::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) rr[e] = __float_as_uint(__uint_as_float(rr[e]) * alpha);
            tmem_st16(lane_base + o_col + q * 16, rr);
          }
          tc::tmem_wait_st();
          if (grow) { l *= alpha; m = m_tile; }
        }
        const uint64_t sc2 = f2(a.scale_log2, a.scale_log2), nm2 = f2(-m, -m);
        uint64_t lsum = 0ull;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t w[16];
          if (32 * q < hi_max) {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const uint64_t z = fma_f32x2(f2(x[32 * q + 2 * e], x[32 * q + 2 * e + 1]), sc2, nm2);
              const float p0 = ex2(f32x2_lo(z)), p1 = ex2(f32x2_hi(z));
              lsum = add_f32x2(lsum, f2(p0, p1));
              w[e] = pack_bf16x2(p0, p1);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) w[e] = 0u;
          }
          tmem_st16(lane_base + s_col + q * 16, w);
          if (q == 1) {
            tc::tmem_wait_st();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_half[s]);
          }
        }
        l += f32x2_lo(lsum) + f32x2_hi(lsum);
        tc::tmem_wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[s]);
      }
      if (!ok) break;
      if ((*s_bad >> (pieces & 31)) & 1u) l = NAN;                      // a page id outside the pool: no result
      if (c > 0 && !warp_wait(&o_full[s], used)) { ok = false; break; }
      tc::fence_after_sync();
      if (pc.halves && s == 1) {
        // slot 0 takes it from here: it reads both O
        if (shared > 0 && !warp_wait(ml_free, shared - 1)) { ok = false; break; }
        ml[t] = make_float2(m, l);
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(ml_full);
      } else {
        float w0 = 1.f, w1 = 0.f;                                       // weights of the two slots' O
        if (pc.halves) {
          if (!warp_wait(ml_full, shared)) { ok = false; break; }
          const float2 other = ml[t];
          const float M = fmaxf(m, other.x);
          w0 = ex2(m - M);
          w1 = ex2(other.x - M);
          l = fmaf(l, w0, other.y * w1);
          m = M;
        }
#pragma unroll
        for (int q = 0; q < DV / 32; ++q) {
          uint32_t r0[32];
          if (c > 0) {
            tc::tmem_ld32(lane_base + o_col + 32 * q, r0);
            tc::tmem_wait_ld();
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) x[32 * q + e] = c > 0 ? __uint_as_float(r0[e]) : 0.f;
        }
        if (pc.halves && pc.c[1] > 0) {
          tc::fence_after_sync();
#pragma unroll
          for (int q = 0; q < DV / 32; ++q) {
            uint32_t r0[32];
            tc::tmem_ld32(lane_base + o_col + 128 + 32 * q, r0);
            tc::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) x[32 * q + e] = fmaf(x[32 * q + e], w0, w1 * __uint_as_float(r0[e]));
          }
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          if (c > 0) mbar_arrive(&o_free[s]);
          if (pc.halves) {
            if (pc.c[1] > 0) mbar_arrive(&o_free[1]);
            mbar_arrive(ml_free);
          }
        }
        if (pc.whole) {
          // O / l in 16-column chunks, transposed through the staging tile so that a store instruction writes whole sectors of
          // 16 rows (piece k of row r at position k ^ ((r >> 2) & 1): no bank conflicts)
          const float inv = l == 0.f ? 0.f : 1.0f / l;
          const int my_row = row_ok ? (p.s.t0 + token) * a.Hq + p.g * G + t % G : -1;
          uint16_t* orow[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int rr = __shfl_sync(FULL_MASK, my_row, (lane >> 1) + 16 * i);
            orow[i] = rr < 0 ? nullptr : reinterpret_cast<uint16_t*>(a.out) + (int64_t)rr * DV + (lane & 1) * 8;
          }
#pragma unroll
          for (int q = 0; q < DV / 16; ++q) {
#pragma unroll
            for (int k2 = 0; k2 < 2; ++k2) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float y0 = x[16 * q + 8 * k2 + 2 * e], y1 = x[16 * q + 8 * k2 + 2 * e + 1];
                w[e] = l == 0.f ? 0u : pack_bf16x2(y0 * inv, y1 * inv);
              }
              *reinterpret_cast<uint4*>(stage + lane * 32 + ((k2 ^ ((lane >> 2) & 1)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int rr = (lane >> 1) + 16 * i, k2 = lane & 1;
              const uint4 v = *reinterpret_cast<const uint4*>(stage + rr * 32 + ((k2 ^ ((rr >> 2) & 1)) << 4));
              if (orow[i] != nullptr) *reinterpret_cast<uint4*>(orow[i] + 16 * q) = v;
            }
            __syncwarp();
          }
        } else {
          // a part, rows fastest: [2 slots][DV / 4][128 rows] float4, and (maximum, sum)
          const int part = blockIdx.x * 2 + (run.x0 >= p.at ? 0 : 1);
          float4* dst = reinterpret_cast<float4*>(a.part_acc) + ((int64_t)part * 2 + s) * (DV / 4) * BM + t;
#pragma unroll
          for (int q = 0; q < DV / 4; ++q) dst[q * BM] = make_float4(x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]);
          reinterpret_cast<float2*>(a.part_ml)[((int64_t)part * 2 + s) * BM + t] = make_float2(m, l);
          // the unit's first run tells the joining kernel where the parts are
          if (s == 0 && t == 0 && pc.st0 == 0) {
            PagedJoin j;
            j.first = part;
            j.last = run.of(p.at + p.n_steps - 1);
            j.t0 = p.s.t0; j.T = p.s.T; j.g = p.g; j.rt = 2 * p.rt; j.halves = pc.halves;
            a.joins[blockIdx.x] = j;
          }
        }
      }
      tiles += c;
      used += c > 0;
      shared += pc.halves;
      ++pieces;
      if (*s_abort) { ok = false; break; }      // (a piece that is through is written again: NaN)
    }
    if (!ok) *s_abort = 1;
    if (!ok || __any_sync(FULL_MASK, *s_odd != 0)) mend_rows<DV>(walk, run_begin, a, cut, run, s, t, !ok);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == MMA_WARP) tc::tmem_dealloc(tmem, TMEM_COLS);
}

// Joins the parts of a unit that several runs share: CTA (run that the unit begins in, slot and 16 of its columns), a
// thread a row.
constexpr int JOIN_COLS = 16;
template <int DV>
__global__ void __launch_bounds__(BM)
attn_paged_join_kernel(const __grid_constant__ PagedArgs a) {
  griddep_wait();                               // inputs of this launch are complete from here on
  griddep_launch_dependents();
  const PagedJoin j = a.joins[blockIdx.x];
  const int s = blockIdx.y / (DV / JOIN_COLS), c0 = blockIdx.y % (DV / JOIN_COLS) * JOIN_COLS, t = threadIdx.x;
  if (j.last < 0 || (j.halves && s == 1)) return;
  const int G = a.Hq / a.Hkv, tpt = BM / G, token = (j.rt + s) * tpt + t / G;
  if (t >= tpt * G || token >= j.T) return;
  const float2* ml = reinterpret_cast<const float2*>(a.part_ml) + (int64_t)s * BM + t;
  const float4* acc = reinterpret_cast<const float4*>(a.part_acc) + ((int64_t)s * (DV / 4) + c0 / 4) * BM + t;
  const int run0 = blockIdx.x, n = j.last - run0 + 1;
  auto part = [&](int i) { return i == 0 ? j.first : 2 * (run0 + i); };
  float M = M_NONE, L = 0.f;
  for (int i = 0; i < n; ++i) M = fmaxf(M, ml[(int64_t)part(i) * 2 * BM].x);
  float4 o[JOIN_COLS / 4];
#pragma unroll
  for (int q = 0; q < JOIN_COLS / 4; ++q) o[q] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const float2 x = ml[(int64_t)part(i) * 2 * BM];
    const float w = ex2(x.x - M);
    L = fmaf(x.y, w, L);
    if (x.y == 0.f) continue;                   // a part in which the row saw nothing
#pragma unroll
    for (int q = 0; q < JOIN_COLS / 4; ++q) {
      const float4 v = acc[((int64_t)part(i) * 2 * (DV / 4) + q) * BM];
      o[q].x = fmaf(v.x, w, o[q].x); o[q].y = fmaf(v.y, w, o[q].y);
      o[q].z = fmaf(v.z, w, o[q].z); o[q].w = fmaf(v.w, w, o[q].w);
    }
  }
  const float inv = L == 0.f ? 0.f : 1.0f / L;
  uint4* out = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.out) +
                                        ((int64_t)(j.t0 + token) * a.Hq + j.g * G + t % G) * DV + c0);
#pragma unroll
  for (int h = 0; h < JOIN_COLS / 8; ++h) {
    const float4 u = o[2 * h], v = o[2 * h + 1];
    out[h] = make_uint4(pack_bf16x2(u.x * inv, u.y * inv), pack_bf16x2(u.z * inv, u.w * inv), pack_bf16x2(v.x * inv, v.y * inv),
                        pack_bf16x2(v.z * inv, v.w * inv));
  }
}

template <int D, int DV>
cudaError_t launch_d(const PagedArgs& a, int runs, cudaStream_t s) {
  constexpr int SMEM = Layout<D, DV>::SMEM;
  static DeviceOnce configured;
  cudaError_t e;
  if (!configured.done()) {
    e = cudaFuncSetAttribute(attn_paged_chunk_kernel<D, DV>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (e != cudaSuccess) return e;
    // with fewer registers at launch the softmax warpgroups' setmaxnreg.inc could never be satisfied
    cudaFuncAttributes fa;
    if ((e = cudaFuncGetAttributes(&fa, attn_paged_chunk_kernel<D, DV>)) != cudaSuccess) return e;
    if (fa.numRegs != REGS_LAUNCH) return cudaErrorInvalidDeviceFunction;
    configured.mark();
  }
  const int rows = std::min(1 << a.page_shift, BN), G = a.Hq / a.Hkv;
  CUtensorMap mk, mv, mq;
  if ((e = paged_pool_map(&mk, a.k, a, D, a.page_stride, rows)) != cudaSuccess) return e;
  if ((e = paged_pool_map(&mv, a.v, a, DV, a.page_stride_v, rows)) != cudaSuccess) return e;
  if ((e = paged_query_map(&mq, a, D, G, BM / G)) != cudaSuccess) return e;
  return launch_pdl(attn_paged_chunk_kernel<D, DV>, dim3(runs), dim3(THREADS), (size_t)SMEM, s, a, mk, mv, mq);
}

}  // namespace

cudaError_t launch_attn_paged_chunk(const PagedArgs& a, int Dk, int Dv, int runs, cudaStream_t s, unsigned* n_launches) {
  cudaError_t e = Dk == 64 ? launch_d<64, 64>(a, runs, s) : (Dk == 128 ? launch_d<128, 128>(a, runs, s) : launch_d<192, 128>(a, runs, s));
  if (e != cudaSuccess) return e;
  ++*n_launches;
  if (runs == 1) return e;                      // no unit is shared
  const dim3 grid(runs, 2 * Dv / JOIN_COLS);
  e = Dv == 64 ? launch_pdl(attn_paged_join_kernel<64>, grid, dim3(BM), 0, s, a) : launch_pdl(attn_paged_join_kernel<128>, grid, dim3(BM), 0, s, a);
  if (e == cudaSuccess) ++*n_launches;
  return e;
}

// Steps of a sequence of T tokens and L slots in units of two row tiles, per KV head (as CutPairs counts them).
void attn_paged_chunk_load(int T, int L, int G, int64_t* steps, int64_t* units) {
  const int tpt = BM / G, tiles = (T + tpt - 1) / tpt;
  for (int z = 0; 2 * z < tiles; ++z) {
    const int last = std::min(2 * z + 1, tiles - 1);
    const int seen = std::min(std::max(L - T + std::min(T, (last + 1) * tpt), 0), L), n = (seen + BN - 1) / BN;
    *steps += std::max(1, 2 * z + 1 < tiles ? n : (n + 1) / 2);
    ++*units;
  }
}

}  // namespace kva
