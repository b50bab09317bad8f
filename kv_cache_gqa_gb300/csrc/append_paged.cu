// QK-Norm + RoPE + write of a ragged batch of new tokens into a paged cache (kv_cache_append_paged).
//
// A CTA takes one token (few tokens: a part of its rows) or eight, a warp each (long appends), whose angles its
// threads evaluate once.  A q or K row of D values belongs to SW lanes of a warp (SW = 8, 16 or 32 for rows up
// to 64, 128 or 256 wide), 8 values a lane: 4 of each half where the whole row turns as one block, else 8 in a row.  V, which is
// only copied, goes 256 values a warp whatever the row's width.  A warp walks its q, K and V sets in order with AHEAD of them on their way; the cosines,
// sines and norm weights of its dims stay in registers.  The token's sequence is found by a search of 32 probes
// at a time in token_start, its slot is L - T + i, and the table names the page; the rows' loads go out first.
//
// Bound: long appends by HBM in principle (24 chunks of 64 to 1024 tokens, 16/8 heads of 128, 149 MB: 45 us, 3.3 TB/s), in fact by
// the instructions and the latency of a row (load, sum over its lanes, turn) at 32 warps an SM (55% of issue slots, a third of DRAM's
// throughput), and by a last round of CTAs that is two thirds full.  There: 3 / 4 / 5 CTAs an SM 51 / 45 / 45 us, with the turn
// through shared memory 53 / 47 / 59 (and 2 / 3 / 4 / 6 sets ahead 47 / 49 / 50 / 57; a CTA a token 83).  The same rows in other forms: no
// turn 33.5 us, sections 45, 2D 47, the last 64 dims interleaved 43.5; float32 in and out (299 MB) 49, 57, 60 and 56 us.  64 tokens:
// latency (4.4 us).
//
// Method: the append of the decode step (Youtu-VL-4B ncnn port, step 6) with per-head RMSNorm and rotate-half
// RoPE (Penguin-VL ncnn port, sections 2.1 and 4.2; Youtu-VL-4B ncnn port, implementation difficulty 2).
// The reference has no cache in pages and no scaled positions.
#include <algorithm>

#include "append_rows.cuh"
#include "launch.h"

namespace kva {

namespace {

constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;
constexpr int TOKENS = WARPS;    // of a CTA in a long append
constexpr int MAX_D = 256;

// The sequence of token t: the last b with start[b] <= t, by 32 probes at a time (whole warp).
__device__ __forceinline__ int sequence_of(const int32_t* start, int B, int t, int lane) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, probe = lo + step * lane;
    const bool below = probe < hi && start[probe] <= t;
    lo += step * max(__popc(__ballot_sync(FULL_MASK, below)) - 1, 0);
    hi = min(lo + step, hi);
  }
  return lo;
}

// How a row's rotated pairs (d, d + half) lie in the lanes.  PAIRED: the whole row turns as one block, and a lane holds 4 dims
// of each half, so pairs meet in its registers.  ALIGNED: the rotated range and its halves (quarters for 2D) are multiples of
// 8 dims, the lane's 8 partners a piece of the row's copy in shared memory.  GENERAL: partners one by one.
enum Turn { GENERAL, ALIGNED, PAIRED };

// 4 elements at p and 4 at p + gap
__device__ __forceinline__ void load_halves(Raw8<float>& x, const float* p, int gap) {
  x.a = __ldg(reinterpret_cast<const float4*>(p));
  x.b = __ldg(reinterpret_cast<const float4*>(p + gap));
}
__device__ __forceinline__ void load_halves(Raw8<bf16_t>& x, const bf16_t* p, int gap) {
  const uint2 lo = __ldg(reinterpret_cast<const uint2*>(p)), hi = __ldg(reinterpret_cast<const uint2*>(p + gap));
  x.a = make_uint4(lo.x, lo.y, hi.x, hi.y);
}
__device__ __forceinline__ void store_halves(float* p, int gap, const float (&y)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(y[0], y[1], y[2], y[3]);
  *reinterpret_cast<float4*>(p + gap) = make_float4(y[4], y[5], y[6], y[7]);
}
__device__ __forceinline__ void store_halves(bf16_t* p, int gap, const float (&y)[8]) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
  *reinterpret_cast<uint2*>(p + gap) = make_uint2(pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
}

template <typename InT, typename OutT, int SW, Turn TURN, int TOK>
__global__ void __launch_bounds__(THREADS, 4)
append_paged_kernel(const __grid_constant__ AppendPagedArgs a) {
  constexpr int AHEAD = 2;                              // sets of a warp on their way
  constexpr int RPW = 32 / SW;                          // q or K rows a warp holds
  constexpr int WPT = WARPS / TOK;                      // warps per token
  constexpr int LD = SW * 8 + (RPW > 1 ? SW : 0);       // the rows of a warp start in different banks
  __shared__ __align__(16) float s_cos[TOK][MAX_ROPE_FREQ];
  __shared__ __align__(16) float s_sin[TOK][MAX_ROPE_FREQ];
  __shared__ __align__(16) float s_row[TURN == PAIRED ? 1 : WARPS][RPW][LD];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int sub = lane / SW, sl = lane % SW, e0 = TURN == PAIRED ? sl * 4 : sl * 8;   // the lane's first dim
  const int tl = warp / WPT, t0 = blockIdx.x * TOK, t = t0 + tl;
  const int Dk = a.Dk, Dv = a.Dv, Hkv = a.Hkv, Hq = a.Hq;
  const int ro = a.rot_offset, rw = a.rot_dim, half = rw / 2, kind_r = a.rope.kind;
  const bool rotate = kind_r != KVA_ROPE_NONE, norm = a.q_w != nullptr;
  griddep_wait();                               // inputs of this launch are complete from here on

  // Sets of the token's rows: kind 0 q, 1 K (RPW heads, lanes by dims), 2 V (256 values, 8 a lane).
  // This lane's unit (head, or 8 values of V) in set i of a kind is unit0 + i * per, of `units`.
  const int step = WPT * gridDim.z, start = blockIdx.z * WPT + warp % WPT;
  const int pieces = Hkv * (Dv / 8);
  const int sets_q = (Hq + RPW - 1) / RPW, sets_k = (Hkv + RPW - 1) / RPW, sets_v = (pieces + 31) / 32;
  auto units = [&](int kind) { return kind == 0 ? Hq : (kind == 1 ? Hkv : pieces); };
  auto sets = [&](int kind) { return kind == 0 ? sets_q : (kind == 1 ? sets_k : sets_v); };
  const bool in_row = sl * 8 < Dk;
  // the walk that loads: kind, set, and this lane's unit and address in it
  struct Walk { int kind, set, unit; const InT* p; };
  auto enter = [&](Walk& w, int set) {          // the first set >= start of the walk's kind, or of a later one
    w.set = set;
    while (w.kind < 3 && w.set >= sets(w.kind)) { w.set -= sets(w.kind); ++w.kind; }
    if (w.kind == 2) {
      w.unit = w.set * 32 + lane;
      w.p = reinterpret_cast<const InT*>(a.v) + t * a.v_stride + (int64_t)w.unit * 8;
    } else {
      w.unit = w.set * RPW + sub;
      w.p = reinterpret_cast<const InT*>(w.kind ? a.k : a.q) + t * (w.kind ? a.k_stride : a.q_stride) +
            (int64_t)w.unit * Dk + e0;
    }
  };
  auto fetch = [&](Walk& w, Raw8<InT>& x) {      // the walk's set, then on to the next
    x.zero();
    if (w.kind > 2) return;
    if (w.unit < units(w.kind) && (w.kind == 2 || in_row)) {
      if (TURN == PAIRED && w.kind < 2) load_halves(x, w.p, Dk / 2);
      else x.load(w.p);
    }
    w.set += step;
    if (w.set < sets(w.kind)) {
      const int by = step * (w.kind == 2 ? 32 : RPW);
      w.unit += by;
      w.p += (int64_t)by * (w.kind == 2 ? 8 : Dk);
    } else {
      enter(w, w.set);
    }
  };
  Walk walk{0, 0, 0, nullptr};
  Raw8<InT> ahead[AHEAD];
  if (t < a.T) {
    enter(walk, start);
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) fetch(walk, ahead[i]);
  }
  if (rotate)                                           // the angles, behind the first loads
    for (int j = tid; j < half * min(TOK, a.T - t0); j += THREADS) {
      const int tt = TOK == 1 ? 0 : j / half, f = j - tt * half;
      const int32_t p = a.pos[(int64_t)(t0 + tt) * a.rope.n_axes + a.rope.axis[f]];
      float c, s;
      rotation(p, a.rope.inv_hi[f], a.rope.inv_lo[f], a.rope.inv[f], &c, &s);
      s_cos[tt][f] = c * a.magnitude;
      s_sin[tt][f] = s * a.magnitude;
    }
  // the token's place: its row of a head in K and V of the page, or none
  int64_t at_k = -1, at_v = 0;
  if (t < a.T) {
    const int b = sequence_of(a.start, a.B, t, lane), first = a.start[b], n = a.start[b + 1] - first;
    const int64_t slot = (int64_t)a.lengths[b] - n + (t - first);
    if (t >= first && t - first < n && slot >= 0 && slot < a.slots) {
      const int page = a.table[(int64_t)b * a.table_stride + (slot >> a.page_shift)];
      const int64_t in = slot & ((1 << a.page_shift) - 1);
      if (page >= 0 && page < a.n_pages) {
        at_k = page * a.page_stride + in * Dk;
        at_v = page * a.page_stride_v + in * Dv;
      }
    }
  }
  __syncthreads();
  if (t >= a.T) return;

  // this lane's angles and its partner piece (ALIGNED): outputs d0.. of the rotated range
  const int d0 = e0 - ro;
  const bool turns = rotate && d0 >= 0 && d0 < rw;
  const int block = kind_r == KVA_ROPE_2D ? half : rw, hb = block / 2;   // blocks turn apart; halves pair up
  bool low = true;
  int partner = 0;
  uint64_t cs[4] = {}, sn[4] = {};
  if (TURN == PAIRED && rotate && in_row) {
    const ulonglong2 c = *reinterpret_cast<const ulonglong2*>(&s_cos[tl][e0]), v = *reinterpret_cast<const ulonglong2*>(&s_sin[tl][e0]);
    cs[0] = c.x; cs[1] = c.y;
    sn[0] = v.x; sn[1] = v.y;
    sn[2] = v.x ^ 0x8000000080000000ull; sn[3] = v.y ^ 0x8000000080000000ull;
  }
  if (TURN == ALIGNED && turns) {
    const int bi = d0 >= block ? 1 : 0, d = d0 - bi * block;
    low = d < hb;
    const int j0 = bi * hb + (low ? d : d - hb);
    partner = kind_r == KVA_ROPE_INTERLEAVED ? ro + 2 * j0 : ro + (low ? d0 + hb : d0 - hb);
    shared_pairs(&s_cos[tl][j0], cs);
    shared_pairs(&s_sin[tl][j0], sn);
    if (low) {                                          // y = x cos - p sin there
#pragma unroll
      for (int i = 0; i < 4; ++i) sn[i] ^= 0x8000000080000000ull;
    }
  }
  float* row = s_row[TURN == PAIRED ? 0 : warp][sub];
  const float inv_d = 1.0f / (float)Dk;
  uint64_t x[4] = {}, wv[4] = {};
  auto mirror = [&]() {
    reinterpret_cast<ulonglong2*>(row + e0)[0] = make_ulonglong2(x[0], x[1]);
    reinterpret_cast<ulonglong2*>(row + e0)[1] = make_ulonglong2(x[2], x[3]);
    __syncwarp();
  };
  auto apply_norm = [&]() {                             // squares in the lanes, then over the row's lanes
    uint64_t q = 0ull;
#pragma unroll
    for (int i = 0; i < 4; ++i) q = fma_f32x2(x[i], x[i], q);
    float ss = f32x2_lo(q) + f32x2_hi(q);
#pragma unroll
    for (int o = 1; o < SW; o <<= 1) ss += __shfl_xor_sync(FULL_MASK, ss, o);
    const float r = rsqrtf(fmaf(ss, inv_d, a.eps));
    const uint64_t r2 = pack_f32x2(r, r);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = mul_f32x2(mul_f32x2(x[i], r2), wv[i]);
  };
  auto turn = [&]() {
    if constexpr (TURN == PAIRED) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint64_t lo = x[i], hi = x[2 + i];
        x[i] = sum_of_products(lo, cs[i], hi, sn[2 + i]);
        x[2 + i] = sum_of_products(hi, cs[i], lo, sn[i]);
      }
      return;
    }
    mirror();
    if constexpr (TURN == ALIGNED) {
      if (turns) {
        if (kind_r == KVA_ROPE_INTERLEAVED) {           // inputs 2 j0 .. 2 j0 + 15 are 8 pairs
          uint64_t q[8];
          ulonglong2 two;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            two = reinterpret_cast<const ulonglong2*>(row + partner)[i];
            q[2 * i] = two.x; q[2 * i + 1] = two.y;
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint64_t ev = pack_f32x2(f32x2_lo(q[2 * i]), f32x2_lo(q[2 * i + 1]));
            const uint64_t od = pack_f32x2(f32x2_hi(q[2 * i]), f32x2_hi(q[2 * i + 1]));
            x[i] = sum_of_products(low ? ev : od, cs[i], low ? od : ev, sn[i]);
          }
        } else {
          uint64_t p[4];
          shared_pairs(row + partner, p);
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] = sum_of_products(x[i], cs[i], p[i], sn[i]);
        }
      }
    } else {
      float y[8];
      unpack_pairs(x, y);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int dd = d0 + i;
        if (dd < 0 || dd >= rw) continue;
        const int bi = dd / block, d = dd - bi * block;
        const bool lo = d < hb;
        const int j = bi * hb + (lo ? d : d - hb);
        const float c = s_cos[tl][j], v = lo ? -s_sin[tl][j] : s_sin[tl][j];
        const bool inter = kind_r == KVA_ROPE_INTERLEAVED;
        const float own = inter ? row[ro + 2 * j + (lo ? 0 : 1)] : y[i];
        const float other = inter ? row[ro + 2 * j + (lo ? 1 : 0)] : row[ro + (lo ? dd + hb : dd - hb)];
        y[i] = __fadd_rn(__fmul_rn(own, c), __fmul_rn(other, v));
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = pack_f32x2(y[2 * i], y[2 * i + 1]);
    }
    __syncwarp();                                       // buffer reads done before it is written again
  };

  int set = start;                                      // runs on from kind to kind, as the walk does
#pragma unroll
  for (int kind = 0; kind < 3; ++kind) {
    const bool qk = kind < 2;
    const int per = qk ? RPW : 32;
    if (norm && qk && in_row && set < sets(kind)) {
      Raw8<float> w;
      const float* from = (kind ? a.k_w : a.q_w) + e0;
      if constexpr (TURN == PAIRED) load_halves(w, from, Dk / 2);
      else w.load(from);
      w.pairs(wv);
    }
    int unit = set * per + (qk ? sub : lane);
    for (; set < sets(kind); set += step, unit += step * per) {
      ahead[0].pairs(x);
#pragma unroll
      for (int i = 0; i + 1 < AHEAD; ++i) ahead[i] = ahead[i + 1];
      fetch(walk, ahead[AHEAD - 1]);
      const bool on = unit < units(kind) && (!qk || in_row);
      if (qk) {
        if (norm && !a.after_rope) apply_norm();
        if (rotate) turn();
        if (norm && a.after_rope) apply_norm();
      }
      if (!on) continue;
      float y[8];
      unpack_pairs(x, y);
      if (kind == 0) {
        OutT* to = reinterpret_cast<OutT*>(a.q_out) + ((int64_t)t * Hq + unit) * Dk + e0;
        if constexpr (TURN == PAIRED) store_halves(to, Dk / 2, y);
        else store8(to, y);
      } else if (at_k >= 0) {
        if (kind == 1) {
          OutT* to = reinterpret_cast<OutT*>(a.kc) + at_k + ((int64_t)unit << a.page_shift) * Dk + e0;
          if constexpr (TURN == PAIRED) store_halves(to, Dk / 2, y);
          else store8(to, y);
        } else {
          const int head = unit / (Dv / 8), d = (unit - head * (Dv / 8)) * 8;
          store8(reinterpret_cast<OutT*>(a.vc) + at_v + ((int64_t)head << a.page_shift) * Dv + d, y);
        }
      }
    }
    set -= sets(kind);
  }
  griddep_launch_dependents();
}

constexpr int SMS = 152;          // grids are sized for the whole GPU; fewer SMs only take longer

template <typename InT, typename OutT, Turn TURN, int TOK>
cudaError_t launch_t(const AppendPagedArgs& a, cudaStream_t s) {
  const int D = a.Dk, rpw = D <= 64 ? 4 : (D <= 128 ? 2 : 1);
  const int64_t sets = (a.Hq + rpw - 1) / rpw + (int64_t)((a.Hkv + rpw - 1) / rpw) + ((int64_t)a.Hkv * a.Dv + 255) / 256;
  // few tokens spread their rows over CTAs, about two per SM
  const int64_t ctas = (a.T + TOK - 1) / TOK, most = (sets + WARPS / TOK - 1) / (WARPS / TOK);
  const int groups = (int)std::max<int64_t>(1, std::min<int64_t>(most, 2 * SMS / ctas));
  const dim3 grid((unsigned)ctas, 1, groups);
  if (D <= 64) return launch_pdl(append_paged_kernel<InT, OutT, 8, TURN, TOK>, grid, dim3(THREADS), 0, s, a);
  if (D <= 128) return launch_pdl(append_paged_kernel<InT, OutT, 16, TURN, TOK>, grid, dim3(THREADS), 0, s, a);
  return launch_pdl(append_paged_kernel<InT, OutT, 32, TURN, TOK>, grid, dim3(THREADS), 0, s, a);
}

// A token per warp once that leaves four CTAs per SM.
template <typename InT, typename OutT, Turn TURN>
cudaError_t launch_w(const AppendPagedArgs& a, cudaStream_t s) {
  return a.T >= 4 * TOKENS * SMS ? launch_t<InT, OutT, TURN, TOKENS>(a, s) : launch_t<InT, OutT, TURN, 1>(a, s);
}

template <typename InT, typename OutT>
cudaError_t launch_a(const AppendPagedArgs& a, cudaStream_t s) {
  const bool one_block = a.rope.kind != KVA_ROPE_2D && a.rope.kind != KVA_ROPE_INTERLEAVED;
  if (one_block && a.rot_offset == 0 && a.rot_dim == a.Dk) return launch_w<InT, OutT, PAIRED>(a, s);
  const int unit = a.rope.kind == KVA_ROPE_2D ? 32 : 16;
  return a.rot_offset % 8 == 0 && a.rot_dim % unit == 0 ? launch_w<InT, OutT, ALIGNED>(a, s) : launch_w<InT, OutT, GENERAL>(a, s);
}

}  // namespace

cudaError_t launch_append_paged(const AppendPagedArgs& a, kva_dtype in_dtype, kva_dtype cache_dtype, cudaStream_t s) {
  if (a.Dk > MAX_D || a.Dv > MAX_D || a.rot_dim / 2 > MAX_ROPE_FREQ) return cudaErrorInvalidValue;
  if (in_dtype == KVA_BF16)
    return cache_dtype == KVA_BF16 ? launch_a<bf16_t, bf16_t>(a, s) : launch_a<bf16_t, float>(a, s);
  return cache_dtype == KVA_BF16 ? launch_a<float, bf16_t>(a, s) : launch_a<float, float>(a, s);
}

}  // namespace kva
