// The 4-bit cache's write and read-back: QK-Norm + RoPE + quantisation fused into the cache write
// (kv_cache_append_q4), and the expansion of listed slots into a bf16 or float32 cache
// (kv_cache_expand_q4).  Layout and quantiser: kva_cache_q4 in kv_attn.h.
//
// Append: a CTA takes one token (few tokens: a part of its rows) or eight, a warp each (long appends), whose
// angles its threads evaluate once.  A q or K row of D values belongs to SW lanes of a warp (SW = 8, 16
// or 32 for rows up to 64, 128 or 256 wide), 8 consecutive values a lane, so the 64 values of a
// quantisation group sit in 8 consecutive lanes: the group's minimum and maximum are three shuffles
// each, a lane's 8 codes are one 32-bit word of the cache, and a group's first lane writes its scale and
// midpoint.  V is only quantised, so a warp takes 4 of its groups whatever the row's width.  A warp walks
// its q, K and V sets in order with two of them on their way; the cosines, sines and norm weights of its
// dims stay in registers.  A lane's 8 values rotate as one piece where the rotated range and its
// halves are multiples of 8 dims.
//
// A code is decided by a rounding: a value that is off by an ulp of float32 becomes the neighbouring code
// once in about 10^6, which is as near to it (scale / 2 either way).  The quotients are correctly rounded,
// because bf16 values often lie on a tie exactly.  The steps before them are float32 with their usual errors: squares in 32
// strided sums and then pairwise, a row's factor from rsqrtf (2 ulp; for rows of 192 the inverse of D is rounded too),
// products and sums of the rotation rounded apart, cosines and sines as rotation() below says.  The order of
// the sums is this kernel's choice; the definition fixes none.
//
// Bound: issue slots.  512 tokens in 28 caches (16 + 8 + 8 heads of 128, bf16): 160 MB in 93 us, 63% of the
// slots used with three CTAs an SM (two: 131 us with the read-back instead of 113; four, at 64 registers: 113, and
// 114 instead of 94 where rows are 192 wide).  Its read-back, 75 MB in 20 us, uses 74%.
//
// Method: the append of the decode step (Youtu-VL-4B ncnn port, step 6) with per-head RMSNorm and
// rotate-half RoPE (Penguin-VL ncnn port, sections 2.1 and 4.2; Youtu-VL-4B ncnn port,
// implementation difficulty 2).  The pages hold their caches in 16 or 32 bits; the 4-bit form has
// no counterpart there.
#include <algorithm>

#include "append_rows.cuh"
#include "launch.h"

namespace kva {

namespace {

constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;
constexpr int TOKENS = WARPS;    // of a CTA in a long append
constexpr int MAX_D = 256;

// Sum of squares of a row of D values in shared memory, by its SW lanes: strided sums l, l + 32, ... (the
// lanes read without bank conflicts), then pairs of neighbouring sums.
template <int SW>
__device__ __forceinline__ float sum_squares(const float* row, int D, int sl) {
  constexpr int NL = 32 / SW;                             // strided sums a lane keeps
  float v[NL];
#pragma unroll
  for (int j = 0; j < NL; ++j) {
    float f[4] = {0.f, 0.f, 0.f, 0.f};
    for (int i = 0; i < D; i += 128)
#pragma unroll
      for (int m = 0; m < 4; ++m)
        if (i + 32 * m < D) {
          const float x = row[i + 32 * m + sl + SW * j], q = __fmul_rn(x, x);
          f[m] = i == 0 ? q : __fadd_rn(f[m], q);
        }
    v[j] = __fadd_rn(__fadd_rn(__fadd_rn(f[0], f[1]), f[2]), f[3]);
#pragma unroll
    for (int o = 1; o < SW; o <<= 1) v[j] = __fadd_rn(v[j], __shfl_xor_sync(FULL_MASK, v[j], o));
  }
  if constexpr (NL == 1) return v[0];
  else if constexpr (NL == 2) return __fadd_rn(v[0], v[1]);
  else return __fadd_rn(__fadd_rn(v[0], v[1]), __fadd_rn(v[2], v[3]));
}

// a / b for a correctly rounded inverse r of b: one correction of the product makes it the correctly
// rounded quotient (Markstein, "Computation of elementary functions on the IBM RISC System/6000").
__device__ __forceinline__ float quotient(float a, float b, float r) {
  const float q = a * r;
  return fmaf(fmaf(-q, b, a), r, q);
}

// Quantise the 8 values of this lane (four pairs), whose group of 64 is the lane's aligned set of 8
// lanes.  Returns the code word; *par = (scale, mid) packed for the group's first lane.
__device__ __forceinline__ uint32_t quantise8(const uint64_t (&x)[4], uint32_t* par) {
  float lo = f32x2_lo(x[0]), hi = lo;
  uint64_t probe = 0ull;                                // sums of 0 x: NaN if an element is NaN (which fminf drops) or infinite
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    lo = fminf(fminf(lo, f32x2_lo(x[i])), f32x2_hi(x[i]));
    hi = fmaxf(fmaxf(hi, f32x2_lo(x[i])), f32x2_hi(x[i]));
    probe = fma_f32x2(x[i], 0ull, probe);
  }
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) {
    lo = fminf(lo, __shfl_xor_sync(FULL_MASK, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(FULL_MASK, hi, o));
  }
  const float all = f32x2_lo(probe) + f32x2_hi(probe);
  const unsigned any = __ballot_sync(FULL_MASK, all != all);
  const bool odd = ((any >> (threadIdx.x & 24)) & 0xffu) != 0;
  // the scale is rounded up, so 15 steps cover the spread; one below bf16's normal range is 0
  float scale = __bfloat162float(__float2bfloat16_ru(quotient(hi - lo, 15.0f, 1.0f / 15.0f)));
  if (scale < 1.17549435e-38f) scale = 0.f;
  float mid = __bfloat162float(__float2bfloat16_rn(fmaf(8.0f, scale, lo)));
  if (odd || !(scale <= 3.402823466e38f) || !(fabsf(mid) <= 3.402823466e38f)) scale = mid = __uint_as_float(0x7fc00000u);
  const float inv = scale > 0.f ? __frcp_rn(scale) : 0.f;
  const uint64_t m2 = pack_f32x2(-mid, -mid), s2 = pack_f32x2(-scale, -scale), i2 = pack_f32x2(inv, inv);
  const uint64_t magic = pack_f32x2(12582920.f, 12582920.f);
  uint32_t w = 0;
#pragma unroll
  for (int i = 3; i >= 0; --i) {
    // quotients (as quotient()), not products with the inverse: bf16 inputs meet exact half steps, which
    // round to even.  Adding 1.5 * 2^23 + 8 leaves 0x4b400000 + code; the constants go at the end.
    const uint64_t d = add_f32x2(x[i], m2), q = mul_f32x2(d, i2), f = fma_f32x2(fma_f32x2(q, s2, d), i2, q);
    const uint64_t c = add_f32x2(pack_f32x2(fminf(fmaxf(f32x2_lo(f), -8.f), 7.f), fminf(fmaxf(f32x2_hi(f), -8.f), 7.f)), magic);
    w = w * 16u + (uint32_t)(c >> 32);
    w = w * 16u + (uint32_t)c;
  }
  w -= 0x4b400000u * 0x11111111u;
  *par = (__float_as_uint(scale) >> 16) | (__float_as_uint(mid) & 0xffff0000u);   // both are bf16 values
  return w;
}

// ALIGNED: the rotated range and its halves (quarters for 2D) are multiples of 8 dims.
template <typename InT, typename QOutT, int SW, bool ALIGNED, int TOK>
__global__ void __launch_bounds__(THREADS, 3)
append_q4_kernel(const __grid_constant__ AppendQ4Args a) {
  constexpr int RPW = 32 / SW;                          // q or K rows a warp holds
  constexpr int WPT = WARPS / TOK;                      // warps per token
  constexpr int LD = SW * 8 + (RPW > 1 ? SW : 0);       // the rows of a warp start in different banks
  __shared__ __align__(16) float s_cos[TOK][MAX_ROPE_FREQ];
  __shared__ __align__(16) float s_sin[TOK][MAX_ROPE_FREQ];
  __shared__ __align__(16) float s_row[WARPS][RPW][LD];

  const int n = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int sub = lane / SW, sl = lane % SW, e0 = sl * 8;
  const int tl = warp / WPT, t0 = blockIdx.x * TOK, t = t0 + tl;
  const int Dk = a.c.Dk, Dv = a.c.Dv, Hkv = a.c.Hkv, Hq = a.q ? a.Hq : 0, Gk = Dk / Q4_GROUP, Gv = Dv / Q4_GROUP;
  const int ro = a.rot_offset, rw = a.rot_dim, half = rw / 2, kind_r = a.rope.kind;
  const bool rotate = kind_r != KVA_ROPE_NONE, norm = a.q_w != nullptr;
  const int64_t tok = (int64_t)n * a.T + t;
  griddep_wait();                               // inputs of this launch are complete from here on

  // Sets of the token's rows: kind 0 q, 1 K (RPW heads, lanes by dims), 2 V (4 quantisation groups, lanes
  // by groups).  This lane's unit in set i of a kind is unit0 + i * per, of `units`.
  const int step = WPT * gridDim.z, start = blockIdx.z * WPT + warp % WPT;
  const int sets_q = (Hq + RPW - 1) / RPW, sets_k = (Hkv + RPW - 1) / RPW, sets_v = (Hkv * Gv + 3) / 4;
  auto units = [&](int kind) { return kind == 0 ? Hq : (kind == 1 ? Hkv : Hkv * Gv); };
  auto sets = [&](int kind) { return kind == 0 ? sets_q : (kind == 1 ? sets_k : sets_v); };
  const bool in_row = e0 < Dk;
  // the walk that loads: kind, set, and this lane's unit and address in it
  struct Walk { int kind, set, unit; const InT* p; };
  auto enter = [&](Walk& w, int set) {          // the first set >= start of the walk's kind, or of a later one
    w.set = set;
    while (w.kind < 3 && w.set >= sets(w.kind)) { w.set -= sets(w.kind); ++w.kind; }
    if (w.kind == 2) {
      w.unit = w.set * 4 + (lane >> 3);
      w.p = reinterpret_cast<const InT*>(a.v) + tok * Hkv * Dv + (int64_t)w.unit * Q4_GROUP + 8 * (lane & 7);
    } else {
      w.unit = w.set * RPW + sub;
      w.p = reinterpret_cast<const InT*>(w.kind ? a.k : a.q) + (tok * (w.kind ? Hkv : Hq) + w.unit) * Dk + e0;
    }
  };
  auto fetch = [&](Walk& w, Raw8<InT>& x) {      // the walk's set, then on to the next
    x.zero();
    if (w.kind > 2) return;
    if (w.kind == 2) {
      if (w.unit < units(2)) x.load(w.p);
    } else if (in_row && w.unit < units(w.kind)) {
      x.load(w.p);
    }
    w.set += step;
    if (w.set < sets(w.kind)) {
      const int by = step * (w.kind == 2 ? 4 : RPW);
      w.unit += by;
      w.p += by * (w.kind == 2 ? Q4_GROUP : Dk);
    } else {
      enter(w, w.set);
    }
  };
  Walk walk{0, 0, 0, nullptr};
  Raw8<InT> ahead[2];
  if (t < a.T) {
    enter(walk, start);
    fetch(walk, ahead[0]);
    fetch(walk, ahead[1]);
  }
  if (rotate)                                           // the angles, behind the first loads
    for (int j = tid; j < half * min(TOK, a.T - t0); j += THREADS) {
      const int tt = TOK == 1 ? 0 : j / half, f = j - tt * half;
      const int32_t p = a.pos[(int64_t)n * a.pos_stride + (int64_t)(t0 + tt) * a.rope.n_axes + a.rope.axis[f]];
      rotation(p, a.rope.inv_hi[f], a.rope.inv_lo[f], a.rope.inv[f], &s_cos[tt][f], &s_sin[tt][f]);
    }
  __syncthreads();
  if (t >= a.T) return;

  const int slot = a.slot[(int64_t)n * a.slot_stride + t];
  const bool in_cache = slot >= 0 && slot < a.c.capacity;
  // this lane's angles and its partner piece (ALIGNED): outputs d0.. of the rotated range
  const int d0 = e0 - ro;
  const bool turns = rotate && d0 >= 0 && d0 < rw;
  const int block = kind_r == KVA_ROPE_2D ? half : rw, hb = block / 2;   // blocks turn apart; halves pair up
  bool low = true;
  int partner = 0;
  uint64_t cs[4] = {}, sn[4] = {};
  if (ALIGNED && turns) {
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
  float* row = s_row[warp][sub];
  const float inv_d = 1.0f / (float)Dk;
  uint64_t x[4] = {}, wv[4] = {};
  auto mirror = [&]() {
    reinterpret_cast<ulonglong2*>(row + e0)[0] = make_ulonglong2(x[0], x[1]);
    reinterpret_cast<ulonglong2*>(row + e0)[1] = make_ulonglong2(x[2], x[3]);
    __syncwarp();
  };
  auto apply_norm = [&]() {                             // the row is in shared memory
    const float r = rsqrtf(__fadd_rn(__fmul_rn(sum_squares<SW>(row, Dk, sl), inv_d), a.eps));
    const uint64_t r2 = pack_f32x2(r, r);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = mul_f32x2(mul_f32x2(x[i], r2), wv[i]);
    __syncwarp();                                       // buffer reads done before it is written again
  };
  auto turn = [&]() {
    mirror();
    if constexpr (ALIGNED) {
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
    __syncwarp();
  };

  int set = start;                                      // runs on from kind to kind, as the walk does
#pragma unroll
  for (int kind = 0; kind < 3; ++kind) {
    const bool qk = kind < 2;
    const int G = kind == 1 ? Gk : Gv, per = qk ? RPW : 4;
    if (norm && qk && in_row && set < sets(kind)) {
      Raw8<float> w;
      w.load((kind ? a.k_w : a.q_w) + (int64_t)n * a.w_stride + e0);
      w.pairs(wv);
    }
    int unit = set * per + (qk ? sub : lane >> 3);
    for (; set < sets(kind); set += step, unit += step * per) {
      ahead[0].pairs(x);
      ahead[0] = ahead[1];
      fetch(walk, ahead[1]);
      const bool on = unit < units(kind) && (!qk || in_row);
      if (qk) {
        if (norm && !a.after_rope) { mirror(); apply_norm(); }
        if (rotate) turn();
        if (norm && a.after_rope) { mirror(); apply_norm(); }
      }
      if (kind == 0) {
        if (on) {
          float y[8];
          unpack_pairs(x, y);
          store8(reinterpret_cast<QOutT*>(a.q_out) + (tok * Hq + unit) * Dk + e0, y);
        }
      } else {
        uint32_t par;
        const uint32_t word = quantise8(x, &par);       // every lane: shuffles
        const int head = qk ? unit : (G == 1 ? unit : (G == 2 ? unit >> 1 : (G == 4 ? unit >> 2 : unit / 3)));
        const int group = qk ? sl >> 3 : unit - head * G;
        if (on && in_cache) {
          const int64_t at = ((int64_t)n * a.c.inst_rows + (int64_t)head * a.c.capacity + slot) * G + group;
          (qk ? a.c.k : a.c.v)[8 * (at - group) + (lane & 7) * G + group] = word;
          if ((lane & 7) == 0) (qk ? a.c.ks : a.c.vs)[at] = par;
        }
      }
    }
    set -= sets(kind);
  }
  // a long append must not have its SMs taken by a waiting persistent kernel
  griddep_launch_dependents();
}

// Read-back: a CTA takes EX_SLOTS slots of one KV head, a thread one word of 8 codes at a time;
// consecutive threads take consecutive words.  Words of a row (8 to 32) and groups (1 to 4) divide the
// small indices by a multiplication.
constexpr int EX_SLOTS = 64;
template <typename OutT>
__global__ void __launch_bounds__(THREADS)
expand_q4_kernel(const __grid_constant__ ExpandQ4Args a) {
  const int n = blockIdx.z, g = blockIdx.y, t0 = blockIdx.x * EX_SLOTS, nt = min(EX_SLOTS, a.T - t0);
  __shared__ int s_slot[EX_SLOTS];
  griddep_wait();
  if ((int)threadIdx.x < nt) s_slot[threadIdx.x] = a.slot[(int64_t)n * a.slot_stride + t0 + threadIdx.x];
  __syncthreads();
  const int64_t row0 = (int64_t)n * a.c.inst_rows + (int64_t)g * a.c.capacity;
#pragma unroll
  for (int half = 0; half < 2; ++half) {                // K, then V
    const int D = half ? a.c.Dv : a.c.Dk, words = D / 8, G = D / Q4_GROUP;
    const uint32_t* codes = half ? a.c.v : a.c.k;
    const uint32_t* pars = half ? a.c.vs : a.c.ks;
    OutT* dst = reinterpret_cast<OutT*>(half ? a.dv : a.dk) + (int64_t)n * (half ? a.d_stride_v : a.d_stride) +
                ((int64_t)g * a.d_capacity + a.d_first + t0) * D;
    const uint32_t inv_words = 65536u / words + 1, inv_g = 65536u / G + 1;   // exact below 2^11 words, 32 groups
    constexpr int U = 4;                                // words in flight per thread
    for (int i0 = threadIdx.x; i0 < nt * words; i0 += U * THREADS) {
      uint32_t code[U], par[U];
      int t[U], first[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t i = i0 + u * THREADS;
        t[u] = (int)((i * inv_words) >> 16);
        const uint32_t w = i - t[u] * words, blk = (w * inv_g) >> 16, grp = w - blk * G;
        first[u] = Q4_GROUP * grp + 8 * blk;
        const int slot = (int)i < nt * words ? s_slot[t[u]] : -1;
        if (slot < 0 || slot >= a.c.capacity) { t[u] = -1; continue; }
        code[u] = __ldg(codes + (row0 + slot) * words + w);
        par[u] = __ldg(pars + (row0 + slot) * G + grp);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (t[u] < 0) continue;
        const float scale = bf16_lo(par[u]), mid = bf16_hi(par[u]);
        float y[8];
        // a code in the low byte of 0x4b000000 is 2^23 + code; 2^23 + 8 is taken off
        const uint32_t even = code[u] & 0x0f0f0f0fu, odd = (code[u] >> 4) & 0x0f0f0f0fu;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t b = __byte_perm(e & 1 ? odd : even, 0x4b000000u, 0x7440 + e / 2);
          y[e] = fmaf(scale, __uint_as_float(b) - 8388616.f, mid);
        }
        store8(dst + (int64_t)t[u] * D + first[u], y);
      }
    }
  }
  griddep_launch_dependents();
}

constexpr int SMS = 152;          // grids are sized for the whole GPU; fewer SMs only take longer

template <typename InT, typename QOutT, bool ALIGNED, int TOK>
cudaError_t launch_t(const AppendQ4Args& a, cudaStream_t s) {
  const int D = a.c.Dk, rpw = D <= 64 ? 4 : (D <= 128 ? 2 : 1);
  const int64_t sets = ((a.q ? a.Hq : 0) + rpw - 1) / rpw + (int64_t)((a.c.Hkv + rpw - 1) / rpw) +
                       ((int64_t)a.c.Hkv * (a.c.Dv / Q4_GROUP) + 3) / 4;
  // few tokens spread their rows over CTAs, about two per SM
  const int64_t ctas = (int64_t)((a.T + TOK - 1) / TOK) * a.N, most = (sets + WARPS / TOK - 1) / (WARPS / TOK);
  const int groups = (int)std::max<int64_t>(1, std::min<int64_t>(most, 2 * SMS / ctas));
  const dim3 grid((a.T + TOK - 1) / TOK, a.N, groups);
  if (D <= 64) return launch_pdl(append_q4_kernel<InT, QOutT, 8, ALIGNED, TOK>, grid, dim3(THREADS), 0, s, a);
  if (D <= 128) return launch_pdl(append_q4_kernel<InT, QOutT, 16, ALIGNED, TOK>, grid, dim3(THREADS), 0, s, a);
  return launch_pdl(append_q4_kernel<InT, QOutT, 32, ALIGNED, TOK>, grid, dim3(THREADS), 0, s, a);
}

// A token per warp once that leaves four CTAs per SM.
template <typename InT, typename QOutT, bool ALIGNED>
cudaError_t launch_w(const AppendQ4Args& a, cudaStream_t s) {
  return (int64_t)a.T * a.N >= (int64_t)4 * TOKENS * SMS ? launch_t<InT, QOutT, ALIGNED, TOKENS>(a, s)
                                                                  : launch_t<InT, QOutT, ALIGNED, 1>(a, s);
}

template <typename InT, typename QOutT>
cudaError_t launch_a(const AppendQ4Args& a, cudaStream_t s) {
  const int unit = a.rope.kind == KVA_ROPE_2D ? 32 : 16;
  return a.rot_offset % 8 == 0 && a.rot_dim % unit == 0 ? launch_w<InT, QOutT, true>(a, s) : launch_w<InT, QOutT, false>(a, s);
}

}  // namespace

cudaError_t launch_append_q4(const AppendQ4Args& a, kva_dtype in_dtype, kva_dtype q_out_dtype, cudaStream_t s) {
  if (a.c.Dk > MAX_D || a.c.Dv > MAX_D || a.rot_dim / 2 > MAX_ROPE_FREQ || a.N > 65535) return cudaErrorInvalidValue;
  if (in_dtype == KVA_BF16)
    return q_out_dtype == KVA_BF16 ? launch_a<bf16_t, bf16_t>(a, s) : launch_a<bf16_t, float>(a, s);
  return q_out_dtype == KVA_BF16 ? launch_a<float, bf16_t>(a, s) : launch_a<float, float>(a, s);
}

cudaError_t launch_expand_q4(const ExpandQ4Args& a, kva_dtype dst_dtype, cudaStream_t s) {
  const dim3 grid((a.T + EX_SLOTS - 1) / EX_SLOTS, a.c.Hkv, a.N);
  if (dst_dtype == KVA_BF16) return launch_pdl(expand_q4_kernel<bf16_t>, grid, dim3(THREADS), 0, s, a);
  return launch_pdl(expand_q4_kernel<float>, grid, dim3(THREADS), 0, s, a);
}

}  // namespace kva
