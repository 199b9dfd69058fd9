// Router selection that two experts leave only in the order of their exact keys,
// for any number of tokens.
//
// The logits are tensor-core products (m16n8k16, fp32 sums): a CTA takes 16
// tokens, its eight warps split d and add up in warp order.  The instruction
// sums 32 columns at a time, from zero, and ordinary fp32 additions join those
// sums: what it may lose of its addends is then a share of those 32 products,
// not of all that came before them (see logit_tol).  Each warp then selects two
// of the tokens in fp32.
// Where two of a token's K + 1 best keys (or the last kept and the first dropped
// group) lie closer than a bound on those sums' errors allows to tell, it selects
// in fp64, with the logits of the experts in question summed again in fp64 (a
// product of two bf16 numbers is exact in fp32).  How often that is, for random
// rows, and what the kernel takes with 2048 of them (the second line: 3001):
//     8 experts, width 4096                       0.6 % of the tokens     24 us
//    64 experts, width 2048                       4 %                     46 us
//   128 experts, width 4096, 2 of 4 groups        10 %                   279 us
//   256 experts, width 7168                       14 %                   295 us
//   256 experts, width 7168, 2 of 8 groups        14 %                  1152 us
// Reading x takes 2 to 5 us; in the narrow routers what is left is the few fp64
// tokens, each a chain of about 8 us, one of which most CTAs have.  With groups one
// token in 100 (4 groups) or 50 (8 groups) leaves open which groups are kept: its
// warp then sums every expert's logit, two at a time, and the launch lasts as long as
// that takes.  (Sums carried through the whole width need a bound that is larger and
// grows with it; under one that did not hold they took 1794 us for the last line and
// 215 for the one before, where most of the time is now the products'.)  The
// squared lengths of the router's rows, made in this kernel on the way, cost 20 us
// more than in a kernel of their own (64 experts).
//
// Scores, selection bias, group limit and gates as in the routing kernels
// (jsqmd.com "第11章 MoE模型推理" 11.1.1, 11.3.3; ybb.press "MoE 推理工程深层实战"
// 2.3); ties go to the lower index, a NaN key ranks as -inf.
#include <math.h>

#include <atomic>

#include "common.cuh"
#include "kernels.h"
#include "pdl.cuh"
#include "route_select.cuh"

namespace moe {

namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kWarps = 8;
constexpr int kTokens = 16;  // of a CTA

struct ExactParams {
  int S, d, E, K, score_fn, renormalize, num_groups, topk_groups;
  float tau;
  const __nv_bfloat16* x;
  const __nv_bfloat16* w;
  const float* wsq;  // [E]: squared lengths of the router's rows
  const float* router_bias;
  const float* sel_bias;
  int32_t* topk_idx;
  float* topk_w;
  float* cand_key;
  float* score_out;
  StatusBlock* status;
};

__device__ __forceinline__ double neg_inf() { return __longlong_as_double(0xfff0000000000000ll); }

__device__ __forceinline__ double warp_sum_d(double v) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(kFull, v, off);
  return v;
}

__device__ __forceinline__ float warp_sum_f(float v) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(kFull, v, off);
  return v;
}

// Largest (v, lowest idx) over the warp.
__device__ __forceinline__ void warp_best(double& v, int& idx) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) {
    const double ov = __shfl_xor_sync(kFull, v, off);
    const int oi = __shfl_xor_sync(kFull, idx, off);
    if (ov > v || (ov == v && oi < idx)) {
      v = ov;
      idx = oi;
    }
  }
}

// The q-th of 8 bf16 values.
__device__ __forceinline__ float bf16_at(const uint4& v, int q) {
  const uint32_t w = q < 2 ? v.x : q < 4 ? v.y : q < 6 ? v.z : v.w;
  return __uint_as_float((q & 1) ? (w & 0xFFFF0000u) : (w << 16));
}

// fp64 logits of n <= 2 experts e[], by a warp; four steps' loads at a time.
__device__ void exact_logits(const ExactParams& p, const __nv_bfloat16* xr, const int (&e)[2], int n, double (&out)[2]) {
  const int lane = lane_id();
  double acc[2] = {0.0, 0.0};
  const __nv_bfloat16* wr[2] = {p.w + static_cast<int64_t>(e[0]) * p.d, p.w + static_cast<int64_t>(e[n - 1]) * p.d};
  for (int c = lane * 8; c < p.d; c += 1024) {
    uint4 x[4], w[4][2];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x[k] = ldg16_if(xr + c + 256 * k, c + 256 * k < p.d);
#pragma unroll
      for (int i = 0; i < 2; ++i) w[k][i] = ldg16_if(wr[i] + c + 256 * k, c + 256 * k < p.d);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int q = 0; q < 8; ++q)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          acc[i] += static_cast<double>(__fmul_rn(bf16_at(x[k], q), bf16_at(w[k][i], q)));
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (i < n)
      out[i] = warp_sum_d(acc[i]) + (p.router_bias != nullptr ? static_cast<double>(__ldg(p.router_bias + e[i])) : 0.0);
}

template <int NI>
struct Token {
  double logit[NI];  // expert 32 i + lane
};

template <int NI>
__device__ __forceinline__ void put(Token<NI>& t, int e, double v) {
#pragma unroll
  for (int i = 0; i < NI; ++i)
    if (32 * i + lane_id() == e) t.logit[i] = v;
}

__device__ __forceinline__ double score_of(const ExactParams& p, double l) {
  if (p.score_fn == MOE_SCORE_SIGMOID) return 1.0 / (1.0 + exp(-l));
  return p.tau == 1.0f ? l : l / static_cast<double>(p.tau);
}

__device__ __forceinline__ double key_of(const ExactParams& p, double l, int e) {
  double k = score_of(p, l);
  if (p.sel_bias != nullptr) k += static_cast<double>(__ldg(p.sel_bias + e));
  return isnan(k) ? neg_inf() : k;
}

// Candidates of the kept groups; gap: distance between the last kept and the
// first dropped group score.
template <int NI>
__device__ void group_limit(const ExactParams& p, const double (&key)[NI], bool (&cand)[NI], double* gap) {
  *gap = __longlong_as_double(0x7ff0000000000000ll);
  if (p.num_groups <= 1) return;
  const int lane = lane_id(), gs = p.E / p.num_groups;
  // group score of (register i, lane)'s own group
  double sum[NI];
  if (gs >= 32) {
    const int r = gs >> 5;  // registers per group
#pragma unroll
    for (int i = 0; i < NI; ++i) sum[i] = 0.0;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const double s = warp_sum_d(32 * i + lane < p.E ? key[i] : 0.0);
#pragma unroll
      for (int j = 0; j < NI; ++j)
        if (j / r == i / r) sum[j] += s;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      double s = key[i];
      for (int off = gs >> 1; off >= 1; off >>= 1) s += __shfl_xor_sync(kFull, s, off);
      sum[i] = s;
    }
  }
  bool chosen[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    if (isnan(sum[i])) sum[i] = neg_inf();
    chosen[i] = false;
  }
  double last = 0.0;
  for (int round = 0; round <= p.topk_groups && round < p.num_groups; ++round) {
    double bv = neg_inf();
    int bg = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int g = (32 * i + lane) / gs;
      if (32 * i + lane < p.E && !chosen[i] && (sum[i] > bv || (sum[i] == bv && g < bg))) {
        bv = sum[i];
        bg = g;
      }
    }
    warp_best(bv, bg);
    if (round == p.topk_groups) {
      *gap = last - bv;
      break;
    }
    last = bv;
#pragma unroll
    for (int i = 0; i < NI; ++i)
      if ((32 * i + lane) / gs == bg) chosen[i] = true;
  }
#pragma unroll
  for (int i = 0; i < NI; ++i) cand[i] = cand[i] && chosen[i];
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Squared lengths of the router's rows, a warp per row; `zero`: four
// words that a later kernel of the call counts in.
__global__ void __launch_bounds__(128) router_norm_kernel(const __nv_bfloat16* w, int E, int d, float* wsq, int* zero) {
  const int e = blockIdx.x * 4 + (threadIdx.x >> 5);
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0 && threadIdx.x < 4) zero[threadIdx.x] = 0;
  if (e >= E) return;
  float sq = 0.0f;
#pragma unroll 4
  for (int c = lane_id() * 8; c < d; c += 256) {
    const uint4 v = ldg16(w + static_cast<int64_t>(e) * d + c);
#pragma unroll
    for (int q = 0; q < 8; ++q) sq = fmaf(bf16_at(v, q), bf16_at(v, q), sq);
  }
  sq = warp_sum_f(sq);
  if (lane_id() == 0) wsq[e] = sq;
}

// fp32 logits of the CTA's tokens against NT tiles of 8 experts from e0 on, into
// out[16][E], and on the way the tokens' squared lengths.  A piece is 32 columns
// of d (quad lane q takes columns 8 q ..: the order of a sum's terms is free),
// the next pieces' loads under way during a piece's products.
template <int NT>
__device__ void tile_logits(const ExactParams& p, int t0, int e0, float (*part)[kTokens][64], float (*sq)[kTokens],
                            float* out) {
  const int warp = threadIdx.x >> 5, lane = lane_id(), q = lane & 3, g = lane >> 2;
  const __nv_bfloat16 *ap[2], *bp[NT];
#pragma unroll
  for (int i = 0; i < 2; ++i) ap[i] = p.x + static_cast<int64_t>(min(t0 + g + 8 * i, p.S - 1)) * p.d;
#pragma unroll
  for (int j = 0; j < NT; ++j) bp[j] = p.w + static_cast<int64_t>(min(e0 + 8 * j + g, p.E - 1)) * p.d;
  float acc[NT][4], xs[2] = {0.0f, 0.0f};
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int v = 0; v < 4; ++v) acc[j][v] = 0.0f;
  struct Piece {
    uint4 a[2], b[NT];
  };
  auto load = [&](Piece& pc, int k) {
    const bool in = k + 8 * q < p.d;
#pragma unroll
    for (int i = 0; i < 2; ++i) pc.a[i] = ldg16_if(ap[i] + k + 8 * q, in);
#pragma unroll
    for (int j = 0; j < NT; ++j) pc.b[j] = ldg16_if(bp[j] + k + 8 * q, in);
  };
  auto add = [&](const Piece& pc) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int v = 0; v < 8; ++v) xs[i] = fmaf(bf16_at(pc.a[i], v), bf16_at(pc.a[i], v), xs[i]);
    float c[NT][4];  // from zero: logit_tol counts on it; all first halves, then all second ones, so that none waits
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int v = 0; v < 4; ++v) c[j][v] = 0.0f;
      mma_bf16(c[j], pc.a[0].x, pc.a[1].x, pc.a[0].y, pc.a[1].y, pc.b[j].x, pc.b[j].y);
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) mma_bf16(c[j], pc.a[0].z, pc.a[1].z, pc.a[0].w, pc.a[1].w, pc.b[j].z, pc.b[j].w);
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int v = 0; v < 4; ++v) acc[j][v] += c[j][v];
  };
  constexpr int kAhead = NT <= 2 ? 4 : 2;  // pieces in flight
  Piece pc[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead - 1; ++i) load(pc[i], (warp + i * kWarps) * 32);
  for (int k = warp * 32; k < p.d; k += 32 * kAhead * kWarps) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      load(pc[(i + kAhead - 1) % kAhead], k + (i + kAhead - 1) * 32 * kWarps);
      add(pc[i]);
    }
  }
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int v = 0; v < 4; ++v) part[warp][g + 8 * (v >> 1)][8 * j + 2 * q + (v & 1)] = acc[j][v];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    xs[i] += __shfl_xor_sync(kFull, xs[i], 1);
    xs[i] += __shfl_xor_sync(kFull, xs[i], 2);
    if (q == 0) sq[warp][g + 8 * i] = xs[i];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kTokens * 8 * NT; i += 32 * kWarps) {
    const int t = i / (8 * NT), c = i % (8 * NT);
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += part[w][t][c];
    if (e0 + c < p.E) out[t * p.E + e0 + c] = s;
  }
  __syncthreads();
}

// Bound on the errors of a token's fp32 logits, in units of u = 2^-24 |x| |w|.
//   32 columns: two instructions of 16 products and an accumulator.  PTX promises
//   additions of at least single precision in any order and with any rounding, so
//   each is off by at most 2^-23 of its addends' magnitudes: (15 + 16) 2^-23 m with
//   m the sum of the 32 products' magnitudes.  (Seen on a B200: addends cut to
//   2^-25 of the largest, the sum to 2^-23: less than that.)  Over all columns the m
//   add up to at most |x| |w|: 62 u.
//   Joining them: a rounding of 2^-24 of a partial sum, itself at most |x| |w|, for
//   every 256 columns (eight warps take turns) and for the eight warps: d / 256 + 9 u.
// With room for the second-order terms 96 + d / 256 u; the factor behind covers the
// lengths' own fp32 sums (chains of d / 32 additions).  Squares below fp32's range
// (elements below 2^-74) take less than 2^-58 from a length for any 32-bit d, products
// below it less than 2^-95 from a sum; squares above it make the bound infinite, which
// decides nothing.
__device__ __forceinline__ float logit_tol(const ExactParams& p, float xsq) {
  float w = 0.0f;
  for (int e = lane_id(); e < p.E; e += 32) w = fmaxf(w, __ldg(p.wsq + e));
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) w = fmaxf(w, __shfl_xor_sync(kFull, w, off));
  const float d = static_cast<float>(p.d);
  return (d * 0x1p-8f + 96.0f) * 0x1p-24f * (1.01f + d * 0x1p-28f) * (sqrtf(xsq) + 0x1p-58f) * (sqrtf(w) + 0x1p-58f) +
         0x1p-95f;
}

// The token's selection by one warp, from its fp32 logits (without the bias), in
// fp32; false, with nothing written, where that cannot tell.
template <int NI>
__device__ bool select_fast(const ExactParams& p, int tok, const float* approx, float tol) {
  using namespace route_detail;
  const int lane = lane_id();
  const float kNegInf = __int_as_float(0xff800000);
  float score[NI], key[NI];
  bool valid[NI], cand[NI];
  bool bad = false;
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int e = 32 * i + lane;
    valid[i] = e < p.E;
    float l = kNegInf;
    if (valid[i]) {
      l = approx[e];
      if (p.router_bias != nullptr) l += __ldg(p.router_bias + e);
      bad |= !isfinite(l);
    }
    score[i] = p.score_fn == MOE_SCORE_SIGMOID ? 1.0f / (1.0f + expf(-l)) : p.tau == 1.0f ? l : l / p.tau;
    key[i] = score[i];
    if (valid[i] && p.sel_bias != nullptr) key[i] += __ldg(p.sel_bias + e);
    if (!valid[i]) key[i] = kNegInf;
    bad |= valid[i] && !isfinite(key[i]);
    cand[i] = valid[i];
    if (valid[i]) top = fmaxf(top, fabsf(key[i]) + fabsf(score[i]) + fabsf(l));
  }
  if (__any_sync(kFull, bad)) return false;
  // a key's error: the logit's, and the roundings of the router bias, the score (which repeats the one before it 1 / tau
  // times as large) and the selection bias, each of a few 2^-24 of its own result: a large score may hide in a small key
  const float err = tol * (p.score_fn == MOE_SCORE_SIGMOID ? 0.25f : 1.0f / p.tau) + warp_max(top) * 0x1p-21f;
  if (p.num_groups > 1) {
    const int gs = p.E / p.num_groups;
    float sum[NI];
    if (gs >= 32) {
      const int r = gs >> 5;
#pragma unroll
      for (int i = 0; i < NI; ++i) sum[i] = 0.0f;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const float s = warp_sum(valid[i] ? key[i] : 0.0f);
#pragma unroll
        for (int j = 0; j < NI; ++j)
          if (j / r == i / r) sum[j] += s;
      }
    } else {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        float s = key[i];
        for (int off = gs >> 1; off >= 1; off >>= 1) s += __shfl_xor_sync(kFull, s, off);
        sum[i] = s;
      }
    }
    float last = 0.0f;
    uint32_t chosen = 0;
    for (int round = 0; round <= p.topk_groups && round < p.num_groups; ++round) {
      float bv = kNegInf;
      int bg = 0x7fffffff;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int g = (32 * i + lane) / gs;
        if (valid[i] && !((chosen >> i) & 1u) && (sum[i] > bv || (sum[i] == bv && g < bg))) {
          bv = sum[i];
          bg = g;
        }
      }
      warp_argmax(bv, bg);
      if (round == p.topk_groups) {
        // sums of gs keys, with the roundings of their own additions
        if (!(last - bv > 4.0f * gs * err)) return false;  // (a bound that overflowed decides nothing either)
        break;
      }
      last = bv;
#pragma unroll
      for (int i = 0; i < NI; ++i)
        if ((32 * i + lane) / gs == bg) chosen |= 1u << i;
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) cand[i] = cand[i] && ((chosen >> i) & 1u);
  }
  int my_e = 0;
  float mine = 0.0f, last = 0.0f;
  for (int k = 0; k <= p.K; ++k) {
    float bv = kNegInf;
    int be = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int e = 32 * i + lane;
      if (cand[i] && (key[i] > bv || (key[i] == bv && e < be))) {
        bv = key[i];
        be = e;
      }
    }
    warp_argmax(bv, be);
    if (be >= p.E) break;  // fewer than K + 1 candidates
    if (k > 0 && !(last - bv > 2.0f * err)) return false;
    last = bv;
    float sc = 0.0f;
#pragma unroll
    for (int i = 0; i < NI; ++i)
      if (32 * i + lane == be) {
        cand[i] = false;
        sc = score[i];
      }
    sc = __shfl_sync(kFull, sc, be & 31);
    if (lane == k) {
      my_e = be;
      mine = sc;
    }
  }
  const bool in = lane < p.K;
  const float g = gate_of<NI>(score, valid, mine, in, p.score_fn, p.renormalize);
  if (in) {
    p.topk_idx[static_cast<int64_t>(tok) * p.K + lane] = my_e;
    p.topk_w[static_cast<int64_t>(tok) * p.K + lane] = g;
  }
  return true;
}

// The same in fp64, with exact logits of everyone who is in question.
template <int NI>
__device__ __noinline__ void select_token(const ExactParams& p, int tok, const float* approx, float err) {
  const int lane = lane_id();
  const __nv_bfloat16* xr = p.x + static_cast<int64_t>(tok) * p.d;
  Token<NI> t;
  double key[NI];
  bool cand[NI], valid[NI];
  double gap;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int e = 32 * i + lane;
    valid[i] = e < p.E;
    t.logit[i] = neg_inf();
    if (valid[i]) {
      t.logit[i] = static_cast<double>(approx[e]);
      if (p.router_bias != nullptr) t.logit[i] += static_cast<double>(__ldg(p.router_bias + e));
      bad |= !isfinite(t.logit[i]);
    }
    cand[i] = valid[i];
    key[i] = valid[i] ? key_of(p, t.logit[i], e) : neg_inf();
  }
  bool settled = false;  // cand holds everyone who may be picked
  // a token with an infinity or a NaN keeps these logits: none of its sums means more
  if (!__any_sync(kFull, bad)) {
    group_limit<NI>(p, key, cand, &gap);
    const double slope = p.score_fn == MOE_SCORE_SIGMOID ? 0.25 : 1.0 / static_cast<double>(p.tau);
    const double tol = slope * static_cast<double>(err);
    if (!(gap > 2.0 * tol * (p.E / p.num_groups)) || !isfinite(tol)) {
      // which groups are kept is open, or the bound overflowed: every expert's exact logit
      for (int e0 = 0; e0 < p.E; e0 += 2) {
        const int n = min(2, p.E - e0);
        const int e[2] = {e0, min(e0 + 1, p.E - 1)};
        double v[2];
        exact_logits(p, xr, e, n, v);
        put<NI>(t, e[0], v[0]);
        if (n == 2) put<NI>(t, e[1], v[1]);
      }
    } else {
      // the K + 1 best keys, and everyone else who might beat the last of them
      double last = neg_inf();
      uint32_t taken = 0;
      for (int k = 0; k <= p.K; ++k) {
        double bv = neg_inf();
        int be = 0x7fffffff;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const int e = 32 * i + lane;
          if (cand[i] && !((taken >> i) & 1u) && (key[i] > bv || (key[i] == bv && e < be))) {
            bv = key[i];
            be = e;
          }
        }
        warp_best(bv, be);
        if (be >= p.E) break;
        last = bv;
#pragma unroll
        for (int i = 0; i < NI; ++i)
          if (32 * i + lane == be) taken |= 1u << i;
      }
#pragma unroll
      for (int i = 0; i < NI; ++i) cand[i] = cand[i] && (((taken >> i) & 1u) || key[i] >= last - 2.0 * tol);
      // of those, the ones closer to another than their errors: only their logits are in question
      uint32_t open = 0;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        uint32_t left = __ballot_sync(kFull, cand[i]);
        while (left) {
          const int src = __ffs(left) - 1;
          left &= left - 1;
          const double k = __shfl_sync(kFull, key[i], src);
#pragma unroll
          for (int m = 0; m < NI; ++m)
            if (cand[m] && !(m == i && lane == src) && fabs(key[m] - k) <= 2.0 * tol) open |= 1u << m;
        }
      }
      int pend[2] = {0, 0}, np = 0;
      auto flush = [&]() {
        if (np == 0) return;
        double v[2];
        exact_logits(p, xr, pend, np, v);
        put<NI>(t, pend[0], v[0]);
        if (np == 2) put<NI>(t, pend[1], v[1]);
        np = 0;
      };
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        uint32_t left = __ballot_sync(kFull, (open >> i) & 1u);
        while (left) {
          const int e = 32 * i + __ffs(left) - 1;
          left &= left - 1;
          if (np == 0)
            pend[0] = e;
          else
            pend[1] = e;
          if (++np == 2) flush();
        }
      }
      flush();
      settled = true;
    }
  }
  double score[NI];
  bool some[NI];
  bad = false;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    bad |= valid[i] && !isfinite(t.logit[i]);
    score[i] = score_of(p, t.logit[i]);
    key[i] = valid[i] ? key_of(p, t.logit[i], 32 * i + lane) : neg_inf();
  }
  bad = __any_sync(kFull, bad);
  if (bad && lane == 0) report(p.status, MOE_STATUS_NONFINITE_LOGIT, MOE_CNT_NONFINITE);
#pragma unroll
  for (int i = 0; i < NI; ++i) some[i] = settled ? cand[i] : valid[i];
  if (!settled) group_limit<NI>(p, key, some, &gap);
  if (p.cand_key != nullptr) {
    // re-routing looks at every candidate: the kept groups' experts, exact or not
    bool in[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) in[i] = valid[i];
    group_limit<NI>(p, key, in, &gap);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int64_t at = static_cast<int64_t>(tok) * p.E + 32 * i + lane;
      if (valid[i]) {
        p.cand_key[at] = in[i] ? static_cast<float>(key[i]) : static_cast<float>(neg_inf());
        p.score_out[at] = static_cast<float>(score[i]);
      }
    }
  }
  int my_e = 0;
  double mine = 0.0;
  for (int k = 0; k < p.K; ++k) {
    double bv = neg_inf();
    int be = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int e = 32 * i + lane;
      if (some[i] && (key[i] > bv || (key[i] == bv && e < be))) {
        bv = key[i];
        be = e;
      }
    }
    warp_best(bv, be);
    double sc = 0.0;
#pragma unroll
    for (int i = 0; i < NI; ++i)
      if (32 * i + lane == be) {
        some[i] = false;
        sc = score[i];
      }
    sc = __shfl_sync(kFull, sc, be & 31);
    if (lane == k) {
      my_e = be;
      mine = sc;
    }
  }
  const bool in = lane < p.K;
  float g;
  if (p.score_fn == MOE_SCORE_SOFTMAX) {
    double top = in ? mine : neg_inf();
    if (!p.renormalize) {
#pragma unroll
      for (int i = 0; i < NI; ++i)
        if (valid[i]) top = fmax(top, score[i]);
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) top = fmax(top, __shfl_xor_sync(kFull, top, off));
    const float ex = in ? expf(static_cast<float>(mine - top)) : 0.0f;
    float s = ex;
    if (!p.renormalize) {
      s = 0.0f;
#pragma unroll
      for (int i = 0; i < NI; ++i)
        if (valid[i]) s += expf(static_cast<float>(score[i] - top));
    }
    g = ex / warp_sum_f(s);
  } else {
    const double s = p.renormalize ? warp_sum_d(in ? mine : 0.0) : 1.0;
    g = static_cast<float>(mine / s);
  }
  if (in) {
    p.topk_idx[static_cast<int64_t>(tok) * p.K + lane] = my_e;
    p.topk_w[static_cast<int64_t>(tok) * p.K + lane] = g;
  }
}

template <int NI>
__global__ void __launch_bounds__(32 * kWarps, 2) route_exact_kernel(const ExactParams p) {
  __shared__ float part[kWarps][kTokens][64];
  __shared__ float sq[kWarps][kTokens];
  extern __shared__ float logits[];  // [16][E]
  const int warp = threadIdx.x >> 5, t0 = blockIdx.x * kTokens;
  pdl_wait();
  pdl_trigger();
  for (int e0 = 0; e0 < p.E; e0 += 64) {
    const int left = p.E - e0;
    if (NI == 1 && left <= 8)
      tile_logits<1>(p, t0, e0, part, sq, logits);
    else if (left <= 16)
      tile_logits<2>(p, t0, e0, part, sq, logits);
    else if (left <= 32)
      tile_logits<4>(p, t0, e0, part, sq, logits);
    else
      tile_logits<8>(p, t0, e0, part, sq, logits);
  }
  for (int i = warp; i < kTokens; i += kWarps) {
    if (t0 + i >= p.S) break;
    float xsq = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) xsq += sq[w][i];
    const float tol = logit_tol(p, xsq);
    // (re-routing reads every candidate's key: the fp64 path writes them)
    if (p.cand_key != nullptr || !select_fast<NI>(p, t0 + i, logits + i * p.E, tol))
      select_token<NI>(p, t0 + i, logits + i * p.E, tol);
  }
}

template <int NI>
cudaError_t launch_ni(const ExactParams& p, cudaStream_t stream) {
  if (NI == 8) {  // 16 x 256 logits beside the static arrays exceed the default 48 KB
    static std::atomic<uint64_t> attr_set{0};  // one bit per device ordinal (host threads may launch concurrently)
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !(attr_set.load(std::memory_order_relaxed) & (1ull << dev))) {
      e = cudaFuncSetAttribute(route_exact_kernel<NI>, cudaFuncAttributeMaxDynamicSharedMemorySize, kTokens * 256 * 4);
      if (e != cudaSuccess) return e;
      if (dev < 64) attr_set.fetch_or(1ull << dev, std::memory_order_relaxed);
    }
  }
  const cudaError_t e = launch_pdl(route_exact_kernel<NI>, dim3((p.S + kTokens - 1) / kTokens), dim3(32 * kWarps),
                                   static_cast<size_t>(kTokens) * p.E * 4, stream, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_route_exact(const RouteArgs& a, float* wsq, int* zero, cudaStream_t stream) {
  if (a.S <= 0) return cudaSuccess;
  const auto* w = static_cast<const __nv_bfloat16*>(a.w_router);
  const cudaError_t e = launch_pdl(router_norm_kernel, dim3((a.E + 3) / 4), dim3(128), 0, stream, w, a.E, a.d, wsq, zero);
  if (e != cudaSuccess) return e;
  ExactParams p{a.S, a.d, a.E, a.K, a.score_fn, a.renormalize, a.num_groups, a.topk_groups, a.tau,
                static_cast<const __nv_bfloat16*>(a.x), w, wsq,
                a.router_bias, a.sel_bias, a.topk_idx, a.topk_w, a.cand_key_out, a.score_out, a.status};
  if (a.E <= 32) return launch_ni<1>(p, stream);
  if (a.E <= 64) return launch_ni<2>(p, stream);
  if (a.E <= 128) return launch_ni<4>(p, stream);
  return launch_ni<8>(p, stream);
}

}  // namespace moe
