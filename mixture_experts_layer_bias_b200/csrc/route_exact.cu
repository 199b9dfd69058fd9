// Router selection on fp64 keys for any number of tokens, a warp per token.
//
// A product of two bf16 numbers is exact in fp64, so their fp64 sum gives each
// logit to about 2^-52 of its terms: two experts change places only where the
// exact keys do.  Up to 32 experts, every logit is summed that way, a CTA per 4
// tokens: its four warps split d and take 4 tokens x 4 experts at a time, 16
// fp64 multiply-adds for 4 conversions of tokens and 4 of weights, these by
// integer operations (the conversion instruction, 16 a clock and SM, would bound
// a dot product on its own).  Above, the fp32 logits of the tensor-core
// GEMM select the K + 1 best experts first; those, and every expert that the
// GEMM's error bound leaves within reach of the last of them, get exact logits,
// and the selection and the gates are made from the exact ones only: K + 1 dot
// products a token instead of E.
//
// Scores, selection bias, group limit and gates as in the routing kernels
// (jsqmd.com "第11章 MoE模型推理" 11.1.1, 11.3.3; ybb.press "MoE 推理工程深层实战"
// 2.3); ties go to the lower index, a NaN key ranks as -inf.
#include <math.h>

#include "common.cuh"
#include "kernels.h"
#include "pdl.cuh"

namespace moe {

namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kWarps = 4;  // and tokens of a CTA

struct ExactParams {
  int S, d, E, K, score_fn, renormalize, num_groups, topk_groups;
  float tau;
  const __nv_bfloat16* x;
  const __nv_bfloat16* w;
  const float* approx;  // E > 32: [S][E] fp32 logits without the bias
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

// A bf16 (its bits in the upper half of `w`) as a double times 2^-896, by
// moving its fields: exact for every finite value, subnormals included; an
// infinity or a NaN becomes one.
__device__ __forceinline__ double bf16_bits_to_f64(uint32_t w) {
  uint32_t hi = (w >> 3) & 0x0FFFE000u;  // exponent and mantissa at the bottom of a double's exponent field
  if (hi >= 0x0FF00000u) hi |= 0x7FF00000u;
  return __hiloint2double(static_cast<int>(hi | (w & 0x80000000u)), 0);
}
constexpr double kUnscale = 0x1p896;

// The q-th of 8 bf16 values, as the bits of a float.
__device__ __forceinline__ uint32_t bf16_at(const uint4& v, int q) {
  const uint32_t w = q < 2 ? v.x : q < 4 ? v.y : q < 6 ? v.z : v.w;
  return (q & 1) ? (w & 0xFFFF0000u) : (w << 16);
}

// Exact logits of n <= 4 experts e[]; with NORMS also the largest squared length
// of their rows and that of the token (fp32: a bound needs no more).
template <bool NORMS>
__device__ __forceinline__ void exact_logits(const ExactParams& p, const __nv_bfloat16* xr, const int (&e)[4], int n,
                                             double (&out)[4], float* wnorm, float* xnorm) {
  const int lane = lane_id();
  double acc[4] = {0.0, 0.0, 0.0, 0.0};
  float sq[4] = {0.f, 0.f, 0.f, 0.f}, xq = 0.0f;
  const __nv_bfloat16* wr[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) wr[i] = p.w + static_cast<int64_t>(e[i < n ? i : 0]) * p.d;
  uint4 xv, wv[4], xn, wn[4];  // this step's pieces and the next one's
  auto load = [&](int c, uint4& x, uint4 (&w)[4]) {
    x = ldg16_if(xr + c, c < p.d);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = ldg16_if(wr[i] + c, c < p.d && i < n);
  };
  auto add = [&](const uint4& x, const uint4 (&w)[4]) {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const float xf = __uint_as_float(bf16_at(x, q));
      if (NORMS) xq = fmaf(xf, xf, xq);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float wf = __uint_as_float(bf16_at(w[i], q));
        acc[i] += static_cast<double>(__fmul_rn(xf, wf));  // the product is exact in fp32
        if (NORMS) sq[i] = fmaf(wf, wf, sq[i]);
      }
    }
  };
  load(lane * 8, xv, wv);
  for (int c = lane * 8; c < p.d; c += 512) {
    load(c + 256, xn, wn);
    add(xv, wv);
    load(c + 512, xv, wv);
    add(xn, wn);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i < n) {
      out[i] = warp_sum_d(acc[i]) + (p.router_bias != nullptr ? static_cast<double>(__ldg(p.router_bias + e[i])) : 0.0);
      if (NORMS) *wnorm = fmaxf(*wnorm, warp_sum_f(sq[i]));
    }
  }
  if (NORMS) *xnorm = warp_sum_f(xq);
}

template <int NI>
struct Token {
  double logit[NI];  // expert 32 i + lane
  uint32_t exact;    // bit i: logit[i] is exact
};

template <int NI>
__device__ __forceinline__ void put(Token<NI>& t, int e, double v) {
#pragma unroll
  for (int i = 0; i < NI; ++i)
    if (32 * i + lane_id() == e) {
      t.logit[i] = v;
      t.exact |= 1u << i;
    }
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

// Logits of the CTA's 4 tokens against all experts (at most 32), into out[4][E].
__device__ void all_logits(const ExactParams& p, int t0, double (*part)[16], double* out) {
  const int warp = threadIdx.x >> 5, lane = lane_id();
  const __nv_bfloat16* xr[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) xr[i] = p.x + static_cast<int64_t>(min(t0 + i, p.S - 1)) * p.d;
  for (int e0 = 0; e0 < p.E; e0 += 4) {
    const __nv_bfloat16* wr[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) wr[i] = p.w + static_cast<int64_t>(min(e0 + i, p.E - 1)) * p.d;
    double acc[16];  // [token][expert]
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = 0.0;
    for (int c = (warp * 32 + lane) * 8; c < p.d; c += kWarps * 256) {
      uint4 xv[4], wv[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) xv[i] = ldg16_if(xr[i] + c, true);
#pragma unroll
      for (int i = 0; i < 4; ++i) wv[i] = ldg16_if(wr[i] + c, true);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        double xd[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) xd[i] = static_cast<double>(__uint_as_float(bf16_at(xv[i], q)));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const double wd = bf16_bits_to_f64(bf16_at(wv[j], q));
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[i * 4 + j] = fma(xd[i], wd, acc[i * 4 + j]);
        }
      }
    }
    // reduce-scatter over the warp: lanes i and i + 16 end with the warp's sum of value i
#pragma unroll
    for (int s = 8; s >= 1; s >>= 1) {
      const bool upper = (lane & s) != 0;
#pragma unroll
      for (int i = 0; i < s; ++i) {
        const double send = upper ? acc[i] : acc[i + s], keep = upper ? acc[i + s] : acc[i];
        acc[i] = keep + __shfl_xor_sync(kFull, send, s);
      }
    }
    acc[0] += __shfl_xor_sync(kFull, acc[0], 16);
    if (lane < 16) part[warp][lane] = acc[0];
    __syncthreads();
    if (threadIdx.x < 16) {
      const int e = e0 + (lane & 3);
      if (e < p.E)
        out[(lane >> 2) * p.E + e] = ((part[0][lane] + part[1][lane]) + (part[2][lane] + part[3][lane])) * kUnscale +
                                     (p.router_bias != nullptr ? static_cast<double>(__ldg(p.router_bias + e)) : 0.0);
    }
    __syncthreads();
  }
}

template <int NI>
__global__ void __launch_bounds__(kWarps * 32, NI <= 2 ? 5 : 4) route_exact_kernel(const ExactParams p) {
  __shared__ double part[kWarps][16];
  __shared__ double direct[kWarps * kRouteExactAll];
  const int lane = lane_id();
  const int tok = blockIdx.x * kWarps + (threadIdx.x >> 5);
  pdl_wait();
  pdl_trigger();
  if (NI == 1) all_logits(p, blockIdx.x * kWarps, part, direct);
  if (tok >= p.S) return;
  const __nv_bfloat16* xr = p.x + static_cast<int64_t>(tok) * p.d;
  Token<NI> t;
  t.exact = 0;
  auto all_exact = [&]() {
    for (int e0 = 0; e0 < p.E; e0 += 4) {
      const int n = min(4, p.E - e0);
      const int e[4] = {e0, e0 + 1, e0 + 2, e0 + 3};
      double v[4];
      exact_logits<false>(p, xr, e, n, v, nullptr, nullptr);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < n) put<NI>(t, e[i], v[i]);
    }
  };
  double key[NI];
  bool cand[NI], valid[NI];
  double gap;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    valid[i] = 32 * i + lane < p.E;
    t.logit[i] = neg_inf();
  }
  if (NI == 1) {
    if (valid[0]) t.logit[0] = direct[(threadIdx.x >> 5) * p.E + lane];
    t.exact = 1;
  } else {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int e = 32 * i + lane;
      if (valid[i]) {
        t.logit[i] = static_cast<double>(__ldg(p.approx + static_cast<int64_t>(tok) * p.E + e));
        if (p.router_bias != nullptr) t.logit[i] += static_cast<double>(__ldg(p.router_bias + e));
        bad |= !isfinite(t.logit[i]);
      }
    }
    // a token with an infinity or a NaN keeps the GEMM's logits: none of its sums means more
    if (!__any_sync(kFull, bad)) {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        cand[i] = valid[i];
        key[i] = valid[i] ? key_of(p, t.logit[i], 32 * i + lane) : neg_inf();
      }
      group_limit<NI>(p, key, cand, &gap);
      // exact logits of the K + 1 best by the GEMM's logits
      float xn = 0.0f, wn = 0.0f;
      double last = neg_inf();
      int pend[4] = {0, 0, 0, 0}, np = 0;
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
        const bool found = be < p.E;
        if (found) {
#pragma unroll
          for (int i = 0; i < NI; ++i)
            if (32 * i + lane == be) taken |= 1u << i;
          last = bv;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (i == np) pend[i] = be;
          ++np;
        }
        if (np == 4 || ((k == p.K || !found) && np > 0)) {
          double v[4];
          if (k < 4)
            exact_logits<true>(p, xr, pend, np, v, &wn, &xn);
          else
            exact_logits<false>(p, xr, pend, np, v, nullptr, nullptr);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (i < np) put<NI>(t, pend[i], v[i]);
          np = 0;
        }
        if (!found) break;
      }
      // The GEMM adds d / 16 products of 16 terms, each addition off by at most 2^-23 of the sum's largest part, which
      // is at most |x| |w|; the first picks' row lengths stand for all rows'.  Twice that, in the key's units.
      const double slope = p.score_fn == MOE_SCORE_SIGMOID ? 0.25 : 1.0 / static_cast<double>(p.tau);
      const double tol = 2.0 * slope * (p.d / 16 + 16) * 0x1p-23 * sqrt(static_cast<double>(xn) * wn);
      if (gap <= 2.0 * tol * (p.E / p.num_groups)) {
        all_exact();
      } else {
        // everyone else who might beat the last of them
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          uint32_t near = __ballot_sync(kFull, cand[i] && !((taken >> i) & 1u) && key[i] >= last - 2.0 * tol);
          while (near) {
            const int src = __ffs(near) - 1;
            near &= near - 1;
            const int e[4] = {32 * i + src, 0, 0, 0};
            double v[4];
            exact_logits<false>(p, xr, e, 1, v, nullptr, nullptr);
            if (lane == src) {
              t.logit[i] = v[0];
              t.exact |= 1u << i;
            }
          }
        }
        // experts whose logits stayed approximate are out of the running
#pragma unroll
        for (int i = 0; i < NI; ++i)
          if (!((t.exact >> i) & 1u)) cand[i] = false;
      }
    }
  }
  // selection from what is exact
  double score[NI];
  bool some[NI];
  bad = false;
  bool refined = false;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    bad |= valid[i] && !isfinite(t.logit[i]);
    score[i] = score_of(p, t.logit[i]);
    key[i] = valid[i] ? key_of(p, t.logit[i], 32 * i + lane) : neg_inf();
    refined |= valid[i] && !((t.exact >> i) & 1u);
  }
  bad = __any_sync(kFull, bad);
  refined = __any_sync(kFull, refined) && !bad;  // some logits are approximate: cand holds the exact ones of the kept groups
  if (bad && lane == 0) report(p.status, MOE_STATUS_NONFINITE_LOGIT, MOE_CNT_NONFINITE);
#pragma unroll
  for (int i = 0; i < NI; ++i) some[i] = refined ? cand[i] : valid[i];
  if (!refined) group_limit<NI>(p, key, some, &gap);
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
cudaError_t launch_ni(const ExactParams& p, cudaStream_t stream) {
  const cudaError_t e =
      launch_pdl(route_exact_kernel<NI>, dim3((p.S + kWarps - 1) / kWarps), dim3(kWarps * 32), 0, stream, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_route_exact(const RouteArgs& a, cudaStream_t stream) {
  if (a.S <= 0) return cudaSuccess;
  ExactParams p{a.S, a.d, a.E, a.K, a.score_fn, a.renormalize, a.num_groups, a.topk_groups, a.tau,
                static_cast<const __nv_bfloat16*>(a.x), static_cast<const __nv_bfloat16*>(a.w_router), nullptr,
                a.router_bias, a.sel_bias, a.topk_idx, a.topk_w, a.cand_key_out, a.score_out, a.status};
  if (a.E > kRouteExactAll) {
    const cudaError_t e = launch_router_logits(a, stream);
    if (e != cudaSuccess) return e;
    p.approx = a.logits_scratch;
  }
  if (a.E <= 32) return launch_ni<1>(p, stream);
  if (a.E <= 64) return launch_ni<2>(p, stream);
  if (a.E <= 128) return launch_ni<4>(p, stream);
  return launch_ni<8>(p, stream);
}

}  // namespace moe
