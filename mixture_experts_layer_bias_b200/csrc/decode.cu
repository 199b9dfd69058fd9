// The whole MoE layer for a few tokens (at most MOE_DECODE_MAX_TOKENS) in one
// cooperative kernel, one CTA per SM, optionally with low-rank adapters of
// many requests beside the expert projections.
//
// jsqmd.com "第11章 MoE模型推理" 11.1.1: y = sum_{i in TopK} g_i(x) E_i(x).
// With a handful of tokens the layer is bound by reading the touched experts'
// weights once, and a chain of kernels leaves HBM idle at every boundary.
// Here the steps are phases of one grid, separated by grid barriers:
//   route    logits, a warp per (expert, 8 tokens); with E4M3 weights also the
//            tokens' row codes; then every CTA selects all tokens by itself
//            and builds the expert groups in shared memory (no barrier)
//   adapt    (adapters) u = A x of every (token, expert) row
//   up       hidden = act(x W_in), a warp per (expert, column)
//   down     y = sum_k g_k hidden_k W_out, a warp per column
#include <math.h>

#include "common.cuh"
#include "kernels.h"
#include "route_select.cuh"
#include "row_coding.cuh"

namespace moe {

namespace {

using route_detail::select_topk;
using route_detail::SelectParams;
using route_detail::warp_sum;

constexpr int kThreads = 384;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxSlabs = 257;
constexpr int kRouteTokens = 8;  // tokens per warp of the logits

// Grid barrier state, in the workspace's first 256 bytes behind the status
// block.  `arrived` counts arrivals within one call; the last CTA to leave
// the kernel sets both words back to zero.
struct GridSync {
  uint32_t arrived;
  uint32_t left;
};
constexpr size_t kSyncOffset = 128;
static_assert(sizeof(StatusBlock) <= kSyncOffset, "the grid barrier sits behind the status block");

struct Ws {
  size_t logits, xq, xs, hidden, hq, hs, u_in, u_out, total;
};

size_t up256(size_t v) { return (v + 255) & ~size_t(255); }

Ws ws_layout(int S, int d, int E, int K, int h, int ns, int terms, int rank) {
  Ws L;
  size_t o = 256;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = up256(o + bytes);
    return at;
  };
  const size_t rows = static_cast<size_t>(S) * (K + ns);
  L.logits = take(static_cast<size_t>(S) * E * 4);
  L.xq = take(static_cast<size_t>(terms) * S * d);
  L.xs = take(terms ? static_cast<size_t>(S) * 4 : 0);
  L.hidden = take(rows * h * 2);
  L.hq = take(static_cast<size_t>(terms) * rows * h);
  L.hs = take(terms ? rows * 4 : 0);
  L.u_in = take(rows * 2 * rank * 4);
  L.u_out = take(rows * rank * 4);
  L.total = o;
  return L;
}

struct Params {
  DecodeArgs a;
  float* logits;
  uint8_t* xq;
  float* xs;
  __nv_bfloat16* hidden;
  uint8_t* hq;
  float* hs;
  float* u_in;
  float* u_out;
  StatusBlock* status;
  GridSync* sync;
};

// Shared-memory tables of one CTA: the selection and the expert groups.
struct Tables {
  int idx[MOE_DECODE_MAX_TOKENS * 32];        // [S][K]
  float gate[MOE_DECODE_MAX_TOKENS * 32];     // [S][K]
  uint16_t row_slot[MOE_DECODE_MAX_TOKENS * 33];  // row -> slot t*K + k (shared rows: token)
  int first[kMaxSlabs + 1];                   // active group -> its first row
  int slab[kMaxSlabs];                        // active group -> weight slab
  int adapter[MOE_DECODE_MAX_TOKENS];         // token -> adapter or -1
  int warp_sums[kWarps];
  int active;
  int abort;
};

__device__ __forceinline__ uint32_t ld_acquire(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

// Every CTA of the grid arrives; false when the wait gave up.
__device__ bool grid_barrier(const Params& p, Tables& t, uint32_t phase) {
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    atomicAdd(&p.sync->arrived, 1);
    const uint32_t want = phase * gridDim.x;
    if (ld_acquire(&p.sync->arrived) < want) {
      const uint64_t t0 = globaltimer_ns();
      while (ld_acquire(&p.sync->arrived) < want) {
        if (globaltimer_ns() - t0 > kWaitLimitNs) {
          t.abort = 1;
          report(p.status, MOE_STATUS_TIMEOUT, MOE_CNT_TIMEOUT);
          break;
        }
      }
    }
  }
  __syncthreads();
  return t.abort == 0;
}

__device__ void leave(const Params& p) {
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    if (atomicAdd(&p.sync->left, 1) == gridDim.x - 1) {
      p.sync->arrived = 0;
      p.sync->left = 0;
    }
  }
}

__device__ __forceinline__ float e4m3_value(uint32_t c) {
  const float m = coding::e4m3_magnitude(c);
  return (c & 0x80u) ? -m : m;
}

// Sum over a warp of w[k] * row[k] for one weight row: bf16 operands, or E4M3
// weight codes against the row's one or two terms.
__device__ float warp_dot(const void* w, const void* row, int n, int terms) {
  float acc = 0.0f;
  const int lane = lane_id();
  if (terms == 0) {
    for (int c = lane * 8; c < n; c += 256) {
      float a[8], b[8];
      coding::bf16x8_to_f32(ldg16(static_cast<const __nv_bfloat16*>(w) + c), a);
      coding::bf16x8_to_f32(__ldcg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(row) + c)), b);
#pragma unroll
      for (int j = 0; j < 8; ++j) acc = fmaf(a[j], b[j], acc);
    }
  } else {
    const auto* wc = static_cast<const uint8_t*>(w);
    const auto* rc = static_cast<const uint8_t*>(row);
    for (int c = lane * 4; c < n; c += 128) {
      const uint32_t q = __ldg(reinterpret_cast<const uint32_t*>(wc + c));
      const uint32_t r1 = __ldcg(reinterpret_cast<const uint32_t*>(rc + c));
      const uint32_t r2 = terms == 2 ? __ldcg(reinterpret_cast<const uint32_t*>(rc + n + c)) : 0u;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        acc = fmaf(e4m3_value(q >> (8 * j)), e4m3_value(r1 >> (8 * j)) + e4m3_value(r2 >> (8 * j)), acc);
    }
  }
  return warp_sum(acc);
}

// scale * sum_r u[r] B[a][slab][n][r], by a warp.
__device__ float warp_delta(const LoraParams& l, int m, int slabs, int a, int slab, int out, int n, const float* u) {
  const auto* b = static_cast<const __nv_bfloat16*>(l.b[m]) +
                  ((static_cast<int64_t>(a) * slabs + slab) * out + n) * l.r;
  float acc = 0.0f;
  for (int i = lane_id(); i < l.r; i += 32) acc = fmaf(to_f32(b[i]), __ldcg(u + i), acc);
  return warp_sum(acc) * __ldg(l.scale + a);
}

template <int NI>
__device__ void select_tokens(const Params& p, Tables& t, const SelectParams& sp) {
  const int warp = threadIdx.x >> 5, lane = lane_id();
  for (int tok = warp; tok < p.a.S; tok += kWarps) {
    float l[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int e = 32 * i + lane;
      l[i] = e < p.a.E ? __ldcg(p.logits + static_cast<int64_t>(tok) * p.a.E + e) : 0.0f;
    }
    select_topk<NI>(l, sp, tok);
  }
}

// Router logits and, with E4M3 weights, the tokens' codes.
__device__ void route_phase(const Params& p) {
  const DecodeArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = lane_id();
  const int tb = (a.S + kRouteTokens - 1) / kRouteTokens;
  const int dots = a.E * tb, items = dots + (a.terms ? a.S : 0);
  const auto* x = static_cast<const __nv_bfloat16*>(a.x);
  for (int i = blockIdx.x + gridDim.x * warp; i < items; i += gridDim.x * kWarps) {
    if (i >= dots) {
      const int t = i - dots;
      coding::code_row<32>(x + static_cast<int64_t>(t) * a.d, p.xq + static_cast<int64_t>(t) * a.terms * a.d,
                           p.xs + t, a.d, a.terms, lane);
      continue;
    }
    const int e = i % a.E, t0 = (i / a.E) * kRouteTokens;
    const auto* w = static_cast<const __nv_bfloat16*>(a.w_router) + static_cast<int64_t>(e) * a.d;
    float acc[kRouteTokens];
#pragma unroll
    for (int j = 0; j < kRouteTokens; ++j) acc[j] = 0.0f;
    for (int c = lane * 8; c < a.d; c += 256) {
      float wf[8];
      coding::bf16x8_to_f32(ldg16(w + c), wf);
#pragma unroll
      for (int j = 0; j < kRouteTokens; ++j) {
        if (t0 + j < a.S) {
          float xf[8];
          coding::bf16x8_to_f32(ldg16(x + static_cast<int64_t>(t0 + j) * a.d + c), xf);
#pragma unroll
          for (int q = 0; q < 8; ++q) acc[j] = fmaf(wf[q], xf[q], acc[j]);
        }
      }
    }
    const float bias = a.router_bias != nullptr ? __ldg(a.router_bias + e) : 0.0f;
#pragma unroll
    for (int j = 0; j < kRouteTokens; ++j) {
      const float s = warp_sum(acc[j]);
      if (lane == 0 && t0 + j < a.S) p.logits[static_cast<int64_t>(t0 + j) * a.E + e] = __fadd_rn(s, bias);
    }
  }
}

// Selection of every token and the group tables, by each CTA for itself.
__device__ void tables_phase(const Params& p, Tables& t) {
  const DecodeArgs& a = p.a;
  const int tid = threadIdx.x, lane = lane_id(), warp = tid >> 5;
  SelectParams sp{a.E,        a.K,    a.score_fn, a.renormalize, a.num_groups, a.topk_groups, a.tau,
                  a.sel_bias, t.idx,  t.gate,     blockIdx.x == 0 ? p.status : nullptr, nullptr, nullptr};
  if (a.E <= 32)
    select_tokens<1>(p, t, sp);
  else if (a.E <= 64)
    select_tokens<2>(p, t, sp);
  else if (a.E <= 128)
    select_tokens<4>(p, t, sp);
  else
    select_tokens<8>(p, t, sp);
  if (a.lora.n > 0) {
    for (int i = tid; i < a.S; i += kThreads) {
      int id = __ldg(a.lora.ids + i);
      if (id < -1 || id >= a.lora.n) {
        if (blockIdx.x == 0) report(p.status, MOE_STATUS_BAD_ADAPTER, -1);
        id = -1;
      }
      t.adapter[i] = id;
    }
  }
  __syncthreads();
  // thread e: the rows of expert e, in slot order
  const int slots = a.S * a.K, slabs = a.E + a.num_shared;
  int count = 0;
  if (tid < a.E) {
    for (int i = 0; i < slots; ++i) count += t.idx[i] == tid;
  } else if (tid < slabs) {
    count = a.S;
  }
  // exclusive prefix over the slabs of (rows, active groups)
  const int v = count | (count > 0 ? 1 << 16 : 0);
  int incl = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o = __shfl_up_sync(0xFFFFFFFFu, incl, off);
    if (lane >= off) incl += o;
  }
  if (lane == 31) t.warp_sums[warp] = incl;
  __syncthreads();
  int before = incl - v;
  for (int w = 0; w < warp; ++w) before += t.warp_sums[w];
  const int row0 = before & 0xFFFF, group = before >> 16;
  if (tid < slabs && count > 0) {
    t.first[group] = row0;
    t.slab[group] = tid;
    if (tid < a.E) {
      int r = row0;
      for (int i = 0; i < slots; ++i)
        if (t.idx[i] == tid) t.row_slot[r++] = static_cast<uint16_t>(i);
    } else {
      for (int i = 0; i < a.S; ++i) t.row_slot[row0 + i] = static_cast<uint16_t>(i);
    }
  }
  if (tid == kThreads - 1) {
    const int all = before + v;
    t.active = all >> 16;
    t.first[all >> 16] = all & 0xFFFF;
  }
  if (blockIdx.x == 0) {
    if (a.counts != nullptr && tid < a.E) a.counts[tid] = count;
    for (int i = tid; i < slots; i += kThreads) {
      if (a.topk_idx != nullptr) a.topk_idx[i] = t.idx[i];
      if (a.topk_w != nullptr) a.topk_w[i] = t.gate[i];
    }
  }
  __syncthreads();
}

struct Row {
  int token;
  float gate;
};

// Codes of one hidden row by a warp.  The row was written by this grid, so it
// is read at L2 (ld.global.cg), twice: maximum, then codes.
__device__ void code_hidden_row(const __nv_bfloat16* src, uint8_t* dst, float* scale, int n, int terms) {
  const int lane = lane_id();
  uint32_t acc = 0;
  for (int c = lane * 8; c < n; c += 256) acc = coding::absmax_bits8(acc, __ldcg(reinterpret_cast<const uint4*>(src + c)));
  const uint32_t bits = __reduce_max_sync(0xFFFFFFFFu, max(acc & 0xFFFFu, acc >> 16));
  float s, m;
  coding::row_scale(terms, __uint_as_float(bits << 16), bits > 0x7F80u, bits >= 0x7F80u, s, m);
  for (int c = lane * 8; c < n; c += 256)
    coding::code_piece(__ldcg(reinterpret_cast<const uint4*>(src + c)), dst, n, c, terms, s, m);
  if (lane == 0) *scale = s;
}

// The row `r` of the active group with slab `slab`.
__device__ __forceinline__ Row row_at(const Params& p, const Tables& t, int slab, int r) {
  const int s = t.row_slot[r];
  if (slab == p.a.E) return Row{s, 1.0f};
  return Row{s / p.a.K, t.gate[s]};
}

__device__ __forceinline__ int group_of_row(const Tables& t, int r) {
  int lo = 0, hi = t.active;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.first[mid] <= r)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// u[row][m][i] = A_m[a][slab][i] . row for the pairs m0 .. m0 + nm - 1.
__device__ void adapter_inner(const Params& p, const Tables& t, int m0, int nm) {
  const LoraParams& l = p.a.lora;
  const int rows = t.first[t.active], slabs = p.a.E + p.a.num_shared;
  const int warp = threadIdx.x >> 5;
  const int n = m0 == 2 ? p.a.h : p.a.d;
  float* out = m0 == 2 ? p.u_out : p.u_in;
  for (int i = blockIdx.x + gridDim.x * warp; i < rows * nm * l.r; i += gridDim.x * kWarps) {
    const int j = i % l.r, m = m0 + (i / l.r) % nm, r = i / (l.r * nm);
    if (l.a[m] == nullptr) continue;
    const int slab = t.slab[group_of_row(t, r)];
    const int token = row_at(p, t, slab, r).token, ad = t.adapter[token];
    if (ad < 0) continue;
    const auto* w = static_cast<const __nv_bfloat16*>(l.a[m]) + ((static_cast<int64_t>(ad) * slabs + slab) * l.r + j) * n;
    const __nv_bfloat16* src = m0 == 2 ? p.hidden + static_cast<int64_t>(r) * n
                                       : static_cast<const __nv_bfloat16*>(p.a.x) + static_cast<int64_t>(token) * n;
    const float v = warp_dot(w, src, n, 0);
    if (lane_id() == 0) out[(static_cast<int64_t>(r) * nm + (m - m0)) * l.r + j] = v;
  }
}

__device__ void up_phase(const Params& p, const Tables& t) {
  const DecodeArgs& a = p.a;
  const int warp = threadIdx.x >> 5, slabs = a.E + a.num_shared;
  const int wb = a.terms ? 1 : 2;
  const bool swiglu = a.activation == MOE_ACT_SWIGLU;
  for (int64_t i = blockIdx.x + gridDim.x * warp; i < static_cast<int64_t>(t.active) * a.h; i += gridDim.x * kWarps) {
    const int g = static_cast<int>(i / a.h), n = static_cast<int>(i % a.h), slab = t.slab[g];
    const int64_t ch = static_cast<int64_t>(slab) * a.h + n;
    for (int r = t.first[g]; r < t.first[g + 1]; ++r) {
      const int token = row_at(p, t, slab, r).token;
      const void* src = a.terms ? static_cast<const void*>(p.xq + static_cast<int64_t>(token) * a.terms * a.d)
                                : static_cast<const void*>(static_cast<const __nv_bfloat16*>(a.x) +
                                                           static_cast<int64_t>(token) * a.d);
      const float rs = a.terms ? __ldcg(p.xs + token) : 1.0f;
      float v[2] = {0.0f, 0.0f};
      for (int m = swiglu ? 0 : 1; m < 2; ++m) {
        const int q = swiglu ? m : 0;
        v[m] = rs * warp_dot(static_cast<const char*>(a.w_in[q]) + ch * a.d * wb, src, a.d, a.terms);
        if (a.terms) v[m] *= __ldg(a.s_in[q] + ch);
        if (a.lora.n > 0 && a.lora.a[m] != nullptr && t.adapter[token] >= 0)
          v[m] += warp_delta(a.lora, m, slabs, t.adapter[token], slab, a.h, n,
                             p.u_in + (static_cast<int64_t>(r) * 2 + m) * a.lora.r);
      }
      float out;
      if (swiglu) {
        out = v[0] / (1.0f + __expf(-v[0])) * v[1];
      } else {
        const float z = v[1] + __ldg(a.b_in + ch);
        out = 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
      }
      if (lane_id() == 0) p.hidden[static_cast<int64_t>(r) * a.h + n] = __float2bfloat16_rn(out);
    }
  }
}

__device__ void down_phase(const Params& p, const Tables& t) {
  const DecodeArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = lane_id(), slabs = a.E + a.num_shared;
  const int wb = a.terms ? 1 : 2;
  auto* y = static_cast<__nv_bfloat16*>(a.y);
  for (int n = blockIdx.x + gridDim.x * warp; n < a.d; n += gridDim.x * kWarps) {
    float acc[2] = {0.0f, 0.0f};  // tokens lane, lane + 32
    for (int g = 0; g < t.active; ++g) {
      const int slab = t.slab[g];
      const int64_t ch = static_cast<int64_t>(slab) * a.d + n;
      for (int r = t.first[g]; r < t.first[g + 1]; ++r) {
        const Row row = row_at(p, t, slab, r);
        const void* src = a.terms ? static_cast<const void*>(p.hq + static_cast<int64_t>(r) * a.terms * a.h)
                                  : static_cast<const void*>(p.hidden + static_cast<int64_t>(r) * a.h);
        float v = warp_dot(static_cast<const char*>(a.w_out) + ch * a.h * wb, src, a.h, a.terms);
        if (a.terms) v *= __ldcg(p.hs + r) * __ldg(a.s_out + ch);
        if (a.lora.n > 0 && a.lora.a[2] != nullptr && t.adapter[row.token] >= 0)
          v += warp_delta(a.lora, 2, slabs, t.adapter[row.token], slab, a.d, n,
                          p.u_out + static_cast<int64_t>(r) * a.lora.r);
        if (a.b_out != nullptr) v += __ldg(a.b_out + ch);
        if ((row.token & 31) == lane) acc[row.token >> 5] += row.gate * v;
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (lane + 32 * i < a.S) y[static_cast<int64_t>(lane + 32 * i) * a.d + n] = __float2bfloat16_rn(acc[i]);
  }
}

__global__ void __launch_bounds__(kThreads, 1) decode_kernel(const Params p) {
  extern __shared__ uint8_t smem[];
  Tables& t = *reinterpret_cast<Tables*>(smem);
  const DecodeArgs& a = p.a;
  if (threadIdx.x == 0) t.abort = 0;
  uint32_t phase = 0;
  route_phase(p);
  bool ok = grid_barrier(p, t, ++phase);
  if (ok) {
    tables_phase(p, t);
    if (a.lora.n > 0) {
      adapter_inner(p, t, 0, 2);
      ok = grid_barrier(p, t, ++phase);
    }
  }
  if (ok) {
    up_phase(p, t);
    ok = grid_barrier(p, t, ++phase);
  }
  if (ok && (a.terms || a.lora.n > 0)) {
    if (a.terms) {
      const int rows = t.first[t.active];
      for (int r = blockIdx.x + gridDim.x * (threadIdx.x >> 5); r < rows; r += gridDim.x * kWarps)
        code_hidden_row(p.hidden + static_cast<int64_t>(r) * a.h, p.hq + static_cast<int64_t>(r) * a.terms * a.h,
                        p.hs + r, a.h, a.terms);
    }
    if (a.lora.n > 0 && a.lora.a[2] != nullptr) adapter_inner(p, t, 2, 1);
    ok = grid_barrier(p, t, ++phase);
  }
  if (ok) down_phase(p, t);
  leave(p);
}

}  // namespace

size_t decode_workspace_bytes(int S, int d, int E, int K, int h, int num_shared, int terms, int lora_rank) {
  return ws_layout(S, d, E, K, h, num_shared, terms, lora_rank).total;
}

cudaError_t launch_decode(const DecodeArgs& a, cudaStream_t stream) {
  const Ws L = ws_layout(a.S, a.d, a.E, a.K, a.h, a.num_shared, a.terms, a.lora.n > 0 ? a.lora.r : 0);
  char* ws = static_cast<char*>(a.ws);
  Params p;
  p.a = a;
  p.logits = reinterpret_cast<float*>(ws + L.logits);
  p.xq = reinterpret_cast<uint8_t*>(ws + L.xq);
  p.xs = reinterpret_cast<float*>(ws + L.xs);
  p.hidden = reinterpret_cast<__nv_bfloat16*>(ws + L.hidden);
  p.hq = reinterpret_cast<uint8_t*>(ws + L.hq);
  p.hs = reinterpret_cast<float*>(ws + L.hs);
  p.u_in = reinterpret_cast<float*>(ws + L.u_in);
  p.u_out = reinterpret_cast<float*>(ws + L.u_out);
  p.status = reinterpret_cast<StatusBlock*>(ws);
  p.sync = reinterpret_cast<GridSync*>(ws + kSyncOffset);
  const int grid = a.num_sms < kDecodeMaxCtas ? a.num_sms : kDecodeMaxCtas;
  void* args[] = {&p};
  return cudaLaunchCooperativeKernel(reinterpret_cast<void*>(decode_kernel), dim3(grid), dim3(kThreads), args,
                                     sizeof(Tables), stream);
}

}  // namespace moe
