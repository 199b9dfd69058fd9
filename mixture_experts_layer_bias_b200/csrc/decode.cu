// The whole MoE layer for a few tokens (at most MOE_DECODE_MAX_TOKENS) in one
// cooperative kernel, one CTA per SM, optionally with low-rank adapters of
// many requests beside the expert projections.
//
// jsqmd.com "第11章 MoE模型推理" 11.1.1: y = sum_{i in TopK} g_i(x) E_i(x).
// With a handful of tokens the layer is bound by reading the touched experts'
// weights once, and a chain of kernels leaves HBM idle at every boundary.
// Here the steps are phases of one grid:
//   route    logits in fp64, a few warps per (expert, 8 tokens); with E4M3 weights
//            also the tokens' row codes; then the selection and the expert
//            groups, which every CTA builds in its own shared memory
//   up       hidden = act(x W_in)
//   down     y = sum_k g_k hidden_k W_out
//
// Logits and selection keys are fp64 (bf16 products are exact in fp32, their
// sum is not), so the choice between two experts is that of the exact keys
// however close they are.
//
// The two products run on the 5th-generation tensor cores with the WEIGHTS as
// the M = 128 operand and a group's tokens as the N = 16 .. 128 columns, so no
// row of the product is padding and a weight byte goes HBM -> shared memory
// -> tensor core without passing through registers.  A step is one 128-byte
// swizzle row of K (64 bf16 or 128 E4M3) of two 128-row weight tiles that share
// one token tile: gate and up rows of the same 128 hidden columns (SwiGLU), or
// 256 neighbouring output columns.  All steps of a phase, in the order (group,
// tile, k) for up and (tile, group, k) for down, are cut into one range of
// equal cost per CTA (see step_cost), whatever the group sizes are.  A tile
// cut by a range border goes through fp32 partial sums in the workspace: in the
// up phase whichever of its CTAs comes last adds them up, in the down phase the
// whole grid adds them at the end, together with the gate-weighted sum over a
// token's experts.  Both add in CTA order, so results do not depend on timing.
//
// Token tile of the up phase: while all tokens fit into the 16 columns that an
// MMA has at least, every group uses all of them, straight from x.  Otherwise
// the token rows (or codes) are first copied group by group and a group's
// columns are its own tokens.  (Gathering the rows by TMA, four at a time,
// held the up phase at 4.8 TB/s for one token.)
//
// Roles (384 threads): warp 0 feeds a ring of stages by TMA, warp 1 issues the
// MMAs, warps 4 - 11 are the epilogue, two per TMEM lane quarter (2 and 3 help it
// with the adapters).  The weights of
// the down phase do not depend on the hidden rows, so the producer fills the
// whole ring with them while the up phase drains and the grid waits for the last
// hidden row.
//
// E4M3 weights: the tokens' codes (one or two per element, see quant.cu) are
// separate columns of the same product, added in the epilogue.  The codes of a
// hidden row need the row's maximum: it is kept by integer atomics (order does
// not matter) while the up phase stores the bf16 hidden rows, and the epilogue
// warps write the codes between the phases.
//
// Adapters: while the tensor cores start on a phase, warps 2 - 11 of the whole grid
// take the inner products u = A x (up) or A hidden (down) and then the
// outer ones scale * B u, in equal shares, into fp32 buffers; the epilogue adds
// those to a tile's final sums.  (Made by the epilogue itself, tile by tile, the
// outer products kept the CTAs of the busiest expert 150 us longer than the others.)
//
// Every wait is bounded: a CTA that gives up reports MOE_STATUS_TIMEOUT, lets
// its copies and MMAs in flight finish, frees its TMEM and leaves; the others'
// waits then run out too.
#include <math.h>

#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "gemm_common.cuh"
#include "kernels.h"
#include "row_coding.cuh"

namespace moe {

namespace {

constexpr int kThreads = 384;
constexpr int kWarps = kThreads / 32;
constexpr int kEpiWarp0 = 4;  // epilogue warps 4 .. 11
constexpr int kEpiThreads = kThreads - 32 * kEpiWarp0;
constexpr int kLoraWarp0 = 2;  // warps 2 .. 11 take the adapters' products
constexpr int kLoraWarps = kWarps - kLoraWarp0;
constexpr int kMaxSlabs = 257;
constexpr int kRouteTokens = 8;  // tokens per item of the logits
constexpr int kMaxStages = 8;
constexpr int kMaxSlices = 8;  // of K, in the adapters' inner products
constexpr int kTileBytes = 128 * 128;  // one weight tile of a step: 128 rows x 128 bytes of K
constexpr int kTmemCols = 512;
constexpr int kAccs = 16;  // accumulator pairs in flight, 2 x 16 .. 2 x 128 columns each
constexpr size_t kSmemLimit = 232448;  // 227 KB per CTA

// Grid-wide arrival counters, in the workspace's first 256 bytes behind the
// status block: they count up within one call; the last CTA to leave the
// kernel sets them back to zero.
enum Arrival { kRouted, kSelected, kPacked, kInnerUp, kOuterUp, kHidden, kCoded, kInnerDown, kOuterDown, kSummed, kNumArrivals };
struct GridSync {
  uint32_t arrived[kNumArrivals];
  uint32_t left;
};
constexpr size_t kSyncOffset = 128;
static_assert(sizeof(StatusBlock) <= kSyncOffset, "the arrival counters sit behind the status block");
static_assert(kSyncOffset + sizeof(GridSync) <= 256, "the arrival counters sit in the initialised block");

struct Ws {
  size_t logits, idx, gate, xq, xs, xp, hidden, amax, hq, hs, u_in, u_out, d_in, d_out, outs, joins, partial, total;
};

size_t up256(size_t v) { return (v + 255) & ~size_t(255); }

// Whether the up phase's token tile holds all tokens (see above).
__host__ __device__ constexpr bool all_tokens(int S, int terms) { return S * (terms == 2 ? 2 : 1) <= 16; }

Ws ws_layout(int S, int d, int E, int K, int h, int ns, int terms, int rank) {
  Ws L;
  size_t o = 256;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = up256(o + bytes);
    return at;
  };
  const size_t rows = static_cast<size_t>(S) * (K + ns);
  L.logits = take(static_cast<size_t>(S) * E * 8);
  L.idx = take(static_cast<size_t>(S) * K * 4);
  L.gate = take(static_cast<size_t>(S) * K * 4);
  L.xq = take(static_cast<size_t>(terms) * S * d);
  L.xs = take(terms ? static_cast<size_t>(S) * 4 : 0);
  L.xp = take(all_tokens(S, terms) ? 0 : rows * d * (terms ? terms : 2));
  L.hidden = take(rows * h * 2);
  L.amax = take(terms ? rows * 4 : 0);
  L.hq = take(static_cast<size_t>(terms) * rows * h);
  L.hs = take(terms ? rows * 4 : 0);
  L.u_in = take(kMaxSlices * rows * 2 * rank * 4);
  L.u_out = take(kMaxSlices * rows * rank * 4);
  L.d_in = take(rank ? rows * 2 * h * 4 : 0);
  L.d_out = take(rank ? rows * d * 4 : 0);
  L.outs = take(rows * d * 4);
  // per CTA: a counter for the cut up tile that begins in it, and two tiles' partial sums
  L.joins = take(kDecodeMaxCtas * 4);
  L.partial = take(static_cast<size_t>(kDecodeMaxCtas) * 2 * S * 256 * 4);
  L.total = o;
  return L;
}

struct Params {
  DecodeArgs a;
  double* logits;
  int* idx;     // the selection, where it is made by several CTAs
  float* gate;
  uint8_t* xq;
  float* xs;
  uint8_t* xp;  // token rows or codes, group by group
  __nv_bfloat16* hidden;
  uint32_t* amax;
  uint8_t* hq;
  float* hs;
  float* u_in;   // adapters: inner products by slice of K [slice][row][2][r], [slice][row][r]
  float* u_out;
  float* d_in;   // outer products [row][2][h], [row][d]
  float* d_out;
  float* outs;   // expert outputs [row][d] (down tiles that lie in one CTA)
  uint32_t* joins;
  float* partial;
  StatusBlock* status;
  GridSync* sync;
  int stages, stage_bytes, ring_bytes;
  int stream_weights;  // weights leave L2 first
  int test_stall;      // test hook: the producer delivers nothing (the bounded waits must give up)
};

// Shared-memory control block of one CTA; the selection's arrays follow it.
struct Ctl {
  uint64_t full_w[kMaxStages];
  uint64_t full_b[kMaxStages];
  uint64_t empty[kMaxStages];
  uint64_t tfull[kAccs];
  uint64_t tempty[kAccs];
  uint64_t drain;
  int acc_begin[kAccs], acc_end[kAccs];  // TMEM columns of the units in flight (the MMA thread's)
  uint32_t tmem_base;
  int abort;
  int active;
  int last;
  int others_done[2];  // of a cut up tile's parts: all but this CTA's (by the unit's parity)
  int warp_sums[kWarps];
  int warp_costs[kWarps];
  int first[kMaxSlabs + 1];            // active group -> its first row
  int row0[kMaxSlabs];                 // slab -> its first row
  int group[kMaxSlabs];                // slab -> its active group
  int weight[kMaxSlabs + 1];           // active group -> sum of the step costs of the groups before it
  int begin[2][kDecodeMaxCtas + 1];    // phase, CTA -> its first step
  int slab[kMaxSlabs];                 // active group -> weight slab
  uint64_t mask[kMaxSlabs];            // active group -> its tokens
  uint64_t tokens_of[kMaxSlabs];       // slab -> its tokens
  int adapter[MOE_DECODE_MAX_TOKENS];  // token -> adapter or -1
  float scale[MOE_DECODE_MAX_TOKENS];  // E4M3: token -> its codes' scale
};

// Scratch of the routing, in the ring before its first copy.
struct Scratch {
  uint64_t key[kThreads];   // ordered keys
  double score[kThreads];   // gate sources
  double sum[kThreads];     // logits: warp sums; selection: group scores, then the picks' gate sources
  int idx[MOE_DECODE_MAX_TOKENS * 32];     // [S][K]
  float gate[MOE_DECODE_MAX_TOKENS * 32];  // [S][K]
};

struct Tables {
  Ctl* c;
  Scratch* scratch;
  float* row_gate;     // row -> its gate
  float* row_scale;    // E4M3: row -> its codes' scale (tokens, then hidden rows)
  uint16_t* row_tok;   // row -> its token
  uint16_t* row_grp;   // row -> its active group
  uint16_t* slot_row;  // [S][K]: slot -> its row
};

size_t tables_bytes(int S, int K, int ns) {
  const size_t rows = static_cast<size_t>(S) * (K + ns);
  return ((sizeof(Ctl) + 15) & ~size_t(15)) + ((rows * 12 + static_cast<size_t>(S) * K * 2 + 15) & ~size_t(15));
}

__device__ __forceinline__ uint32_t ld_acquire(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

// One thread: wait until every CTA has arrived at `k`.
__device__ bool wait_arrivals(const Params& p, Arrival k, volatile int* abort_flag) {
  const uint32_t* word = &p.sync->arrived[k];
  if (ld_acquire(word) >= gridDim.x) return true;
  const uint64_t t0 = globaltimer_ns();
  while (ld_acquire(word) < gridDim.x) {
    if (*abort_flag) return false;
    if (globaltimer_ns() - t0 > kWaitLimitNs) return false;
  }
  return true;
}

__device__ __forceinline__ void give_up(const Params& p, volatile int* abort_flag) {
  *abort_flag = 1;
  report(p.status, MOE_STATUS_TIMEOUT, MOE_CNT_TIMEOUT);
}

// A barrier (`id`) of the warps from WARP0 on; true when any of them passes
// `failed`.  Its answer is the same for all, so they leave a loop together or not
// at all.
template <int WARP0>
__device__ __forceinline__ bool any_of(bool failed) {
  int any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.s32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %3, %2, p;\n\t"
      "selp.s32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"(static_cast<int>(failed)), "n"(kThreads - 32 * WARP0), "n"(WARP0 == kEpiWarp0 ? 1 : 2)
      : "memory");
  return any != 0;
}
__device__ __forceinline__ bool epi_any(bool failed) { return any_of<kEpiWarp0>(failed); }

// The warps from WARP0 on arrive at `k` for their CTA once their writes are done
// (written by the generic proxy, read by other CTAs through either).
template <int WARP0 = kEpiWarp0>
__device__ __forceinline__ void epi_arrive(const Params& p, Arrival k) {
  fence_proxy_async_global();
  any_of<WARP0>(false);
  if (threadIdx.x == 32 * WARP0) {
    __threadfence();  // (the barrier before it makes this cover every warp's writes)
    atomicAdd(&p.sync->arrived[k], 1);
  }
}

// They wait for `k`; false (for all of them) when it gave up.
template <int WARP0 = kEpiWarp0>
__device__ __forceinline__ bool epi_wait(const Params& p, Arrival k, volatile int* abort_flag) {
  bool failed = false;
  if (threadIdx.x == 32 * WARP0 && !wait_arrivals(p, k, abort_flag)) {
    give_up(p, abort_flag);
    failed = true;
  }
  return !any_of<WARP0>(failed);
}

// Every thread of every CTA: false when the wait gave up.
__device__ bool grid_barrier(const Params& p, Ctl& c, Arrival k) {
  fence_proxy_async_global();
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    atomicAdd(&p.sync->arrived[k], 1);
    if (!wait_arrivals(p, k, &c.abort)) give_up(p, &c.abort);
  }
  __syncthreads();
  fence_proxy_async_global();
  return c.abort == 0;
}

// The last CTA to leave sets the counters back for the next call.
__device__ void leave(const Params& p) {
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    if (atomicAdd(&p.sync->left, 1) == gridDim.x - 1) {
      for (int i = 0; i < kNumArrivals; ++i) p.sync->arrived[i] = 0;
      p.sync->left = 0;
    }
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
  return v;
}

// Router logits, a team of a CTA's warps per (expert, 8 tokens), striding over d in
// 16-byte pieces: a bf16 product is exact in fp32 and is summed in fp64.  (64 tokens
// and 64 experts: 124 us for the layer with teams of 3 warps in one round, 128 with
// the whole CTA in four.)  With E4M3 weights also the tokens' codes, a warp per token, by the CTAs from the
// other end of the grid.  The join counters and row maxima start at zero.
__device__ void route_phase(const Params& p, Scratch& c) {
  const DecodeArgs& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = lane_id();
  const int rows = a.S * (a.K + a.num_shared);
  for (int i = blockIdx.x * kThreads + tid; i < kDecodeMaxCtas || (a.terms && i < rows); i += gridDim.x * kThreads) {
    if (i < kDecodeMaxCtas) p.joins[i] = 0;
    if (a.terms && i < rows) p.amax[i] = 0;
  }
  const auto* x = static_cast<const __nv_bfloat16*>(a.x);
  if (a.terms) {
    for (int t = (gridDim.x - 1 - blockIdx.x) + gridDim.x * warp; t < a.S; t += gridDim.x * kWarps)
      coding::code_row<32>(x + static_cast<int64_t>(t) * a.d, p.xq + static_cast<int64_t>(t) * a.terms * a.d,
                           p.xs + t, a.d, a.terms, lane);
  }
  const int items = a.E * ((a.S + kRouteTokens - 1) / kRouteTokens);
  int team = kWarps;  // warps of an item: as many as leave one round of items
  while (team > 1 && items > static_cast<int>(gridDim.x) * (kWarps / team)) team = kWarps / (kWarps / team + 1);
  const int teams = kWarps / team, mine = warp / team, rank = (warp - mine * team) * 32 + lane;
  for (int i0 = blockIdx.x * teams; i0 < items; i0 += gridDim.x * teams) {
    const int i = i0 + mine;
    const int e = i % a.E, t0 = (i / a.E) * kRouteTokens, nt = i < items ? min(kRouteTokens, a.S - t0) : 0;
    const auto* w = static_cast<const __nv_bfloat16*>(a.w_router) + static_cast<int64_t>(e) * a.d;
    const auto* xt = x + static_cast<int64_t>(t0) * a.d;
    double acc[kRouteTokens];
#pragma unroll
    for (int j = 0; j < kRouteTokens; ++j) acc[j] = 0.0;
    for (int k = rank * 8; k < a.d && nt > 0; k += team * 256) {
      float wf[8];
      uint4 xv[kRouteTokens];
      const uint4 wv = ldg16(w + k);
#pragma unroll
      for (int j = 0; j < kRouteTokens; ++j)
        if (j < nt) xv[j] = ldg16(xt + static_cast<int64_t>(j) * a.d + k);
      coding::bf16x8_to_f32(wv, wf);
#pragma unroll
      for (int j = 0; j < kRouteTokens; ++j) {
        if (j < nt) {
          float xf[8];
          coding::bf16x8_to_f32(xv[j], xf);
#pragma unroll
          for (int q = 0; q < 8; ++q) acc[j] += static_cast<double>(__fmul_rn(wf[q], xf[q]));
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kRouteTokens; ++j) {
      if (j < nt) {
        double v = acc[j];
        for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
        if (lane == 0) c.sum[warp * kRouteTokens + j] = v;
      }
    }
    __syncthreads();
    if (rank < nt) {
      double v = a.router_bias != nullptr ? static_cast<double>(__ldg(a.router_bias + e)) : 0.0;
      for (int k = 0; k < team; ++k) v += c.sum[(mine * team + k) * kRouteTokens + rank];
      p.logits[static_cast<int64_t>(t0 + rank) * a.E + e] = v;
    }
    __syncthreads();
  }
}

// A double as an unsigned integer of the same order; all results are above 0.
__device__ __forceinline__ uint64_t ordered(double v) {
  const uint64_t b = static_cast<uint64_t>(__double_as_longlong(v));
  return (b >> 63) ? ~b : b | (uint64_t(1) << 63);
}

// Tokens that a CTA selects at once: a thread per (token, expert).
__device__ __forceinline__ int select_width(int E) {
  int w = 8;
  while (w < E) w <<= 1;
  return w;
}

// Selection of the tokens t0 .. t0 + n - 1 (n * width <= kThreads) by the whole
// CTA: an expert's slot is the number of candidates with a larger key (ties to
// the lower index; a NaN key ranks as -inf).  Scores, group limit and gates as
// in the routing kernels, with fp64 keys.
__device__ void select_tokens(const Params& p, Scratch& c, int t0, int n, int width, int* idx, float* gate, bool report_bad) {
  const DecodeArgs& a = p.a;
  const int tid = threadIdx.x, j = tid / width, e = tid % width;
  const double kNegInf = __longlong_as_double(0xfff0000000000000ll);
  const bool in = j < n && e < a.E;
  double score = 0.0, key = kNegInf;
  if (in) {
    const double l = __ldcg(p.logits + static_cast<int64_t>(t0 + j) * a.E + e);
    score = a.score_fn == MOE_SCORE_SIGMOID ? 1.0 / (1.0 + exp(-l)) : (a.tau == 1.0f ? l : l / static_cast<double>(a.tau));
    key = a.sel_bias != nullptr ? score + static_cast<double>(__ldg(a.sel_bias + e)) : score;
    if (isnan(key)) key = kNegInf;
    c.score[tid] = score;
    c.key[tid] = ordered(key);
    if (report_bad) {
      // one report per token: by its first bad expert
      if (!isfinite(l)) {
        bool first = true;
        for (int q = 0; q < e && first; ++q)
          first = isfinite(__ldcg(p.logits + static_cast<int64_t>(t0 + j) * a.E + q));
        if (first) report(p.status, MOE_STATUS_NONFINITE_LOGIT, MOE_CNT_NONFINITE);
      }
    }
  }
  __syncthreads();
  if (a.num_groups > 1) {
    const int gs = a.E / a.num_groups;
    double s = 0.0;
    if (j < n && e < a.num_groups) {
      for (int q = 0; q < gs; ++q) {
        const uint64_t o = c.key[j * width + e * gs + q];
        s += __longlong_as_double(static_cast<long long>((o >> 63) ? o ^ (uint64_t(1) << 63) : ~o));
      }
      if (isnan(s)) s = kNegInf;
      c.sum[tid] = s;
    }
    __syncthreads();
    bool kept = false;
    if (in) {
      const int g = e / gs;
      const double mine = c.sum[j * width + g];
      int rank = 0;
      for (int q = 0; q < a.num_groups; ++q) {
        const double o = c.sum[j * width + q];
        rank += o > mine || (o == mine && q < g);
      }
      kept = rank < a.topk_groups;
    }
    __syncthreads();
    if (in && !kept) c.key[tid] = 0;  // below every candidate
    __syncthreads();
  }
  const uint64_t mine_key = in ? c.key[tid] : 0;
  if (mine_key != 0) {  // a candidate: its slot is the number of better ones
    const uint64_t mine = mine_key;
    int rank = 0;
    const uint64_t* keys = c.key + j * width;
    if (a.num_groups > 1) {
      const int gs = a.E / a.num_groups;
      for (int g = 0; g < a.num_groups; ++g) {
        if (keys[g * gs] == 0) continue;  // a dropped group
        for (int q = g * gs; q < (g + 1) * gs; ++q) rank += keys[q] > mine || (keys[q] == mine && q < e);
      }
    } else {
      for (int q = 0; q < a.E; ++q) rank += keys[q] > mine || (keys[q] == mine && q < e);
    }
    if (rank < a.K) {
      idx[(t0 + j) * a.K + rank] = e;
      c.sum[j * width + rank] = score;  // (the group scores have been read)
    }
  }
  __syncthreads();
  if (j < n && e < a.K) {
    const double* picks = c.sum + j * width;
    const double mine = picks[e];
    float g;
    if (a.score_fn == MOE_SCORE_SOFTMAX) {
      const double* from = a.renormalize ? picks : c.score + j * width;
      const int m = a.renormalize ? a.K : a.E;
      double top = kNegInf;
      bool nan = false;
      for (int q = 0; q < m; ++q) {
        top = fmax(top, from[q]);
        nan |= isnan(from[q]);
      }
      float sum = 0.0f;
      for (int q = 0; q < m; ++q) sum += expf(static_cast<float>(from[q] - top));
      g = expf(static_cast<float>(mine - top)) / sum;
      if (nan) g = __int_as_float(0x7fc00000);
    } else if (a.renormalize) {
      double sum = 0.0;
      for (int q = 0; q < a.K; ++q) sum += picks[q];
      g = static_cast<float>(mine / sum);
    } else {
      g = static_cast<float>(mine);
    }
    gate[(t0 + j) * a.K + e] = g;
  }
  __syncthreads();
}

// What a step of a group with this many tokens costs: its weight bytes and, for
// every 16 columns of its token tile, about a tenth of that again (measured on 64
// tokens over 64 E4M3 experts: 52 us for a CTA's steps with one box of columns, 67
// with three, 75 with five; that shape alone is behind the numbers, bf16 weights and
// other widths use them as they are).  Groups that share a dense tile all cost the same.
__device__ __forceinline__ int step_cost(const DecodeArgs& a, int tokens) {
  return all_tokens(a.S, a.terms) ? 1 : 9 + (tokens * (a.terms == 2 ? 2 : 1) + 15) / 16;
}

// Selection and the group tables in this CTA's shared memory.  Up to two rounds
// of tokens are selected by every CTA for itself; more are spread over the CTAs
// (a grid barrier costs less than a third round).  False: a wait gave up.
__device__ bool tables_phase(const Params& p, const Tables& t) {
  const DecodeArgs& a = p.a;
  Ctl& c = *t.c;
  Scratch& sc = *t.scratch;
  const int tid = threadIdx.x, lane = lane_id(), warp = tid >> 5;
  const int slots = a.S * a.K, slabs = a.E + a.num_shared;
  const int width = select_width(a.E), per = kThreads / width, rounds = (a.S + per - 1) / per;
  for (int i = tid; i < slabs; i += kThreads) c.tokens_of[i] = 0;
  // a token's adapter and its codes' scale, loaded while the selection runs
  const bool adapted = a.lora.n > 0 && tid < a.S;
  const int id = adapted ? __ldg(a.lora.ids + tid) : -1;
  const float scale = a.terms && tid < a.S ? __ldcg(p.xs + tid) : 1.0f;
  if (rounds <= 2) {
    for (int r = 0; r < rounds; ++r)
      select_tokens(p, sc, r * per, min(per, a.S - r * per), width, sc.idx, sc.gate, blockIdx.x == 0);
  } else {
    for (int r = blockIdx.x; r < rounds; r += gridDim.x)
      select_tokens(p, sc, r * per, min(per, a.S - r * per), width, p.idx, p.gate, true);
    if (!grid_barrier(p, c, kSelected)) return false;
    for (int i = tid; i < slots; i += kThreads) {
      sc.idx[i] = __ldcg(p.idx + i);
      sc.gate[i] = __ldcg(p.gate + i);
    }
    __syncthreads();
  }
  // an expert's tokens as a 64-bit mask: its rows are the set bits in token order
  for (int i = tid; i < slots; i += kThreads)
    atomicOr(reinterpret_cast<uint32_t*>(c.tokens_of + sc.idx[i]) + (i / a.K >> 5), 1u << (i / a.K & 31));
  if (tid == kThreads - 1 && a.num_shared) c.tokens_of[a.E] = a.S == 64 ? ~uint64_t(0) : (uint64_t(1) << a.S) - 1;
  if (tid < a.S) {
    const bool known = id >= -1 && id < a.lora.n;
    if (adapted && !known && blockIdx.x == 0) report(p.status, MOE_STATUS_BAD_ADAPTER, -1);
    c.adapter[tid] = adapted && known ? id : -1;
    c.scale[tid] = scale;
  }
  __syncthreads();
  // exclusive prefix over the slabs of (rows, active groups)
  const uint64_t mask = tid < slabs ? c.tokens_of[tid] : 0;
  const int count = __popcll(mask);
  const int v = count | (count > 0 ? 1 << 16 : 0);
  const int cost = count > 0 ? step_cost(a, count) : 0;
  int incl = v, costs = cost;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o = __shfl_up_sync(0xFFFFFFFFu, incl, off), oc = __shfl_up_sync(0xFFFFFFFFu, costs, off);
    if (lane >= off) {
      incl += o;
      costs += oc;
    }
  }
  if (lane == 31) {
    c.warp_sums[warp] = incl;
    c.warp_costs[warp] = costs;
  }
  __syncthreads();
  int before = incl - v;
  costs -= cost;
  for (int w = 0; w < warp; ++w) {
    before += c.warp_sums[w];
    costs += c.warp_costs[w];
  }
  const int row0 = before & 0xFFFF, group = before >> 16;
  if (count > 0) {
    c.first[group] = row0;
    c.slab[group] = tid;
    c.mask[group] = mask;
    c.weight[group] = costs;
  }
  if (tid < slabs) {
    c.row0[tid] = row0;
    c.group[tid] = group;
  }
  if (tid == kThreads - 1) {
    const int all = before + v;
    c.active = all >> 16;
    c.first[all >> 16] = all & 0xFFFF;
    c.weight[all >> 16] = costs + cost;
  }
  __syncthreads();
  for (int i = tid; i < slots + a.S * a.num_shared; i += kThreads) {
    const bool shared = i >= slots;
    const int tok = shared ? i - slots : i / a.K;
    const int e = shared ? a.E : sc.idx[i];
    const int r = c.row0[e] + __popcll(c.tokens_of[e] & ((uint64_t(1) << tok) - 1));
    t.row_tok[r] = static_cast<uint16_t>(tok);
    t.row_grp[r] = static_cast<uint16_t>(c.group[e]);
    t.row_gate[r] = shared ? 1.0f : sc.gate[i];
    if (!shared) t.slot_row[i] = static_cast<uint16_t>(r);
    if (a.terms) t.row_scale[r] = c.scale[tok];
  }
  if (blockIdx.x == 0) {
    if (a.counts != nullptr && tid < a.E) a.counts[tid] = count;
    for (int i = tid; i < slots; i += kThreads) {
      if (a.topk_idx != nullptr) a.topk_idx[i] = sc.idx[i];
      if (a.topk_w != nullptr) a.topk_w[i] = sc.gate[i];
    }
  }
  fence_proxy_async_smem();  // the scratch lies where the first copies land
  __syncthreads();
  if (all_tokens(a.S, a.terms)) return true;
  // token rows or codes, group by group: a warp per row
  const int rows = slots + a.S * a.num_shared, bytes = a.d * (a.terms ? a.terms : 2);
  for (int r = blockIdx.x + gridDim.x * warp; r < rows; r += gridDim.x * kWarps) {
    const int tok = t.row_tok[r];
    const auto* src = reinterpret_cast<const uint4*>(
        (a.terms ? p.xq : static_cast<const uint8_t*>(a.x)) + static_cast<int64_t>(tok) * bytes);
    auto* dst = reinterpret_cast<uint4*>(p.xp + static_cast<int64_t>(r) * bytes);
    for (int i = lane; i < bytes / 16; i += 128) {
      uint4 q[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (i + 32 * k < bytes / 16) q[k] = __ldcg(src + i + 32 * k);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (i + 32 * k < bytes / 16) dst[i + 32 * k] = q[k];
    }
  }
  return grid_barrier(p, c, kPacked);
}

// This warp's share [lo, hi) of n items that the grid's warps 2 .. 11 divide.
__device__ __forceinline__ void warp_share(int n, int& lo, int& hi) {
  const int warps = gridDim.x * kLoraWarps, w = ((threadIdx.x >> 5) - kLoraWarp0) * gridDim.x + blockIdx.x;
  const int q = n / warps, r = n - q * warps;
  lo = w * q + min(w, r);
  hi = lo + q + (w < r ? 1 : 0);
}

// Slices of K of the inner products: about two items for every warp of the grid.
__device__ __forceinline__ int inner_slices(int items, int pieces) {
  const int warps = gridDim.x * kLoraWarps;
  return max(1, min(min(kMaxSlices, pieces), 2 * warps / max(items, 1)));
}

// Warps 2 .. 11: u[slice][row][m][i] = A_m[a][slab][i] . row over a slice of K, for
// the pairs m0 .. m0 + nm - 1.  An item is (row, pair, 8 values, slice): the row's
// pieces of 256 meet eight rows of A, nine loads per lane and piece; a warp
// streams through its items' pieces with the next one's loads always under way.
__device__ void adapter_inner(const Params& p, const Tables& t, int m0, int nm) {
  const LoraParams& l = p.a.lora;
  const int rows = t.c->first[t.c->active], slabs = p.a.E + p.a.num_shared, blocks = l.r / 8;
  const int lane = lane_id();
  const int n = m0 == 2 ? p.a.h : p.a.d, pieces = (n + 255) / 256;
  float* out = m0 == 2 ? p.u_out : p.u_in;
  const int slices = inner_slices(rows * nm * blocks, pieces);
  int lo, hi;
  warp_share(rows * nm * blocks * slices, lo, hi);
  struct Cursor {
    int item, piece, end;
    const __nv_bfloat16 *w, *src;  // w nullptr: nothing to do for this item
  };
  auto seek = [&](Cursor& c) {  // to the item's rows
    const int s = c.item % slices, i = c.item / slices;
    const int j = i % blocks * 8, m = m0 + i / blocks % nm, r = i / (blocks * nm);
    c.piece = pieces * s / slices;
    c.end = pieces * (s + 1) / slices;
    c.w = nullptr;
    if (c.item >= hi || l.a[m] == nullptr) return;
    const int token = t.row_tok[r], ad = t.c->adapter[token], slab = t.c->slab[t.row_grp[r]];
    if (ad < 0) return;
    c.w = static_cast<const __nv_bfloat16*>(l.a[m]) + ((static_cast<int64_t>(ad) * slabs + slab) * l.r + j) * n;
    c.src = m0 == 2 ? p.hidden + static_cast<int64_t>(r) * n
                    : static_cast<const __nv_bfloat16*>(p.a.x) + static_cast<int64_t>(token) * n;
  };
  auto next = [&](Cursor& c) {
    if (++c.piece == c.end || c.w == nullptr) {
      do {
        ++c.item;
        seek(c);
      } while (c.w == nullptr && c.item < hi);
    }
  };
  struct Piece {
    uint4 x, w[8];
  };
  auto load = [&](const Cursor& c, Piece& pc) {
    const int col = c.piece * 256 + lane * 8;
    const bool in = c.w != nullptr && col < n;
#pragma unroll
    for (int k = 0; k < 8; ++k) pc.w[k] = ldg16_if(c.w + static_cast<int64_t>(k) * n + col, in);
    pc.x = in ? __ldcg(reinterpret_cast<const uint4*>(c.src + col)) : make_uint4(0, 0, 0, 0);
  };
  float acc[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) acc[k] = 0.0f;
  auto add = [&](const Cursor& c, const Piece& pc) {
    float xf[8];
    coding::bf16x8_to_f32(pc.x, xf);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float wf[8];
      coding::bf16x8_to_f32(pc.w[k], wf);
#pragma unroll
      for (int q = 0; q < 8; ++q) acc[k] = fmaf(wf[q], xf[q], acc[k]);
    }
    if (c.piece + 1 < c.end) return;
    float v = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float s = warp_sum(acc[k]);
      if (lane == k) v = s;
      acc[k] = 0.0f;
    }
    const int s = c.item % slices, i = c.item / slices;
    if (lane < 8) out[(static_cast<int64_t>(s) * rows * nm + i / blocks) * l.r + i % blocks * 8 + lane] = v;
  };
  Cursor c0{lo, 0, 0, nullptr, nullptr};
  if (lo < hi) seek(c0);
  if (c0.w == nullptr) next(c0);
  Piece p0, p1;
  load(c0, p0);
  while (c0.w != nullptr) {
    Cursor c1 = c0;
    next(c1);
    load(c1, p1);
    add(c0, p0);
    if (c1.w == nullptr) break;
    c0 = c1;
    next(c0);
    load(c0, p0);
    add(c1, p1);
  }
}

// Warps 2 .. 11: out[row][m][n] = scale * sum_i u[row][m][i] B_m[a][slab][n][i].
// r / 8 neighbouring lanes (rounded up to a power of two) take 16 bytes each of a
// column's row of B and add up by shuffles; eight loads per lane make a batch of
// columns, the next batch's under way, and a warp takes an equal run of batches.
__device__ void adapter_outer(const Params& p, const Tables& t, int m0, int nm) {
  const LoraParams& l = p.a.lora;
  const int rows = t.c->first[t.c->active], slabs = p.a.E + p.a.num_shared, lane = lane_id();
  const int n = m0 == 2 ? p.a.d : p.a.h;
  const float* us = m0 == 2 ? p.u_out : p.u_in;
  float* out = m0 == 2 ? p.d_out : p.d_in;
  int width = 1;
  while (width * 8 < l.r) width *= 2;  // lanes of a column
  const int sub = lane & (width - 1), per = 32 / width, first = lane / width, batch = 8 * per;
  const int batches = (n + batch - 1) / batch;
  const bool holds = sub * 8 < l.r;
  const int slices = inner_slices(rows * nm * (l.r / 8), ((m0 == 2 ? p.a.h : p.a.d) + 255) / 256);
  int lo, hi;
  warp_share(rows * nm * batches, lo, hi);
  while (lo < hi) {
    const int at = lo / batches, m = m0 + at % nm, r = at / nm;  // at = r * nm + m - m0
    const int b0 = lo - at * batches, b1 = min(batches, b0 + hi - lo);
    lo += b1 - b0;
    const int ad = t.c->adapter[t.row_tok[r]];
    if (ad < 0) continue;
    float* o = out + static_cast<int64_t>(at) * n;
    const int c1 = min(n, b1 * batch);
    if (l.a[m] == nullptr) {
      for (int c = b0 * batch + lane; c < c1; c += 32) o[c] = 0.0f;
      continue;
    }
    const auto* w = static_cast<const __nv_bfloat16*>(l.b[m]) +
                    (static_cast<int64_t>(ad) * slabs + t.c->slab[t.row_grp[r]]) * n * l.r + sub * 8;
    auto load = [&](int c, uint4 (&v)[8]) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int col = c + k * per;
        v[k] = ldg16_if(w + static_cast<int64_t>(col) * l.r, holds && col < c1);
      }
    };
    uint4 v0[8], v1[8];
    load(b0 * batch + first, v0);
    float uf[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) uf[q] = 0.0f;
    for (int k = 0; k < slices && holds; ++k) {
      const float* src = us + (static_cast<int64_t>(k) * rows * nm + at) * l.r + sub * 8;
      const float4 a0 = __ldcg(reinterpret_cast<const float4*>(src)), a1 = __ldcg(reinterpret_cast<const float4*>(src + 4));
      uf[0] += a0.x;
      uf[1] += a0.y;
      uf[2] += a0.z;
      uf[3] += a0.w;
      uf[4] += a1.x;
      uf[5] += a1.y;
      uf[6] += a1.z;
      uf[7] += a1.w;
    }
    const float scale = __ldg(l.scale + ad);
    auto finish = [&](int c, const uint4 (&v)[8]) {
      float s[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        float f[8];
        coding::bf16x8_to_f32(v[k], f);
        s[k] = 0.0f;
#pragma unroll
        for (int q = 0; q < 8; ++q) s[k] = fmaf(f[q], uf[q], s[k]);
      }
      for (int off = width >> 1; off >= 1; off >>= 1) {  // the eight sums' shuffles overlap
#pragma unroll
        for (int k = 0; k < 8; ++k) s[k] += __shfl_xor_sync(0xFFFFFFFFu, s[k], off);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int col = c + k * per;
        if (sub == 0 && col < c1) o[col] = s[k] * scale;
      }
    };
    for (int c = b0 * batch + first; c - first < c1; c += 2 * batch) {
      load(c + batch, v1);
      finish(c, v0);
      load(c + 2 * batch, v0);
      finish(c + batch, v1);  // past the end: stores nothing
    }
  }
}

// Epilogue warps: the hidden rows' codes from their maxima, a warp per 512 columns of a row.
__device__ void code_hidden(const Params& p, const Tables& t) {
  const DecodeArgs& a = p.a;
  const int rows = t.c->first[t.c->active], pieces = (a.h + 511) / 512;
  const int warp = (threadIdx.x >> 5) - kEpiWarp0;
  for (int i = blockIdx.x + gridDim.x * warp; i < rows * pieces; i += gridDim.x * (kEpiThreads / 32)) {
    const int r = i / pieces, piece = i - r * pieces, c0 = piece * 512 + lane_id() * 8, c1 = c0 + 256;
    const __nv_bfloat16* src = p.hidden + static_cast<int64_t>(r) * a.h;
    uint8_t* dst = p.hq + static_cast<int64_t>(r) * a.terms * a.h;
    const uint32_t bits = __ldcg(p.amax + r);
    uint4 v0 = make_uint4(0, 0, 0, 0), v1 = v0;
    if (c0 < a.h) v0 = __ldcg(reinterpret_cast<const uint4*>(src + c0));
    if (c1 < a.h) v1 = __ldcg(reinterpret_cast<const uint4*>(src + c1));
    float s, m;
    coding::row_scale(a.terms, __uint_as_float(bits << 16), bits > 0x7F80u, bits >= 0x7F80u, s, m);
#pragma unroll 1
    for (int k = 0; k < 2; ++k) {
      const int col = k == 0 ? c0 : c1;
      if (col < a.h) coding::code_piece(k == 0 ? v0 : v1, dst, a.h, col, a.terms, s, m);
    }
    if (piece == 0 && lane_id() == 0) p.hs[r] = s;
  }
}

// The steps of one phase (32 bits: checked on the host), cut into `parts` ranges
// of about equal cost; this CTA's is [lo, hi).
struct Phase {
  int nk;     // steps of a tile (its K)
  int total;
  int parts;  // CTAs that have steps: every one of them at least one
  const int* begin;
  int lo, hi;

  __device__ __forceinline__ int begin_of(int c) const { return begin[c]; }
  // the CTA whose range holds step s
  __device__ __forceinline__ int part_of(int s) const {
    int a = 0, b = parts;  // begin[a] <= s < begin[b]
    while (b - a > 1) {
      const int m = (a + b) >> 1;
      if (begin[m] <= s)
        a = m;
      else
        b = m;
    }
    return a;
  }
  // ... and the last one of a tile's, from its first one
  __device__ __forceinline__ int last_part(int c, int s) const {
    while (begin[c + 1] <= s) ++c;
    return c;
  }
};

// Half of the threads: the ranges of a phase of `tiles` tiles per group, tile after
// tile within a group (up), or group after group within a tile (down).
__device__ void cut_phase(Ctl& c, int ph, int tiles, int nk, bool equal) {
  const int total = c.active * tiles * nk, parts = min(total, static_cast<int>(gridDim.x));
  const int weight = c.weight[c.active];
  for (int i = threadIdx.x % (kThreads / 2); i <= parts; i += kThreads / 2) {
    int s;
    if (equal || total < 4 * parts || i == parts) {
      // equal costs, or too few steps to weigh them (a range must not be empty): equal numbers, the longer ones first
      const int q = total / parts, r = total - q * parts;
      s = i * q + min(i, r);
    } else {
      // the first step that starts at or after this share of the cost; a range costs at least four average steps,
      // more than any one step
      const int64_t all = static_cast<int64_t>(weight) * tiles * nk;
      int64_t at = all * i / parts;
      const int64_t row = static_cast<int64_t>(weight) * nk;  // down: one tile, all groups
      int j = 0;
      if (ph == 1) {
        j = static_cast<int>(at / row);
        at -= j * row;
      }
      const int64_t unit = ph == 0 ? static_cast<int64_t>(tiles) * nk : nk;  // steps of a group in a row
      int lo = 0, hi = c.active;  // the group that holds the cost `at`
      while (hi - lo > 1) {
        const int m = (lo + hi) >> 1;
        if (c.weight[m] * unit <= at)
          lo = m;
        else
          hi = m;
      }
      const int w = c.weight[lo + 1] - c.weight[lo];
      const int64_t k = (at - c.weight[lo] * unit + w - 1) / w;
      s = ph == 0 ? static_cast<int>(lo * unit + k) : static_cast<int>((static_cast<int64_t>(j) * c.active + lo) * nk + k);
    }
    c.begin[ph][i] = s;
  }
}

__device__ __forceinline__ Phase phase_of(const Ctl& c, int ph, int tiles, int nk) {
  Phase f;
  f.nk = nk;
  f.total = c.active * tiles * nk;
  f.parts = min(f.total, static_cast<int>(gridDim.x));
  f.begin = c.begin[ph];
  const int i = min(static_cast<int>(blockIdx.x), f.parts);
  f.lo = f.begin[i];
  f.hi = i < f.parts ? f.begin[i + 1] : f.lo;
  return f;
}

// The part of one tile that lies in a range.
struct Unit {
  int tile, k0, k1;
};

__device__ __forceinline__ Unit unit_at(const Phase& f, int s) {
  Unit u;
  u.tile = s / f.nk;
  u.k0 = s - u.tile * f.nk;
  u.k1 = min(f.nk, u.k0 + f.hi - s);
  return u;
}

// Partial tile of CTA c with part of the steps from s0 on, element [tok][half *
// 128 + n]: 0 where the steps from s0 on began before its range, else 1.
__device__ __forceinline__ float* partial_of(const Params& p, const Phase& f, int c, int s0) {
  return p.partial + (static_cast<int64_t>(c) * 2 + (f.begin_of(c) > s0 ? 0 : 1)) * p.a.S * 256;
}

// The epilogue warps have written this CTA's part of an up tile that the CTAs
// c0 .. c1 share: true for all of them when it was the last one.
__device__ __forceinline__ bool join_last(const Params& p, const Tables& t, int c0, int c1) {
  epi_any(false);
  if (threadIdx.x == 32 * kEpiWarp0) {
    __threadfence();
    t.c->last = atomicAdd(p.joins + c0, 1) == static_cast<uint32_t>(c1 - c0);
    __threadfence();
  }
  epi_any(false);
  return t.c->last != 0;
}

// Ring position: stage and how often the ring has gone round.
struct Slot {
  int stage = 0;
  uint32_t round = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++stage == stages) {
      stage = 0;
      round ^= 1;
    }
  }
};

// Warp 0.  Weight tiles and token tiles have barriers of their own, so a stage's
// weights can be under way before its tokens exist.
struct Producer {
  const Params& p;
  const Tables& t;
  uint8_t* ring;
  Slot w, b;
  uint64_t hint;
  uint32_t armed_w = 0, armed_b = 0, round_w = 0, round_b = 0;  // barriers armed, and their last rounds

  __device__ Producer(const Params& p_, const Tables& t_, uint8_t* ring_)
      : p(p_), t(t_), ring(ring_), hint(p_.stream_weights ? l2_evict_first() : l2_evict_normal()) {}

  // Two weight tiles: rows n0 of slab `slab` of w0, and rows n1 of w1.
  __device__ bool weights(const CUtensorMap* w0, const CUtensorMap* w1, int k, int n0, int n1, int slab) {
    const int lane = lane_id();
    Ctl& c = *t.c;
    bool ok = true;
    if (lane == 0) ok = mbar_wait(&c.empty[w.stage], w.round ^ 1u, &c.abort);
    ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
    if (!ok) return false;
    uint8_t* st = ring + w.stage * p.stage_bytes;
    if (lane == 0) {
      mbar_arrive_expect_tx(&c.full_w[w.stage], 2 * kTileBytes);
      tma_load_3d_hint(st, w0, k, n0, slab, &c.full_w[w.stage], hint);
      tma_load_3d_hint(st + kTileBytes, w1, k, n1, slab, &c.full_w[w.stage], hint);
    }
    armed_w |= 1u << w.stage;
    round_w = (round_w & ~(1u << w.stage)) | (w.round << w.stage);
    w.next(p.stages);
    return true;
  }

  // Token tile: `boxes` boxes of 16 rows from `row` on.
  __device__ void tokens(const CUtensorMap* m, int k, int row, int boxes) {
    const int lane = lane_id();
    Ctl& c = *t.c;
    uint8_t* dst = ring + b.stage * p.stage_bytes + 2 * kTileBytes;
    if (lane == 0) mbar_arrive_expect_tx(&c.full_b[b.stage], boxes * 2048);
    __syncwarp();
    if (lane < boxes) tma_load_2d(dst + lane * 2048, m, k, row + 16 * lane, &c.full_b[b.stage]);
    arm_b();
  }

  __device__ __forceinline__ void arm_b() {
    armed_b |= 1u << b.stage;
    round_b = (round_b & ~(1u << b.stage)) | (b.round << b.stage);
    b.next(p.stages);
  }

  // Lets every copy in flight land (each barrier's last armed round).
  __device__ void settle() {
    if (lane_id() != 0) return;
    int never = 0;
    for (int i = 0; i < p.stages; ++i) {
      if (armed_w & (1u << i)) mbar_wait(&t.c->full_w[i], (round_w >> i) & 1u, &never);
      if (armed_b & (1u << i)) mbar_wait(&t.c->full_b[i], (round_b >> i) & 1u, &never);
    }
  }
};

__device__ __forceinline__ int up_tiles_of(const DecodeArgs& a) {
  return a.activation == MOE_ACT_SWIGLU ? (a.h + 127) / 128 : (a.h + 255) / 256;
}

__device__ void produce(const Params& p, const Tables& t, uint8_t* ring, const Phase& up, const Phase& down,
                        const CUtensorMap* m_in0, const CUtensorMap* m_in1, const CUtensorMap* m_out,
                        const CUtensorMap* m_x, const CUtensorMap* m_hidden) {
  const DecodeArgs& a = p.a;
  Ctl& c = *t.c;
  const int bk = a.terms ? 128 : 64, terms = a.terms == 2 ? 2 : 1;
  const bool pair = a.activation == MOE_ACT_SWIGLU, dense = all_tokens(a.S, a.terms);
  const int tiles = up_tiles_of(a);
  Producer pr(p, t, ring);
  bool ok = true;
  for (int s = up.lo; s < up.hi && ok;) {
    const Unit u = unit_at(up, s);
    const int g = u.tile / tiles, j = u.tile - g * tiles, slab = c.slab[g];
    const int n0 = pair ? j * 128 : j * 256, n1 = pair ? n0 : n0 + 128;
    const int row = dense ? 0 : c.first[g] * terms;
    const int boxes = dense ? 1 : ((c.first[g + 1] - c.first[g]) * terms + 15) / 16;
    for (int k = u.k0; k < u.k1; ++k) {
      if (!(ok = pr.weights(m_in0, m_in1, k * bk, n0, n1, slab))) break;
      pr.tokens(m_x, k * bk, row, boxes);
    }
    s += u.k1 - u.k0;
  }
  // down: the first `ahead` steps' weights go out before the hidden rows are known to be complete
  const int ahead = min(down.hi - down.lo, p.stages);
  for (int pass = 0; pass < 2 && ok; ++pass) {
    const int end = pass == 0 ? down.lo + ahead : down.hi;
    if (pass == 1) {
      if (lane_id() == 0) ok = wait_arrivals(p, a.terms ? kCoded : kHidden, &c.abort);
      ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
      fence_proxy_async_global();
    }
    int tile = down.lo / down.nk, k = down.lo - tile * down.nk;
    int j = tile / c.active, g = tile - j * c.active;
    for (int s = down.lo; s < end && ok; ++s) {
      if (pass == 0 || s >= down.lo + ahead)
        ok = pr.weights(m_out, m_out, k * bk, j * 256, j * 256 + 128, c.slab[g]);
      if (pass == 1 && ok)
        pr.tokens(m_hidden, k * bk, c.first[g] * terms, ((c.first[g + 1] - c.first[g]) * terms + 15) / 16);
      if (++k == down.nk) {
        k = 0;
        if (++g == c.active) {
          g = 0;
          ++j;
        }
      }
    }
  }
  if (!ok && lane_id() == 0) give_up(p, &c.abort);
  pr.settle();  // also where all went out: the MMA warp may give up before it has seen the last ones land
}

// TMEM columns of the units' accumulator pairs, one after another around the 512:
// the MMA thread and the epilogue warps follow the same sequence.  Small groups
// take few columns, so up to 16 units run ahead of the epilogue (while its warps
// are still at the adapters' products, above all).
struct AccRing {
  int tail = 0;
  __device__ __forceinline__ int take(int n) {  // n columns per tile
    const int at = tail + 2 * n > kTmemCols ? 0 : tail;
    tail = at + 2 * n;
    return at;
  }
};

// MMA columns of a group's token tile.
__device__ __forceinline__ int tile_cols(const Params& p, const Ctl& c, int ph, int g) {
  const int terms = p.a.terms == 2 ? 2 : 1;
  if (ph == 0 && all_tokens(p.a.S, p.a.terms)) return 16;
  return ((c.first[g + 1] - c.first[g]) * terms + 15) & ~15;
}

// Warp 1, one lane.
__device__ void multiply(const Params& p, const Tables& t, uint8_t* ring, const Phase& up, const Phase& down) {
  const DecodeArgs& a = p.a;
  Ctl& c = *t.c;
  const int tiles = up_tiles_of(a);
  Slot at;
  AccRing ring_cols;
  int local = 0, drained = 0;  // units issued, units whose accumulators the epilogue has read
  bool ok = true;
  for (int ph = 0; ph < 2 && ok; ++ph) {
    const Phase& f = ph == 0 ? up : down;
    for (int s = f.lo; s < f.hi && ok; ++local) {
      const Unit u = unit_at(f, s);
      const int g = ph == 0 ? u.tile / tiles : u.tile % c.active;
      const int n = tile_cols(p, c, ph, g);
      const uint32_t idesc = a.terms ? idesc_e4m3_f32(128, n) : idesc_bf16_f32(128, n);
      const int acc = local % kAccs, col = ring_cols.take(n);
      // the columns are free once every unit in flight that holds some of them has been read (oldest first)
      while (ok) {
        bool free = local - drained < kAccs;
        for (int o = drained; o < local && free; ++o)
          free = c.acc_end[o % kAccs] <= col || c.acc_begin[o % kAccs] >= col + 2 * n;
        if (free) break;
        ok = mbar_wait(&c.tempty[drained % kAccs], (drained / kAccs) & 1, &c.abort);
        ++drained;
      }
      if (!ok) break;
      c.acc_begin[acc] = col;
      c.acc_end[acc] = col + 2 * n;
      tc_fence_after();
      const uint32_t d0 = c.tmem_base + col, d1 = d0 + n;
      for (int k = u.k0; k < u.k1; ++k) {
        if (!(ok = mbar_wait(&c.full_w[at.stage], at.round, &c.abort))) break;
        if (!(ok = mbar_wait(&c.full_b[at.stage], at.round, &c.abort))) break;
        tc_fence_after();
        const uint32_t w = smem_u32(ring + at.stage * p.stage_bytes), b = w + 2 * kTileBytes;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const uint32_t on = (k > u.k0 || kk > 0) ? 1u : 0u;
          const uint64_t bd = smem_desc_sw128(b + kk * 32);
          if (a.terms) {
            tc_mma_f8(d0, smem_desc_sw128(w + kk * 32), bd, idesc, on);
            tc_mma_f8(d1, smem_desc_sw128(w + kTileBytes + kk * 32), bd, idesc, on);
          } else {
            tc_mma_f16(d0, smem_desc_sw128(w + kk * 32), bd, idesc, on);
            tc_mma_f16(d1, smem_desc_sw128(w + kTileBytes + kk * 32), bd, idesc, on);
          }
        }
        tc_commit(&c.empty[at.stage]);
        at.next(p.stages);
      }
      if (!ok) break;
      tc_commit(&c.tfull[acc]);
      s += u.k1 - u.k0;
    }
  }
  tc_commit(&c.drain);  // every MMA issued must finish before TMEM is released
  int never = 0;
  mbar_wait(&c.drain, 0, &never);
  if (!ok) give_up(p, &c.abort);
}

// Eight accumulator columns -> the sums of their tokens: 8, or 4 of two terms each.
template <int TERMS>
__device__ __forceinline__ void load_sums(uint32_t taddr, float (&v)[TERMS == 2 ? 4 : 8]) {
  uint32_t r[8];
  tmem_ld_32x32b_x8(taddr, r);
  tmem_ld_wait();
  if (TERMS == 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(r[2 * i]) + __uint_as_float(r[2 * i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < (TERMS == 2 ? 4 : 8); ++i) v[i] = __uint_as_float(r[i]);
  }
}

// Hidden value from a row's final sums v0, v1 (gate and up, or v0 alone): the
// row's scale rs and the column's cs0, cs1 (1 without E4M3 weights), the
// adapters' share d0, d1, bias, activation.  The quick division (off by two units
// in the last place; 0 where the sigmoid is below 2^-126) has no branches, so the
// rows of a chunk overlap.
template <bool PAIR>
__device__ __forceinline__ float hidden_value(float rs, float cs0, float cs1, float bias, float v0, float v1, float d0,
                                              float d1) {
  v0 = fmaf(v0, rs * cs0, d0);
  if (PAIR) {
    v1 = fmaf(v1, rs * cs1, d1);
    return __fdividef(v0, 1.0f + __expf(-v0)) * v1;
  }
  const float z = v0 + bias;
  return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
}

// One hidden element of a tile: tile column `n` (0..127) of half `m`.
__device__ __forceinline__ int hidden_col(bool pair, int j, int m, int n) { return pair ? j * 128 + n : j * 256 + m * 128 + n; }

// Hidden rows of a CTA's tiles.  The 8 columns that a warp reads from its
// accumulators at once are the chunk of rows that it finishes at once: every step
// runs over the whole chunk before the next one, because two warps per scheduler
// hide little of one row's chain of instructions.  A cut tile's parts meet in the
// CTA that comes last: mostly it finds the others' parts complete when it starts on
// its own and adds them to the sums in its registers; else all parts go through
// memory.  Either way they are added in CTA order.
template <bool PAIR, int TERMS>
__device__ bool epilogue_up(const Params& p, const Tables& t, const Phase& f, int& local, AccRing& cols_ring) {
  const DecodeArgs& a = p.a;
  Ctl& c = *t.c;
  constexpr int kPer = TERMS == 2 ? 4 : 8;  // rows of a chunk
  const int warp = threadIdx.x >> 5, lane = lane_id(), q = warp & 3, half = (warp - kEpiWarp0) >> 2;
  const bool dense = all_tokens(a.S, TERMS);
  const int tiles = up_tiles_of(a);
  const int nl = q * 32 + lane;
  const bool outer = a.lora.n > 0 && (a.lora.a[0] != nullptr || a.lora.a[1] != nullptr);
  bool outer_ready = !outer;
  for (int s = f.lo; s < f.hi; ++local) {
    const Unit u = unit_at(f, s);
    s += u.k1 - u.k0;
    const int g = u.tile / tiles, j = u.tile - g * tiles, slab = c.slab[g];
    const int row0 = c.first[g], cnt = c.first[g + 1] - row0;
    const bool whole = u.k0 == 0 && u.k1 == f.nk;
    const int s0 = u.tile * f.nk;
    const int c0 = whole ? 0 : f.part_of(s0), c1 = whole ? 0 : f.last_part(c0, s0 + f.nk - 1);
    float* part = partial_of(p, f, blockIdx.x, s0);
    if (!outer_ready) {
      if (!epi_wait(p, kOuterUp, &c.abort)) return false;
      outer_ready = true;
    }
    const int n = hidden_col(PAIR, j, half, nl);
    const bool in = n < a.h;
    float cs0 = 1.0f, cs1 = 1.0f, bias = 0.0f;  // the column's scales or bias, loaded while the sums are made
    if (in) {
      const int64_t ch = static_cast<int64_t>(slab) * a.h + n;
      if (TERMS) {
        cs0 = __ldg(a.s_in[0] + ch);
        cs1 = __ldg(a.s_in[1] + ch);
      }
      if (!PAIR) bias = __ldg(a.b_in + ch);
    }
    const int acc = local % kAccs, acc_n = tile_cols(p, c, 0, g), acc_col = cols_ring.take(acc_n);
    int& all_there = c.others_done[local & 1];  // (two: a slow warp may still look at the unit before)
    if (threadIdx.x == 32 * kEpiWarp0)
      all_there = !whole && ld_acquire(p.joins + c0) == static_cast<uint32_t>(c1 - c0);
    const bool failed = !mbar_wait(&c.tfull[acc], (local / kAccs) & 1, &c.abort);
    if (epi_any(failed)) {
      if (threadIdx.x == 32 * kEpiWarp0) give_up(p, &c.abort);
      return false;
    }
    tc_fence_after();
    const bool complete = whole || all_there;
    const uint32_t tb = c.tmem_base + acc_col + (static_cast<uint32_t>(q * 32) << 16);
    const uint64_t mask = c.mask[g];
    const int cols = dense ? a.S : cnt;  // tokens in the tile's columns
    // the adapters' share of the rows r, and their hidden values from complete sums
    auto shares = [&](const int (&r)[kPer], float (&d0)[kPer], float (&d1)[kPer]) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        d0[i] = d1[i] = 0.0f;
        if (outer && in && r[i] >= 0 && c.adapter[t.row_tok[r[i]]] >= 0) {
          const float* d = p.d_in + static_cast<int64_t>(r[i]) * 2 * a.h + n;
          d0[i] = __ldcg(d + (PAIR ? 0 : a.h));
          if (PAIR) d1[i] = __ldcg(d + a.h);
        }
      }
    };
    auto finish = [&](const int (&r)[kPer], const float (&v0)[kPer], const float (&v1)[kPer], const float (&d0)[kPer],
                      const float (&d1)[kPer]) {
      __nv_bfloat16 hv[kPer];
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        hv[i] = __float2bfloat16_rn(hidden_value<PAIR>(TERMS && r[i] >= 0 ? t.row_scale[r[i]] : 1.0f, cs0, cs1, bias,
                                                       v0[i], PAIR ? v1[i] : 0.0f, d0[i], d1[i]));
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (in && r[i] >= 0) p.hidden[static_cast<int64_t>(r[i]) * a.h + n] = hv[i];
      if (TERMS) {  // the rows' maxima: lane i raises that of row r[i]
        uint32_t top = 0;
        int at = -1;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, in ? __bfloat16_as_ushort(hv[i]) & 0x7FFFu : 0u);
          if (lane == i) {
            top = m;
            at = r[i];
          }
        }
        if (at >= 0) atomicMax(p.amax + at, top);
      }
    };
    // v0, v1 become the sums over the parts c0 .. c1 in that order, this CTA's own from v0, v1 (own) or from memory as
    // well; kBatch parts' loads are in flight together
    auto add_parts = [&](const int (&r)[kPer], bool own, float (&v0)[kPer], float (&v1)[kPer]) {
      constexpr int kBatch = PAIR && TERMS != 2 ? 2 : 4;
      float sum0[kPer], sum1[kPer];
#pragma unroll
      for (int i = 0; i < kPer; ++i) sum0[i] = sum1[i] = 0.0f;
      for (int cc = c0; cc <= c1; cc += kBatch) {
        float q0[kBatch][kPer], q1[kBatch][kPer];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          const bool mine = own && cc + b == static_cast<int>(blockIdx.x), load = cc + b <= c1 && !mine;
          const float* src = partial_of(p, f, min(cc + b, c1), s0) + nl + (PAIR ? 0 : half * 128);
#pragma unroll
          for (int i = 0; i < kPer; ++i) {
            q0[b][i] = mine ? v0[i] : 0.0f;
            if (load && r[i] >= 0) q0[b][i] = __ldcg(src + (r[i] - row0) * 256);
            if (PAIR) {
              q1[b][i] = mine ? v1[i] : 0.0f;
              if (load && r[i] >= 0) q1[b][i] = __ldcg(src + (r[i] - row0) * 256 + 128);
            }
          }
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
#pragma unroll
          for (int i = 0; i < kPer; ++i) {
            sum0[i] += q0[b][i];
            if (PAIR) sum1[i] += q1[b][i];
          }
      }
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        v0[i] = sum0[i];
        if (PAIR) v1[i] = sum1[i];
      }
    };
    // SwiGLU: the two halves of the warps take alternate chunks of columns, both tiles; else one tile each
    for (int ch = PAIR ? half : 0; ch * kPer < cols; ch += PAIR ? 2 : 1) {
      float v0[kPer], v1[kPer], d0[kPer], d1[kPer];
      int r[kPer];  // the columns' rows (-1: none)
      uint32_t some = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int col = ch * kPer + i;
        r[i] = col < cols ? row0 + col : -1;
        if (dense) r[i] = col < cols && ((mask >> col) & 1) ? row0 + __popcll(mask & ((uint64_t(1) << col) - 1)) : -1;
        some |= r[i] >= 0;
      }
      if (!some) continue;
      if (complete) shares(r, d0, d1);
      load_sums<TERMS>(tb + (PAIR ? 0 : half * acc_n) + ch * 8, v0);
      if (PAIR) load_sums<TERMS>(tb + acc_n + ch * 8, v1);
      if (!complete) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          if (r[i] < 0) continue;
          float* o = part + (r[i] - row0) * 256 + nl;
          o[PAIR ? 0 : half * 128] = v0[i];
          if (PAIR) o[128] = v1[i];
        }
        continue;
      }
      if (!whole) add_parts(r, true, v0, v1);
      finish(r, v0, v1, d0, d1);
    }
    tc_fence_before();
    mbar_arrive(&c.tempty[acc]);
    if (complete || !join_last(p, t, c0, c1)) continue;
    const int step = PAIR ? 2 * kPer : kPer;
    for (int i0 = PAIR ? half * kPer : 0; i0 < cnt; i0 += step) {
      float v0[kPer], v1[kPer], d0[kPer], d1[kPer];
      int r[kPer];
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        r[i] = i0 + i < cnt ? row0 + i0 + i : -1;
        v0[i] = v1[i] = 0.0f;  // (this CTA's part comes from memory too)
      }
      shares(r, d0, d1);
      add_parts(r, false, v0, v1);
      finish(r, v0, v1, d0, d1);
    }
  }
  return true;
}

template <int TERMS>
__device__ bool epilogue_down(const Params& p, const Tables& t, const Phase& f, int& local, AccRing& cols_ring) {
  const DecodeArgs& a = p.a;
  Ctl& c = *t.c;
  const int warp = threadIdx.x >> 5, lane = lane_id(), q = warp & 3, half = (warp - kEpiWarp0) >> 2;
  constexpr int kPer = TERMS == 2 ? 4 : 8;    // rows of a chunk
  const int nl = half * 128 + q * 32 + lane;  // this thread's column of the tile
  const bool outer = a.lora.n > 0 && a.lora.a[2] != nullptr;
  bool outer_ready = !outer;
  for (int s = f.lo; s < f.hi; ++local) {
    const Unit u = unit_at(f, s);
    s += u.k1 - u.k0;
    const int j = u.tile / c.active, g = u.tile - j * c.active, slab = c.slab[g];
    const int row0 = c.first[g], cnt = c.first[g + 1] - row0, n = j * 256 + nl;
    const bool in = n < a.d, whole = u.k0 == 0 && u.k1 == f.nk, first = u.k0 == 0;
    if (!outer_ready && first) {  // the tile's first steps take the adapters' share
      if (!epi_wait(p, kOuterDown, &c.abort)) return false;
      outer_ready = true;
    }
    const int64_t och = static_cast<int64_t>(slab) * a.d + n;
    const float cs = TERMS && in ? __ldg(a.s_out + och) : 1.0f;
    const float bias = a.b_out != nullptr && in && first ? __ldg(a.b_out + och) : 0.0f;
    const int acc = local % kAccs, acc_n = tile_cols(p, c, 1, g), acc_col = cols_ring.take(acc_n);
    const bool failed = !mbar_wait(&c.tfull[acc], (local / kAccs) & 1, &c.abort);
    if (epi_any(failed)) {
      if (threadIdx.x == 32 * kEpiWarp0) give_up(p, &c.abort);
      return false;
    }
    tc_fence_after();
    const uint32_t tb = c.tmem_base + acc_col + half * acc_n + (static_cast<uint32_t>(q * 32) << 16);
    // a whole tile's sums are the expert's outputs, a part's are added up at the end
    float* dst = whole ? p.outs + static_cast<int64_t>(row0) * a.d + n
                       : partial_of(p, f, blockIdx.x, u.tile * f.nk) + nl;
    const int64_t stride = whole ? a.d : 256;
    for (int ch = 0; ch * kPer < cnt; ++ch) {
      float v[kPer], dd[kPer];
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int tk = ch * kPer + i;
        dd[i] = bias;
        if (tk < cnt && outer && first && in && c.adapter[t.row_tok[row0 + tk]] >= 0)
          dd[i] += __ldcg(p.d_out + static_cast<int64_t>(row0 + tk) * a.d + n);
      }
      load_sums<TERMS>(tb + ch * 8, v);
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int tk = ch * kPer + i;
        if (tk < cnt && in) dst[tk * stride] = TERMS ? fmaf(v[i], t.row_scale[row0 + tk] * cs, dd[i]) : v[i] + dd[i];
      }
    }
    tc_fence_before();
    mbar_arrive(&c.tempty[acc]);
  }
  return true;
}

// Each down tile's first CTA and how many more hold parts of it, into shared memory
// (the ring, idle once this CTA's own products are done).
__device__ void list_parts(const Phase& f, uchar2* parts) {
  for (int i = threadIdx.x - 32 * kEpiWarp0; i < f.total / f.nk; i += kEpiThreads) {
    const int c0 = f.part_of(i * f.nk);
    parts[i] = make_uchar2(c0, f.last_part(c0, i * f.nk + f.nk - 1) - c0);
  }
}

// y[t] = sum_k gate_k * expert output of its k-th row (+ the shared expert's), four
// columns per thread of the grid: whole tiles' outputs, or the parts of a cut tile
// in CTA order, four parts' loads in flight together.
__device__ void combine(const Params& p, const Tables& t, const Phase& f, const uchar2* parts) {
  const DecodeArgs& a = p.a;
  const Ctl& c = *t.c;
  const int quads = a.d / 4, slots = a.S * a.K, tid = threadIdx.x - 32 * kEpiWarp0;
  auto* y = static_cast<__nv_bfloat16*>(a.y);
  for (int i = blockIdx.x * kEpiThreads + tid; i < a.S * quads; i += gridDim.x * kEpiThreads) {
    const int tk = i / quads, n = (i - tk * quads) * 4, j = n / 256;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int k = 0; k < a.K + a.num_shared; ++k) {
      const int r = k < a.K ? t.slot_row[tk * a.K + k] : slots + tk;
      const int g = t.row_grp[r], tile = j * c.active + g;
      const uchar2 pt = parts[tile];
      const float gate = t.row_gate[r];
      const int64_t at = static_cast<int64_t>(r - c.first[g]) * 256 + n % 256;
      const float* src = pt.y == 0 ? p.outs + static_cast<int64_t>(r) * a.d + n : partial_of(p, f, pt.x, tile * f.nk) + at;
      float4 o = __ldcg(reinterpret_cast<const float4*>(src));
      for (int cc = 1; cc <= pt.y; cc += 4) {
        float4 q[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          q[b] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (cc + b <= pt.y)
            q[b] = __ldcg(reinterpret_cast<const float4*>(partial_of(p, f, pt.x + cc + b, tile * f.nk) + at));
        }
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          o.x += q[b].x;
          o.y += q[b].y;
          o.z += q[b].z;
          o.w += q[b].w;
        }
      }
      v.x = fmaf(gate, o.x, v.x);
      v.y = fmaf(gate, o.y, v.y);
      v.z = fmaf(gate, o.z, v.z);
      v.w = fmaf(gate, o.w, v.w);
    }
    *reinterpret_cast<uint2*>(y + static_cast<int64_t>(tk) * a.d + n) =
        make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
  }
}

// Warps 2 .. 11: the adapters' share of a phase; false when a wait gave up.  (33
// tokens with 32 adapters of rank 64 over fine E4M3 experts: 233 us; 242 with the
// epilogue's eight warps alone, or with one copy of this code that is called.)
__device__ __forceinline__ bool adapter_products(const Params& p, const Tables& t, int m0, int nm, Arrival inner, Arrival outer) {
  adapter_inner(p, t, m0, nm);
  epi_arrive<kLoraWarp0>(p, inner);
  if (!epi_wait<kLoraWarp0>(p, inner, &t.c->abort)) return false;
  adapter_outer(p, t, m0, nm);
  epi_arrive<kLoraWarp0>(p, outer);
  return true;
}

// Warps 4 .. 11; with adapters also warps 2 and 3, which help with their products.
template <bool PAIR, int TERMS>
__device__ void epilogue(const Params& p, const Tables& t, const Phase& up, const Phase& down, uint8_t* ring) {
  const DecodeArgs& a = p.a;
  Ctl& c = *t.c;
  int local = 0;
  AccRing cols;
  const bool inner_up = a.lora.n > 0 && (a.lora.a[0] != nullptr || a.lora.a[1] != nullptr);
  const bool inner_down = a.lora.n > 0 && a.lora.a[2] != nullptr;
  const bool helper = threadIdx.x < 32 * kEpiWarp0;
  if (inner_up && !adapter_products(p, t, 0, 2, kInnerUp, kOuterUp)) return;
  bool ok = true;
  if (!helper) {
    ok = epilogue_up<PAIR, TERMS>(p, t, up, local, cols);
    if (ok) epi_arrive(p, kHidden);
    if (ok && (TERMS || inner_down)) ok = epi_wait(p, kHidden, &c.abort);
  }
  // (the helpers wait here for the hidden rows, and learn it if there will be none)
  if (inner_down ? any_of<kLoraWarp0>(!ok) : !ok) return;
  if (!helper && TERMS) {
    code_hidden(p, t);
    epi_arrive(p, kCoded);
  }
  if (inner_down && !adapter_products(p, t, 2, 1, kInnerDown, kOuterDown)) return;
  if (helper) return;
  if (TERMS) {  // the hidden rows' scales
    if (!epi_wait(p, kCoded, &c.abort)) return;
    for (int r = threadIdx.x - 32 * kEpiWarp0; r < c.first[c.active]; r += kEpiThreads) t.row_scale[r] = __ldcg(p.hs + r);
    epi_any(false);
  }
  if (!epilogue_down<TERMS>(p, t, down, local, cols)) return;
  epi_arrive(p, kSummed);
  auto* parts = reinterpret_cast<uchar2*>(ring);
  list_parts(down, parts);
  if (!epi_wait(p, kSummed, &c.abort)) return;  // (its barrier also closes the table)
  combine(p, t, down, parts);
}

__global__ void __launch_bounds__(kThreads, 1)
    decode_kernel(const __grid_constant__ CUtensorMap m_in0, const __grid_constant__ CUtensorMap m_in1,
                  const __grid_constant__ CUtensorMap m_out, const __grid_constant__ CUtensorMap m_x,
                  const __grid_constant__ CUtensorMap m_hidden, const __grid_constant__ Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const DecodeArgs& a = p.a;
  Tables t;
  uint8_t* at = ring + p.ring_bytes;
  t.c = reinterpret_cast<Ctl*>(at);
  t.scratch = reinterpret_cast<Scratch*>(ring);
  at += (sizeof(Ctl) + 15) & ~size_t(15);
  const int rows = a.S * (a.K + a.num_shared);
  t.row_gate = reinterpret_cast<float*>(at);
  t.row_scale = t.row_gate + rows;
  t.row_tok = reinterpret_cast<uint16_t*>(t.row_scale + rows);
  t.row_grp = t.row_tok + rows;
  t.slot_row = t.row_grp + rows;
  Ctl& c = *t.c;
  const int warp = threadIdx.x >> 5;
  if (warp == 1) {
    if (lane_id() == 0) {
      for (int i = 0; i < p.stages; ++i) {
        mbar_init(&c.full_w[i], 1);
        mbar_init(&c.full_b[i], 1);
        mbar_init(&c.empty[i], 1);
      }
      for (int i = 0; i < kAccs; ++i) {
        mbar_init(&c.tfull[i], 1);
        mbar_init(&c.tempty[i], kEpiThreads);
      }
      mbar_init(&c.drain, 1);
      c.abort = 0;
      fence_mbar_init();
    }
    __syncwarp();
    tmem_alloc(&c.tmem_base, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  route_phase(p, *t.scratch);
  if (grid_barrier(p, c, kRouted) && tables_phase(p, t)) {
    const bool pair = a.activation == MOE_ACT_SWIGLU;
    const int bk = a.terms ? 128 : 64;
    const int up_nk = (a.d + bk - 1) / bk, down_nk = (a.h + bk - 1) / bk;
    const bool equal = all_tokens(a.S, a.terms);
    const int ph = threadIdx.x >= kThreads / 2;
    cut_phase(c, ph, ph == 0 ? up_tiles_of(a) : (a.d + 255) / 256, ph == 0 ? up_nk : down_nk, equal);
    __syncthreads();
    const Phase up = phase_of(c, 0, up_tiles_of(a), up_nk);
    const Phase down = phase_of(c, 1, (a.d + 255) / 256, down_nk);
    if (warp == 0 && !p.test_stall)
      produce(p, t, ring, up, down, &m_in0, pair ? &m_in1 : &m_in0, &m_out, &m_x, &m_hidden);
    else if (warp == 1 && lane_id() == 0)
      multiply(p, t, ring, up, down);
    else if (warp >= (a.lora.n > 0 ? kLoraWarp0 : kEpiWarp0)) {
      if (a.terms == 2)
        epilogue<true, 2>(p, t, up, down, ring);
      else if (a.terms == 1)
        epilogue<true, 1>(p, t, up, down, ring);
      else if (pair)
        epilogue<true, 0>(p, t, up, down, ring);
      else
        epilogue<false, 0>(p, t, up, down, ring);
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(c.tmem_base, kTmemCols);
  }
  leave(p);
}

}  // namespace

size_t decode_workspace_bytes(int S, int d, int E, int K, int h, int num_shared, int terms, int lora_rank) {
  return ws_layout(S, d, E, K, h, num_shared, terms, lora_rank).total;
}

namespace {

// Bytes of a stage: two weight tiles, then the columns of the largest possible group.
int stage_bytes_of(int S, int terms) { return 2 * kTileBytes + ((S * (terms == 2 ? 2 : 1) + 15) & ~15) * 128; }

int stages_of(int S, int K, int ns, int terms) {
  const size_t room = kSmemLimit - 1024 - tables_bytes(S, K, ns);
  return std::min<int>(kMaxStages, static_cast<int>(room / stage_bytes_of(S, terms)));
}

}  // namespace

bool decode_supported(int S, int d, int E, int K, int h, int num_shared, int terms) {
  if (S <= 0) return true;
  const int stages = stages_of(S, K, num_shared, terms);
  const int64_t ring = static_cast<int64_t>(stages) * stage_bytes_of(S, terms);
  if (stages < 2 || ring < static_cast<int64_t>(sizeof(Scratch))) return false;
  // steps and tiles are counted in 32 bits; the combine's table of tiles lies in the ring
  const int64_t bk = terms ? 128 : 64, groups = std::min<int64_t>(E, static_cast<int64_t>(S) * K) + num_shared;
  const int64_t up = groups * ((h + 127) / 128) * ((d + bk - 1) / bk), down = groups * ((d + 255) / 256) * ((h + bk - 1) / bk);
  return up <= (1 << 30) && down <= (1 << 30) && 2 * groups * ((d + 255) / 256) <= ring;
}

#ifdef MOE_B200_TEST_HOOKS
// Failure-detection test hook (the test build only): the next n launches run
// with a producer that delivers nothing, so their waits give up.
namespace {
int g_stall_decode = 0;
}
extern "C" void moe_test_stall_decode(int n) { g_stall_decode = n > 0 ? n : 0; }
#endif

cudaError_t launch_decode(const DecodeArgs& a, cudaStream_t stream) {
  static std::atomic<uint64_t> attr_set{0};  // one bit per device ordinal (host threads may launch concurrently)
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(attr_set.load(std::memory_order_relaxed) & (1ull << dev))) {
    e = cudaFuncSetAttribute(decode_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmemLimit));
    if (e != cudaSuccess) return e;
    if (dev < 64) attr_set.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  const Ws L = ws_layout(a.S, a.d, a.E, a.K, a.h, a.num_shared, a.terms, a.lora.n > 0 ? a.lora.r : 0);
  char* ws = static_cast<char*>(a.ws);
  Params p;
  p.a = a;
  p.logits = reinterpret_cast<double*>(ws + L.logits);
  p.idx = reinterpret_cast<int*>(ws + L.idx);
  p.gate = reinterpret_cast<float*>(ws + L.gate);
  p.xq = reinterpret_cast<uint8_t*>(ws + L.xq);
  p.xs = reinterpret_cast<float*>(ws + L.xs);
  p.xp = reinterpret_cast<uint8_t*>(ws + L.xp);
  p.hidden = reinterpret_cast<__nv_bfloat16*>(ws + L.hidden);
  p.amax = reinterpret_cast<uint32_t*>(ws + L.amax);
  p.hq = reinterpret_cast<uint8_t*>(ws + L.hq);
  p.hs = reinterpret_cast<float*>(ws + L.hs);
  p.u_in = reinterpret_cast<float*>(ws + L.u_in);
  p.u_out = reinterpret_cast<float*>(ws + L.u_out);
  p.d_in = reinterpret_cast<float*>(ws + L.d_in);
  p.d_out = reinterpret_cast<float*>(ws + L.d_out);
  p.outs = reinterpret_cast<float*>(ws + L.outs);
  p.joins = reinterpret_cast<uint32_t*>(ws + L.joins);
  p.partial = reinterpret_cast<float*>(ws + L.partial);
  p.status = reinterpret_cast<StatusBlock*>(ws);
  p.sync = reinterpret_cast<GridSync*>(ws + kSyncOffset);
  const int terms = a.terms == 2 ? 2 : 1, eb = a.terms ? 1 : 2;
  if (!decode_supported(a.S, a.d, a.E, a.K, a.h, a.num_shared, a.terms)) return cudaErrorInvalidValue;
  const size_t fixed = 1024 + tables_bytes(a.S, a.K, a.num_shared);
  p.stage_bytes = stage_bytes_of(a.S, a.terms);
  p.stages = stages_of(a.S, a.K, a.num_shared, a.terms);
  p.ring_bytes = p.stages * p.stage_bytes;
  p.test_stall = 0;
#ifdef MOE_B200_TEST_HOOKS
  if (g_stall_decode > 0) {
    --g_stall_decode;
    p.test_stall = 1;
  }
#endif
  const int slabs = a.E + a.num_shared;
  const int64_t rows = static_cast<int64_t>(a.S) * (a.K + a.num_shared);
  CUtensorMap in0, in1, out, mx, mh;
  if (!gemm::make_slab_map(&in0, a.w_in[0], slabs, a.h, a.d, eb) || !gemm::make_slab_map(&out, a.w_out, slabs, a.d, a.h, eb))
    return cudaErrorInvalidValue;
  in1 = in0;
  if (a.w_in[1] != nullptr && !gemm::make_slab_map(&in1, a.w_in[1], slabs, a.h, a.d, eb)) return cudaErrorInvalidValue;
  // token rows: all of x (or its codes), or the rows copied group by group; boxes of 16 rows
  const bool dense = all_tokens(a.S, a.terms);
  const void* xrows = !dense ? p.xp : a.terms ? static_cast<const void*>(p.xq) : a.x;
  if (!gemm::make_map(&mx, xrows, (dense ? a.S : rows) * terms, a.d, 16, eb) ||
      !gemm::make_map(&mh, a.terms ? static_cast<const void*>(p.hq) : p.hidden, rows * terms, a.h, 16, eb))
    return cudaErrorInvalidValue;
  // Each weight byte is read once per call.  Where the touched experts exceed half of the 126 MB L2, their lines are
  // marked to leave first, which keeps the kernel's code, the router weights and the activations there between calls;
  // a smaller layer may find its weights in L2 the next time.
  const int64_t touched = std::min<int64_t>(a.E, static_cast<int64_t>(a.S) * a.K) + a.num_shared;
  const int mats = a.activation == MOE_ACT_SWIGLU ? 3 : 2;
  p.stream_weights = touched * mats * a.h * a.d * eb > (int64_t(63) << 20);
  const int grid = a.num_sms < kDecodeMaxCtas ? a.num_sms : kDecodeMaxCtas;
  void* args[] = {&in0, &in1, &out, &mx, &mh, &p};
  return cudaLaunchCooperativeKernel(reinterpret_cast<void*>(decode_kernel), dim3(grid), dim3(kThreads), args,
                                     p.ring_bytes + fixed, stream);
}

}  // namespace moe
