// Low-rank adapters of many requests beside the grouped expert projections:
// per row (token t, expert e, adapter a)
//   u = A[a][e] row            r values
//   delta = scale[a] B[a][e] u added to the projection's fp32 sums by the
//                              grouped GEMM's epilogue
// A warp per inner product, a thread per output element.
#include "common.cuh"
#include "gemm_common.cuh"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kRows = 64;  // rows per work unit
constexpr int kThreads = 256;

struct Smem {
  int start[gemm::kMaxGroups + 1];
  int ad[kRows];
};

// Exclusive prefix of the groups' tiles (of kRows rows) by warp 0.
__device__ void tile_starts(const LoraRowsArgs& a, Smem& s) {
  if (threadIdx.x < 32) {
    const int lane = lane_id();
    int carry = 0;
    for (int base = 0; base < a.num_groups; base += 32) {
      const int g = base + lane;
      int tiles = 0;
      if (g < a.num_groups) {
        const GroupEntry ge = a.groups[g];
        const bool ok = ge.rows > 0 && ge.expert >= 0 && ge.expert < a.slabs && ge.out_row0 >= 0 &&
                        static_cast<int64_t>(ge.out_row0) + ge.rows <= a.rows;
        tiles = ok ? (ge.rows + kRows - 1) / kRows : 0;
      }
      int incl = tiles;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, incl, off);
        if (lane >= off) incl += o;
      }
      if (g < a.num_groups) s.start[g] = carry + incl - tiles;
      carry += __shfl_sync(0xFFFFFFFFu, incl, 31);
    }
    if (lane == 0) s.start[a.num_groups] = carry;
  }
  __syncthreads();
}

__global__ void __launch_bounds__(kThreads) lora_rows_kernel(const LoraRowsArgs a, int outer) {
  __shared__ Smem s;
  tile_starts(a, s);
  const int tiles = s.start[a.num_groups];
  const int warp = threadIdx.x >> 5, lane = lane_id(), r = a.lora.r;
  for (int tt = blockIdx.x; tt < tiles; tt += gridDim.x) {
    int lo = 0, hi = a.num_groups;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s.start[mid] <= tt)
        lo = mid;
      else
        hi = mid;
    }
    const GroupEntry ge = a.groups[lo];
    const int i0 = (tt - s.start[lo]) * kRows, n = min(kRows, ge.rows - i0);
    const bool shared = ge.expert == a.shared_slab;
    __syncthreads();
    if (threadIdx.x < n) {
      const int i = i0 + threadIdx.x;
      const int token = shared ? i : a.token_of_row[ge.out_row0 + i];
      int id = -1;
      if (token >= 0 && token < a.S) id = a.lora.ids[token];
      if (id < -1 || id >= a.lora.n) {
        report(a.status, MOE_STATUS_BAD_ADAPTER, -1);
        id = -1;
      }
      s.ad[threadIdx.x] = id;
    }
    __syncthreads();
    if (!outer) {
      for (int j = warp; j < n * a.pairs * r; j += kThreads / 32) {
        const int q = j % r, m = (j / r) % a.pairs, i = j / (r * a.pairs);
        const int id = s.ad[i];
        if (id < 0 || a.lora.a[a.m0 + m] == nullptr) continue;
        const int64_t row = ge.out_row0 + i0 + i;
        const auto* w = static_cast<const __nv_bfloat16*>(a.lora.a[a.m0 + m]) +
                        ((static_cast<int64_t>(id) * a.slabs + ge.expert) * r + q) * a.K;
        const __nv_bfloat16* x;
        if (shared && a.src_shared != nullptr)
          x = static_cast<const __nv_bfloat16*>(a.src_shared) + static_cast<int64_t>(i0 + i) * a.K;
        else
          x = static_cast<const __nv_bfloat16*>(a.src) + (a.src_by_token ? a.token_of_row[row] : row) * a.K;
        float acc = 0.0f;
        for (int c = lane * 8; c < a.K; c += 256) {
          float wf[8], xf[8];
          unpack16<__nv_bfloat16>(ldg16(w + c), wf);
          unpack16<__nv_bfloat16>(ldg16(x + c), xf);
#pragma unroll
          for (int k = 0; k < 8; ++k) acc = fmaf(wf[k], xf[k], acc);
        }
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) acc += __shfl_xor_sync(0xFFFFFFFFu, acc, off);
        if (lane == 0)
          static_cast<__nv_bfloat16*>(a.u)[(row * a.pairs + m) * r + q] = __float2bfloat16_rn(acc);
      }
    } else {
      const int cols = a.pairs * a.N;
      for (int64_t j = threadIdx.x; j < static_cast<int64_t>(n) * cols; j += kThreads) {
        const int i = static_cast<int>(j / cols), c = static_cast<int>(j % cols), m = c / a.N, col = c % a.N;
        const int id = s.ad[i];
        const int64_t row = ge.out_row0 + i0 + i;
        float acc = 0.0f;
        if (id >= 0 && a.lora.b[a.m0 + m] != nullptr) {
          const auto* b = static_cast<const __nv_bfloat16*>(a.lora.b[a.m0 + m]) +
                          ((static_cast<int64_t>(id) * a.slabs + ge.expert) * a.N + col) * r;
          const auto* u = static_cast<const __nv_bfloat16*>(a.u) + (row * a.pairs + m) * r;
          for (int k = 0; k < r; ++k) acc = fmaf(to_f32(b[k]), to_f32(u[k]), acc);
          acc *= a.lora.scale[id];
        }
        static_cast<__nv_bfloat16*>(a.delta)[row * cols + c] = __float2bfloat16_rn(acc);
      }
    }
  }
}

}  // namespace

cudaError_t launch_lora_rows(const LoraRowsArgs& a, cudaStream_t stream) {
  if (a.num_groups <= 0 || a.num_groups > gemm::kMaxGroups) return cudaErrorInvalidValue;
  const int64_t bound = a.max_total_rows / kRows + a.num_groups;
  const int64_t cap = static_cast<int64_t>(a.num_sms) * 8;
  const dim3 grid(static_cast<unsigned>(bound < cap ? bound : cap));
  for (int outer = 0; outer < 2; ++outer) {
    lora_rows_kernel<<<grid, kThreads, 0, stream>>>(a, outer);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace moe
