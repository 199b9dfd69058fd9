// Low-rank adapters of many requests beside the grouped expert projections:
// per row (token t, expert e, adapter a)
//   u = A[a][e] row                r values
//   delta = scale[a] B[a][e] u     added to the projection's fp32 sums by the
//                                  grouped GEMM's epilogue
// Requests share the experts, not the adapters, so the rows are first sorted by
// (expert, adapter) into tiles of up to 64 rows that share one pair of adapter
// matrices (lora_plan_kernel, once per call).  A tile's products then run on
// m16n8k16 tensor-core instructions: both are bound by memory (the rows are
// read once, the deltas written once, and an adapter's matrices are read once
// per tile), and r = 8 .. 128 columns would leave most of a tcgen05 tile empty.
//
// Operand fragments are loaded straight from global memory, 16 (inner) or 8
// (outer) bytes per lane: a product's sum over k does not depend on the order
// of k, so lane quad q takes 8 (4) neighbouring k for the fragment slots that
// the instruction gives it, the same for both operands.
#include "common.cuh"
#include "gemm_common.cuh"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kRows = kLoraTileRows;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPlanThreads = 1024;

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Exclusive prefix of v over the block's threads, and the total.
__device__ int block_prefix(int v, int* warp_sums, int* total) {
  const int lane = lane_id(), warp = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o = __shfl_up_sync(0xFFFFFFFFu, incl, off);
    if (lane >= off) incl += o;
  }
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  int before = incl - v, all = 0;
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    if (w < warp) before += warp_sums[w];
    all += warp_sums[w];
  }
  *total = all;
  __syncthreads();
  return before;
}

// One CTA per group: counts its rows by adapter, lays the adapters' rows out one
// after another and cuts them into tiles.  Where a group's tiles and list
// entries lie, and the order of an adapter's rows, depend on timing; no result
// does (a row's products never meet another row's).
__global__ void __launch_bounds__(kPlanThreads) lora_plan_kernel(const LoraPlanArgs a) {
  __shared__ int hist[kLoraMaxAdapters];  // rows of each adapter, then its next entry
  __shared__ int warp_sums[kPlanThreads / 32];
  __shared__ int base_tile, base_row;
  const GroupEntry ge = a.groups[blockIdx.x];
  const bool ok = ge.rows > 0 && ge.rows <= a.S && ge.expert >= 0 && ge.expert < a.slabs && ge.out_row0 >= 0 &&
                  static_cast<int64_t>(ge.out_row0) + ge.rows <= a.rows;
  if (!ok) return;  // the GEMM reports it
  const int tid = threadIdx.x, n = a.lora.n;
  const bool shared = ge.expert == a.shared_slab;
  for (int i = tid; i < n; i += kPlanThreads) hist[i] = 0;
  __syncthreads();
  auto adapter_of = [&](int i, int& token) {
    token = shared ? i : a.token_of_row[ge.out_row0 + i];
    return token >= 0 && token < a.S ? a.lora.ids[token] : -1;
  };
  for (int i = tid; i < ge.rows; i += kPlanThreads) {
    int token;
    int id = adapter_of(i, token);
    if (id < -1 || id >= n) {
      report(a.status, MOE_STATUS_BAD_ADAPTER, -1);
      id = -1;
    }
    a.plan.has[ge.out_row0 + i] = id >= 0;
    if (id >= 0) atomicAdd(&hist[id], 1);
  }
  __syncthreads();
  // this thread's adapters: a run of `per`
  const int per = (n + kPlanThreads - 1) / kPlanThreads, a0 = min(tid * per, n), a1 = min(a0 + per, n);
  int rows = 0, tiles = 0;
  for (int i = a0; i < a1; ++i) {
    rows += hist[i];
    tiles += (hist[i] + kRows - 1) / kRows;
  }
  int all_rows, all_tiles;
  int row = block_prefix(rows, warp_sums, &all_rows);
  int tile = block_prefix(tiles, warp_sums, &all_tiles);
  if (tid == 0) {
    base_tile = all_tiles > 0 ? atomicAdd(&a.plan.counts[0], all_tiles) : 0;
    base_row = all_rows > 0 ? atomicAdd(&a.plan.counts[1], all_rows) : 0;
  }
  __syncthreads();
  row += base_row;
  tile += base_tile;
  for (int i = a0; i < a1; ++i) {
    const int c = hist[i];
    for (int k = 0; k < c; k += kRows) a.plan.tiles[tile++] = LoraTile{ge.expert, i, row + k, min(kRows, c - k)};
    hist[i] = row;
    row += c;
  }
  __syncthreads();
  for (int i = tid; i < ge.rows; i += kPlanThreads) {
    int token;
    const int id = adapter_of(i, token);
    if (id >= 0 && id < n) a.plan.list[atomicAdd(&hist[id], 1)] = make_int2(ge.out_row0 + i, token);
  }
}

// Inner products of one (tile, slice of K) per unit.  N = pairs * r columns in
// blocks of 32; warp w takes block w % nb and, of the slice, every kslices-th
// piece of 32 k; the warps of a block add up in a fixed order through shared
// memory.
struct InnerShape {
  int splits;  // slices of K
  int chunk;   // k of a slice (a multiple of 32)
};

__global__ void __launch_bounds__(kThreads, 1) lora_inner_kernel(const LoraRowsArgs a, const InnerShape sh) {
  __shared__ float red[kWarps][32][33];  // half of the rows at a time
  __shared__ const __nv_bfloat16* rowp[kRows];
  const int lane = lane_id(), warp = threadIdx.x >> 5, r = a.lora.r, q = lane & 3, gq = lane >> 2;
  const int cols = a.pairs * r, nb = (cols + 31) / 32, kslices = kWarps / nb;
  const int block = warp % nb, kslice = warp / nb;
  const int units = a.plan.counts[0] * sh.splits;
  for (int un = blockIdx.x; un < units; un += gridDim.x) {
    const LoraTile tile = a.plan.tiles[un / sh.splits];
    const int split = un % sh.splits, k0 = split * sh.chunk, k1 = min(a.K, k0 + sh.chunk);
    __syncthreads();
    if (threadIdx.x < kRows) {
      const int2 e = a.plan.list[tile.pos + min(static_cast<int>(threadIdx.x), tile.rows - 1)];
      const __nv_bfloat16* p;
      if (tile.expert == a.shared_slab && a.src_shared != nullptr)
        p = static_cast<const __nv_bfloat16*>(a.src_shared) + static_cast<int64_t>(e.y) * a.K;
      else
        p = static_cast<const __nv_bfloat16*>(a.src) + static_cast<int64_t>(a.src_by_token ? e.y : e.x) * a.K;
      rowp[threadIdx.x] = p;
    }
    __syncthreads();
    // rows of A for this lane's column of each 8-column tile of the block (nullptr: no such column or no pair)
    const __nv_bfloat16* bp[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int col = block * 32 + j * 8 + gq, m = col / r;
      bp[j] = nullptr;
      if (col < cols && a.lora.a[a.m0 + m] != nullptr)
        bp[j] = static_cast<const __nv_bfloat16*>(a.lora.a[a.m0 + m]) +
                ((static_cast<int64_t>(tile.adapter) * a.slabs + tile.expert) * r + (col - m * r)) * a.K;
    }
    const int mt = (tile.rows + 15) / 16;
    float acc[4][4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[i][j][v] = 0.0f;
    if (kslice < kslices) {
      const uint4 zero = make_uint4(0, 0, 0, 0);
      for (int k = k0 + kslice * 32; k < k1; k += kslices * 32) {
        const int c = k + 8 * q;  // this lane's 8 k (K is a multiple of 8)
        const bool in = c < k1;
        uint4 av[4][2], bv[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) bv[j] = in && bp[j] != nullptr ? ldg16(bp[j] + c) : zero;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          av[i][0] = in && i < mt ? ldg16(rowp[i * 16 + gq] + c) : zero;
          av[i][1] = in && i < mt ? ldg16(rowp[i * 16 + gq + 8] + c) : zero;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (i < mt) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              mma_bf16(acc[i][j], av[i][0].x, av[i][1].x, av[i][0].y, av[i][1].y, bv[j].x, bv[j].y);
              mma_bf16(acc[i][j], av[i][0].z, av[i][1].z, av[i][0].w, av[i][1].w, bv[j].z, bv[j].w);
            }
          }
        }
      }
    }
    // accumulator (i, j): rows 16 i + gq (+ 8), columns 8 j + 2 q (+ 1) of the block
    float* u = a.u + (static_cast<int64_t>(split) * a.max_total_rows + tile.pos) * cols;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (32 * h < tile.rows) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int v = 0; v < 4; ++v)
              red[warp][i * 16 + gq + (v >> 1) * 8][j * 8 + 2 * q + (v & 1)] = acc[2 * h + i][j][v];
        __syncthreads();
        for (int i = threadIdx.x; i < min(32, tile.rows - 32 * h) * cols; i += kThreads) {
          const int row = i / cols, col = i - row * cols, b = col / 32;
          float s = 0.0f;
          for (int k = 0; k < kslices; ++k) s += red[k * nb + b][row][col - b * 32];
          u[static_cast<int64_t>(32 * h + row) * cols + col] = s;
        }
        __syncthreads();
      }
    }
  }
}

// Outer products of one (tile, kOuterCols columns of one pair) per unit.  The
// tile's u (the slices' sums, rounded to bf16) sits in shared memory; warp w
// makes 32 columns at a time.  Its column c of the 8-column tile j stands for
// column 8 (c / 2) + 2 j + c % 2 of the 32, so that a lane ends with 8
// neighbouring columns of its rows: one 16-byte store each.
constexpr int kOuterCols = 2048;

__global__ void __launch_bounds__(kThreads) lora_outer_kernel(const LoraRowsArgs a, int splits) {
  __shared__ __align__(16) __nv_bfloat16 us[kRows][MOE_LORA_MAX_RANK + 8];
  __shared__ int64_t out_row[kRows];
  const int lane = lane_id(), warp = threadIdx.x >> 5, r = a.lora.r, q = lane & 3, gq = lane >> 2;
  const int cols = a.pairs * r, rp = (r + 15) & ~15;
  const int blocks = (a.N + kOuterCols - 1) / kOuterCols;
  const int units = a.plan.counts[0] * a.pairs * blocks;
  for (int un = blockIdx.x; un < units; un += gridDim.x) {
    const LoraTile tile = a.plan.tiles[un / (a.pairs * blocks)];
    const int m = un / blocks % a.pairs, n0 = un % blocks * kOuterCols;
    __syncthreads();
    if (threadIdx.x < kRows)
      out_row[threadIdx.x] = a.plan.list[tile.pos + min(static_cast<int>(threadIdx.x), tile.rows - 1)].x;
    for (int i = threadIdx.x; i < kRows * rp; i += kThreads) {
      const int row = i / rp, c = i - row * rp;
      float s = 0.0f;
      if (row < tile.rows && c < r && a.lora.a[a.m0 + m] != nullptr) {
        const float* src = a.u + static_cast<int64_t>(tile.pos + row) * cols + m * r + c;
        for (int k = 0; k < splits; ++k) s += __ldg(src + static_cast<int64_t>(k) * a.max_total_rows * cols);
      }
      us[row][c] = __float2bfloat16_rn(s);
    }
    __syncthreads();
    const float scale = __ldg(a.lora.scale + tile.adapter);
    const auto* b = static_cast<const __nv_bfloat16*>(a.lora.b[a.m0 + m]);
    if (b != nullptr) b += (static_cast<int64_t>(tile.adapter) * a.slabs + tile.expert) * a.N * r;
    const int mt = (tile.rows + 15) / 16;
    for (int n = n0 + warp * 32; n < min(a.N, n0 + kOuterCols); n += kWarps * 32) {
      float acc[4][4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[i][j][v] = 0.0f;
      for (int k = 0; k < rp; k += 16) {
        uint2 bv[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int col = n + 8 * (gq >> 1) + 2 * j + (gq & 1);
          bv[j] = b != nullptr && col < a.N && k + 4 * q < r
                      ? __ldg(reinterpret_cast<const uint2*>(b + static_cast<int64_t>(col) * r + k + 4 * q))
                      : make_uint2(0, 0);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (i < mt) {
            const uint2 u0 = *reinterpret_cast<const uint2*>(&us[i * 16 + gq][k + 4 * q]);
            const uint2 u1 = *reinterpret_cast<const uint2*>(&us[i * 16 + gq + 8][k + 4 * q]);
#pragma unroll
            for (int j = 0; j < 4; ++j) mma_bf16(acc[i][j], u0.x, u1.x, u0.y, u1.y, bv[j].x, bv[j].y);
          }
        }
      }
      const int col = n + 8 * q;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int hi = 0; hi < 2; ++hi) {
          const int row = i * 16 + gq + hi * 8;
          if (row < tile.rows && col < a.N) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = pack_bf16x2(acc[i][j][2 * hi] * scale, acc[i][j][2 * hi + 1] * scale);
            stg16(static_cast<__nv_bfloat16*>(a.delta) + (out_row[row] * a.pairs + m) * a.N + col,
                  make_uint4(w[0], w[1], w[2], w[3]));
          }
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_lora_plan(const LoraPlanArgs& a, cudaStream_t stream) {
  if (a.num_groups <= 0 || a.num_groups > gemm::kMaxGroups || a.lora.n > kLoraMaxAdapters) return cudaErrorInvalidValue;
  cudaError_t e = cudaMemsetAsync(a.plan.counts, 0, 2 * sizeof(int), stream);
  if (e != cudaSuccess) return e;
  lora_plan_kernel<<<a.num_groups, kPlanThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_lora_rows(const LoraRowsArgs& a, cudaStream_t stream) {
  if (a.max_total_rows <= 0) return cudaSuccess;
  // slices of K: about two units per SM when every tile is full, at least 256 k each
  const int64_t tiles = (a.max_total_rows + kRows - 1) / kRows;
  int splits = static_cast<int>((2 * a.num_sms + tiles - 1) / tiles);
  if (splits > kLoraMaxSplits) splits = kLoraMaxSplits;
  if (splits > a.K / 256) splits = a.K / 256 > 0 ? a.K / 256 : 1;
  const int chunk = ((a.K + splits - 1) / splits + 31) & ~31;
  splits = (a.K + chunk - 1) / chunk;
  // the tile count is known on the device only: at most one per row
  const int64_t inner = a.max_total_rows * splits, outer = a.max_total_rows * a.pairs * ((a.N + kOuterCols - 1) / kOuterCols);
  lora_inner_kernel<<<static_cast<unsigned>(inner < a.num_sms * 2 ? inner : a.num_sms * 2), kThreads, 0, stream>>>(
      a, InnerShape{splits, chunk});
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  lora_outer_kernel<<<static_cast<unsigned>(outer < a.num_sms * 4 ? outer : a.num_sms * 4), kThreads, 0, stream>>>(
      a, splits);
  return cudaGetLastError();
}

}  // namespace moe
