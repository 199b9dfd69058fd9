// Low-rank adapters of many requests beside the grouped expert projections:
// per row (token t, expert e, adapter a)
//   u = A[a][e] row                r values
//   delta = scale[a] B[a][e] u     added to the projection's fp32 sums by the
//                                  grouped GEMM's epilogue
// Requests share the experts, not the adapters, so the rows are first sorted by
// (expert, adapter) into tiles of up to 32 rows that share one pair of adapter
// matrices (lora_plan_kernel, once per call).  A tile's products then run on
// m16n8k16 tensor-core instructions: both are bound by memory (the rows are
// read once, the deltas written once, and an adapter's matrices are read once
// per tile), and r = 8 .. 128 columns would leave most of a tcgen05 tile empty.
//
// Operand fragments are loaded straight from global memory, 16 (inner) or 8
// (outer) bytes per lane: a product's sum over k does not depend on the order
// of k, so lane quad q takes 8 (4) neighbouring k for the fragment slots that
// the instruction gives it, the same for both operands.
#include <algorithm>

#include "common.cuh"
#include "gemm_common.cuh"
#include "kernels.h"
#include "pdl.cuh"

namespace moe {

namespace {

constexpr int kRows = kLoraTileRows;
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
  __shared__ int base_tile, base_row, refused;
  pdl_wait();
  pdl_trigger();
  const GroupEntry ge = a.groups[blockIdx.x];
  const bool ok = ge.rows > 0 && ge.expert >= 0 && ge.expert < a.slabs && ge.out_row0 >= 0 &&
                  static_cast<int64_t>(ge.out_row0) + ge.rows <= a.rows;
  if (!ok) return;  // empty, or the GEMM skips it and says so
  const int tid = threadIdx.x, n = a.lora.n;
  const bool shared = ge.expert == a.shared_slab;
  // Group tables made from a caller's offsets may overlap: whoever claims rows that
  // x_perm, token_of_row or the lists do not have is left without adapters.
  auto refuse = [&]() {
    if (tid == 0) report(a.status, MOE_STATUS_BAD_GROUP, -1);
    for (int i = tid; i < ge.rows; i += kPlanThreads) a.plan.has[ge.out_row0 + i] = 0;
  };
  if (ge.rows > a.S || (!shared && static_cast<int64_t>(ge.out_row0) + ge.rows > a.routed_rows)) {
    refuse();
    return;
  }
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
    const unsigned long long at = all_rows > 0 ? atomicAdd(a.plan.rows, static_cast<unsigned long long>(all_rows)) : 0;
    refused = at + all_rows > static_cast<unsigned long long>(a.max_total_rows);
    base_row = static_cast<int>(at);
    base_tile = all_tiles > 0 && !refused ? atomicAdd(a.plan.tile_count, all_tiles) : 0;
  }
  __syncthreads();
  if (refused) {
    refuse();
    return;
  }
  row += base_row;
  tile += base_tile;
  for (int i = a0; i < a1; ++i) {
    const int c = hist[i];
    hist[i] = tile * kRows;  // the adapter's next entry
    for (int k = 0; k < c; k += kRows) a.plan.tiles[tile++] = LoraTile{ge.expert, i, row + k, min(kRows, c - k)};
    row += c;
  }
  __syncthreads();
  for (int i = tid; i < ge.rows; i += kPlanThreads) {
    int token;
    const int id = adapter_of(i, token);
    if (id >= 0 && id < n) a.plan.list[atomicAdd(&hist[id], 1)] = make_int2(ge.out_row0 + i, token);
  }
}

// A tile and its rows in shared memory, loaded one unit ahead: the entries of
// tile i are list[32 i ..], so tile and rows load side by side.
struct TileRows {
  LoraTile tile;
  int2 row[kRows];
};
struct MetaRegs {
  LoraTile tile;
  int2 row;
};
__device__ __forceinline__ MetaRegs meta_load(const LoraPlan& p, int tile) {
  MetaRegs m{};
  if (threadIdx.x < kRows) m.row = p.list[tile * kRows + threadIdx.x];  // (entries past the tile's rows: not used)
  if (threadIdx.x == 0) m.tile = p.tiles[tile];
  return m;
}
__device__ __forceinline__ void meta_store(TileRows& t, const MetaRegs& m) {
  if (threadIdx.x < kRows) t.row[threadIdx.x] = m.row;
  if (threadIdx.x == 0) t.tile = m.tile;
}

// Inner products of one (tile, slice of K) per unit.  N = pairs * r columns in
// blocks of 32; warp w takes block w % nb and every kslices-th part of the slice,
// pieces of 32 k with the next piece's loads under way during a piece's products;
// the warps of a block add up in a fixed order through shared memory.  (With 16
// warps per SM the loop is bound by its own instructions as much as by loads, so
// the whole pieces have no conditions and constant offsets.  Two pieces of fragments
// beside the accumulators and pointers are more than the 128 registers that 16 warps
// leave a thread: it spills 432 bytes, 244 with eight warps to a CTA.)  Measured
// inside the layer on 24,008 rows over 64 E4M3 experts, 12 adapters of rank 32: 62 us
// for gate and up (K = 2048; 215 MB from HBM, 33 us at the copy rate), 38 us for down
// (K = 1408; 132 MB, 20 us).  What bounds it is the way from L2: a tile of 32 rows
// reads its 64 (or 32) rows of A again, and a load of a fragment touches eight lines.
template <int V>
struct Const {
  static constexpr int value = V;
};
struct InnerShape {
  int splits;  // slices of K
  int chunk;   // k of a slice
  int part;    // k of a warp's part of it (a multiple of 32)
};

template <int W>  // warps of a CTA: 4, or 8 for more than 4 blocks of columns
__global__ void __launch_bounds__(32 * W, 16 / W) lora_inner_kernel(const LoraRowsArgs a, const InnerShape sh) {
  __shared__ float red[W][kRows][33];
  __shared__ TileRows meta[2];
  const int lane = lane_id(), warp = threadIdx.x >> 5, r = a.lora.r, q = lane & 3, gq = lane >> 2;
  const int cols = a.pairs * r, nb = (cols + 31) / 32, kslices = W / nb;
  const int block = warp % nb, kslice = warp / nb;
  pdl_wait();
  pdl_trigger();
  const int units = *a.plan.tile_count * sh.splits;
  if (blockIdx.x < units) meta_store(meta[0], meta_load(a.plan, blockIdx.x / sh.splits));
  __syncthreads();
  for (int un = blockIdx.x, buf = 0; un < units; un += gridDim.x, buf ^= 1) {
    const LoraTile tile = meta[buf].tile;
    const int split = un % sh.splits, k0 = split * sh.chunk, k1 = min(a.K, k0 + sh.chunk);
    const int next = un + gridDim.x;
    MetaRegs ahead{};
    if (next < units) ahead = meta_load(a.plan, next / sh.splits);
    auto row_of = [&](int i) {
      const int2 e = meta[buf].row[min(i, tile.rows - 1)];
      if (tile.expert == a.shared_slab && a.src_shared != nullptr)
        return static_cast<const __nv_bfloat16*>(a.src_shared) + static_cast<int64_t>(e.y) * a.K;
      return static_cast<const __nv_bfloat16*>(a.src) + static_cast<int64_t>(a.src_by_token ? e.y : e.x) * a.K;
    };
    // rows of A for this lane's column of each 8-column tile of the block (columns that do not exist, or whose pair does
    // not, read another one's row and are not stored)
    const __nv_bfloat16* bp[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int col = min(block * 32 + j * 8 + gq, cols - 1), m = col / r;
      const void* base = a.lora.a[a.m0 + m] != nullptr ? a.lora.a[a.m0 + m] : a.lora.a[a.m0 + (m ^ 1)];
      bp[j] = static_cast<const __nv_bfloat16*>(base) +
              ((static_cast<int64_t>(tile.adapter) * a.slabs + tile.expert) * r + (col - m * r)) * a.K;
    }
    const bool two = tile.rows > 16;
    const __nv_bfloat16* ap[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      ap[i][0] = row_of(i * 16 + gq);
      ap[i][1] = row_of(i * 16 + gq + 8);
    }
    float acc[2][4][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[i][j][v] = 0.0f;
    struct Piece {
      uint4 a[2][2], b[4];
    };
    auto load = [&](Piece& pc, auto off) {  // whole piece, `off` pieces from the pointers on
      constexpr int kBytes = decltype(off)::value * 64;
#pragma unroll
      for (int j = 0; j < 4; ++j) pc.b[j] = ldg16_at<kBytes>(bp[j]);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        pc.a[i][0] = ldg16_at<kBytes>(ap[i][0]);
        pc.a[i][1] = ldg16_at<kBytes>(ap[i][1]);
      }
    };
    auto products = [&](const Piece& pc) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (i == 0 || two) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            mma_bf16(acc[i][j], pc.a[i][0].x, pc.a[i][1].x, pc.a[i][0].y, pc.a[i][1].y, pc.b[j].x, pc.b[j].y);
            mma_bf16(acc[i][j], pc.a[i][0].z, pc.a[i][1].z, pc.a[i][0].w, pc.a[i][1].w, pc.b[j].z, pc.b[j].w);
          }
        }
      }
    };
    auto advance = [&](int k) {
#pragma unroll
      for (int j = 0; j < 4; ++j) bp[j] += k;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        ap[i][0] += k;
        ap[i][1] += k;
      }
    };
    if (kslice < kslices) {
      const int kb = k0 + kslice * sh.part, ke = min(k1, kb + sh.part);  // this warp's k
      int pieces = ke > kb ? (ke - kb) / 32 : 0;
      const int rest = ke > kb ? (ke - kb) & 31 : 0;
      advance(kb + 8 * q);  // this lane's 8 k of the first piece
      Piece p0, p1;
      if (pieces > 0) load(p0, Const<0>{});
      for (; pieces > 4; pieces -= 4) {
        load(p1, Const<1>{});
        products(p0);
        load(p0, Const<2>{});
        products(p1);
        load(p1, Const<3>{});
        products(p0);
        load(p0, Const<4>{});
        products(p1);
        advance(128);
      }
      for (; pieces > 0; --pieces) {
        if (pieces > 1) load(p1, Const<1>{});
        products(p0);
        p0 = p1;
        advance(32);
      }
      if (rest) {  // the last k of K, a multiple of 8
        const bool in = 8 * q < rest;
#pragma unroll
        for (int j = 0; j < 4; ++j) p0.b[j] = ldg16_if(bp[j], in);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          p0.a[i][0] = ldg16_if(ap[i][0], in);
          p0.a[i][1] = ldg16_if(ap[i][1], in);
        }
        products(p0);
      }
    }
    // accumulator (i, j): rows 16 i + gq (+ 8), columns 8 j + 2 q (+ 1) of the block
    float* u = a.u + (static_cast<int64_t>(split) * a.max_total_rows + tile.pos) * cols;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int v = 0; v < 4; ++v) red[warp][i * 16 + gq + (v >> 1) * 8][j * 8 + 2 * q + (v & 1)] = acc[i][j][v];
    if (next < units) meta_store(meta[buf ^ 1], ahead);
    __syncthreads();
    for (int row = warp; row < tile.rows; row += W) {
      for (int b = 0; b < nb; ++b) {
        const int col = b * 32 + lane;
        float s = 0.0f;
        for (int k = 0; k < kslices; ++k) s += red[k * nb + b][row][lane];
        if (col < cols) u[static_cast<int64_t>(row) * cols + col] = s;
      }
    }
    __syncthreads();
  }
}

// Outer products of one (tile, block of columns of every pair) per unit.  The
// tile's u (the slices' sums, rounded to bf16) sits in shared memory; warp w
// makes 32 columns of a pair at a time, the next columns' rows of B under way
// during the products.  Its column c of the 8-column tile j stands for column 8
// (c / 2) + 2 j + c % 2 of the 32, so that a lane ends with 8 neighbouring
// columns of its rows: one 16-byte store each.  Measured as above: 82 us for gate
// and up (N = 1408 each: 125 MB of deltas and 138 MB from HBM, 40 us at the copy
// rate), 55 us for down (N = 2048).  u is summed in fp32 over all of K and rounded
// once, to the type that the instruction multiplies, and the deltas are bf16: each
// rounding is at most a 2^-8 share of what the adapters add.  Two bf16 terms of u
// would double the products, fp32 deltas the traffic that bounds this kernel.
constexpr int kOuterThreads = 128;
constexpr int kOuterWarps = kOuterThreads / 32;

template <int KSTEPS>  // 16-k steps of the rank kept in registers: r <= 16 KSTEPS
__global__ void __launch_bounds__(kOuterThreads, KSTEPS <= 2 ? 6 : 4) lora_outer_kernel(const LoraRowsArgs a, int splits, int block) {
  __shared__ __align__(16) __nv_bfloat16 us[2][kRows][16 * KSTEPS + 8];
  __shared__ TileRows meta[2];
  const int lane = lane_id(), warp = threadIdx.x >> 5, r = a.lora.r, q = lane & 3, gq = lane >> 2;
  const int cols = a.pairs * r, rp = 16 * KSTEPS;
  const int blocks = (a.N + block - 1) / block;
  pdl_wait();
  pdl_trigger();
  const int units = *a.plan.tile_count * blocks;
  if (blockIdx.x < units) meta_store(meta[0], meta_load(a.plan, blockIdx.x / blocks));
  __syncthreads();
  for (int un = blockIdx.x, buf = 0; un < units; un += gridDim.x, buf ^= 1) {
    const LoraTile tile = meta[buf].tile;
    const int n0 = un % blocks * block, nc = min(a.N - n0, block);
    const int next = un + gridDim.x;
    MetaRegs ahead{};
    if (next < units) ahead = meta_load(a.plan, next / blocks);
    // rows of B of 32 columns: item `it` of the unit is column group it / pairs of pair it % pairs
    const int items = (nc + 31) / 32 * a.pairs;
    uint2 bv[KSTEPS][4];
    auto load_b = [&](int it) {
      const int m = it % a.pairs, n = n0 + it / a.pairs * 32;
      const auto* b = static_cast<const __nv_bfloat16*>(a.lora.b[a.m0 + m]);
      const bool any = it < items && b != nullptr;
      if (any) b += (static_cast<int64_t>(tile.adapter) * a.slabs + tile.expert) * a.N * r;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int col = n + 8 * (gq >> 1) + 2 * j + (gq & 1);
#pragma unroll
        for (int k = 0; k < KSTEPS; ++k)
          bv[k][j] = ldg8_if(b + static_cast<int64_t>(col) * r + 16 * k + 4 * q, any && col < a.N && 16 * k + 4 * q < r);
      }
    };
    load_b(warp);
    for (int i = threadIdx.x; i < a.pairs * kRows * rp; i += kOuterThreads) {
      const int m = i / (kRows * rp), row = i / rp % kRows, c = i % rp;
      float s = 0.0f;
      if (row < tile.rows && c < r && a.lora.a[a.m0 + m] != nullptr) {
        const float* src = a.u + static_cast<int64_t>(tile.pos + row) * cols + m * r + c;
        for (int k = 0; k < splits; ++k) s += __ldg(src + static_cast<int64_t>(k) * a.max_total_rows * cols);
      }
      us[m][row][c] = __float2bfloat16_rn(s);
    }
    __syncthreads();
    const float scale = __ldg(a.lora.scale + tile.adapter);
    const bool two = tile.rows > 16;
    for (int it = warp; it < items; it += kOuterWarps) {
      const int m = it % a.pairs, n = n0 + it / a.pairs * 32;
      float acc[2][4][4];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[i][j][v] = 0.0f;
#pragma unroll
      for (int k = 0; k < KSTEPS; ++k) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (i == 0 || two) {
            const uint2 u0 = *reinterpret_cast<const uint2*>(&us[m][i * 16 + gq][16 * k + 4 * q]);
            const uint2 u1 = *reinterpret_cast<const uint2*>(&us[m][i * 16 + gq + 8][16 * k + 4 * q]);
#pragma unroll
            for (int j = 0; j < 4; ++j) mma_bf16(acc[i][j], u0.x, u1.x, u0.y, u1.y, bv[k][j].x, bv[k][j].y);
          }
        }
      }
      load_b(it + kOuterWarps);
      const int col = n + 8 * q;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int hi = 0; hi < 2; ++hi) {
          const int row = i * 16 + gq + hi * 8;
          if (row < tile.rows && col < a.N) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = pack_bf16x2(acc[i][j][2 * hi] * scale, acc[i][j][2 * hi + 1] * scale);
            const int64_t at = static_cast<int64_t>(meta[buf].row[row].x) * a.pairs + m;
            stg16(static_cast<__nv_bfloat16*>(a.delta) + at * a.N + col, make_uint4(w[0], w[1], w[2], w[3]));
          }
        }
      }
    }
    if (next < units) meta_store(meta[buf ^ 1], ahead);
    __syncthreads();
  }
}

template <int W>
cudaError_t launch_inner(const LoraRowsArgs& a, int splits, int chunk, int nb, cudaStream_t stream) {
  const int kslices = W / nb, part = ((chunk + kslices - 1) / kslices + 31) & ~31;
  // the tile count is known on the device only: at most one per row
  const int64_t units = a.max_total_rows * splits, cap = static_cast<int64_t>(16 / W) * a.num_sms;
  return launch_pdl(lora_inner_kernel<W>, dim3(static_cast<unsigned>(units < cap ? units : cap)), dim3(32 * W), 0, stream, a,
                    InnerShape{splits, chunk, part});
}

template <int KSTEPS>
cudaError_t launch_outer(const LoraRowsArgs& a, int splits, cudaStream_t stream) {
  // Columns of a unit: a multiple of 128 (32 per warp), at most 2048, fewer where there are few tiles (full ones at
  // least; a small batch has more, shorter ones): about six units per SM.
  const int64_t tiles = (a.max_total_rows + kRows - 1) / kRows;
  const int64_t want = (6 * a.num_sms + tiles - 1) / tiles;
  const int block = static_cast<int>(std::min<int64_t>(2048, std::max<int64_t>(128, (a.N / want + 127) / 128 * 128)));
  const int64_t units = a.max_total_rows * ((a.N + block - 1) / block);
  const int64_t cap = static_cast<int64_t>(KSTEPS <= 2 ? 6 : 4) * a.num_sms;
  return launch_pdl(lora_outer_kernel<KSTEPS>, dim3(static_cast<unsigned>(units < cap ? units : cap)), dim3(kOuterThreads),
                    0, stream, a, splits, block);
}

}  // namespace

cudaError_t launch_lora_plan(const LoraPlanArgs& a, cudaStream_t stream) {
  if (a.num_groups <= 0 || a.num_groups > gemm::kMaxGroups || a.lora.n > kLoraMaxAdapters) return cudaErrorInvalidValue;
  cudaError_t e = cudaSuccess;
  if (!a.counts_zeroed) {
    if ((e = cudaMemsetAsync(a.plan.tile_count, 0, 16, stream)) != cudaSuccess) return e;
    lora_plan_kernel<<<a.num_groups, kPlanThreads, 0, stream>>>(a);  // (behind a memset: no dependent launch)
  } else {
    e = launch_pdl(lora_plan_kernel, dim3(a.num_groups), dim3(kPlanThreads), 0, stream, a);
  }
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_lora_rows(const LoraRowsArgs& a, cudaStream_t stream) {
  if (a.max_total_rows <= 0) return cudaSuccess;
  int splits = lora_splits(a.max_total_rows, a.K, a.num_sms);
  const int chunk = ((a.K + splits - 1) / splits + 31) & ~31;
  splits = (a.K + chunk - 1) / chunk;
  const int nb = (a.pairs * a.lora.r + 31) / 32;
  cudaError_t e = nb <= 4 ? launch_inner<4>(a, splits, chunk, nb, stream) : launch_inner<8>(a, splits, chunk, nb, stream);
  if (e != cudaSuccess) return e;
  if (a.lora.r <= 16)
    e = launch_outer<1>(a, splits, stream);
  else if (a.lora.r <= 32)
    e = launch_outer<2>(a, splits, stream);
  else if (a.lora.r <= 64)
    e = launch_outer<4>(a, splits, stream);
  else
    e = launch_outer<8>(a, splits, stream);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace moe
