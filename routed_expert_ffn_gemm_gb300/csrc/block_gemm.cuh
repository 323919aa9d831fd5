// Shared by the block product's kernels (block_gemm.cu, block_gemm_many.cu).
#pragma once

#include <atomic>

#include "ptx.cuh"
#include "train.cuh"

namespace moe {
namespace block_gemm {

constexpr int kMaxGroups = 1024;
constexpr int kBand = 16;                     // row tiles that share a pass over the weights
constexpr int kOutBytes = 2048;               // staging of an accumulating warp: 32 rows of 64 bytes

struct Params {
  int R, K, N, E, MT, KB, NB;
  int out_f32;
  const float* a_scales;
  const float* w_scales;
  const int32_t* offsets;
  void* out;
  int* status;
  long long timeout_ns;
};

struct Maps {
  CUtensorMap w;     // 128 of the reduction x 128 channels (block_gemm_many.cu: 64)
  CUtensorMap a[5];  // boxes of 8 << i rows
  CUtensorMap out;   // 32 rows of 64 bytes
};

// Where unit u is: row tiles of ROWS rows come first inside bands of kBand, so
// that a weight tile is read from memory once while the band's rows stay in
// L2.
struct Place {
  int g, tiles, mt, row0, n_valid;
};
template <int ROWS>
__device__ __forceinline__ Place place_of(int u, const int* offs, const int* prefix, int E, int MT) {
  const int t = u / MT;
  int lo = 0, hi = E - 1;  // the expert whose tiles hold t
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (prefix[mid] <= t) lo = mid; else hi = mid - 1;
  }
  Place x;
  x.g = lo;
  x.tiles = prefix[lo + 1] - prefix[lo];
  const int l = u - prefix[lo] * MT;
  const int band = l / (kBand * MT), rem = l - band * (kBand * MT);
  const int wide = min(kBand, x.tiles - band * kBand);
  x.mt = rem / wide;
  x.row0 = offs[lo] + (band * kBand + rem % wide) * ROWS;
  x.n_valid = min(ROWS, offs[lo + 1] - x.row0);
  return x;
}

// Group ranges, clamped into [0, R] and ordered, and the prefix of their
// counts of ROWS-row tiles, in shared memory.  The whole CTA calls this and
// synchronises afterwards.
template <int ROWS>
__device__ __forceinline__ void row_tiles(const Params& p, int* offs, int* prefix, int threads) {
  const int lane = threadIdx.x & 31;
  for (int g = threadIdx.x; g <= p.E; g += threads) {
    int o = p.offsets[g];
    if (o < 0 || o > p.R) {
      set_device_status(p.status, MOE_ERR_DEVICE_BOUNDS);
      o = o < 0 ? 0 : p.R;
    }
    offs[g] = o;
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    ordered_offsets(offs, p.E, p.status);
    int run = 0;
    for (int g0 = 0; g0 < p.E; g0 += 32) {
      const int g = g0 + lane;
      const int n = g < p.E ? (offs[g + 1] - offs[g] + ROWS - 1) / ROWS : 0;
      int incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      if (g < p.E) prefix[g] = run + incl - n;
      run += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) prefix[p.E] = run;
  }
}

// All lanes of the warp wait; the warp agrees on the outcome.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, uint64_t deadline, volatile int* abort) {
  return __all_sync(0xffffffffu, ptx::mbar_wait_bounded(bar, parity, deadline, abort)) != 0;
}

// One warp's accumulators to memory, rows on M: the lane's row is r0 + lane of
// the unit, acc[i][j] channel ch0 + STRIDE i + j.  64 bytes of each row at a
// time, staged in BUFS buffers in turn: by a TMA store when all 32 rows are
// the unit's (it clips the channels past N), else row by row.
// 16-byte chunk c of row r sits at c ^ ((r >> 1) & 3), as the store's 64-byte
// swizzle has it.
template <int BUFS, int CHUNKS, int STRIDE>
__device__ __forceinline__ void store_rows_m(const Params& p, const CUtensorMap* map, int row0, int n_valid,
                                             const float (&acc)[CHUNKS][32], int r0, int ch0, uint8_t* out0) {
  const int lane = threadIdx.x & 31;
  if (r0 >= n_valid) return;
  if (BUFS > 1 && lane == 0) ptx::bulk_wait_read<0>();  // (the unit before may have ended on either buffer)
  const bool whole = r0 + 32 <= n_valid;
  const int es = p.out_f32 ? 4 : 2, per = 64 / es;  // channels in 64 bytes
  uint8_t* out = static_cast<uint8_t*>(p.out) + (size_t)(row0 + r0) * p.N * es;
#pragma unroll
  for (int i = 0; i < CHUNKS; ++i) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (k == 1 && !p.out_f32) break;
      const int ch = ch0 + STRIDE * i + k * per;
      if (ch >= p.N) break;
      uint8_t* outb = out0 + ((p.out_f32 ? 2 * i + k : i) % BUFS) * kOutBytes;
      if (lane == 0) ptx::bulk_wait_read<BUFS - 1>();  // the store before has read this buffer
      __syncwarp();
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint4 v;
        if (p.out_f32) {
          const float* f = &acc[i][16 * k + 4 * c];
          v = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
        } else {
          float f[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) f[j] = acc[i][8 * c + j];
          v = bf16_pack(f);
        }
        *reinterpret_cast<uint4*>(outb + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4)) = v;
      }
      if (whole) {
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          ptx::tma_store_2d(map, ptx::smem_u32(outb), ch, row0 + r0);
          ptx::bulk_commit();
        }
        continue;
      }
      __syncwarp();
      const int c = lane & 3;
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const int r = 8 * h + (lane >> 2);
        const uint4 t = *reinterpret_cast<const uint4*>(outb + r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
        if (r0 + r < n_valid && ch + c * (16 / es) < p.N)
          *reinterpret_cast<uint4*>(out + (size_t)r * p.N * es + (size_t)ch * es + c * 16) = t;
      }
      __syncwarp();
    }
  }
}

// Launches one cluster of CLUSTER CTAs for each unit, up to what is resident
// at once: the grids are persistent, and not every SM finds its partners.
// `known`: resident clusters per device, one value, written once.
template <int CLUSTER, typename Kernel, typename P, typename M>
moe_status launch_clusters(Kernel kern, std::atomic<int> (&known)[64], int smem, long long units, int num_sms,
                           cudaStream_t s, const P& p, const M& maps) {
  constexpr int kThreads = 384;
  int dev = 0;
  MOE_TRY_CUDA(cudaGetDevice(&dev));
  if (dev < 0 || dev >= 64) return MOE_ERR_UNSUPPORTED;
  int n = known[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    MOE_TRY_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(CLUSTER);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = CLUSTER;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    MOE_TRY_CUDA(cudaOccupancyMaxActiveClusters(&n, kern, &cfg));
    if (n < 1) return MOE_ERR_UNSUPPORTED;
    known[dev].store(n, std::memory_order_relaxed);
  }
  long long clusters = n < num_sms / CLUSTER ? n : num_sms / CLUSTER;
  if (units < clusters) clusters = units;
  MOE_TRY_CUDA(launch_kc(CLUSTER, kern, dim3((unsigned)clusters * CLUSTER), dim3(kThreads), smem, s, p, maps));
  return MOE_OK;
}

}  // namespace block_gemm

// From this many rows an expert on average the product runs on
// block_gemm_many.cu.  64 experts of 7168 x 4096, us there and in
// block_gemm.cu: 80 rows 379 and 358, 100 rows 381 and 394, 120 rows 385 and
// 395, 160 rows 386 and 437; 90 rows unevenly spread 401 and 377; one expert
// with 100 rows 31 and 35.  The average counts experts without rows, which
// the host cannot see: 90 rows on average with half of the experts empty 198
// and 224.
constexpr long long kManyRows = 100;
moe_status block_gemm_many_launch(const block_gemm::Params& p, const block_gemm::Maps& maps, bool transposed,
                                  int num_sms, cudaStream_t s);

}  // namespace moe
