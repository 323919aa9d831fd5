// 8-bit blocks: rows as E4M3 codes with one scale for each block of 128
// columns, and SwiGLU with a checkpoint in that form.
//
// 16 lanes hold a block, 8 consecutive elements each (16 bytes of bf16): the
// block's maximum is four shuffles, each element is read once, stays in
// registers until its block's scale is known, and is written once.  All
// three kernels are bound by memory: a row's bytes are needed once and the
// arithmetic hides behind them.
#include "train.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kGroups = kThreads / 16;  // blocks of 128 columns that a CTA holds at a time

template <bool F32>
__device__ __forceinline__ void load8(const void* x, size_t at, float (&v)[8]) {
  if constexpr (F32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(x) + at);
    const float4 a = p[0], b = p[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    bf16_values(*reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(x) + at), v);
  }
}

// A 16-lane group's place: block `t` of rows of nb blocks.  Lanes past the
// row's end (or a group past the last block) hold zeros and write nothing.
struct Place {
  uint32_t row, kb, col;
  bool live;  // this lane's 8 columns exist
};
__device__ __forceinline__ Place place_of(uint32_t t, uint32_t tasks, uint32_t nb, uint32_t cols) {
  Place p;
  p.row = t / nb;
  p.kb = t - p.row * nb;
  p.col = p.kb * kQBlock + (threadIdx.x & 15u) * 8u;
  p.live = t < tasks && p.col < cols;
  return p;
}

// U blocks of each group in flight per step: all loads are issued before the
// first block's maximum is reduced.
template <bool F32, bool POW2, int U>
__global__ void __launch_bounds__(kThreads) quantize_blocks_kernel(const void* __restrict__ x, uint32_t tasks,
                                                                   uint32_t nb, uint32_t cols, int64_t ldx,
                                                                   uint8_t* __restrict__ codes,
                                                                   float* __restrict__ scales) {
  griddep_begin();
  const uint32_t step = gridDim.x * kGroups;
  // (both groups of a warp take the same number of steps: `t` of its first)
  const uint32_t first = blockIdx.x * kGroups + (threadIdx.x >> 5) * 2u, mine = (threadIdx.x >> 4) & 1u;
  for (uint32_t t = first; t < tasks; t += U * step) {
    float v[U][8];
    Place p[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      p[i] = place_of(t + i * step + mine, tasks, nb, cols);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
      if (p[i].live) load8<F32>(x, (size_t)p[i].row * ldx + p[i].col, v[i]);
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const BlockScale sc = block_scale<POW2>(block_amax(v[i]));
      if (!p[i].live) continue;
      *reinterpret_cast<uint2*>(codes + (size_t)p[i].row * cols + p[i].col) = block_codes(v[i], sc.r);
      if ((threadIdx.x & 15u) == 0u) scales[(size_t)p[i].row * nb + p[i].kb] = sc.s;
    }
  }
}

// sigmoid(g) from the hardware's exponential and reciprocal (a few units of
// 2^-22 relative): 0 for g far below zero, where exp(-g) overflows.
__device__ __forceinline__ float sigmoid(float g) { return __frcp_rn(1.f + __expf(-g)); }

__global__ void __launch_bounds__(kThreads) swiglu_save_kernel(const SwigluSaveArgs a, uint32_t tasks, uint32_t nb) {
  griddep_begin();
  const uint32_t step = gridDim.x * kGroups, f = (uint32_t)a.f;
  const uint32_t first = blockIdx.x * kGroups + (threadIdx.x >> 5) * 2u, mine = (threadIdx.x >> 4) & 1u;
  const size_t plane = (size_t)a.R * f, splane = (size_t)a.R * nb;
  for (uint32_t t = first; t < tasks; t += step) {
    const Place p = place_of(t + mine, tasks, nb, f);
    float g[8] = {}, u[8] = {}, h[8];
    if (p.live) {
      load8<false>(a.g, (size_t)p.row * a.ld + p.col, g);
      load8<false>(a.u, (size_t)p.row * a.ld + p.col, u);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = g[i] * sigmoid(g[i]) * u[i];
    const size_t at = (size_t)p.row * f + p.col, sat = (size_t)p.row * nb + p.kb;
    const bool lead = p.live && (threadIdx.x & 15u) == 0u;
    if (a.h != nullptr && p.live) reinterpret_cast<uint4*>(a.h)[at / 8] = bf16_pack(h);
    if (a.codes != nullptr) {
      const BlockScale sc = block_scale<false>(block_amax(h));
      if (p.live) *reinterpret_cast<uint2*>(a.codes + at) = block_codes(h, sc.r);
      if (lead) a.scales[sat] = sc.s;
    }
    const BlockScale sg = block_scale<true>(block_amax(g)), su = block_scale<true>(block_amax(u));
    if (p.live) {
      *reinterpret_cast<uint2*>(a.saved + at) = block_codes(g, sg.r);
      *reinterpret_cast<uint2*>(a.saved + plane + at) = block_codes(u, su.r);
    }
    if (lead) {
      a.saved_scales[sat] = sg.s;
      a.saved_scales[splane + sat] = su.s;
    }
  }
}

__global__ void __launch_bounds__(kThreads) swiglu_backward_kernel(const SwigluBackwardArgs a, uint32_t tasks,
                                                                   uint32_t nb) {
  griddep_begin();
  const uint32_t step = gridDim.x * kGroups, f = (uint32_t)a.f;
  const uint32_t first = blockIdx.x * kGroups + (threadIdx.x >> 5) * 2u, mine = (threadIdx.x >> 4) & 1u;
  const size_t plane = (size_t)a.R * f, splane = (size_t)a.R * nb;
  for (uint32_t t = first; t < tasks; t += step) {
    const Place p = place_of(t + mine, tasks, nb, f);
    const size_t at = (size_t)p.row * f + p.col, sat = (size_t)p.row * nb + p.kb;
    float g[8] = {}, u[8] = {}, dh[8] = {}, h[8];
    if (p.live) {
      e4m3_values(*reinterpret_cast<const uint2*>(a.saved + at), g);
      e4m3_values(*reinterpret_cast<const uint2*>(a.saved + plane + at), u);
      load8<false>(a.dh, at, dh);
      const float sg = a.saved_scales[sat], su = a.saved_scales[splane + sat];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        g[i] *= sg;
        u[i] *= su;
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float sig = sigmoid(g[i]), silu = g[i] * sig;
      h[i] = silu * u[i];
      const float dg = dh[i] * u[i] * (sig * (1.f + g[i] * (1.f - sig)));
      u[i] = dh[i] * silu;  // du
      g[i] = dg;
    }
    if (p.live) {
      const size_t to = (size_t)p.row * a.ld + p.col;
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.dg) + to) = bf16_pack(g);
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.du) + to) = bf16_pack(u);
      if (a.h != nullptr) reinterpret_cast<uint4*>(a.h)[at / 8] = bf16_pack(h);
    }
    if (a.codes != nullptr) {  // f % 128 == 0: dg's blocks, then du's
      const BlockScale sg = block_scale<false>(block_amax(g)), su = block_scale<false>(block_amax(u));
      if (p.live) {
        uint8_t* c = a.codes + (size_t)p.row * 2 * f + p.col;
        *reinterpret_cast<uint2*>(c) = block_codes(g, sg.r);
        *reinterpret_cast<uint2*>(c + f) = block_codes(u, su.r);
        if ((threadIdx.x & 15u) == 0u) {
          float* s = a.scales + (size_t)p.row * 2 * nb + p.kb;
          s[0] = sg.s;
          s[nb] = su.s;
        }
      }
    }
  }
}

// CTAs for `tasks` blocks: enough to fill the SMs with 8 CTAs each.
int grid_of(uint32_t tasks, int num_sms) {
  const uint32_t want = (tasks + kGroups - 1) / kGroups, most = 8u * (uint32_t)num_sms;
  return (int)(want < most ? want : most);
}

// Blocks of rows x nb, or 0 when their count (with a last partial step past
// it) does not fit 32 bits.
uint32_t task_count(int rows, int nb) {
  const uint64_t n = (uint64_t)rows * (uint64_t)nb;
  return n <= 0x7fffffffull ? (uint32_t)n : 0u;
}

}  // namespace

moe_status quantize_blocks_launch(const void* x, bool f32, bool pow2, int rows, int cols, int64_t ldx,
                                  uint8_t* codes, float* scales, int num_sms, cudaStream_t s) {
  const int nb = ceil_div(cols, kQBlock);
  const uint32_t tasks = task_count(rows, nb);
  if (tasks == 0u) return MOE_ERR_UNSUPPORTED;
  constexpr int U = 2;
  auto kern = f32 ? (pow2 ? quantize_blocks_kernel<true, true, U> : quantize_blocks_kernel<true, false, U>)
                  : (pow2 ? quantize_blocks_kernel<false, true, U> : quantize_blocks_kernel<false, false, U>);
  MOE_TRY_CUDA(launch_k(kern, dim3(grid_of(tasks, num_sms)), dim3(kThreads), 0, s, x, tasks, (uint32_t)nb,
                        (uint32_t)cols, ldx, codes, scales));
  return MOE_OK;
}

moe_status swiglu_save_launch(const SwigluSaveArgs& a, int num_sms, cudaStream_t s) {
  const int nb = ceil_div(a.f, kQBlock);
  const uint32_t tasks = task_count(a.R, nb);
  if (tasks == 0u) return MOE_ERR_UNSUPPORTED;
  MOE_TRY_CUDA(launch_k(swiglu_save_kernel, dim3(grid_of(tasks, num_sms)), dim3(kThreads), 0, s, a, tasks,
                        (uint32_t)nb));
  return MOE_OK;
}

moe_status swiglu_backward_launch(const SwigluBackwardArgs& a, int num_sms, cudaStream_t s) {
  const int nb = ceil_div(a.f, kQBlock);
  const uint32_t tasks = task_count(a.R, nb);
  if (tasks == 0u) return MOE_ERR_UNSUPPORTED;
  MOE_TRY_CUDA(launch_k(swiglu_backward_kernel, dim3(grid_of(tasks, num_sms)), dim3(kThreads), 0, s, a, tasks,
                        (uint32_t)nb));
  return MOE_OK;
}

}  // namespace moe
