// 8-bit blocks: rows as E4M3 codes with one scale for each block of 128
// columns, and SwiGLU with a checkpoint in that form.
//
// 16 lanes hold a block, 8 consecutive elements each (16 bytes of bf16): the
// block's maximum is four shuffles, each element is read once, stays in
// registers until its block's scale is known, and is written once.  All
// three kernels are bound by memory: a row's bytes are needed once and the
// arithmetic hides behind them.  Measured: quantiser 65536 x 2048 bf16 69 us
// (5.9 TB/s; a copy has 6.8); SwiGLU 32768 x 2048 with its checkpoint 105 us
// (4.5 TB/s: three blocks' codes an element, the arithmetic shows), its
// gradient with codes and h 144 us (5.6 TB/s).  Small calls are 4 to 6 us.
#include "train.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kGroups = kThreads / 16;  // blocks of 128 columns that a CTA holds at a time

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

// U blocks of each group in flight per step (an even number): all loads are
// issued before the first block's maximum is reduced.
template <bool F32, bool POW2, int U>
__global__ void __launch_bounds__(kThreads, 4) quantize_blocks_kernel(const void* __restrict__ x, uint32_t tasks,
                                                                   uint32_t nb, uint32_t cols, int64_t ldx,
                                                                   uint8_t* __restrict__ codes,
                                                                   float* __restrict__ scales) {
  griddep_begin();
  const uint32_t step = gridDim.x * kGroups;
  // (both groups of a warp take the same number of steps: `t` of its first)
  const uint32_t first = blockIdx.x * kGroups + (threadIdx.x >> 5) * 2u, mine = (threadIdx.x >> 4) & 1u;
  for (uint32_t t = first; t < tasks; t += U * step) {
    uint4 q[U][F32 ? 2 : 1];
    Place p[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      p[i] = place_of(t + i * step + mine, tasks, nb, cols);
      const size_t at = (size_t)p[i].row * ldx + p[i].col;
#pragma unroll
      for (int h = 0; h < (F32 ? 2 : 1); ++h)
        q[i][h] = p[i].live ? __ldg(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(x) + at * (F32 ? 4 : 2)) + h)
                            : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int i = 0; i < U; i += 2) {
      float v[2][8];
      uint32_t m[2];
      BlockScale sc[2];
      if constexpr (F32) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            v[k][4 * h] = __uint_as_float(q[i + k][h].x);
            v[k][4 * h + 1] = __uint_as_float(q[i + k][h].y);
            v[k][4 * h + 2] = __uint_as_float(q[i + k][h].z);
            v[k][4 * h + 3] = __uint_as_float(q[i + k][h].w);
          }
        block_amax(v, m);
      } else {
        bf16_values(q[i][0], v[0]);
        bf16_values(q[i + 1][0], v[1]);
        block_amax_bf16(q[i][0], q[i + 1][0], v, m);
      }
      if constexpr (POW2) {
        sc[0] = pow2_scale(m[0]);
        sc[1] = pow2_scale(m[1]);
      } else {
        amax_scales(m, sc);
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const Place& o = p[i + k];
        if (!o.live) continue;
        *reinterpret_cast<uint2*>(codes + (size_t)o.row * cols + o.col) = block_codes(v[k], sc[k].r);
        if ((threadIdx.x & 15u) == 0u) scales[(size_t)o.row * nb + o.kb] = sc[k].s;
      }
    }
  }
}

__global__ void __launch_bounds__(kThreads, 4) swiglu_save_kernel(const SwigluSaveArgs a, uint32_t tasks, uint32_t nb) {
  griddep_begin();
  const uint32_t step = gridDim.x * kGroups, f = (uint32_t)a.f;
  const uint32_t first = blockIdx.x * kGroups + (threadIdx.x >> 5) * 2u, mine = (threadIdx.x >> 4) & 1u;
  const size_t plane = (size_t)a.R * f, splane = (size_t)a.R * nb;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  Place p = place_of(first + mine, tasks, nb, f);
  auto load = [&](const void* x) {
    return p.live ? __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(x) +
                                                          (size_t)p.row * a.ld + p.col))
                  : zero;
  };
  uint4 qg = load(a.g), qu = load(a.u);
  for (uint32_t t = first; t < tasks; t += step) {
    const Place o = p;
    const uint4 cg = qg, cu = qu;
    p = place_of(t + step + mine, tasks, nb, f);  // the next block is on its way during this one
    qg = load(a.g);
    qu = load(a.u);
    float gu[2][8], h[1][8];
    bf16_values(cg, gu[0]);
    bf16_values(cu, gu[1]);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[0][i] = gu[0][i] * sigmoid(gu[0][i]) * gu[1][i];
    const size_t at = (size_t)o.row * f + o.col, sat = (size_t)o.row * nb + o.kb;
    const bool lead = o.live && (threadIdx.x & 15u) == 0u;
    if (a.h != nullptr && o.live) reinterpret_cast<uint4*>(a.h)[at / 8] = bf16_pack(h[0]);
    if (a.codes != nullptr) {
      uint32_t m[1];
      BlockScale sc[1];
      block_amax(h, m);
      amax_scales(m, sc);
      if (o.live) *reinterpret_cast<uint2*>(a.codes + at) = block_codes(h[0], sc[0].r);
      if (lead) a.scales[sat] = sc[0].s;
    }
    uint32_t m[2];
    block_amax_bf16(cg, cu, gu, m);
    const BlockScale sg = pow2_scale(m[0]), su = pow2_scale(m[1]);
    if (o.live) {
      *reinterpret_cast<uint2*>(a.saved + at) = block_codes(gu[0], sg.r);
      *reinterpret_cast<uint2*>(a.saved + plane + at) = block_codes(gu[1], su.r);
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
    float d[2][8] = {}, dh[8] = {}, h[8];  // g and u, then dg and du
    if (p.live) {
      const uint2 cg = __ldg(reinterpret_cast<const uint2*>(a.saved + at));
      const uint2 cu = __ldg(reinterpret_cast<const uint2*>(a.saved + plane + at));
      const uint4 qh = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.dh) + at));
      const float sg = a.saved_scales[sat], su = a.saved_scales[splane + sat];
      e4m3_values(cg, d[0]);
      e4m3_values(cu, d[1]);
      bf16_values(qh, dh);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        d[0][i] *= sg;
        d[1][i] *= su;
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float g = d[0][i], u = d[1][i], sig = sigmoid(g), silu = g * sig;
      h[i] = silu * u;
      d[0][i] = dh[i] * u * (sig * (1.f + g * (1.f - sig)));
      d[1][i] = dh[i] * silu;
    }
    if (p.live) {
      const size_t to = (size_t)p.row * a.ld + p.col;
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.dg) + to) = bf16_pack(d[0]);
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.du) + to) = bf16_pack(d[1]);
      if (a.h != nullptr) reinterpret_cast<uint4*>(a.h)[at / 8] = bf16_pack(h);
    }
    if (a.codes != nullptr) {  // f % 128 == 0: dg's blocks, then du's
      uint32_t m[2];
      BlockScale sc[2];
      block_amax(d, m);
      amax_scales(m, sc);
      if (p.live) {
        uint8_t* c = a.codes + (size_t)p.row * 2 * f + p.col;
        *reinterpret_cast<uint2*>(c) = block_codes(d[0], sc[0].r);
        *reinterpret_cast<uint2*>(c + f) = block_codes(d[1], sc[1].r);
        if ((threadIdx.x & 15u) == 0u) {
          float* s = a.scales + (size_t)p.row * 2 * nb + p.kb;
          s[0] = sc[0].s;
          s[nb] = sc[1].s;
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
  constexpr int U = 4;
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
