// Declarations shared by the translation units of the expert-training
// operators: 8-bit block quantisation, SwiGLU with 8-bit checkpoints, the
// block-scaled grouped product, the grouped weight gradient, router losses.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace moe {

constexpr int kQBlock = 128;  // columns (and, for weights, rows) that share a scale

inline __host__ __device__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

// ---------------------------------------------------------------------------
// E4M3 codes of a block's values
// ---------------------------------------------------------------------------

// The smallest block maximum that a scale follows: below it the scale of
// 2^-100 is kept, so that scales and their inverses stay normal fp32 numbers.
constexpr uint32_t kMinAmaxBits = 27u << 23;  // 2^-100

struct BlockScale {
  float s;  // the scale that is stored
  float r;  // what values are multiplied by before rounding to E4M3
};

// Scale of a block from the bits of its largest finite magnitude a: s = 2^p
// with a / 2^p in (224, 448], r = 2^-p exactly.
__device__ __forceinline__ BlockScale pow2_scale(uint32_t amax_bits) {
  const uint32_t b = max(amax_bits, kMinAmaxBits);
  // a = 1.m * 2^(E - 127); p = E - 135 while 1.m <= 1.75, else E - 134
  const uint32_t e = (b >> 23) + ((b & 0x7fffffu) > 0x600000u ? 1u : 0u);
  if (amax_bits == 0u) return {1.f, 1.f};
  return {__uint_as_float((e - 8u) << 23), __uint_as_float((262u - e) << 23)};
}

// s = a / 448 and r = 448 / a, each correctly rounded, for the blocks that
// the 16 lanes hold (N of them, each amax known to all lanes): a lane does
// one of the 2 N divisions.  Every lane of the warp calls this.
template <int N>
__device__ __forceinline__ void amax_scales(const uint32_t (&amax_bits)[N], BlockScale (&out)[N]) {
  constexpr int EACH = 16 / (2 * N);  // lanes that do the same division
  const int which = (threadIdx.x & 15) / EACH;
  float a = __uint_as_float(max(amax_bits[0], kMinAmaxBits));
#pragma unroll
  for (int i = 1; i < N; ++i)
    if (which >= 2 * i) a = __uint_as_float(max(amax_bits[i], kMinAmaxBits));
  const bool scale = (which & 1) == 0;
  const float q = __fdiv_rn(scale ? a : 448.f, scale ? 448.f : a);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float s = __shfl_sync(0xffffffffu, q, 2 * i * EACH, 16);
    const float r = __shfl_sync(0xffffffffu, q, (2 * i + 1) * EACH, 16);
    out[i] = amax_bits[i] == 0u ? BlockScale{1.f, 1.f} : BlockScale{s, r};
  }
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

// The largest magnitudes of N blocks over the 16 lanes that hold 8 values of
// each, as bits.  E4M3 has no infinity: infinities and NaN do not count
// toward the maximum and become NaN here (and so in the codes).  Every lane
// of the warp calls this.
template <int N>
__device__ __forceinline__ void finite_amax(float (&v)[N][8], uint32_t (&m)[N]) {
#pragma unroll
  for (int n = 0; n < N; ++n) {
    m[n] = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t a = abs_bits(v[n][i]);
      if (a < 0x7f800000u)
        m[n] = max(m[n], a);
      else
        v[n][i] = __uint_as_float(0x7fffffffu);
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m[n] = max(m[n], __shfl_xor_sync(0xffffffffu, m[n], o));
  }
}
template <int N>
__device__ __forceinline__ void block_amax(float (&v)[N][8], uint32_t (&m)[N]) {
  uint32_t top = 0u;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    m[n] = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) m[n] = max(m[n], abs_bits(v[n][i]));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m[n] = max(m[n], __shfl_xor_sync(0xffffffffu, m[n], o));
    top = max(top, m[n]);
  }
  if (__any_sync(0xffffffffu, top >= 0x7f800000u)) finite_amax(v, m);  // rare: some value is not finite
}
// The same of two blocks of bf16 values (8 of each in a and b, as stored):
// the maxima travel as the halves of one word.
__device__ __forceinline__ void block_amax_bf16(const uint4& a, const uint4& b, float (&v)[2][8], uint32_t (&m)[2]) {
  auto top = [](const uint4& q) {  // of the even and of the odd elements
    return __vmaxu2(__vmaxu2(q.x & 0x7fff7fffu, q.y & 0x7fff7fffu), __vmaxu2(q.z & 0x7fff7fffu, q.w & 0x7fff7fffu));
  };
  const uint32_t ta = top(a), tb = top(b);
  uint32_t t = __vmaxu2(__byte_perm(ta, tb, 0x5410), __byte_perm(ta, tb, 0x7632));  // a's low, b's high
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) t = __vmaxu2(t, __shfl_xor_sync(0xffffffffu, t, o));
  m[0] = t << 16;
  m[1] = t & 0xffff0000u;
  if (__any_sync(0xffffffffu, max(m[0], m[1]) >= 0x7f800000u)) finite_amax(v, m);
}

__device__ __forceinline__ uint2 block_codes(const float (&v)[8], float r) {
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = e4m3_pair(v[2 * i] * r, v[2 * i + 1] * r);
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// The two E4M3 codes in the low 16 bits as fp32 (exact).
__device__ __forceinline__ float2 e4m3_pair_values(uint32_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Eight E4M3 codes as fp32 (exact).
__device__ __forceinline__ void e4m3_values(uint2 c, float (&v)[8]) {
  const uint32_t w[4] = {c.x & 0xffffu, c.x >> 16, c.y & 0xffffu, c.y >> 16};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = e4m3_pair_values(w[i]);
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

__device__ __forceinline__ void bf16_values(uint4 q, float (&v)[8]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 bf16_pack(const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// ---------------------------------------------------------------------------
// row groups
// ---------------------------------------------------------------------------

// One warp: offs[0..E] in shared memory (each within the rows already) made
// non-decreasing, so that groups never overlap; a decreasing offset is
// recorded as MOE_ERR_DEVICE_BOUNDS.
__device__ __forceinline__ void ordered_offsets(int* offs, int E, int* status) {
  const int lane = threadIdx.x & 31;
  int top = 0;
  for (int g0 = 0; g0 <= E; g0 += 32) {
    const int g = g0 + lane, o = g <= E ? offs[g] : 0;
    int m = max(o, top);
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, m, s);
      if (lane >= s) m = max(m, v);
    }
    if (g <= E && m != o) {
      offs[g] = m;
      set_device_status(status, MOE_ERR_DEVICE_BOUNDS);
    }
    top = __shfl_sync(0xffffffffu, m, 31);
  }
  __syncwarp();
}

// ---------------------------------------------------------------------------
// launchers
// ---------------------------------------------------------------------------

moe_status quantize_blocks_launch(const void* x, bool f32, bool pow2, int rows, int cols, int64_t ldx,
                                  uint8_t* codes, float* scales, int num_sms, cudaStream_t s);

struct SwigluSaveArgs {
  int R, f;
  const void* g;
  const void* u;
  int64_t ld;
  void* h;             // nullable
  uint8_t* codes;      // nullable, with scales
  float* scales;
  uint8_t* saved;      // [2, R, f]
  float* saved_scales; // [2, R, ceil(f/128)]
};
moe_status swiglu_save_launch(const SwigluSaveArgs& a, int num_sms, cudaStream_t s);

struct SwigluBackwardArgs {
  int R, f;
  const uint8_t* saved;
  const float* saved_scales;
  const void* dh;
  void* dg;
  void* du;
  int64_t ld;
  void* h;             // nullable
  uint8_t* codes;      // nullable, [R, 2f], with scales [R, 2f/128]
  float* scales;
};
moe_status swiglu_backward_launch(const SwigluBackwardArgs& a, int num_sms, cudaStream_t s);

struct RouterLossArgs {
  int T, E, k;
  const float* logits;
  const int32_t* idx;
  const uint8_t* mask;  // nullable
  float balance, z;
  float* loss;          // [2]
  int32_t* counts;      // [E + 1]
  float* lse;           // [T]
  void* workspace;
  int num_sms;
  int* status;
};
size_t router_losses_workspace(int T, int E, int num_sms);
moe_status router_losses_launch(const RouterLossArgs& a, cudaStream_t s);

struct RouterLossGradArgs {
  int T, E, k;
  const float* logits;
  const int32_t* idx;
  const uint8_t* mask;   // nullable
  float balance, z;
  const int32_t* counts;
  const float* lse;
  const float* grad;     // nullable
  const float* w;        // nullable, with dw
  const float* dw;
  float* dlogits;
  int num_sms;
  int* status;
};
moe_status router_losses_backward_launch(const RouterLossGradArgs& a, cudaStream_t s);

struct BlockGemmArgs {
  int R, K, N, E;
  bool transposed, out_f32;
  const uint8_t* a;
  const float* a_scales;
  const int32_t* offsets;
  const uint8_t* w;
  const float* w_scales;
  void* out;
  int num_sms;
  int* status;
  long long timeout_ns;
};
moe_status block_gemm_launch(const BlockGemmArgs& a, cudaStream_t s);

struct WgradArgs {
  int R, N, K, E;
  const void* dy;
  int64_t ld_dy;
  const void* x;          // bf16, or E4M3 codes with x_scales
  const float* x_scales;  // nullable
  const int32_t* offsets;
  void* dw;
  bool out_f32, accumulate;
  int num_sms;
  int* status;
  long long timeout_ns;
};
moe_status grouped_wgrad_launch(const WgradArgs& a, cudaStream_t s);

}  // namespace moe
