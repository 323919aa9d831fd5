// MXFP4: blocks of 32 values in E2M1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their
// negatives) with a power of two 2^(b - 127) each; b = 255 is NaN.  Declarations
// shared by the translation units of the 4-bit and token-movement operators.
#pragma once

#include <cuda_fp16.h>

#include "train.cuh"

namespace moe {

constexpr int kMxBlock = 32;

// The scale byte of a block whose largest magnitude has the bits `amax`:
// p = floor(log2 a) - 2 is the exponent field less 129, so b = p + 127 the field
// less 2 (subnormal magnitudes: the least scale); with `fit` one more where
// a / 2^p in [4, 8) is above 6.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax, bool fit) {
  const int e = (int)(amax >> 23);
  if (amax >= 0x7f800000u) return 255u;
  if (amax == 0u) return 127u;
  return (uint32_t)max(e - 2 + (fit && (amax & 0x7fffffu) > 0x400000u ? 1 : 0), 0);
}

// 2^(127 - b): what values are multiplied by before rounding (exact; always a
// normal number).  0 for a NaN block, whose codes are 0.
__device__ __forceinline__ float mx_inverse(uint32_t b) { return __uint_as_float(b == 255u ? 0u : (254u - b) << 23); }

// 2^(b - 127), NaN for 255.
__device__ __forceinline__ float mx_scale(uint32_t b) {
  return __uint_as_float(b == 0u ? 0x400000u : b == 255u ? 0x7fffffffu : b << 23);
}

// Eight values to codes, the first in the low four bits: nearest, ties to the
// even code, saturating.
__device__ __forceinline__ uint32_t e2m1x8(const float* v) {
  uint32_t w;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}\n"
      : "=r"(w)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return w;
}

// Eight codes as fp32 (exact).
__device__ __forceinline__ void e2m1_values(uint32_t w, float* v) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}\n"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

// N words from global memory, 32 bytes at a time where the address allows.
template <int N, bool WIDE>
__device__ __forceinline__ void load_words(const void* p, uint32_t (&w)[N]) {
  const uint32_t* q = static_cast<const uint32_t*>(p);
  if constexpr (WIDE) {
#pragma unroll
    for (int i = 0; i < N; i += 8)
      asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                   : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3]), "=r"(w[i + 4]), "=r"(w[i + 5]),
                     "=r"(w[i + 6]), "=r"(w[i + 7])
                   : "l"(q + i));
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const uint4 t = *reinterpret_cast<const uint4*>(q + i);
      w[i] = t.x;
      w[i + 1] = t.y;
      w[i + 2] = t.z;
      w[i + 3] = t.w;
    }
  }
}
template <int N, bool WIDE>
__device__ __forceinline__ void store_words(void* p, const uint32_t (&w)[N]) {
  uint32_t* q = static_cast<uint32_t*>(p);
  if constexpr (WIDE) {
#pragma unroll
    for (int i = 0; i < N; i += 8)
      asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(q + i), "r"(w[i]), "r"(w[i + 1]),
                   "r"(w[i + 2]), "r"(w[i + 3]), "r"(w[i + 4]), "r"(w[i + 5]), "r"(w[i + 6]), "r"(w[i + 7])
                   : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) *reinterpret_cast<uint4*>(q + i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
  }
}

// A block as loaded (16 words of bf16 pairs, or 32 of fp32), its largest
// magnitude's bits and its values.
template <bool F32>
struct MxBlock {
  static constexpr int WORDS = F32 ? 32 : 16;
  uint32_t w[WORDS];

  __device__ __forceinline__ uint32_t amax() const {
    uint32_t m = 0u;
    if constexpr (F32) {
#pragma unroll
      for (int i = 0; i < 32; ++i) m = max(m, w[i] & 0x7fffffffu);
      return m;
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
      return max(m << 16, m & 0xffff0000u);
    }
  }
  __device__ __forceinline__ void values(int first, float (&v)[8], float r) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int j = first + i;
      const uint32_t bits = F32 ? w[j % WORDS] : (j & 1) ? w[(j >> 1) % WORDS] & 0xffff0000u : w[(j >> 1) % WORDS] << 16;
      v[i] = __uint_as_float(bits) * r;
    }
  }
  // The scale byte, and the 32 codes.
  __device__ __forceinline__ uint32_t codes(bool fit, uint4& c) const {
    const uint32_t b = mx_scale_byte(amax(), fit);
    const float r = mx_inverse(b);
    uint32_t out[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float v[8];
      values(8 * i, v, r);
      out[i] = b == 255u ? 0u : e2m1x8(v);
    }
    c = make_uint4(out[0], out[1], out[2], out[3]);
    return b;
  }
};

// ---------------------------------------------------------------------------
// launchers
// ---------------------------------------------------------------------------

moe_status quantize_mxfp4_launch(const void* x, bool f32, bool fit, int rows, int cols, int matrix_rows, int64_t ldx,
                                 uint8_t* codes, uint8_t* scales, cudaStream_t s);
moe_status mxfp4_values_launch(const uint8_t* codes, const uint8_t* scales, bool f32, int rows, int cols,
                               int matrix_rows, void* out, cudaStream_t s);

struct SwigluMxArgs {
  int R, f;
  bool fit;
  const void* g;
  const void* u;
  int64_t ld;
  uint8_t* codes;
  uint8_t* scales;
  void* h;  // nullable
};
moe_status swiglu_mxfp4_launch(const SwigluMxArgs& a, cudaStream_t s);

struct DispatchArgs {
  int T, d, E, k;
  bool f32, to_mx, fit;
  const void* x;         // nullable: maps alone
  int64_t ldx;
  const int32_t* idx;
  int32_t* counts;
  int32_t* offsets;
  int32_t* row_token;
  int32_t* inv_row;
  void* rows;            // nullable with x
  uint8_t* row_scales;
  int32_t* chunks;       // workspace
  int num_sms;
  int* status;
};
size_t dispatch_workspace(int T, int E, int k);
moe_status dispatch_launch(const DispatchArgs& a, cudaStream_t s);

struct CombineRowsArgs {
  int T, d, k, R;
  bool f32;
  const void* rows;
  const int32_t* inv_row;
  const float* w;        // nullable: ones
  const void* add;       // nullable
  void* out;
  int num_sms;
  int* status;
};
moe_status combine_rows_launch(const CombineRowsArgs& a, cudaStream_t s);

struct CombineRowsGradArgs {
  int T, d, k, R;
  bool f32;
  const void* d_out;
  const void* rows;      // nullable when dw is
  const int32_t* inv_row;
  const float* w;        // nullable: ones
  void* d_rows;          // nullable
  float* dw;             // nullable
  int num_sms;
  int* status;
};
moe_status combine_rows_backward_launch(const CombineRowsGradArgs& a, cudaStream_t s);

struct MxGemmArgs {
  int R, K, N, E;
  bool out_f32;
  const uint8_t* a;
  const uint8_t* a_scales;
  const int32_t* offsets;
  const uint8_t* w;
  const uint8_t* w_scales;
  void* out;
  int64_t ld_out;
  int num_sms;
  int* status;
  long long timeout_ns;
};
moe_status mxfp4_gemm_launch(const MxGemmArgs& a, cudaStream_t s);

}  // namespace moe
