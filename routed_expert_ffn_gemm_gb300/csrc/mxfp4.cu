// MXFP4 rows and weights: quantiser, its reading back, and SwiGLU to MXFP4.
//
// A lane holds a whole block of 32 columns: it reads 64 bytes of bf16 (128 of
// fp32), finds the block's maximum without its neighbours, and writes 16 bytes
// of codes and one of scale, which lie side by side over the lanes.  Each
// element is read once and written once.  Memory bounds the quantiser and its
// reading back (16 x 4096 x 7168 in bf16 165 and 173 us, 7.2 and 6.9 TB/s;
// 16384 x 7168 in fp32 83 and 95), instructions SwiGLU (65536 x 768 43 us, 5.3
// TB/s: two special functions and some fifteen others an element).
// Scales of weights go by block first ([K/32, N] of a matrix), so there a CTA
// takes 32 rows x 32 blocks and turns the tile's scales in shared memory.
#include "mxfp4.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 32;  // rows and blocks of a tile of weights
constexpr uint64_t kMaxGrid = 1 << 20;

template <bool F32, bool WIDE>
__global__ void __launch_bounds__(kThreads) quantize_rows_kernel(const uint8_t* __restrict__ x, uint32_t tasks,
                                                                 uint32_t nb, int64_t ldx, int fit,
                                                                 uint4* __restrict__ codes,
                                                                 uint8_t* __restrict__ scales) {
  griddep_begin();
  const uint32_t step = gridDim.x * kThreads;
  for (uint32_t t = blockIdx.x * kThreads + threadIdx.x; t < tasks; t += step) {
    const uint32_t row = t / nb, kb = t - row * nb;
    MxBlock<F32> b;
    load_words<MxBlock<F32>::WORDS, WIDE>(x + ((size_t)row * ldx + (size_t)kb * kMxBlock) * (F32 ? 4 : 2), b.w);
    uint4 c;
    scales[t] = (uint8_t)b.codes(fit != 0, c);
    codes[t] = c;
  }
}

// A tile's place: matrix, first row in it, first block.
struct Tile {
  uint32_t m, n0, kb0;
};
__device__ __forceinline__ Tile tile_of(uint32_t t, uint32_t tiles_n, uint32_t tiles_k) {
  const uint32_t m = t / (tiles_n * tiles_k), r = t - m * (tiles_n * tiles_k);
  return {m, r / tiles_k * kTile, r % tiles_k * kTile};
}

template <bool F32, bool WIDE>
__global__ void __launch_bounds__(kThreads) quantize_weights_kernel(const uint8_t* __restrict__ x, uint32_t tiles,
                                                                    uint32_t nb, uint32_t N, int64_t ldx, int fit,
                                                                    uint4* __restrict__ codes,
                                                                    uint8_t* __restrict__ scales) {
  griddep_begin();
  __shared__ __align__(4) uint8_t sc[kTile][kTile + 4];  // [block][row], read four rows at a time
  const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
  const uint32_t tiles_n = (N + kTile - 1) / kTile, tiles_k = (nb + kTile - 1) / kTile;
  for (uint32_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const Tile o = tile_of(t, tiles_n, tiles_k);
    const uint32_t kb = o.kb0 + lane;
#pragma unroll
    for (uint32_t i = 0; i < kTile * 32 / kThreads; ++i) {
      const uint32_t n = o.n0 + warp + i * (kThreads / 32);
      if (n >= N || kb >= nb) continue;
      const size_t row = (size_t)o.m * N + n;
      MxBlock<F32> b;
      load_words<MxBlock<F32>::WORDS, WIDE>(x + (row * ldx + (size_t)kb * kMxBlock) * (F32 ? 4 : 2), b.w);
      uint4 c;
      sc[lane][n - o.n0] = (uint8_t)b.codes(fit != 0, c);
      codes[row * nb + kb] = c;
    }
    __syncthreads();
    const uint32_t k = threadIdx.x >> 3, r = (threadIdx.x & 7u) * 4u;  // four rows of a block
    if (o.kb0 + k < nb) {
      uint8_t* to = scales + ((size_t)o.m * nb + o.kb0 + k) * N + o.n0 + r;
      if ((N & 3u) == 0u) {
        if (o.n0 + r < N) *reinterpret_cast<uint32_t*>(to) = *reinterpret_cast<const uint32_t*>(&sc[k][r]);
      } else {
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i)
          if (o.n0 + r + i < N) to[i] = sc[k][r + i];
      }
    }
    __syncthreads();
  }
}

template <bool F32, bool WIDE>
__device__ __forceinline__ void write_values(uint4 c, uint32_t byte, uint8_t* out) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  const float s = mx_scale(byte);
  uint32_t o[F32 ? 32 : 16];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float v[8];
    e2m1_values(w[i], v);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= s;
    if constexpr (F32) {
#pragma unroll
      for (int j = 0; j < 8; ++j) o[8 * i + j] = __float_as_uint(v[j]);
    } else {
      const uint4 q = bf16_pack(v);
      o[4 * i] = q.x;
      o[4 * i + 1] = q.y;
      o[4 * i + 2] = q.z;
      o[4 * i + 3] = q.w;
    }
  }
  store_words<F32 ? 32 : 16, WIDE>(out, o);
}

template <bool F32, bool WIDE>
__global__ void __launch_bounds__(kThreads) row_values_kernel(const uint4* __restrict__ codes,
                                                              const uint8_t* __restrict__ scales, uint32_t tasks,
                                                              uint8_t* __restrict__ out) {
  griddep_begin();
  const uint32_t step = gridDim.x * kThreads;
  for (uint32_t t = blockIdx.x * kThreads + threadIdx.x; t < tasks; t += step)
    write_values<F32, WIDE>(codes[t], scales[t], out + (size_t)t * kMxBlock * (F32 ? 4 : 2));
}

template <bool F32, bool WIDE>
__global__ void __launch_bounds__(kThreads) weight_values_kernel(const uint4* __restrict__ codes,
                                                                 const uint8_t* __restrict__ scales, uint32_t tiles,
                                                                 uint32_t nb, uint32_t N, uint8_t* __restrict__ out) {
  griddep_begin();
  __shared__ __align__(4) uint8_t sc[kTile][kTile + 4];
  const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
  const uint32_t tiles_n = (N + kTile - 1) / kTile, tiles_k = (nb + kTile - 1) / kTile;
  for (uint32_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const Tile o = tile_of(t, tiles_n, tiles_k);
    const uint32_t k = threadIdx.x >> 3, r = (threadIdx.x & 7u) * 4u;
    if (o.kb0 + k < nb) {
      const uint8_t* from = scales + ((size_t)o.m * nb + o.kb0 + k) * N + o.n0 + r;
      if ((N & 3u) == 0u) {
        if (o.n0 + r < N) *reinterpret_cast<uint32_t*>(&sc[k][r]) = *reinterpret_cast<const uint32_t*>(from);
      } else {
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i)
          if (o.n0 + r + i < N) sc[k][r + i] = from[i];
      }
    }
    __syncthreads();
    const uint32_t kb = o.kb0 + lane;
#pragma unroll
    for (uint32_t i = 0; i < kTile * 32 / kThreads; ++i) {
      const uint32_t n = o.n0 + warp + i * (kThreads / 32);
      if (n >= N || kb >= nb) continue;
      const size_t at = ((size_t)o.m * N + n) * nb + kb;
      write_values<F32, WIDE>(codes[at], sc[lane][n - o.n0], out + at * kMxBlock * (F32 ? 4 : 2));
    }
    __syncthreads();
  }
}

template <bool WIDE>
__global__ void __launch_bounds__(kThreads) swiglu_mxfp4_kernel(const SwigluMxArgs a, uint32_t tasks, uint32_t nb) {
  griddep_begin();
  const uint32_t step = gridDim.x * kThreads;
  for (uint32_t t = blockIdx.x * kThreads + threadIdx.x; t < tasks; t += step) {
    const uint32_t row = t / nb, kb = t - row * nb;
    const size_t at = (size_t)row * a.ld + (size_t)kb * kMxBlock;
    MxBlock<false> g, u;
    load_words<16, WIDE>(static_cast<const __nv_bfloat16*>(a.g) + at, g.w);
    load_words<16, WIDE>(static_cast<const __nv_bfloat16*>(a.u) + at, u.w);
    MxBlock<true> h;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float g0 = __uint_as_float(g.w[i] << 16), g1 = __uint_as_float(g.w[i] & 0xffff0000u);
      h.w[2 * i] = __float_as_uint(g0 * sigmoid(g0) * __uint_as_float(u.w[i] << 16));
      h.w[2 * i + 1] = __float_as_uint(g1 * sigmoid(g1) * __uint_as_float(u.w[i] & 0xffff0000u));
    }
    uint4 c;
    a.scales[t] = (uint8_t)h.codes(a.fit, c);
    reinterpret_cast<uint4*>(a.codes)[t] = c;
    if (a.h != nullptr) {
      uint32_t o[16];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float v[8];
        h.values(8 * i, v, 1.f);
        const uint4 q = bf16_pack(v);
        o[4 * i] = q.x;
        o[4 * i + 1] = q.y;
        o[4 * i + 2] = q.z;
        o[4 * i + 3] = q.w;
      }
      store_words<16, false>(static_cast<uint8_t*>(a.h) + (size_t)t * kMxBlock * 2, o);
    }
  }
}

// CTAs for n of `each` a CTA, one round of them: a fixed grid of 8 CTAs an SM ends
// in a round that is partly empty (SwiGLU of 65536 x 768: 5.05 rounds).
unsigned grid_of(uint64_t n, uint64_t each) {
  const uint64_t want = (n + each - 1) / each;
  return (unsigned)(want < kMaxGrid ? want : kMaxGrid);
}

// Counts that, with a last partial step past them, have to fit 32 bits.
bool fits(uint64_t n) { return n <= 0x7fffffffull; }

bool aligned32(const void* p, int64_t pitch_bytes) {
  return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)pitch_bytes) & 31u) == 0;
}

}  // namespace

moe_status quantize_mxfp4_launch(const void* x, bool f32, bool fit, int rows, int cols, int matrix_rows, int64_t ldx,
                                 uint8_t* codes, uint8_t* scales, cudaStream_t s) {
  const uint32_t nb = (uint32_t)(cols / kMxBlock);
  const uint64_t tasks = (uint64_t)rows * nb;
  if (!fits(tasks)) return MOE_ERR_UNSUPPORTED;
  const bool wide = aligned32(x, ldx * (f32 ? 4 : 2));
  const uint8_t* xb = static_cast<const uint8_t*>(x);
  uint4* cb = reinterpret_cast<uint4*>(codes);
  if (matrix_rows == 0) {
    auto kern = f32 ? (wide ? quantize_rows_kernel<true, true> : quantize_rows_kernel<true, false>)
                    : (wide ? quantize_rows_kernel<false, true> : quantize_rows_kernel<false, false>);
    MOE_TRY_CUDA(launch_k(kern, dim3(grid_of(tasks, kThreads)), dim3(kThreads), 0, s, xb, (uint32_t)tasks, nb,
                          ldx, (int)fit, cb, scales));
    return MOE_OK;
  }
  const uint64_t tiles = (uint64_t)(rows / matrix_rows) * ceil_div(matrix_rows, kTile) * ceil_div((int)nb, kTile);
  auto kern = f32 ? (wide ? quantize_weights_kernel<true, true> : quantize_weights_kernel<true, false>)
                  : (wide ? quantize_weights_kernel<false, true> : quantize_weights_kernel<false, false>);
  MOE_TRY_CUDA(launch_k(kern, dim3(grid_of(tiles, 1)), dim3(kThreads), 0, s, xb, (uint32_t)tiles, nb,
                        (uint32_t)matrix_rows, ldx, (int)fit, cb, scales));
  return MOE_OK;
}

moe_status mxfp4_values_launch(const uint8_t* codes, const uint8_t* scales, bool f32, int rows, int cols,
                               int matrix_rows, void* out, cudaStream_t s) {
  const uint32_t nb = (uint32_t)(cols / kMxBlock);
  const uint64_t tasks = (uint64_t)rows * nb;
  if (!fits(tasks)) return MOE_ERR_UNSUPPORTED;
  const bool wide = aligned32(out, 0);
  const uint4* cb = reinterpret_cast<const uint4*>(codes);
  uint8_t* ob = static_cast<uint8_t*>(out);
  if (matrix_rows == 0) {
    auto kern = f32 ? (wide ? row_values_kernel<true, true> : row_values_kernel<true, false>)
                    : (wide ? row_values_kernel<false, true> : row_values_kernel<false, false>);
    MOE_TRY_CUDA(launch_k(kern, dim3(grid_of(tasks, kThreads)), dim3(kThreads), 0, s, cb, scales,
                          (uint32_t)tasks, ob));
    return MOE_OK;
  }
  const uint64_t tiles = (uint64_t)(rows / matrix_rows) * ceil_div(matrix_rows, kTile) * ceil_div((int)nb, kTile);
  auto kern = f32 ? (wide ? weight_values_kernel<true, true> : weight_values_kernel<true, false>)
                  : (wide ? weight_values_kernel<false, true> : weight_values_kernel<false, false>);
  MOE_TRY_CUDA(launch_k(kern, dim3(grid_of(tiles, 1)), dim3(kThreads), 0, s, cb, scales, (uint32_t)tiles, nb,
                        (uint32_t)matrix_rows, ob));
  return MOE_OK;
}

moe_status swiglu_mxfp4_launch(const SwigluMxArgs& a, cudaStream_t s) {
  const uint32_t nb = (uint32_t)(a.f / kMxBlock);
  const uint64_t tasks = (uint64_t)a.R * nb;
  if (!fits(tasks)) return MOE_ERR_UNSUPPORTED;
  const bool wide = aligned32(a.g, a.ld * 2) && aligned32(a.u, 0);
  auto kern = wide ? swiglu_mxfp4_kernel<true> : swiglu_mxfp4_kernel<false>;
  MOE_TRY_CUDA(launch_k(kern, dim3(grid_of(tasks, kThreads)), dim3(kThreads), 0, s, a, (uint32_t)tasks, nb));
  return MOE_OK;
}

}  // namespace moe
