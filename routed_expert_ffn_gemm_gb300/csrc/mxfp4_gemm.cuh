// Shared by the 4-bit product's kernels.
#pragma once

#include "block_gemm.cuh"
#include "mxfp4.cuh"

namespace moe {
namespace mx_gemm {

using block_gemm::Place;
using block_gemm::kMaxGroups;
using block_gemm::place_of;
using block_gemm::row_tiles;
using block_gemm::warp_wait;

constexpr int kStep = 256;             // of the reduction in a stage: rows of 128 bytes, 8 scales each
constexpr int kAtom = 512;             // scales of 128 rows x 4 blocks as the tensor cores take them

struct Params {
  int R, K, N, E, MT, KS, KB;          // MT: channel tiles, KS: stages of a unit, KB: scale blocks of a row
  int out_f32;
  const uint8_t* a_scales;
  const uint8_t* w_scales;
  const int32_t* offsets;
  void* out;
  int64_t ld_out;
  int* status;
  long long timeout_ns;
};

struct Maps {
  CUtensorMap w;     // 128 channels x 128 bytes (256 codes)
  CUtensorMap a[5];  // boxes of 8 << i rows
};

// How many stages this CTA (or pair) walks in all.
__device__ __forceinline__ long long my_steps(int u_first, int u_step, int units, int KS) {
  return u_first < units ? (long long)((units - 1 - u_first) / u_step + 1) * KS : 0;
}

// A walk over the stages of a CTA's units.
template <int ROWS>
struct Walk {
  const int *offs, *prefix;
  int E, MT, KS, units, u_step;
  int u, ks;
  Place x;
  __device__ __forceinline__ void start(const Params& p, const int* o, const int* pre, int first, int step, int n) {
    offs = o;
    prefix = pre;
    E = p.E;
    MT = p.MT;
    KS = p.KS;
    units = n;
    u_step = step;
    u = first;
    ks = 0;
    if (u < units) x = place_of<ROWS>(u, offs, prefix, E, MT);
  }
  __device__ __forceinline__ bool live() const { return u < units; }
  __device__ __forceinline__ void next() {
    if (++ks < KS) return;
    ks = 0;
    u += u_step;
    if (u < units) x = place_of<ROWS>(u, offs, prefix, E, MT);
  }
};

// The lane's part of the scales of 128 channels x 8 blocks: channels
// ch .. ch + 3 of each block (words along N; N % 16 == 0).  0 past the matrix.
__device__ __forceinline__ void load_weight_scales(const Params& p, int g, int ch, int ks, uint32_t (&w)[8]) {
  const uint8_t* from = p.w_scales + ((size_t)g * p.KB + (size_t)ks * 8) * p.N + ch;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    w[j] = ch < p.N && ks * 8 + j < p.KB ? __ldg(reinterpret_cast<const uint32_t*>(from + (size_t)j * p.N)) : 0u;
}
// ... to two atoms: rows of the lane's four channels from `m` on.
__device__ __forceinline__ void write_weight_scales(uint8_t* atoms, int m, const uint32_t (&w)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t a = __byte_perm(w[4 * h], w[4 * h + 1], 0x5140), b = __byte_perm(w[4 * h + 2], w[4 * h + 3], 0x5140);
    const uint32_t c = __byte_perm(w[4 * h], w[4 * h + 1], 0x7362), d = __byte_perm(w[4 * h + 2], w[4 * h + 3], 0x7362);
    const uint32_t of[4] = {__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632), __byte_perm(c, d, 0x5410),
                            __byte_perm(c, d, 0x7632)};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<uint32_t*>(atoms + h * kAtom + ((m + i) & 31) * 16 + ((m + i) >> 5) * 4) = of[i];
  }
}

// The scales of row `row` (8 blocks), 0 past its end or where it is not `live`.
__device__ __forceinline__ void load_row_scales(const Params& p, bool live, long long row, int ks, uint32_t (&w)[2]) {
  w[0] = w[1] = 0u;
  if (!live) return;
  const uint8_t* from = p.a_scales + (size_t)row * p.KB + (size_t)ks * 8;
  const int n = p.KB - ks * 8;
  if ((p.KB & 3) == 0) {
    w[0] = __ldg(reinterpret_cast<const uint32_t*>(from));
    if (n > 4) w[1] = __ldg(reinterpret_cast<const uint32_t*>(from) + 1);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) w[j >> 2] |= (uint32_t)__ldg(from + j) << (8 * (j & 3));
  }
}

}  // namespace mx_gemm
}  // namespace moe
