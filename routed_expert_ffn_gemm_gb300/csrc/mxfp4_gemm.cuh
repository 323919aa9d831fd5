// Shared by the 4-bit product's kernels.
#pragma once

#include "block_gemm.cuh"
#include "mxfp4.cuh"

namespace moe {
namespace mx_gemm {

using block_gemm::Place;
using block_gemm::kBand;
using block_gemm::kMaxGroups;
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
  CUtensorMap ws;    // weights' scales: 8 blocks of 128 channels (256 for a pair)
  CUtensorMap out;   // 32 rows of 64 bytes (a pair's)
};

// Group ranges, clamped into [0, R] and ordered, and the prefix of their counts
// of ROWS-row tiles, in shared memory, as block_gemm's row_tiles; a lane takes
// consecutive groups, so that there is one scan of each kind over the warp (256
// groups: 0.3 us of a launch instead of 1.4).  The whole CTA calls this and
// synchronises afterwards.
template <int ROWS>
__device__ __forceinline__ void group_tiles(const Params& p, int* offs, int* prefix, int threads) {
  for (int g = threadIdx.x; g <= p.E; g += threads) {
    int o = p.offsets[g];
    if (o < 0 || o > p.R) {
      set_device_status(p.status, MOE_ERR_DEVICE_BOUNDS);
      o = o < 0 ? 0 : p.R;
    }
    offs[g] = o;
  }
  __syncthreads();
  if (threadIdx.x >= 32) return;
  const int lane = threadIdx.x, each = p.E / 32 + 1;
  const int g0 = min(lane * each, p.E + 1), g1 = min(g0 + each, p.E + 1);
  int top = 0;
  for (int g = g0; g < g1; ++g) top = max(top, offs[g]);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, top, o);
    if (lane >= o) top = max(top, v);
  }
  int run = __shfl_up_sync(0xffffffffu, top, 1);
  if (lane == 0) run = 0;
  for (int g = g0; g < g1; ++g) {  // a decreasing offset becomes the largest before it
    const int o = offs[g];
    run = max(run, o);
    if (run != o) {
      offs[g] = run;
      set_device_status(p.status, MOE_ERR_DEVICE_BOUNDS);
    }
  }
  __syncwarp();
  const int e1 = min(g1, p.E);
  int sum = 0;
  for (int g = g0; g < e1; ++g) sum += (offs[g + 1] - offs[g] + ROWS - 1) / ROWS;
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  int at = incl - sum;
  for (int g = g0; g < g1; ++g) {
    prefix[g] = at;
    if (g < p.E) at += (offs[g + 1] - offs[g] + ROWS - 1) / ROWS;
  }
}

// 2^32 / n rounded up, n from 2 to kBand.
static_assert(kBand == 16, "kInverse");
static __constant__ const unsigned kInverse[kBand + 1] = {
    0u,          0u,          0x80000000u, 0x55555556u, 0x40000000u,
    0x33333334u, 0x2aaaaaabu, 0x24924925u, 0x20000000u, 0x1c71c71du,
    0x1999999au, 0x1745d175u, 0x15555556u, 0x13b13b14u,
    0x12492493u, 0x11111112u, 0x10000000u};

// Where a warp's units are, asked in ascending order: block_gemm's place_of (row
// tiles of ROWS rows first inside bands of kBand) in some 100 cycles instead of
// 1200, which every role would spend on every unit (65536 rows on 128 experts of
// 768 x 2048, three stages a unit: 88 us before, 76 here).  The expert is
// sought from the last one on by all lanes at once, and the one division left is
// by a number up to kBand.
template <int ROWS>
struct Units {
  const int *offs, *prefix;
  int E, MT, g;
  __device__ __forceinline__ Units(const Params& p, const int* o, const int* pre)
      : offs(o), prefix(pre), E(p.E), MT(p.MT), g(0) {}

  // (the whole warp)
  __device__ __forceinline__ Place at(int u) {
    const int lane = threadIdx.x & 31;
    for (;;) {  // the last expert that begins at or before u
      const int next = g + 1 + lane;
      const int n = __popc(__ballot_sync(0xffffffffu, next < E && prefix[min(next, E)] * MT <= u));
      g += n;
      if (n < 32) break;
    }
    Place x;
    x.g = g;
    x.tiles = prefix[g + 1] - prefix[g];
    int rem = u - prefix[g] * MT, tile0 = 0;
    if (x.tiles > kBand) {
      tile0 = rem / (kBand * MT) * kBand;
      rem -= tile0 * MT;
    }
    const int wide = min(kBand, x.tiles - tile0);
    // rem / wide: exact by a multiplication with 2^32 / wide rounded up, as
    // rem * kBand < 2^32
    x.mt = wide == 1 ? rem : (int)__umulhi((unsigned)rem, kInverse[wide]);
    x.row0 = offs[g] + (tile0 + rem - x.mt * wide) * ROWS;
    x.n_valid = min(ROWS, offs[g + 1] - x.row0);
    return x;
  }
};

// The scales of 128 channels x 8 blocks from where a copy left them ([8 blocks]
// [PITCH channels]) to two atoms `STEP` bytes apart: each lane turns four
// channels' bytes of four blocks.
template <int PITCH, int STEP>
__device__ __forceinline__ void weight_scale_atoms(const uint8_t* raw, uint8_t* atoms) {
  const int m = 4 * (threadIdx.x & 31);
  uint32_t w[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) w[j] = *reinterpret_cast<const uint32_t*>(raw + j * PITCH + m);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t a = __byte_perm(w[4 * h], w[4 * h + 1], 0x5140), b = __byte_perm(w[4 * h + 2], w[4 * h + 3], 0x5140);
    const uint32_t c = __byte_perm(w[4 * h], w[4 * h + 1], 0x7362), d = __byte_perm(w[4 * h + 2], w[4 * h + 3], 0x7362);
    const uint32_t of[4] = {__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632), __byte_perm(c, d, 0x5410),
                            __byte_perm(c, d, 0x7632)};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<uint32_t*>(atoms + h * STEP + ((m + i) & 31) * 16 + ((m + i) >> 5) * 4) = of[i];
  }
}

// Four words of a row's scales: the 16 blocks from `kb` on, by the widest loads
// that the rows' alignment allows.  0 past the row's end and where it is not
// `live` (blocks past K need any scale that is not NaN: their codes are 0).
__device__ __forceinline__ void load_row_scales(const Params& p, bool live, long long row, int kb, uint32_t (&w)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = 0u;
  if (!live) return;
  const uint8_t* from = p.a_scales + (size_t)row * p.KB + kb;
  const int left = p.KB - kb;
  if ((p.KB & 15) == 0) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(from));
    w[0] = v.x;
    w[1] = v.y;
    w[2] = v.z;
    w[3] = v.w;
  } else if ((p.KB & 7) == 0) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (8 * i < left) {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(from) + i);
        w[2 * i] = v.x;
        w[2 * i + 1] = v.y;
      }
  } else if ((p.KB & 3) == 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (4 * i < left) w[i] = __ldg(reinterpret_cast<const uint32_t*>(from) + i);
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (j < left) w[j >> 2] |= (uint32_t)__ldg(from + j) << (8 * (j & 3));
  }
}

// One warp: the scales of this CTA's rows (32 GROUPS of the unit's ROWS, from
// `first` on) to two atoms a stage; lane 0's arrival on the stage's `raw` tells.
// A lane holds rows lane + 32 i: a word of four blocks of each, side by side, is
// 16 bytes of an atom.  Two stages' scales are one 16-byte load a row, kSets such
// sets are on their way in registers.  The warp that loads must not fence: a
// proxy fence waits for the loads in flight, which made each stage take the 1100
// cycles of a load (16384 rows of 8 experts, 4096 -> 28672: 1120 us with loads in
// front of the fence, 917 with 4-byte asynchronous copies, 626 here).
template <int ROWS, int GROUPS, int STAGES, typename Empty, typename Raw>
__device__ __forceinline__ bool row_scales(const Params& p, const int* offs, const int* prefix, int u_first, int u_step,
                                           int units, int first, uint8_t* atoms, int stage_bytes, Empty empty_bar,
                                           Raw raw_bar, uint64_t deadline, volatile int* abort_flag) {
  constexpr int kSets = 3;
  const int lane = threadIdx.x & 31, pairs = (p.KS + 1) / 2;
  int u = u_first, at = 0;  // what is loaded next
  Units<ROWS> places(p, offs, prefix);
  Place x;
  x.row0 = x.n_valid = 0;
  uint32_t v[kSets][GROUPS][4];
  auto load = [&](uint32_t (&to)[GROUPS][4]) {
    if (u >= units) return;
    if (at == 0) x = places.at(u);
#pragma unroll
    for (int i = 0; i < GROUPS; ++i) {
      const int r = first + lane + 32 * i;
      load_row_scales(p, r < x.n_valid, (long long)x.row0 + r, 16 * at, to[i]);
    }
    if (++at == pairs) {
      at = 0;
      u += u_step;
    }
  };
#pragma unroll
  for (int j = 0; j < kSets; ++j) {
#pragma unroll
    for (int i = 0; i < GROUPS; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) v[j][i][k] = 0u;
    load(v[j]);
  }
  const long long sets = u_first < units ? (long long)((units - 1 - u_first) / u_step + 1) * pairs : 0;
  uint32_t it = 0;
  int pair = 0;
  bool ok = true;
  for (long long i0 = 0; i0 < sets && ok; i0 += kSets) {
#pragma unroll
    for (int j = 0; j < kSets; ++j) {
      if (!ok || i0 + j >= sets) break;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        if (!ok || 2 * pair + half >= p.KS) break;
        const uint32_t s = it % STAGES;
        ok = warp_wait(empty_bar(s), ((it / STAGES) & 1u) ^ 1u, deadline, abort_flag);
        if (!ok) break;
        ++it;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = i < GROUPS ? v[j][i % GROUPS][2 * half + h] : 0u;
          uint8_t* to = atoms + s * stage_bytes + h * kAtom + lane * 16;
          if constexpr (GROUPS > 2)
            *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
          else
            *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[1]);
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(raw_bar(s));
      }
      load(v[j]);
      if (++pair == pairs) pair = 0;
    }
  }
  return ok;
}

}  // namespace mx_gemm

moe_status mxfp4_gemm_many_launch(const mx_gemm::Params& p, const mx_gemm::Maps& maps, int num_sms, cudaStream_t s);

}  // namespace moe
