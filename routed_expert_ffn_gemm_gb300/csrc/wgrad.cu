// Grouped weight gradient: for every expert e,
//
//   dw[e,n,k] = sum over the rows r of e of dy[r,n] x[r,k]      (+ dw[e,n,k])
//
// with dy bf16 and x either bf16 or E4M3 codes with a scale for each 1 x 128
// block (an 8-bit activation checkpoint).  The reduction runs over rows, so
// both operands are MN-major tiles of row-major arrays: 64 rows a stage, and
// the bf16 MMA reads them as they lie.  Codes are multiplied out to bf16 on
// the way: code * scale is exactly a bf16 value when the scale is a power of
// two (4 significant bits, fp32's exponent range); with any other scale it
// is rounded once to bf16.
//
// A unit is 256 x 256 of one expert's dw on a pair of CTAs (cta_group::2:
// 128 dy columns each, x columns split in halves).  Units run in bands of 8
// x tiles, so that the pairs at work share operand columns in L2.
// A group's last rows are followed by another expert's: those rows of the
// last stage are zeroed in shared memory (in both operands: 0 * NaN would
// not vanish) before the MMA reads them.
//
// The tensor cores accumulate 256 rows at a time in tensor memory; chunks
// are added in fp32 registers, so that the error of a long sum stays that
// of rounded fp32 adds.  Results leave through shared memory by TMA stores
// (clipped at the matrix' edge), or TMA adds in L2 when accumulating: each
// element gets one add, so the order cannot matter.
//
// Roles: warp 0 copies, warp 1 issues the MMAs, warps 4..7 prepare stages
// (codes to bf16, zeroed tails), warps 8..15 hold the accumulators.
//
// Bound by the tensor cores with many rows an expert (8 experts of 4096 x
// 14336, 8192 bf16 rows: 605 us, 1.6 PFLOP/s, while the clock holds; about 700
// call after call, under the power cap), by the conversions when those rows
// are codes (875 us), by writing dw with few (116 of 128 experts of 1536 x 2048 in
// fp32, 16384 rows of codes: 284 us, 6.0 TB/s).
#include <atomic>

#include "ptx.cuh"
#include "train.cuh"

namespace moe {
namespace {

constexpr int kThreads = 512;
constexpr int kRows = 64;                     // rows of a stage
constexpr int kChunkStages = 4;               // stages summed in tensor memory
constexpr int kTileBytes = kRows * 128 * 2;   // 128 columns of 64 rows, bf16: two 64-column halves
constexpr int kHalfBytes = kTileBytes / 2;
constexpr int kCodeBytes = kRows * 128;
constexpr int kEpiWarps = 8, kPrepWarps = 4;
constexpr int kBand = 8;
constexpr int kMaxGroups = 1024;
constexpr int kOutBufs = 2, kOutBytes = 32 * 64;  // per accumulating warp: staged boxes of 32 rows of 64 bytes

template <bool CODES>
struct Smem {
  static constexpr int STAGES = CODES ? 4 : 5;
  static constexpr int STAGE_BYTES = 2 * kTileBytes + (CODES ? kCodeBytes : 0);
  static constexpr int OUT_OFF = STAGES * STAGE_BYTES;
  static constexpr int BAR_OFF = OUT_OFF + kEpiWarps * kOutBufs * kOutBytes;
  // full[S], ready[S], empty[S], acc_full[2], acc_empty[2], drain
  static constexpr int NUM_BARS = 3 * STAGES + 5;
  static constexpr int SLOT_OFF = BAR_OFF + 8 * NUM_BARS + 8;
  static constexpr int ABORT_OFF = SLOT_OFF + 8;
  static constexpr int OFFS_OFF = ABORT_OFF + 8;
  static constexpr int BYTES = OFFS_OFF + 4 * (kMaxGroups + 4) + 1024;
  static_assert(BYTES <= 232448, "shared memory budget");
  // every CTA holds all of its SM's tensor memory: never two on one SM
  static_assert(2 * (BYTES + 1024) > 232448 + 1024, "one CTA per SM");
};
constexpr int kRegsLow = 40, kRegsPrep = 80, kRegsHigh = 192;
static_assert(128 * (kRegsLow + kRegsPrep + 2 * kRegsHigh) <= kThreads * 128, "register split");

struct Params {
  int R, N, K, E, NT, KT, KB;
  int out_f32, accumulate;
  const float* x_scales;
  const int32_t* offsets;
  int* status;
  long long timeout_ns;
};

struct Maps {
  CUtensorMap dy, x, dw;
};

struct Unit {
  int g, row0, rows, nt, kt, stages;
};

__device__ __forceinline__ Unit unit_of(int u, const int* offs, const Params& p) {
  Unit x;
  const int per = p.NT * p.KT;
  x.g = u / per;
  const int l = u - x.g * per;
  const int band = l / (kBand * p.NT), rem = l - band * (kBand * p.NT);
  const int wide = min(kBand, p.KT - band * kBand);
  x.nt = rem / wide;
  x.kt = band * kBand + rem % wide;
  x.row0 = offs[x.g];
  x.rows = offs[x.g + 1] - x.row0;
  x.stages = (x.rows + kRows - 1) / kRows;
  return x;
}

__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, uint64_t deadline, volatile int* abort) {
  return __all_sync(0xffffffffu, ptx::mbar_wait_bounded(bar, parity, deadline, abort)) != 0;
}

// 16 codes times their block's scale, as 8 pairs of bf16.  (Shifting a code's
// bits into a bf16 and multiplying by 2^120 times the scale takes as many
// instructions and measured slower, 1099 against 844 us at 8192 rows and 8
// experts of 4096 x 14336.)
__device__ __forceinline__ void codes_to_bf16(const uint32_t (&q)[4], float scale, uint32_t (&y)[8]) {
  const uint64_t s2 = ptx::pack_f32x2(__float_as_uint(scale), __float_as_uint(scale));
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float2 f = e4m3_pair_values(k & 1 ? q[k >> 1] >> 16 : q[k >> 1]);
    float lo, hi;
    ptx::unpack_f32x2(ptx::mul_f32x2(ptx::pack_f32x2(__float_as_uint(f.x), __float_as_uint(f.y)), s2), lo, hi);
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    y[k] = *reinterpret_cast<const uint32_t*>(&v);
  }
}

template <bool CODES>
__global__ void __launch_bounds__(kThreads, 1) wgrad_kernel(const Params p, const __grid_constant__ Maps maps) {
  using S = Smem<CODES>;
  constexpr int kStages = S::STAGES, kStageBytes = S::STAGE_BYTES;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_s = ptx::smem_u32(smem_raw);
  const uint32_t pad = (1024u - (raw_s & 1023u)) & 1023u;
  uint8_t* smem = smem_raw + pad;
  const uint32_t sbase = raw_s + pad, bars = sbase + S::BAR_OFF;
  auto full_bar = [&](int s) { return bars + 8u * s; };
  auto ready_bar = [&](int s) { return bars + 8u * (kStages + s); };
  auto empty_bar = [&](int s) { return bars + 8u * (2 * kStages + s); };
  auto accf_bar = [&](int b) { return bars + 8u * (3 * kStages + b); };
  auto acce_bar = [&](int b) { return bars + 8u * (3 * kStages + 2 + b); };
  const uint32_t drain_bar = bars + 8u * (3 * kStages + 4);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::SLOT_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::ABORT_OFF);
  int* offs = reinterpret_cast<int*>(smem + S::OFFS_OFF);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = ptx::cluster_ctarank();
  const bool leader = rank == 0u;
  auto lead = [&](uint32_t bar) { return ptx::mapa_shared(bar, 0u); };
  const int u_first = (int)(blockIdx.x >> 1), u_step = (int)(gridDim.x >> 1);
  const int units = p.E * p.NT * p.KT;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(full_bar(s), 1);
      ptx::mbar_init(ready_bar(s), 2 * kPrepWarps);
      ptx::mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(accf_bar(b), 1);
      ptx::mbar_init(acce_bar(b), 2 * kEpiWarps);
    }
    ptx::mbar_init(drain_bar, 1);
    *abort_flag = 0;
    ptx::fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    ptx::prefetch_tmap(&maps.dy);
    ptx::prefetch_tmap(&maps.x);
    ptx::prefetch_tmap(&maps.dw);
  }
  if (warp == 1) {
    ptx::tmem_alloc<true>(ptx::smem_u32(tmem_slot), 512);
    ptx::tmem_relinquish<true>();
  }
  griddep_wait();
  griddep_launch_dependents();
  for (int g = threadIdx.x; g <= p.E; g += kThreads) {
    int o = p.offsets[g];
    if (o < 0 || o > p.R) {
      set_device_status(p.status, MOE_ERR_DEVICE_BOUNDS);
      o = o < 0 ? 0 : p.R;
    }
    offs[g] = o;
  }
  __syncthreads();
  if (warp == 0) ordered_offsets(offs, p.E, p.status);
  ptx::tc_fence_before();
  ptx::cluster_sync();
  ptx::tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const uint64_t deadline = ptx::globaltimer_ns() + (uint64_t)p.timeout_ns;

  if (warp < 4) {
    ptx::regs_dec<kRegsLow>();
    if (warp == 0 && lane == 0) {
      // ---------------------------------------------------------- copies
      const uint64_t pol = ptx::policy_evict_normal();
      constexpr uint32_t bytes = kTileBytes + (CODES ? kCodeBytes : kTileBytes);
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      long long issued = 0;
      for (int u = u_first; u < units && ok; u += u_step) {
        const Unit x = unit_of(u, offs, p);
        const int n0 = x.nt * 256 + (int)rank * 128, k0 = x.kt * 256 + (int)rank * 128;
        for (int s = 0; s < x.stages; ++s) {
          if (!ptx::mbar_wait_bounded(empty_bar(stage), phase ^ 1u, deadline, abort_flag)) {
            ok = false;
            break;
          }
          const uint32_t sa = sbase + stage * kStageBytes, fb = full_bar(stage);
          const int row = x.row0 + s * kRows;
          ptx::mbar_arrive_expect_tx(fb, bytes);
          ptx::tma_load_box3(sa, &maps.dy, fb, n0, row, 0, pol);
          ptx::tma_load_box3(sa + kHalfBytes, &maps.dy, fb, n0 + 64, row, 0, pol);
          if (CODES) {
            ptx::tma_load_box3(sa + 2 * kTileBytes, &maps.x, fb, k0, row, 0, pol);
          } else {
            ptx::tma_load_box3(sa + kTileBytes, &maps.x, fb, k0, row, 0, pol);
            ptx::tma_load_box3(sa + kTileBytes + kHalfBytes, &maps.x, fb, k0 + 64, row, 0, pol);
          }
          ++issued;
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // every stage's last arrival from the even CTA, too, before the CTA may leave
      for (long long j = issued > kStages ? issued - kStages : 0; j < issued && ok; ++j)
        ok = ptx::mbar_wait_bounded(empty_bar((int)(j % kStages)), (uint32_t)((j / kStages) & 1), deadline, abort_flag);
      if (!ok) {
        set_device_status(p.status, MOE_ERR_DEVICE_TIMEOUT);
        const uint64_t grace = ptx::globaltimer_ns() + 100000000ull;
        for (long long j = issued > kStages ? issued - kStages : 0; j < issued; ++j)
          while (!ptx::mbar_try_wait(full_bar((int)(j % kStages)), (uint32_t)((j / kStages) & 1)) &&
                 ptx::globaltimer_ns() < grace) {
          }
      }
    } else if (warp == 1 && leader) {
      // ------------------------------------------------------------ MMAs
      // (the whole warp walks the loop and one elected lane issues)
      const uint32_t one = ptx::elect_one() ? 1u : 0u;
      const uint32_t idesc = ptx::idesc_bf16_f32(256, 256) | ptx::kIdescAMn | ptx::kIdescBMn;
      const uint64_t da0 = ptx::sdesc_mn_sw128(sbase, kHalfBytes);
      const uint64_t db0 = ptx::sdesc_mn_sw128(sbase + kTileBytes, kHalfBytes);
      int stage = 0;
      uint32_t phase = 0, it = 0;
      bool ok = true, any = false, seen = false;
      for (int u = u_first; u < units && ok; u += u_step) {
        const Unit x = unit_of(u, offs, p);
        for (int s = 0; s < x.stages; ++s) {
          const uint32_t buf = it & 1u;
          const bool first = s % kChunkStages == 0;
          ok = (!first || ptx::mbar_wait_bounded(acce_bar(buf), ((it >> 1) & 1u) ^ 1u, deadline, abort_flag)) &&
               (seen || ptx::mbar_wait_bounded(ready_bar(stage), phase, deadline, abort_flag));
          ok = __all_sync(0xffffffffu, ok) != 0;
          if (!ok) break;
          ptx::tc_fence_after();
          const uint64_t da = da0 + (uint32_t)(stage * (kStageBytes >> 4)), db = db0 + (uint32_t)(stage * (kStageBytes >> 4));
          const uint32_t d = tmem_base + 256u * buf;
          const int steps = (min(kRows, x.rows - s * kRows) + 15) / 16;
          for (int kk = 0; kk < steps; ++kk)  // 16 rows (two 8-row groups) per instruction
            ptx::mma_f16_pair_one(one, d, da + kk * (2048 >> 4), db + kk * (2048 >> 4), idesc, !first || kk > 0);
          any = true;
          ptx::mma_commit_pair_one(one, empty_bar(stage));
          if (s % kChunkStages == kChunkStages - 1 || s == x.stages - 1) {
            ptx::mma_commit_pair_one(one, accf_bar(buf));
            ++it;
          }
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
          seen = ptx::mbar_test_wait(ready_bar(stage), phase);  // (the answer comes while the MMAs run)
        }
      }
      if (!ok && one) {
        set_device_status(p.status, MOE_ERR_DEVICE_TIMEOUT);
        if (any) {
          ptx::mma_commit_pair(drain_bar);
          const uint64_t grace = ptx::globaltimer_ns() + 100000000ull;
          while (!ptx::mbar_try_wait(drain_bar, 0u) && ptx::globaltimer_ns() < grace) {
          }
        }
      }
    }
  } else if (warp < 8) {
    // --------------------------------------------------- stage preparation
    ptx::regs_dec<kRegsPrep>();
    const int w = warp - 4;
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int u = u_first; u < units && ok; u += u_step) {
      const Unit x = unit_of(u, offs, p);
      // the scales' column block is this CTA's 128 x columns
      const int kb = min(x.kt * 2 + (int)rank, p.KB - 1);
      auto scale_of = [&](int r) {  // row r of the group
        return CODES && r < x.rows ? __ldg(p.x_scales + (size_t)(x.row0 + r) * p.KB + kb) : 0.f;
      };
      float s0 = scale_of(lane), s1 = scale_of(lane + 32);
      for (int s = 0; s < x.stages; ++s) {
        const int valid = min(kRows, x.rows - s * kRows);
        const float n0 = scale_of((s + 1) * kRows + lane), n1 = scale_of((s + 1) * kRows + lane + 32);
        if (!warp_wait(full_bar(stage), phase, deadline, abort_flag)) {
          ok = false;
          break;
        }
        uint8_t* st = smem + stage * kStageBytes;
        if (CODES) {
          // lane: rows lane and lane + 32; warp: code chunks w and w + 4 of a
          // row (16 codes): chunk j sits at j ^ (row & 7), its two bf16
          // chunks at (2 (j & 3) + i) ^ (row & 7) of column half j / 4
          // (all four chunks are read first: one warp a scheduler has to hide the
          // latencies of its own conversions)
          uint4 c[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = lane + 32 * (i >> 1), j = w + 4 * (i & 1);
            c[i] = *reinterpret_cast<const uint4*>(st + 2 * kTileBytes + r * 128 + ((j ^ (r & 7)) << 4));
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = lane + 32 * (i >> 1);
            const uint32_t q[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
            uint32_t y[8];
            codes_to_bf16(q, i >> 1 ? s1 : s0, y);
            if (r >= valid)
#pragma unroll
              for (int k = 0; k < 8; ++k) y[k] = 0u;
            uint8_t* to = st + kTileBytes + (i & 1) * kHalfBytes + r * 128;
            *reinterpret_cast<uint4*>(to + (((2 * w) ^ (r & 7)) << 4)) = make_uint4(y[0], y[1], y[2], y[3]);
            *reinterpret_cast<uint4*>(to + (((2 * w + 1) ^ (r & 7)) << 4)) = make_uint4(y[4], y[5], y[6], y[7]);
          }
        }
        if (valid & 15) {
          // the rows after the group's last, up to the MMA's step: zeros
          const int end = (valid + 15) / 16 * 16, parts = CODES ? 2 : 4;
          for (int i = w * 32 + lane; i < (end - valid) * parts * 8; i += kPrepWarps * 32) {
            const int c = i & 7, part = (i >> 3) % parts, r = valid + (i >> 3) / parts;
            *reinterpret_cast<uint4*>(st + part * kHalfBytes + r * 128 + c * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive_cluster(lead(ready_bar(stage)));
        s0 = n0;
        s1 = n1;
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok && lane == 0) set_device_status(p.status, MOE_ERR_DEVICE_TIMEOUT);
  } else {
    // ------------------------------------------------------- accumulation
    ptx::regs_inc<kRegsHigh>();
    const int q = warp & 3, eg = (warp - 8) >> 2;
    uint8_t* outb = smem + S::OUT_OFF + (warp - 8) * kOutBufs * kOutBytes;
    const uint32_t out_s = ptx::smem_u32(outb);
    const uint32_t tlane = tmem_base + ((uint32_t)(q * 32) << 16);
    uint32_t it = 0, boxes = 0;
    bool ok = true;
    for (int u = u_first; u < units; u += u_step) {
      const Unit x = unit_of(u, offs, p);
      if (x.stages == 0 && p.accumulate) continue;
      uint64_t acc[4][16];  // chunk of 32 columns, pairs
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) acc[i][j] = 0ull;
      for (int s = 0; s < x.stages; s += kChunkStages, ++it) {
        const uint32_t buf = it & 1u;
        if (!warp_wait(accf_bar(buf), (it >> 1) & 1u, deadline, abort_flag)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        const uint32_t at = tlane + 256u * buf + eg * 32;
        uint32_t d[2][16];
        ptx::tmem_ld16(at, d[0]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // the next 16 columns are on their way while 16 are added
            const int n = 2 * i + h, next = n + 1;
            ptx::tmem_ld_wait();
            if (next < 8) {
              ptx::tmem_ld16(at + (next >> 1) * 64 + (next & 1) * 16, d[h ^ 1]);
            } else {  // everything is in registers: the buffer can fill again
              ptx::tc_fence_before();
              __syncwarp();
              if (lane == 0) ptx::mbar_arrive_cluster(lead(acce_bar(buf)));
            }
#pragma unroll
            for (int j = 0; j < 8; ++j)
              acc[i][8 * h + j] = ptx::add_f32x2(acc[i][8 * h + j], ptx::pack_f32x2(d[h][2 * j], d[h][2 * j + 1]));
          }
        }
      }
      if (!ok) break;
      const int n0 = x.nt * 256 + (int)rank * 128 + q * 32;
      if (n0 >= p.N) continue;
      const int per = p.out_f32 ? 16 : 32;  // columns in 64 bytes
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (h == 1 && !p.out_f32) break;
          const int k0 = x.kt * 256 + (2 * i + eg) * 32 + h * per;
          if (k0 >= p.K) break;
          if (lane == 0) ptx::bulk_wait_read<kOutBufs - 1>();  // the box before the last has left its buffer
          __syncwarp();
          const uint32_t ob = (uint32_t)(boxes++ % kOutBufs) * kOutBytes;
          // 16-byte chunk c of row r at c ^ ((r >> 1) & 3): the box' 64-byte swizzle
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint4 v;
            if (p.out_f32) {
              float4 f;
              ptx::unpack_f32x2(acc[i][8 * h + 2 * c], f.x, f.y);
              ptx::unpack_f32x2(acc[i][8 * h + 2 * c + 1], f.z, f.w);
              v = *reinterpret_cast<const uint4*>(&f);
            } else {
              float f[8];
#pragma unroll
              for (int j = 0; j < 4; ++j) ptx::unpack_f32x2(acc[i][4 * c + j], f[2 * j], f[2 * j + 1]);
              v = bf16_pack(f);
            }
            *reinterpret_cast<uint4*>(outb + ob + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4)) = v;
          }
          ptx::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (p.accumulate)
              ptx::tma_add_box3(&maps.dw, out_s + ob, k0, n0, x.g);
            else
              ptx::tma_store_box3(&maps.dw, out_s + ob, k0, n0, x.g);
            ptx::bulk_commit();
          }
        }
      }
    }
    if (lane == 0) ptx::bulk_wait_all();
    if (!ok && lane == 0) set_device_status(p.status, MOE_ERR_DEVICE_TIMEOUT);
  }

  __syncwarp();
  ptx::tc_fence_before();
  ptx::cluster_sync();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc<true>(tmem_base, 512);
  }
}

template <bool CODES>
moe_status launch(const Params& p, const Maps& maps, int num_sms, cudaStream_t s) {
  // resident pairs: the grid is persistent and not every SM finds a partner
  // (one value per device, written once)
  static std::atomic<int> known[64];
  auto kern = wgrad_kernel<CODES>;
  int dev = 0;
  MOE_TRY_CUDA(cudaGetDevice(&dev));
  if (dev < 0 || dev >= 64) return MOE_ERR_UNSUPPORTED;
  int n = known[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    MOE_TRY_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<CODES>::BYTES));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Smem<CODES>::BYTES;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    MOE_TRY_CUDA(cudaOccupancyMaxActiveClusters(&n, kern, &cfg));
    if (n < 1) return MOE_ERR_UNSUPPORTED;
    known[dev].store(n, std::memory_order_relaxed);
  }
  const long long units = (long long)p.E * p.NT * p.KT;
  int grid = 2 * n < num_sms ? 2 * n : num_sms & ~1;
  if (2 * units < grid) grid = (int)(2 * units);
  MOE_TRY_CUDA(launch_kc(2, kern, dim3(grid), dim3(kThreads), Smem<CODES>::BYTES, s, p, maps));
  return MOE_OK;
}

}  // namespace

moe_status grouped_wgrad_launch(const WgradArgs& a, cudaStream_t s) {
  Params p{};
  p.R = a.R;
  p.N = a.N;
  p.K = a.K;
  p.E = a.E;
  p.NT = ceil_div(a.N, 256);
  p.KT = ceil_div(a.K, 256);
  p.KB = ceil_div(a.K, kQBlock);
  p.out_f32 = a.out_f32;
  p.accumulate = a.accumulate;
  p.x_scales = a.x_scales;
  p.offsets = a.offsets;
  p.status = a.status;
  p.timeout_ns = a.timeout_ns;
  if ((long long)a.E * p.NT * p.KT > 0x7fffffffll) return MOE_ERR_UNSUPPORTED;
  const bool codes = a.x_scales != nullptr;
  Maps maps;
  MOE_TRY(make_tmap_3d(&maps.dy, a.dy, 1, a.R, a.N, (uint64_t)a.ld_dy * 2, 2, kRows, 64, 128));
  if (codes)
    MOE_TRY(make_tmap_3d(&maps.x, a.x, 1, a.R, a.K, a.K, 1, kRows, 128, 128));
  else
    MOE_TRY(make_tmap_3d(&maps.x, a.x, 1, a.R, a.K, (uint64_t)a.K * 2, 2, kRows, 64, 128));
  const int es = a.out_f32 ? 4 : 2;
  MOE_TRY(make_tmap_3d(&maps.dw, a.dw, a.E, a.N, a.K, (uint64_t)a.K * es, es, 32, 64 / es, 64));
  return codes ? launch<true>(p, maps, a.num_sms, s) : launch<false>(p, maps, a.num_sms, s);
}

}  // namespace moe
