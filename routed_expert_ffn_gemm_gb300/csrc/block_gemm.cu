// Grouped product of E4M3 rows with E4M3 weights, fp32 scales for blocks of
// 128 along the reduction (rows: 1 x 128, weights: 128 x 128):
//
//   y[r,n] = sum_kb sa[r,kb] sw[e,n/128,kb] sum_{i in block kb} a[r,i] w[e,n,i]
//
// for every row r of expert e.  The inner sum of a block is exact products
// accumulated in fp32 by the tensor cores; the scales change with kb, so a
// block's sum leaves tensor memory before the next one's scale applies and
// is added in fp32 registers: acc += (sa sw) * D.
//
// Orientation: the MMA's M side is output channels (weights are always full
// tiles), its N side rows, so that a few rows cost few columns.  A unit is
// 256 channels x up to 256 rows of one expert on a pair of CTAs (cta_group::2:
// each CTA stages its 128 channels and half of the rows, 32 KB a block, which
// halves the row bytes per SM; at one CTA per tile the 8-bit rate asks L2 for
// more than it gives).  A group's rows are cut into equal tiles of at most
// 256; each unit's rows come by the smallest of four copy boxes that holds
// them.  Units run row tiles first inside bands of 16, so that a weight tile
// is read from memory once while the band's rows stay in L2.
//
// Roles: warp 0 copies (TMA), warp 1 issues the MMAs, warp 2 prepares
// sa * sw of each block in shared memory, warps 4..11 hold the accumulators:
// each warp has 32 channels and alternate chunks of 32 rows.  Two
// accumulator buffers in tensor memory: one fills while the other is read.
//
// Transposed weights ([E, K, N]: the data gradient with the forward's
// arrays) are the same tiles read MN-major by the MMA.
#include <atomic>

#include "ptx.cuh"
#include "train.cuh"

namespace moe {
namespace {

constexpr int kThreads = 384;
constexpr int kBN = 256;                      // most rows of a unit
constexpr int kStages = 5;
constexpr int kABytes = 128 * 128, kBBytes = 128 * 128, kStageBytes = kABytes + kBBytes;
constexpr int kScaleSlots = 8;
constexpr int kEpiWarps = 8;
constexpr int kBand = 16;                     // row tiles that share a pass over the weights
constexpr int kOutPitch = 80;                 // bytes of a staged row of 32 channels (64), padded against conflicts
constexpr int kOutBytes = 32 * kOutPitch;     // per warp: 32 rows
constexpr int kMaxGroups = 1024;
constexpr int kOutOff = kStages * kStageBytes;
constexpr int kScaleOff = kOutOff + kEpiWarps * kOutBytes;
constexpr int kBarOff = kScaleOff + kScaleSlots * kBN * 4;
// full[S], empty[S], acc_full[2], acc_empty[2], scale_full[8], scale_empty[8], drain
constexpr int kNumBars = 2 * kStages + 4 + 2 * kScaleSlots + 1;
constexpr int kSlotOff = kBarOff + 8 * kNumBars;
constexpr int kAbortOff = kSlotOff + 8;
constexpr int kOffsOff = kAbortOff + 8;
constexpr int kPrefixOff = kOffsOff + 4 * (kMaxGroups + 4);
constexpr int kSmemBytes = kPrefixOff + 4 * (kMaxGroups + 4) + 1024;
static_assert(kSmemBytes <= 232448, "shared memory budget");
// every CTA holds all of its SM's tensor memory: never two on one SM
static_assert(2 * (kSmemBytes + 1024) > 232448 + 1024, "one CTA per SM");
// Registers: 384 x 168 at launch; the accumulating warps take what the
// other warpgroup gives back.
constexpr int kRegsLow = 80, kRegsHigh = 208;
static_assert(128 * kRegsLow + 256 * kRegsHigh <= kThreads * 168, "register split");

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
  CUtensorMap w;
  CUtensorMap a[4];  // boxes of 16, 32, 64, 128 rows
};

struct Unit {
  int g, row0, n_valid, n_mma, mt, tiles;
};

__device__ __forceinline__ Unit unit_of(int u, const int* offs, const int* prefix, int E, int MT) {
  const int t = u / MT;
  int lo = 0, hi = E - 1;  // the expert whose tiles hold t
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (prefix[mid] <= t) lo = mid; else hi = mid - 1;
  }
  Unit x;
  x.g = lo;
  x.tiles = prefix[lo + 1] - prefix[lo];
  const int l = u - prefix[lo] * MT;
  const int band = l / (kBand * MT), rem = l - band * (kBand * MT);
  const int wide = min(kBand, x.tiles - band * kBand);
  x.mt = rem / wide;
  const int rt = band * kBand + rem % wide;
  const int cnt = offs[lo + 1] - offs[lo];
  // equal tiles, multiples of 32 rows (the pair splits them in halves of 16)
  const int per = ((cnt + x.tiles - 1) / x.tiles + 31) / 32 * 32;
  x.row0 = offs[lo] + rt * per;
  x.n_valid = min(per, cnt - rt * per);
  x.n_mma = (x.n_valid + 31) / 32 * 32;
  return x;
}

// All lanes of the warp wait; the warp agrees on the outcome.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, uint64_t deadline, volatile int* abort) {
  return __all_sync(0xffffffffu, ptx::mbar_wait_bounded(bar, parity, deadline, abort)) != 0;
}

template <bool TRANS>
__global__ void __launch_bounds__(kThreads, 1) block_gemm_kernel(const Params p, const __grid_constant__ Maps maps) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_s = ptx::smem_u32(smem_raw);
  const uint32_t pad = (1024u - (raw_s & 1023u)) & 1023u;
  uint8_t* smem = smem_raw + pad;
  const uint32_t sbase = raw_s + pad, bars = sbase + kBarOff;
  auto full_bar = [&](int s) { return bars + 8u * s; };
  auto empty_bar = [&](int s) { return bars + 8u * (kStages + s); };
  auto accf_bar = [&](int b) { return bars + 8u * (2 * kStages + b); };
  auto acce_bar = [&](int b) { return bars + 8u * (2 * kStages + 2 + b); };
  auto sfull_bar = [&](int i) { return bars + 8u * (2 * kStages + 4 + i); };
  auto sempty_bar = [&](int i) { return bars + 8u * (2 * kStages + 4 + kScaleSlots + i); };
  const uint32_t drain_bar = bars + 8u * (2 * kStages + 4 + 2 * kScaleSlots);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kSlotOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kAbortOff);
  int* offs = reinterpret_cast<int*>(smem + kOffsOff);
  int* prefix = reinterpret_cast<int*>(smem + kPrefixOff);
  float* scales = reinterpret_cast<float*>(smem + kScaleOff);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = ptx::cluster_ctarank();
  const bool leader = rank == 0u;
  auto lead = [&](uint32_t bar) { return ptx::mapa_shared(bar, 0u); };
  const int u_first = (int)(blockIdx.x >> 1), u_step = (int)(gridDim.x >> 1);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(full_bar(s), 2);  // both producers, on the even CTA's barrier
      ptx::mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(accf_bar(b), 1);
      ptx::mbar_init(acce_bar(b), 2 * kEpiWarps);
    }
    for (int i = 0; i < kScaleSlots; ++i) {
      ptx::mbar_init(sfull_bar(i), 1);
      ptx::mbar_init(sempty_bar(i), kEpiWarps);
    }
    ptx::mbar_init(drain_bar, 1);
    *abort_flag = 0;
    ptx::fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    ptx::prefetch_tmap(&maps.w);
    for (int i = 0; i < 4; ++i) ptx::prefetch_tmap(&maps.a[i]);
  }
  if (warp == 1) {
    ptx::tmem_alloc<true>(ptx::smem_u32(tmem_slot), 512);
    ptx::tmem_relinquish<true>();
  }
  griddep_wait();
  griddep_launch_dependents();

  // group ranges, clamped into [0, R], and the prefix of their tile counts
  for (int g = threadIdx.x; g <= p.E; g += kThreads) {
    int o = p.offsets[g];
    if (o < 0 || o > p.R) {
      set_device_status(p.status, MOE_ERR_DEVICE_BOUNDS);
      o = o < 0 ? 0 : p.R;
    }
    offs[g] = o;
  }
  __syncthreads();
  if (warp == 0) {
    ordered_offsets(offs, p.E, p.status);
    int run = 0;
    for (int g0 = 0; g0 < p.E; g0 += 32) {
      const int g = g0 + lane;
      const int n = g < p.E ? (offs[g + 1] - offs[g] + kBN - 1) / kBN : 0;
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
  ptx::tc_fence_before();
  ptx::cluster_sync();  // (also: the peer's barriers are initialised)
  ptx::tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int units = prefix[p.E] * p.MT;
  const uint64_t deadline = ptx::globaltimer_ns() + (uint64_t)p.timeout_ns;

  if (warp < 4) {
    ptx::regs_dec<kRegsLow>();
    if (warp == 0 && lane == 0) {
      // ---------------------------------------------------------- copies
      const uint64_t once = ptx::policy_evict_first(), keep = ptx::policy_evict_normal();
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      long long issued = 0;
      for (int u = u_first; u < units && ok; u += u_step) {
        const Unit x = unit_of(u, offs, prefix, p.E, p.MT);
        const int half = x.n_mma / 2;
        const int box = half <= 16 ? 0 : half <= 32 ? 1 : half <= 64 ? 2 : 3;
        const CUtensorMap* am = &maps.a[box];
        const uint32_t bytes = kABytes + (16u << box) * 128u;
        const int ch = x.mt * 256 + (int)rank * 128, row = x.row0 + (int)rank * half;
        const uint64_t pol = x.tiles > 1 ? keep : once;
        for (int kb = 0; kb < p.KB; ++kb) {
          if (!ptx::mbar_wait_bounded(empty_bar(stage), phase ^ 1u, deadline, abort_flag)) {
            ok = false;
            break;
          }
          const uint32_t sa = sbase + stage * kStageBytes, fb = lead(full_bar(stage));
          ptx::mbar_arrive_expect_tx_cluster(fb, bytes);
          if (TRANS)
            ptx::tma_load_box3_pair(sa, &maps.w, fb, ch, kb * 128, x.g, pol);
          else
            ptx::tma_load_box3_pair(sa, &maps.w, fb, kb * 128, ch, x.g, pol);
          ptx::tma_load_2d_pair(sa + kABytes, am, fb, kb * 128, row, keep);
          ++issued;
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) {
        set_device_status(p.status, MOE_ERR_DEVICE_TIMEOUT);
        // let issued copies land before shared memory is released
        const uint64_t now = ptx::globaltimer_ns(), grace = now + 100000000ull;
        if (leader) {
          for (long long j = issued > kStages ? issued - kStages : 0; j < issued; ++j)
            while (!ptx::mbar_try_wait(full_bar((int)(j % kStages)), (uint32_t)((j / kStages) & 1)) &&
                   ptx::globaltimer_ns() < grace) {
            }
        } else {  // this CTA's copies complete the peer's barriers: wait a while
          while (ptx::globaltimer_ns() < now + 20000000ull) {
          }
        }
      }
    } else if (warp == 1 && lane == 0 && leader) {
      // ------------------------------------------------------------ MMAs
      int stage = 0;
      uint32_t phase = 0, it = 0;
      bool ok = true;
      for (int u = u_first; u < units && ok; u += u_step) {
        const Unit x = unit_of(u, offs, prefix, p.E, p.MT);
        const uint32_t idesc = ptx::idesc_f16_f32(256, x.n_mma) | (TRANS ? ptx::kIdescAMn : 0u);
        for (int kb = 0; kb < p.KB; ++kb, ++it) {
          const uint32_t buf = it & 1u, acc_phase = (it >> 1) & 1u;
          if (!ptx::mbar_wait_bounded(acce_bar(buf), acc_phase ^ 1u, deadline, abort_flag) ||
              !ptx::mbar_wait_bounded(full_bar(stage), phase, deadline, abort_flag)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          const uint32_t sa = sbase + stage * kStageBytes;
          const uint64_t da = TRANS ? ptx::sdesc_mn_sw128(sa, 16384) : ptx::sdesc_k_sw128(sa);
          const uint64_t db = ptx::sdesc_k_sw128(sa + kABytes);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)  // 32 of the block's 128 per instruction
            ptx::mma_f8_pair(tmem_base + 256u * buf, da + kk * (TRANS ? 4096 >> 4 : 2), db + 2 * kk, idesc, kk > 0);
          ptx::mma_commit_pair(empty_bar(stage));
          ptx::mma_commit_pair(accf_bar(buf));
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) {
        set_device_status(p.status, MOE_ERR_DEVICE_TIMEOUT);
        if (it > 0) {  // MMAs in flight end before tensor memory is freed
          ptx::mma_commit_pair(drain_bar);
          const uint64_t grace = ptx::globaltimer_ns() + 100000000ull;
          while (!ptx::mbar_try_wait(drain_bar, 0u) && ptx::globaltimer_ns() < grace) {
          }
        }
      }
    } else if (warp == 2) {
      // ---------------------------------------- sa * sw of each block
      uint32_t it = 0;
      bool ok = true;
      const bool vec = (p.KB & 3) == 0;
      for (int u = u_first; u < units && ok; u += u_step) {
        const Unit x = unit_of(u, offs, prefix, p.E, p.MT);
        const int nb = min(x.mt * 2 + (int)rank, p.NB - 1);  // (past N: zero weights, never stored)
        for (int kb = 0; kb < p.KB && ok; kb += 4) {
          float v[8][4], w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int k = min(kb + j, p.KB - 1);
            w[j] = __ldg(p.w_scales + (TRANS ? ((size_t)x.g * p.KB + k) * p.NB + nb
                                             : ((size_t)x.g * p.NB + nb) * p.KB + k));
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = lane + 32 * i;
            const float* src = p.a_scales + (size_t)(x.row0 + r) * p.KB + kb;
            if (r >= x.n_valid) {
              v[i][0] = v[i][1] = v[i][2] = v[i][3] = 0.f;
            } else if (vec) {
              const float4 q = __ldg(reinterpret_cast<const float4*>(src));
              v[i][0] = q.x; v[i][1] = q.y; v[i][2] = q.z; v[i][3] = q.w;
            } else {
#pragma unroll
              for (int j = 0; j < 4; ++j) v[i][j] = kb + j < p.KB ? __ldg(src + j) : 0.f;
            }
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (kb + j >= p.KB) break;
            const uint32_t slot = it % kScaleSlots;
            if (!warp_wait(sempty_bar(slot), ((it / kScaleSlots) & 1u) ^ 1u, deadline, abort_flag)) {
              ok = false;
              break;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (32 * i < x.n_mma) scales[slot * kBN + lane + 32 * i] = v[i][j] * w[j];
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(sfull_bar(slot));
            ++it;
          }
        }
      }
      if (!ok && lane == 0) set_device_status(p.status, MOE_ERR_DEVICE_TIMEOUT);
    }
  } else {
    // ------------------------------------------------------- accumulation
    ptx::regs_inc<kRegsHigh>();
    const int q = warp & 3, eg = (warp - 4) >> 2;
    uint8_t* outb = smem + kOutOff + (warp - 4) * kOutBytes;
    const uint32_t out_s = ptx::smem_u32(outb);
    const uint32_t tlane = tmem_base + ((uint32_t)(q * 32) << 16);
    uint32_t it = 0;
    bool ok = true;
    for (int u = u_first; u < units; u += u_step) {
      const Unit x = unit_of(u, offs, prefix, p.E, p.MT);
      // acc[chunk][lane half][column group][lane + 0 / 8]: pairs of rows
      uint64_t acc[4][2][4][2];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][h][j][0] = acc[i][h][j][1] = 0ull;
      for (int kb = 0; kb < p.KB; ++kb, ++it) {
        const uint32_t buf = it & 1u, slot = it % kScaleSlots;
        if (!warp_wait(sfull_bar(slot), (it / kScaleSlots) & 1u, deadline, abort_flag) ||
            !warp_wait(accf_bar(buf), (it >> 1) & 1u, deadline, abort_flag)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        const float* sc = scales + slot * kBN + 2 * (lane & 3);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c0 = (2 * i + eg) * 32;
          if (c0 < x.n_mma) {
            uint32_t d0[16], d1[16];
            ptx::tmem_ld_16x256b_x4(tlane + 256u * buf + c0, d0);
            ptx::tmem_ld_16x256b_x4(tlane + (16u << 16) + 256u * buf + c0, d1);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 s = *reinterpret_cast<const float2*>(sc + c0 + 8 * j);
              const uint64_t s2 = ptx::pack_f32x2(__float_as_uint(s.x), __float_as_uint(s.y));
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                acc[i][0][j][r] =
                    ptx::fma_f32x2(ptx::pack_f32x2(d0[4 * j + 2 * r], d0[4 * j + 2 * r + 1]), s2, acc[i][0][j][r]);
                acc[i][1][j][r] =
                    ptx::fma_f32x2(ptx::pack_f32x2(d1[4 * j + 2 * r], d1[4 * j + 2 * r + 1]), s2, acc[i][1][j][r]);
              }
            }
          }
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          ptx::mbar_arrive_cluster(lead(acce_bar(buf)));
          ptx::mbar_arrive(sempty_bar(slot));
        }
      }
      if (!ok) break;
      const int ch0 = x.mt * 256 + (int)rank * 128 + q * 32;
      if (ch0 >= p.N) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c0 = (2 * i + eg) * 32;
        if (c0 >= x.n_valid) break;
        if (p.out_f32) {
          float* out = static_cast<float*>(p.out);
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                float lo, hi;
                ptx::unpack_f32x2(acc[i][h][j][r], lo, hi);
                const int ch = ch0 + 16 * h + 8 * r + (lane >> 2), c = c0 + 8 * j + 2 * (lane & 3);
                if (ch < p.N) {
                  float* to = out + (size_t)(x.row0 + c) * p.N + ch;
                  if (c < x.n_valid) to[0] = lo;
                  if (c + 1 < x.n_valid) to[p.N] = hi;
                }
              }
        } else {
          // rows of 32 channels through shared memory: 16-byte stores
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t m[4];
#pragma unroll
            for (int o = 0; o < 4; ++o) {  // channels 8o .. 8o + 7
              float lo, hi;
              ptx::unpack_f32x2(acc[i][o >> 1][j][o & 1], lo, hi);
              const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
              m[o] = *reinterpret_cast<const uint32_t*>(&b);
            }
            ptx::stmatrix_x4_trans(out_s + (8 * j + (lane & 7)) * kOutPitch + (lane >> 3) * 16, m[0], m[1], m[2], m[3]);
          }
          __syncwarp();
          __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out);
          const int ch = ch0 + (lane & 3) * 8;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int rr = 8 * k + (lane >> 2), c = c0 + rr;
            const uint4 v = *reinterpret_cast<const uint4*>(outb + rr * kOutPitch + (lane & 3) * 16);
            if (c < x.n_valid && ch < p.N)
              *reinterpret_cast<uint4*>(out + (size_t)(x.row0 + c) * p.N + ch) = v;
          }
          __syncwarp();
        }
      }
    }
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

// CTAs (two per pair) that are resident at once: the grid is persistent and
// not every SM finds a partner.  One value per device, written once.
template <bool TRANS>
moe_status resident_ctas(int* out) {
  static std::atomic<int> known[64];
  int dev = 0;
  MOE_TRY_CUDA(cudaGetDevice(&dev));
  if (dev < 0 || dev >= 64) return MOE_ERR_UNSUPPORTED;
  int n = known[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    auto kern = block_gemm_kernel<TRANS>;
    MOE_TRY_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
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
  *out = 2 * n;
  return MOE_OK;
}

template <bool TRANS>
moe_status launch(const Params& p, const Maps& maps, int num_sms, cudaStream_t s) {
  int ctas = 0;
  MOE_TRY(resident_ctas<TRANS>(&ctas));
  // no more pairs than units can exist: row tiles <= R / 256 + one per group
  const long long tiles = (long long)p.R / kBN + (p.R < p.E ? p.R : p.E);
  const long long units = tiles * p.MT;
  int grid = ctas < num_sms ? ctas : num_sms & ~1;
  if (2 * units < grid) grid = (int)(2 * units);
  MOE_TRY_CUDA(launch_kc(2, block_gemm_kernel<TRANS>, dim3(grid), dim3(kThreads), kSmemBytes, s, p, maps));
  return MOE_OK;
}

}  // namespace

moe_status block_gemm_launch(const BlockGemmArgs& a, cudaStream_t s) {
  Params p{};
  p.R = a.R;
  p.K = a.K;
  p.N = a.N;
  p.E = a.E;
  p.MT = ceil_div(a.N, 256);
  p.KB = ceil_div(a.K, kQBlock);
  p.NB = ceil_div(a.N, kQBlock);
  p.out_f32 = a.out_f32;
  p.a_scales = a.a_scales;
  p.w_scales = a.w_scales;
  p.offsets = a.offsets;
  p.out = a.out;
  p.status = a.status;
  p.timeout_ns = a.timeout_ns;
  if (((long long)a.R / kBN + a.E) * p.MT > 0x7fffffffll) return MOE_ERR_UNSUPPORTED;
  Maps maps;
  if (a.transposed)
    MOE_TRY(make_tmap_3d(&maps.w, a.w, a.E, a.K, a.N, a.N, 1, 128, 128, 128));
  else
    MOE_TRY(make_tmap_3d(&maps.w, a.w, a.E, a.N, a.K, a.K, 1, 128, 128, 128));
  for (int i = 0; i < 4; ++i) MOE_TRY(make_tmap_2d(&maps.a[i], a.a, a.R, a.K, 1, 16u << i, 128, 128));
  return a.transposed ? launch<true>(p, maps, a.num_sms, s) : launch<false>(p, maps, a.num_sms, s);
}

}  // namespace moe
