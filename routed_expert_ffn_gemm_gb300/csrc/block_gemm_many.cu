// The block product (block_gemm.cu) where experts have many rows: a unit is 256
// rows x 256 channels of one expert on a pair of CTAs with one MMA for both
// (cta_group::2, M = 256): each CTA holds 128 rows and the weights of half of
// the channels, 32 KB a block of 128, where MMAs of its own would need 48.
// (Shared memory bounds those: 48 KB written and 48 KB read a block at 128
// bytes a cycle are 768 cycles, the block's MMAs 512.)
//
// Rows are the MMA's M side, so a lane of tensor memory is a row and its scale
// one value a block and 128 channels.  The two halves of 128 channels have two
// buffers of 128 columns each, are issued by a warp each (1 and 3 of the even
// CTA) and added by four warps of each CTA each (4..11), so that one half is
// on its way while the other is read.  Warp 0 of each CTA copies, warp 2
// brings the scales.
//
// What bounds it is the adding warps' chain of waits: a block of 8192 rows x
// 4096 x 14336 takes a pair about 1000 cycles, its MMAs 512, its copies some
// 650, its adds 256 issue slots; two warps a scheduler (128 sums a lane, all
// of the register file) do not hide the waits for a barrier, for tensor memory
// and for shared memory, which MMAs and copies keep busy.  Hence the reads
// ahead: a group's scales at once (460 -> 427 us), the next buffer's barrier
// polled while this one is added (427 -> 415), two staged store boxes (415 ->
// 402), the unit's place handed on by warp 2 instead of searched for in front
// of the stores (12 blocks a unit, 128 experts: 246 -> 234, graph replays; a
// call takes 260).  Measured: 8192 rows of 4 experts 4096 -> 14336 in 395 us,
// 2.4 PFLOP/s;
// clusters of four with an MMA for each CTA and four buffers took 606, a
// quarter of the columns a hand-over 590, one issuing warp for both halves 483.
#include "block_gemm.cuh"

namespace moe {
namespace {

using namespace block_gemm;

constexpr int kThreads = 384;
constexpr int kTileBytes = 128 * 128;         // an operand: 128 rows or channels, 128 codes of the reduction
constexpr int kHalfBytes = kTileBytes / 2;    // 64 channels of each half of 128
constexpr int kStages = 5, kStageBytes = 2 * kTileBytes;
constexpr int kBuffers = 4;                   // of 128 columns: two for each half
constexpr int kGroup = 4, kScaleRing = 3;     // blocks whose scales are handed over at once; such groups in flight
constexpr int kEpiWarps = 8, kChunks = 4;     // chunks of 32 channels of an accumulating warp
constexpr int kOutBufs = 2;                   // staged store boxes of an accumulating warp
constexpr int kOutOff = kStages * kStageBytes;
constexpr int kScaleOff = kOutOff + kEpiWarps * kOutBufs * kOutBytes;
constexpr int kWScaleOff = kScaleOff + kScaleRing * kGroup * 128 * 4;
constexpr int kPlaceOff = kWScaleOff + kScaleRing * kGroup * 8;  // [ring][half][block]
constexpr int kBarOff = kPlaceOff + kScaleRing * 16;             // row0, n_valid, mt of the group's unit
// full[S], empty[S], acc_full[4], acc_empty[4], scale_full[3], scale_empty[3], drain[2]
constexpr int kNumBars = 2 * kStages + 2 * kBuffers + 2 * kScaleRing + 2;
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
constexpr int kRegsLow = 72, kRegsHigh = 216;
static_assert(128 * kRegsLow + 256 * kRegsHigh <= kThreads * 168, "register split");

template <bool TRANS>
__global__ void __launch_bounds__(kThreads, 1) block_gemm_many_kernel(const Params p,
                                                                      const __grid_constant__ Maps maps) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_s = ptx::smem_u32(smem_raw);
  const uint32_t pad = (1024u - (raw_s & 1023u)) & 1023u;
  uint8_t* smem = smem_raw + pad;
  const uint32_t sbase = raw_s + pad, bars = sbase + kBarOff;
  auto full_bar = [&](uint32_t s) { return bars + 8u * s; };
  auto empty_bar = [&](uint32_t s) { return bars + 8u * (kStages + s); };
  auto accf_bar = [&](uint32_t b) { return bars + 8u * (2 * kStages + b); };
  auto acce_bar = [&](uint32_t b) { return bars + 8u * (2 * kStages + kBuffers + b); };
  auto sfull_bar = [&](uint32_t i) { return bars + 8u * (2 * kStages + 2 * kBuffers + i); };
  auto sempty_bar = [&](uint32_t i) { return bars + 8u * (2 * kStages + 2 * kBuffers + kScaleRing + i); };
  auto drain_bar = [&](uint32_t i) { return bars + 8u * (2 * kStages + 2 * kBuffers + 2 * kScaleRing + i); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kSlotOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kAbortOff);
  int* offs = reinterpret_cast<int*>(smem + kOffsOff);
  int* prefix = reinterpret_cast<int*>(smem + kPrefixOff);
  float* scales = reinterpret_cast<float*>(smem + kScaleOff);
  float* wscales = reinterpret_cast<float*>(smem + kWScaleOff);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = ptx::cluster_ctarank();
  const bool leader = rank == 0u;
  auto lead = [&](uint32_t bar) { return ptx::mapa_shared(bar, 0u); };
  const int u_first = (int)(blockIdx.x >> 1), u_step = (int)(gridDim.x >> 1);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(full_bar(s), 2);   // (the even CTA's: both CTAs' copies)
      ptx::mbar_init(empty_bar(s), 2);  // both halves' MMAs
    }
    for (int b = 0; b < kBuffers; ++b) {
      ptx::mbar_init(accf_bar(b), 1);
      ptx::mbar_init(acce_bar(b), kEpiWarps);  // (the even CTA's: a half's four warps of both CTAs)
    }
    for (int i = 0; i < kScaleRing; ++i) {
      ptx::mbar_init(sfull_bar(i), 33);  // each lane's copies, and the unit's place
      ptx::mbar_init(sempty_bar(i), kEpiWarps);
    }
    ptx::mbar_init(drain_bar(0), 1);
    ptx::mbar_init(drain_bar(1), 1);
    *abort_flag = 0;
    ptx::fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    ptx::prefetch_tmap(&maps.w);
    ptx::prefetch_tmap(&maps.a[4]);
    ptx::prefetch_tmap(&maps.out);
  }
  if (warp == 1) {
    ptx::tmem_alloc<true>(ptx::smem_u32(tmem_slot), 512);
    ptx::tmem_relinquish<true>();
  }
  griddep_wait();
  griddep_launch_dependents();
  row_tiles<256>(p, offs, prefix, kThreads);
  ptx::tc_fence_before();
  ptx::cluster_sync();  // (also: the peers' barriers are initialised)
  ptx::tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int units = prefix[p.E] * p.MT;
  const uint64_t deadline = ptx::globaltimer_ns() + (uint64_t)p.timeout_ns;

  if (warp < 4) {
    ptx::regs_dec<kRegsLow>();
    if (warp == 0 && lane == 0) {
      // ---------------------------------------------------------- copies
      const uint64_t keep = ptx::policy_evict_normal();
      uint32_t it = 0;
      bool ok = true;
      for (int u = u_first; u < units && ok; u += u_step) {
        const Place x = place_of<256>(u, offs, prefix, p.E, p.MT);
        const int row = x.row0 + (int)rank * 128, ch = x.mt * 256 + (int)rank * 64;
        for (int kb = 0; kb < p.KB; ++kb, ++it) {
          const uint32_t s = it % kStages;
          if (!ptx::mbar_wait_bounded(empty_bar(s), ((it / kStages) & 1u) ^ 1u, deadline, abort_flag)) {
            ok = false;
            break;
          }
          const uint32_t at = sbase + s * kStageBytes, fb = lead(full_bar(s));
          ptx::mbar_arrive_expect_tx_cluster(fb, kStageBytes);
          ptx::tma_load_2d_pair(at, &maps.a[4], fb, kb * 128, row, keep);
#pragma unroll
          for (int h = 0; h < 2; ++h)
            ptx::tma_load_box3_pair(at + kTileBytes + h * kHalfBytes, &maps.w, fb, TRANS ? ch + 128 * h : kb * 128,
                                    TRANS ? kb * 128 : ch + 128 * h, x.g, keep);
        }
      }
      // every slot's last arrival from the even CTA, too, before the CTA may leave
      for (uint32_t j = it > kStages ? it - kStages : 0; j < it && ok; ++j)
        ok = ptx::mbar_wait_bounded(empty_bar(j % kStages), (j / kStages) & 1u, deadline, abort_flag);
      if (!ok) {
        set_device_status(p.status, MOE_ERR_DEVICE_TIMEOUT);
        // let issued copies land before shared memory is released (the even
        // CTA's barriers tell; the peer's part may never come: the limit ends
        // the wait)
        const uint64_t grace = ptx::globaltimer_ns() + 100000000ull;
        if (leader) {
          for (uint32_t j = it > kStages ? it - kStages : 0; j < it; ++j)
            while (!ptx::mbar_try_wait(full_bar(j % kStages), (j / kStages) & 1u) && ptx::globaltimer_ns() < grace) {
            }
        } else {
          while (ptx::globaltimer_ns() < grace) {
          }
        }
      }
    } else if ((warp & 1) && leader) {
      // ------------------------------- MMAs of channel half `h` for both CTAs
      const uint32_t one = ptx::elect_one() ? 1u : 0u, h = (uint32_t)(warp >> 1);
      const uint32_t idesc = ptx::idesc_f16_f32(256, 128) | (TRANS ? ptx::kIdescBMn : 0u);
      const uint32_t b_s = sbase + kTileBytes + h * kHalfBytes;
      const uint64_t da0 = ptx::sdesc_k_sw128(sbase);
      const uint64_t db0 = TRANS ? ptx::sdesc_mn_sw64(b_s, kHalfBytes) : ptx::sdesc_k_sw128(b_s);
      constexpr uint32_t bstep = TRANS ? 2048 >> 4 : 2;
      const long long mine = u_first < units ? (long long)((units - 1 - u_first) / u_step + 1) * p.KB : 0;
      uint32_t slot = 0, sphase = 0, buf = 0, bphase = 1, seen = 0;
      bool ok = true, any = false;
      for (long long i = 0; i < mine; ++i) {
        ok = ((seen & 1u) || ptx::mbar_wait_bounded(full_bar(slot), sphase, deadline, abort_flag)) &&
             ((seen & 2u) || ptx::mbar_wait_bounded(acce_bar(2 * buf + h), bphase, deadline, abort_flag));
        ok = __all_sync(0xffffffffu, ok) != 0;
        if (!ok) break;
        ptx::tc_fence_after();
        const uint64_t da = da0 + slot * (kStageBytes >> 4), db = db0 + slot * (kStageBytes >> 4);
        const uint32_t d = tmem_base + 128u * (2 * buf + h);
        ptx::mma_f8_pair_one<false>(one, d, da, db, idesc);  // 32 of the block's 128 each
        ptx::mma_f8_pair_one<true>(one, d, da + 2, db + bstep, idesc);
        ptx::mma_f8_pair_one<true>(one, d, da + 4, db + 2 * bstep, idesc);
        ptx::mma_f8_pair_one<true>(one, d, da + 6, db + 3 * bstep, idesc);
        ptx::mma_commit_pair_one(one, accf_bar(2 * buf + h));
        ptx::mma_commit_pair_one(one, empty_bar(slot));
        any = true;
        if (++slot == kStages) {
          slot = 0;
          sphase ^= 1u;
        }
        buf ^= 1u;
        if (buf == 0) bphase ^= 1u;
        // (the answers come while the MMAs run)
        seen = i + 1 < mine ? ptx::mbar_test2(full_bar(slot), sphase, acce_bar(2 * buf + h), bphase) : 0u;
      }
      if (!ok && one) {
        set_device_status(p.status, MOE_ERR_DEVICE_TIMEOUT);
        if (any) {  // MMAs in flight end before tensor memory is freed
          ptx::mma_commit_pair(drain_bar(h));
          const uint64_t grace = ptx::globaltimer_ns() + 100000000ull;
          while (!ptx::mbar_try_wait(drain_bar(h), 0u) && ptx::globaltimer_ns() < grace) {
          }
        }
      }
    } else if (warp == 2) {
      // ------------------------------------------------- scales, by cp.async
      uint32_t it = 0;
      bool ok = true;
      for (int u = u_first; u < units && ok; u += u_step) {
        const Place x = place_of<256>(u, offs, prefix, p.E, p.MT);
        const int rows = min(128, x.n_valid - (int)rank * 128);
        const int nb = min(x.mt * 2 + (lane & 1), p.NB - 1);  // (channels past N: zero weights, never stored)
        const float* wp = p.w_scales + (size_t)x.g * p.KB * p.NB + (TRANS ? (size_t)nb : (size_t)nb * p.KB);
        const float* ap = p.a_scales + (size_t)(x.row0 + (int)rank * 128) * p.KB;
        for (int kb = 0; kb < p.KB; kb += kGroup, ++it) {
          const uint32_t ring = it % kScaleRing;
          if (!warp_wait(sempty_bar(ring), ((it / kScaleRing) & 1u) ^ 1u, deadline, abort_flag)) {
            ok = false;
            break;
          }
          const int n = min(kGroup, p.KB - kb);
          const uint32_t to = sbase + kScaleOff + ring * (kGroup * 128 * 4);
          for (int r = lane; r < rows; r += 32)
#pragma unroll
            for (int j = 0; j < kGroup; ++j)
              if (j < n) ptx::cp_async4(to + (uint32_t)(r * kGroup + j) * 4, ap + (size_t)r * p.KB + kb + j);
          if (lane < 2 * n)
            ptx::cp_async4(sbase + kWScaleOff + ((ring * 2 + (lane & 1)) * kGroup + (lane >> 1)) * 4,
                           wp + (size_t)(kb + (lane >> 1)) * (TRANS ? p.NB : 1));
          ptx::cp_async_arrive_noinc(sfull_bar(ring));
          if (lane == 0) {
            *reinterpret_cast<int4*>(smem + kPlaceOff + ring * 16) = make_int4(x.row0, x.n_valid, x.mt, 0);
            ptx::mbar_arrive(sfull_bar(ring));
          }
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      if (!ok && lane == 0) set_device_status(p.status, MOE_ERR_DEVICE_TIMEOUT);
    }
  } else {
    // ------------------------------------------------------- accumulation
    ptx::regs_inc<kRegsHigh>();
    const int q = warp & 3, h = (warp - 4) >> 2, row = q * 32 + lane;
    uint8_t* outb = smem + kOutOff + (warp - 4) * kOutBufs * kOutBytes;
    const uint32_t at = tmem_base + ((uint32_t)(q * 32) << 16) + h * 128;
    const uint32_t lead_acce = lead(acce_bar((uint32_t)h));
    uint32_t it = 0, sit = 0;
    bool ok = true;
    for (int u = u_first; u < units; u += u_step) {
      float acc[kChunks][32];
#pragma unroll
      for (int i = 0; i < kChunks; ++i)
#pragma unroll
        for (int j = 0; j < 32; ++j) acc[i][j] = 0.f;
      for (int kb0 = 0; kb0 < p.KB; kb0 += kGroup, ++sit) {
        const uint32_t ring = sit % kScaleRing;
        ok = warp_wait(sfull_bar(ring), (sit / kScaleRing) & 1u, deadline, abort_flag);
        if (!ok) break;
        // the group's scales at once: a shared-memory read in front of each
        // block waits behind the memory's other users
        const float4 sa = *reinterpret_cast<const float4*>(scales + (ring * 128 + row) * kGroup);
        const float4 sw = *reinterpret_cast<const float4*>(wscales + (ring * 2 + h) * kGroup);
        float f = sa.x * sw.x, f1 = sa.y * sw.y, f2 = sa.z * sw.z, f3 = sa.w * sw.w;
        const int n = min(kGroup, p.KB - kb0);
        bool seen = ptx::mbar_test_wait(accf_bar(2 * (it & 1u) + h), (it >> 1) & 1u);
#pragma unroll 1
        for (int j = 0; j < n; ++j, ++it) {
          const uint32_t buf = it & 1u;
          ok = __all_sync(0xffffffffu, seen) || warp_wait(accf_bar(2 * buf + h), (it >> 1) & 1u, deadline, abort_flag);
          if (!ok) break;
          ptx::tc_fence_after();
          const uint32_t from = at + 256u * buf;
          uint32_t d[2][32];
          ptx::tmem_ld32(from, d[0]);
#pragma unroll
          for (int t = 0; t < kChunks; ++t) {
            ptx::tmem_ld_wait();
            if (t + 1 < kChunks) {
              ptx::tmem_ld32(from + 32u * (t + 1), d[(t + 1) & 1]);
            } else {  // everything is in registers: the buffer can fill again
              ptx::tc_fence_before();
              __syncwarp();
              if (lane == 0) ptx::mbar_arrive_cluster(lead_acce + 16u * buf);
              seen = ptx::mbar_test_wait(accf_bar(2 * (buf ^ 1u) + h), ((it + 1) >> 1) & 1u);
            }
#pragma unroll
            for (int k = 0; k < 32; ++k) acc[t][k] = fmaf(__uint_as_float(d[t & 1][k]), f, acc[t][k]);
          }
          f = f1;
          f1 = f2;
          f2 = f3;
        }
        if (!ok) break;
        if (kb0 + kGroup >= p.KB) break;  // (the last group's slot tells the unit's place first)
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(sempty_bar(ring));
      }
      if (!ok) break;
      const uint32_t ring = sit++ % kScaleRing;
      const int4 x = *reinterpret_cast<const int4*>(smem + kPlaceOff + ring * 16);
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(sempty_bar(ring));
      store_rows_m<kOutBufs, kChunks, 32>(p, &maps.out, x.x, x.y, acc, (int)rank * 128 + q * 32, x.z * 256 + h * 128,
                                outb);
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

}  // namespace

moe_status block_gemm_many_launch(const Params& p, const Maps& maps, bool transposed, int num_sms, cudaStream_t s) {
  static std::atomic<int> known[2][64];
  const long long units = ((long long)p.R / 256 + (p.R < p.E ? p.R : p.E)) * p.MT;
  return transposed ? launch_clusters<2>(block_gemm_many_kernel<true>, known[1], kSmemBytes, units, num_sms, s, p, maps)
                    : launch_clusters<2>(block_gemm_many_kernel<false>, known[0], kSmemBytes, units, num_sms, s, p, maps);
}

}  // namespace moe
