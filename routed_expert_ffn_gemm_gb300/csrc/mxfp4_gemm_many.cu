// The 4-bit product (mxfp4_gemm.cu) where experts have many rows: a unit is 256
// rows x 256 channels of one expert on a pair of CTAs with one MMA for both
// (cta_group::2, M = 256): each CTA holds 128 rows and the weights of half of
// the channels, and in its tensor memory its rows' scales and all channels'.
//
// Rows are the MMA's M side, so that a lane of tensor memory is a row.  Two
// accumulators of 256 columns and 24 columns of scales are more than the 512
// there are, so the accumulators share 24 columns: the warps that hold them
// read them first, and the next unit's MMAs start behind that.
//
// Roles of each CTA: warp 0 copies codes and the weights' scales, warp 3 brings the
// rows' scales, warp 2 turns the weights' into atoms, warps 4..11 write results (a
// quarter of the rows, half of the channels each); warp 1 of the even CTA issues
// the MMAs.  (A second warp for the atoms changed nothing.)
//
// What bounds it is shared memory: a stage of 256 is 512 cycles of MMAs, while
// copies write 37 KB and MMAs and scale copies read 35 KB, 560 cycles at 128
// bytes a cycle; it takes 620 to 670 (16384 rows on 8 experts of 4096 -> 28672:
// 585 us in bursts, 6.6 PFLOP/s, tensor pipe 73 % busy; 666 under the power cap).
// A tile costs nearly the same whatever its rows: 64 experts of 7168 -> 4096 with
// 256 rows each take 197 us, with 257 293, 384 316, 512 332.  Results in fp32 (twice
// the stores): 65536 rows of 768 -> 2048 85 us in bf16 and 120 in fp32, 16384 rows
// on 8 experts of 4096 -> 28672 608 and 753 (random codes).
// The shared columns cost some 1000 cycles from a unit's last MMA to the next
// one's first.  With few stages a unit the writing warps set the pace: 3300 of
// 3900 cycles of a unit of three (65536 rows on 128 experts of 768 -> 2048: 76
// us).  Results leave by TMA in rows of 64 bytes: 32-byte stores from registers
// took 132 us there, whole lines by plain stores 110 (as shared memory is busy).
#include "mxfp4_gemm.cuh"

namespace moe {
namespace {

using namespace mx_gemm;
using block_gemm::kOutBytes;

constexpr int kThreads = 384;
constexpr int kTileBytes = 128 * 128;  // 128 rows or channels of 256 codes
constexpr int kStages = 5, kStageBytes = 2 * kTileBytes;
constexpr int kAtoms = 6;             // of a stage: rows 2, weights 2 of each 128 channels
constexpr int kEpiWarps = 8, kOutBufs = 2;
constexpr int kScaleOff = kStages * kStageBytes;
constexpr int kRawOff = kScaleOff + kStages * kAtoms * kAtom, kRawBytes = 8 * 256;  // weights' scales as copied
constexpr int kOutOff = kRawOff + kStages * kRawBytes;
constexpr int kBarOff = kOutOff + kEpiWarps * kOutBufs * kOutBytes;
// full[S], empty[S], raw[S], acc_full[2], acc_empty, drain
constexpr int kNumBars = 3 * kStages + 4;
constexpr int kSlotOff = kBarOff + 8 * kNumBars;
constexpr int kAbortOff = kSlotOff + 8;
constexpr int kOffsOff = kAbortOff + 8;
constexpr int kPrefixOff = kOffsOff + 4 * (kMaxGroups + 4);
constexpr int kSmemBytes = kPrefixOff + 4 * (kMaxGroups + 4) + 1024;
static_assert(kSmemBytes <= 232448, "shared memory budget");
// every CTA holds all of its SM's tensor memory: never two on one SM
static_assert(2 * (kSmemBytes + 1024) > 232448 + 1024, "one CTA per SM");
// Tensor memory columns: accumulator b from kAccStep b on, 256 each; scales (rows
// 2 x 4, weights 2 x 4 of each 128 channels) in the last 24.
constexpr uint32_t kAccStep = 232, kScaleCol = 488;
static_assert(kAccStep + 256 <= kScaleCol && kScaleCol + 24 <= 512 && 256 - kAccStep <= 32, "tensor memory");

__global__ void __launch_bounds__(kThreads, 1) mxfp4_gemm_many_kernel(const Params p,
                                                                      const __grid_constant__ Maps maps) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_s = ptx::smem_u32(smem_raw);
  const uint32_t pad = (1024u - (raw_s & 1023u)) & 1023u;
  uint8_t* smem = smem_raw + pad;
  const uint32_t sbase = raw_s + pad, bars = sbase + kBarOff;
  auto full_bar = [&](uint32_t s) { return bars + 8u * s; };
  auto empty_bar = [&](uint32_t s) { return bars + 8u * (kStages + s); };
  auto raw_bar = [&](uint32_t s) { return bars + 8u * (2 * kStages + s); };
  auto accf_bar = [&](uint32_t b) { return bars + 8u * (3 * kStages + b); };
  const uint32_t acce_bar = bars + 8u * (3 * kStages + 2), drain_bar = bars + 8u * (3 * kStages + 3);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kSlotOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kAbortOff);
  int* offs = reinterpret_cast<int*>(smem + kOffsOff);
  int* prefix = reinterpret_cast<int*>(smem + kPrefixOff);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = ptx::cluster_ctarank();
  const bool leader = rank == 0u;
  auto lead = [&](uint32_t bar) { return ptx::mapa_shared(bar, 0u); };
  const int u_first = (int)(blockIdx.x >> 1), u_step = (int)(gridDim.x >> 1);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(raw_bar(s), 2);   // the weights' scales as copied, the rows' atoms
      ptx::mbar_init(full_bar(s), 4);   // (the even CTA's) both CTAs' codes and atoms
      ptx::mbar_init(empty_bar(s), 1);
    }
    ptx::mbar_init(accf_bar(0), 1);
    ptx::mbar_init(accf_bar(1), 1);
    ptx::mbar_init(acce_bar, 2 * kEpiWarps);  // (the even CTA's) both CTAs' warps
    ptx::mbar_init(drain_bar, 1);
    *abort_flag = 0;
    ptx::fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    ptx::prefetch_tmap(&maps.w);
    ptx::prefetch_tmap(&maps.ws);
    ptx::prefetch_tmap(&maps.a[4]);
    ptx::prefetch_tmap(&maps.out);
  }
  if (warp == 1) {
    ptx::tmem_alloc<true>(ptx::smem_u32(tmem_slot), 512);
    ptx::tmem_relinquish<true>();
  }
  griddep_wait();
  griddep_launch_dependents();
  group_tiles<256>(p, offs, prefix, kThreads);
  ptx::tc_fence_before();
  ptx::cluster_sync();  // (also: the peers' barriers are initialised)
  ptx::tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int units = prefix[p.E] * p.MT;
  const uint64_t deadline = ptx::globaltimer_ns() + (uint64_t)p.timeout_ns;
  Units<256> places(p, offs, prefix);

  if (warp == 0) {
    // ---------------------------------------------------------- copies (lane 0)
    const uint64_t keep = ptx::policy_evict_normal();
    uint32_t it = 0;
    bool ok = true;
    for (int u = u_first; u < units && ok; u += u_step) {
      const Place x = places.at(u);
      const int row = x.row0 + (int)rank * 128, ch = x.mt * 256 + (int)rank * 128;
      if (lane == 0)
        for (int ks = 0; ks < p.KS; ++ks, ++it) {
          const uint32_t s = it % kStages;
          if (!ptx::mbar_wait_bounded(empty_bar(s), ((it / kStages) & 1u) ^ 1u, deadline, abort_flag)) {
            ok = false;
            break;
          }
          const uint32_t at = sbase + s * kStageBytes, fb = lead(full_bar(s));
          ptx::mbar_arrive_expect_tx(raw_bar(s), kRawBytes);
          ptx::tma_load_box3(sbase + kRawOff + s * kRawBytes, &maps.ws, raw_bar(s), x.mt * 256, ks * 8, x.g, keep);
          ptx::mbar_arrive_expect_tx_cluster(fb, kStageBytes);
          ptx::tma_load_2d_pair(at, &maps.a[4], fb, ks * 128, row, keep);
          ptx::tma_load_box3_pair(at + kTileBytes, &maps.w, fb, ks * 128, ch, x.g, keep);
        }
      ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
    }
    if (lane == 0) {
      // every slot's last arrival from the even CTA, too, before the CTA may leave
      for (uint32_t j = it > kStages ? it - kStages : 0; j < it && ok; ++j)
        ok = ptx::mbar_wait_bounded(empty_bar(j % kStages), (j / kStages) & 1u, deadline, abort_flag);
      if (!ok) {
        set_device_status(p.status, MOE_ERR_DEVICE_TIMEOUT);
        // let issued copies land before shared memory is released (a stage may
        // never complete, and the odd CTA has no barrier to ask: the limit ends
        // the wait)
        const uint64_t grace = ptx::globaltimer_ns() + 100000000ull;
        while (ptx::globaltimer_ns() < grace) {
        }
      }
    }
  } else if (warp == 1) {
    if (leader) {
      // ------------------------------------------- MMAs for both CTAs
      const uint32_t one = ptx::elect_one() ? 1u : 0u;
      const uint64_t da0 = ptx::sdesc_k_sw128(sbase), db0 = ptx::sdesc_k_sw128(sbase + kTileBytes);
      const uint64_t ds0 = ptx::sdesc_rows16(sbase + kScaleOff);
      constexpr uint32_t idesc[2] = {ptx::idesc_mxf4(256, 256, 0), ptx::idesc_mxf4(256, 256, 1)};
      const uint32_t sc = tmem_base + kScaleCol;
      uint32_t it = 0, n = 0;
      bool ok = true;
      for (int u = u_first; u < units && ok; u += u_step, ++n) {
        const uint32_t d = tmem_base + kAccStep * (n & 1u);
        if (n > 0) ok = warp_wait(acce_bar, (n - 1) & 1u, deadline, abort_flag);
        for (int ks = 0; ks < p.KS && ok; ++ks, ++it) {
          const uint32_t s = it % kStages;
          ok = warp_wait(full_bar(s), (it / kStages) & 1u, deadline, abort_flag);
          if (!ok) break;
          ptx::tc_fence_after();
          const uint64_t ds = ds0 + s * (kAtoms * kAtom >> 4);
#pragma unroll
          for (int i = 0; i < kAtoms; ++i) ptx::tmem_cp_scales_one<true>(one, sc + 4 * i, ds + i * (kAtom >> 4));
          const uint64_t da = da0 + s * (kStageBytes >> 4), db = db0 + s * (kStageBytes >> 4);
          const int left = (p.K - ks * kStep + 63) / 64;  // of the stage's four MMAs of 64
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (i < left)
              ptx::mma_mxf4_one<true>(one, d, da + 2 * i, db + 2 * i, idesc[i & 1], sc + 4 * (i >> 1),
                                      sc + 8 + 8 * (i >> 1), ks + i > 0 ? 1u : 0u);
          ptx::mma_commit_pair_one(one, empty_bar(s));
        }
        if (ok) ptx::mma_commit_pair_one(one, accf_bar(n & 1u));
      }
      if (!ok && one) {
        set_device_status(p.status, MOE_ERR_DEVICE_TIMEOUT);
        if (it > 0) {  // MMAs in flight end before tensor memory is freed
          ptx::mma_commit_pair(drain_bar);
          const uint64_t grace = ptx::globaltimer_ns() + 100000000ull;
          while (!ptx::mbar_try_wait(drain_bar, 0u) && ptx::globaltimer_ns() < grace) {
          }
        }
      }
    }
  } else if (warp == 2) {
    // ------------------------- the weights' scales to atoms, once all have come
    uint32_t it = 0;
    bool ok = true;
    for (int u = u_first; u < units && ok; u += u_step) {
      for (int ks = 0; ks < p.KS; ++ks, ++it) {
        const uint32_t s = it % kStages;
        ok = warp_wait(raw_bar(s), (it / kStages) & 1u, deadline, abort_flag);
        if (!ok) break;
        // (the rows' two atoms, then for each four blocks the atoms of both halves of the channels)
        const uint8_t* raw = smem + kRawOff + s * kRawBytes;
        uint8_t* atoms = smem + kScaleOff + s * (kAtoms * kAtom);
        weight_scale_atoms<256, 2 * kAtom>(raw, atoms + 2 * kAtom);
        weight_scale_atoms<256, 2 * kAtom>(raw + 128, atoms + 3 * kAtom);
        ptx::fence_proxy_async_smem();  // (also for the rows' atoms, which the wait has seen)
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive_cluster(lead(full_bar(s)));
      }
    }
    if (!ok && lane == 0) set_device_status(p.status, MOE_ERR_DEVICE_TIMEOUT);
  } else if (warp == 3) {
    // ---------------------------------------------------- the rows' scales
    const bool ok = row_scales<256, 4, kStages>(p, offs, prefix, u_first, u_step, units, (int)rank * 128,
                                                smem + kScaleOff, kAtoms * kAtom, empty_bar, raw_bar, deadline, abort_flag);
    if (!ok && lane == 0) set_device_status(p.status, MOE_ERR_DEVICE_TIMEOUT);
  } else {
    // ------------------------------------------------------------ results
    const int q = warp & 3, h = (warp - 4) >> 2, r0 = (int)rank * 128 + q * 32;
    uint8_t* out0 = smem + kOutOff + (warp - 4) * kOutBufs * kOutBytes;
    const uint32_t at = tmem_base + ((uint32_t)(q * 32) << 16) + h * 128;
    const uint32_t lead_acce = lead(acce_bar);
    const int es = p.out_f32 ? 4 : 2, per = 64 / es;  // channels in 64 bytes
    uint32_t n = 0, buf = 0;
    bool ok = true;
    for (int u = u_first; u < units; u += u_step, ++n) {
      const Place x = places.at(u);
      const uint32_t b = n & 1u;
      ok = warp_wait(accf_bar(b), (n >> 1) & 1u, deadline, abort_flag);
      if (!ok) break;
      ptx::tc_fence_after();
      // the columns that the accumulators share: the last of the first one's
      // (half 1), the first of the second's (half 0)
      const bool shares = h != (int)b, down = b == 0;
      auto release = [&] {
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive_cluster(lead_acce);
      };
      if (!shares) release();  // (this warp is done with the unit before)
      if (lane == 0) ptx::bulk_wait_read<0>();  // (the unit before may have ended on either buffer)
      const bool whole = r0 + 32 <= x.n_valid;
      uint8_t* out = static_cast<uint8_t*>(p.out) + (size_t)(x.row0 + r0) * p.ld_out * es;
#pragma unroll 1
      for (int t = 0; t < 4; ++t) {
        const int c = down ? 3 - t : t, ch0 = x.mt * 256 + h * 128 + 32 * c;
        uint32_t d[32];
        __syncwarp();
        if (t == 0 || (r0 < x.n_valid && ch0 < p.N)) {
          ptx::tmem_ld32(at + kAccStep * b + 32 * c, d);
          ptx::tmem_ld_wait();
        }
        if (t == 0 && shares) release();
        if (r0 >= x.n_valid || ch0 >= p.N) continue;
#pragma unroll
        for (int k = 0; k < 2; ++k) {  // 64 bytes of each row at a time
          const int ch = ch0 + k * per;
          if ((k == 1 && !p.out_f32) || ch >= p.N) break;
          uint8_t* outb = out0 + buf * kOutBytes;
          buf ^= 1u;
          if (lane == 0) ptx::bulk_wait_read<kOutBufs - 1>();  // the store before the last has read this buffer
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint4 v;
            if (p.out_f32) {
              v = make_uint4(d[16 * k + 4 * i], d[16 * k + 4 * i + 1], d[16 * k + 4 * i + 2], d[16 * k + 4 * i + 3]);
            } else {
              float f[8];
#pragma unroll
              for (int j = 0; j < 8; ++j) f[j] = __uint_as_float(d[8 * i + j]);
              v = bf16_pack(f);
            }
            *reinterpret_cast<uint4*>(outb + lane * 64 + ((i ^ ((lane >> 1) & 3)) << 4)) = v;
          }
          if (whole) {  // (the store clips the channels past N)
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              ptx::tma_store_box3(&maps.out, ptx::smem_u32(outb), ch, x.row0 + r0, 0);
              ptx::bulk_commit();
            }
            continue;
          }
          __syncwarp();
          const int i = lane & 3;
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const int r = 8 * g + (lane >> 2);
            const uint4 v = *reinterpret_cast<const uint4*>(outb + r * 64 + ((i ^ ((r >> 1) & 3)) << 4));
            if (r0 + r < x.n_valid && ch + i * (16 / es) < p.N)
              *reinterpret_cast<uint4*>(out + (size_t)r * p.ld_out * es + (size_t)ch * es + i * 16) = v;
          }
          __syncwarp();
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

}  // namespace

moe_status mxfp4_gemm_many_launch(const Params& p, const Maps& maps, int num_sms, cudaStream_t s) {
  static std::atomic<int> known[64];
  const long long units = ((long long)p.R / 256 + (p.R < p.E ? p.R : p.E)) * p.MT;
  return block_gemm::launch_clusters<2>(mxfp4_gemm_many_kernel, known, kSmemBytes, units, num_sms, s, p, maps);
}

}  // namespace moe
