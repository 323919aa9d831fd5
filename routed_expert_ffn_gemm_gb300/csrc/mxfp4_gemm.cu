// Grouped product of MXFP4 rows with MXFP4 weights on the block-scaled tensor
// core instructions (tcgen05.mma kind::mxf4): E2M1 codes from shared memory, a
// power of two for each 32 codes of a row of either operand from tensor memory;
// the sums over all of K stay in tensor memory.
//
// A unit is 128 channels (the MMA's M side) x up to ROWS rows (N side) of one
// expert.  Roles: warp 0 copies codes and the weights' scales (TMA, 256 of the
// reduction a stage), warp 3 brings the rows' scales into the 512-byte atoms
// that the tensor cores take, warp 2 turns the weights' scales into atoms,
// warp 1 copies atoms to tensor memory and issues the MMAs, warps 4..7 hold a
// quarter of the channels each and write results.  Two accumulators, one filling
// while the other is written.
//
// With few rows the weights are all that moves, and the ring keeps 136 KB of them
// on their way: 512 rows on 256 experts of 2048 -> 7168 288 us (7.0 TB/s, a copy
// has 6.8), one row on each of 8 experts of 7168 -> 4096 25 us (5.0 TB/s with
// launch, prologue and pipeline fill, and 256 units on 152 SMs).  The MMAs would
// take a tenth of that.
#include "mxfp4_gemm.cuh"

namespace moe {
namespace {

using namespace mx_gemm;

constexpr int kThreads = 256;
constexpr int kWeightBytes = 128 * 128, kRawBytes = 8 * 128;

template <int ROWS_>
struct Tile {
  static constexpr int ROWS = ROWS_;
  static constexpr int BOXES = ROWS == 64 ? 4 : 5;   // row boxes 8 << i
  static constexpr int STAGES = ROWS == 64 ? 8 : 6;
  static constexpr int STAGE_BYTES = kWeightBytes + ROWS * 128;
  static constexpr int SCALE_OFF = STAGES * STAGE_BYTES;     // [stage][weights 2, rows 2] atoms
  static constexpr int RAW_OFF = SCALE_OFF + STAGES * 4 * kAtom;  // weights' scales as copied
  static constexpr int BAR_OFF = RAW_OFF + STAGES * kRawBytes;
  // raw[S], full[S], empty[S], acc_full[2], acc_empty[2], drain
  static constexpr int NUM_BARS = 3 * STAGES + 5;
  static constexpr int SLOT_OFF = BAR_OFF + 8 * NUM_BARS;
  static constexpr int ABORT_OFF = SLOT_OFF + 8;
  static constexpr int OFFS_OFF = ABORT_OFF + 8;
  static constexpr int PREFIX_OFF = OFFS_OFF + 4 * (kMaxGroups + 4);
  static constexpr int SMEM_BYTES = PREFIX_OFF + 4 * (kMaxGroups + 4) + 1024;
  static_assert(SMEM_BYTES <= 232448, "shared memory budget");
  // every CTA holds all of its SM's tensor memory: never two on one SM
  static_assert(2 * (SMEM_BYTES + 1024) > 232448 + 1024, "one CTA per SM");
};
// Tensor memory: two accumulators of up to 128 columns, two sets of scales
// (weights 2 x 4 columns, rows 2 x 4 columns).
constexpr uint32_t kAccCols = 128, kScaleCol = 256, kScaleSet = 16;

template <int ROWS>
__global__ void __launch_bounds__(kThreads, 1) mxfp4_gemm_kernel(const Params p, const __grid_constant__ Maps maps) {
  using T = Tile<ROWS>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_s = ptx::smem_u32(smem_raw);
  const uint32_t pad = (1024u - (raw_s & 1023u)) & 1023u;
  uint8_t* smem = smem_raw + pad;
  const uint32_t sbase = raw_s + pad, bars = sbase + T::BAR_OFF;
  auto full_bar = [&](uint32_t s) { return bars + 8u * s; };
  auto empty_bar = [&](uint32_t s) { return bars + 8u * (T::STAGES + s); };
  auto raw_bar = [&](uint32_t s) { return bars + 8u * (2 * T::STAGES + s); };
  auto accf_bar = [&](uint32_t b) { return bars + 8u * (3 * T::STAGES + b); };
  auto acce_bar = [&](uint32_t b) { return bars + 8u * (3 * T::STAGES + 2 + b); };
  const uint32_t drain_bar = bars + 8u * (3 * T::STAGES + 4);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + T::SLOT_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + T::ABORT_OFF);
  int* offs = reinterpret_cast<int*>(smem + T::OFFS_OFF);
  int* prefix = reinterpret_cast<int*>(smem + T::PREFIX_OFF);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int u_first = (int)blockIdx.x, u_step = (int)gridDim.x;

  if (threadIdx.x == 0) {
    for (int s = 0; s < T::STAGES; ++s) {
      ptx::mbar_init(raw_bar(s), 2);  // the weights' scales as copied, the rows' atoms
      ptx::mbar_init(full_bar(s), 2);  // the codes, the scales' atoms
      ptx::mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(accf_bar(b), 1);
      ptx::mbar_init(acce_bar(b), 4);
    }
    ptx::mbar_init(drain_bar, 1);
    *abort_flag = 0;
    ptx::fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    ptx::prefetch_tmap(&maps.w);
    ptx::prefetch_tmap(&maps.ws);
    for (int i = 0; i < T::BOXES; ++i) ptx::prefetch_tmap(&maps.a[i]);
  }
  if (warp == 1) {
    ptx::tmem_alloc<false>(ptx::smem_u32(tmem_slot), 512);
    ptx::tmem_relinquish<false>();
  }
  griddep_wait();
  griddep_launch_dependents();

  group_tiles<ROWS>(p, offs, prefix, kThreads);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int units = prefix[p.E] * p.MT;
  const uint64_t deadline = ptx::globaltimer_ns() + (uint64_t)p.timeout_ns;
  Units<ROWS> places(p, offs, prefix);

  if (warp == 0) {
    // ---------------------------------------------------------- copies (lane 0)
    const uint64_t once = ptx::policy_evict_first(), keep = ptx::policy_evict_normal();
    uint32_t it = 0;
    bool ok = true;
    for (int u = u_first; u < units && ok; u += u_step) {
      const Place x = places.at(u);
      // the box holds the rows; what the MMA reads past it is any earlier stage's, in
      // columns that nobody stores
      int box = 0;
      while (box < T::BOXES - 1 && x.n_valid > 8 << box) ++box;
      const uint32_t bytes = kWeightBytes + (8u << box) * 128u;
      const uint64_t pol = x.tiles > 1 ? keep : once;
      if (lane == 0)
        for (int ks = 0; ks < p.KS; ++ks, ++it) {
          const uint32_t s = it % T::STAGES;
          if (!ptx::mbar_wait_bounded(empty_bar(s), ((it / T::STAGES) & 1u) ^ 1u, deadline, abort_flag)) {
            ok = false;
            break;
          }
          const uint32_t at = sbase + s * T::STAGE_BYTES, fb = full_bar(s), rb = raw_bar(s);
          ptx::mbar_arrive_expect_tx(rb, kRawBytes);
          ptx::tma_load_box3(sbase + T::RAW_OFF + s * kRawBytes, &maps.ws, rb, x.mt * 128, ks * 8, x.g, pol);
          ptx::mbar_arrive_expect_tx(fb, bytes);
          ptx::tma_load_box3(at, &maps.w, fb, ks * 128, x.mt * 128, x.g, pol);
          ptx::tma_load_2d(at + kWeightBytes, &maps.a[box], fb, ks * 128, x.row0, keep);
        }
      ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
    }
    if (lane == 0) {
      // every slot's last arrival, too, before the CTA may leave
      for (uint32_t j = it > T::STAGES ? it - T::STAGES : 0; j < it && ok; ++j)
        ok = ptx::mbar_wait_bounded(empty_bar(j % T::STAGES), (j / T::STAGES) & 1u, deadline, abort_flag);
      if (!ok) {
        set_device_status(p.status, MOE_ERR_DEVICE_TIMEOUT);
        // let issued copies land before shared memory is released (a stage may
        // never complete: the limit ends the wait)
        const uint64_t grace = ptx::globaltimer_ns() + 100000000ull;
        while (ptx::globaltimer_ns() < grace) {
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMAs
    const uint32_t one = ptx::elect_one() ? 1u : 0u;
    const uint64_t da0 = ptx::sdesc_k_sw128(sbase), db0 = ptx::sdesc_k_sw128(sbase + kWeightBytes);
    const uint64_t ds0 = ptx::sdesc_rows16(sbase + T::SCALE_OFF);
    uint32_t it = 0, n = 0;
    bool ok = true;
    for (int u = u_first; u < units && ok; u += u_step, ++n) {
      const Place x = places.at(u);
      const int n_mma = __shfl_sync(0xffffffffu, (x.n_valid + 31) / 32 * 32, 0);
      const uint32_t idesc[2] = {ptx::idesc_mxf4(128, n_mma, 0), ptx::idesc_mxf4(128, n_mma, 1)};
      const uint32_t b = n & 1u, d = tmem_base + kAccCols * b;
      ok = warp_wait(acce_bar(b), ((n >> 1) & 1u) ^ 1u, deadline, abort_flag);
      for (int ks = 0; ks < p.KS && ok; ++ks, ++it) {
        const uint32_t s = it % T::STAGES;
        ok = warp_wait(full_bar(s), (it / T::STAGES) & 1u, deadline, abort_flag);
        if (!ok) break;
        ptx::tc_fence_after();
        const uint32_t sc = tmem_base + kScaleCol + kScaleSet * (it & 1u);
        const uint64_t ds = ds0 + s * (4 * kAtom >> 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) ptx::tmem_cp_scales_one<false>(one, sc + 4 * i, ds + i * (kAtom >> 4));
        const uint64_t da = da0 + s * (T::STAGE_BYTES >> 4), db = db0 + s * (T::STAGE_BYTES >> 4);
        const int left = (p.K - ks * kStep + 63) / 64;  // of the stage's four MMAs of 64
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i < left)
            ptx::mma_mxf4_one<false>(one, d, da + 2 * i, db + 2 * i, idesc[i & 1], sc + 4 * (i >> 1), sc + 8 + 4 * (i >> 1),
                                     ks + i > 0 ? 1u : 0u);
        ptx::mma_commit_one(one, empty_bar(s));
      }
      if (ok) ptx::mma_commit_one(one, accf_bar(b));
    }
    if (!ok && one) {
      set_device_status(p.status, MOE_ERR_DEVICE_TIMEOUT);
      if (it > 0) {  // MMAs in flight end before tensor memory is freed
        ptx::mma_commit(drain_bar);
        const uint64_t grace = ptx::globaltimer_ns() + 100000000ull;
        while (!ptx::mbar_try_wait(drain_bar, 0u) && ptx::globaltimer_ns() < grace) {
        }
      }
    }
  } else if (warp == 2) {
    // ------------------------- the weights' scales to atoms, once all have come
    uint32_t it = 0;
    bool ok = true;
    for (int u = u_first; u < units && ok; u += u_step) {
      for (int ks = 0; ks < p.KS; ++ks, ++it) {
        const uint32_t s = it % T::STAGES;
        ok = warp_wait(raw_bar(s), (it / T::STAGES) & 1u, deadline, abort_flag);
        if (!ok) break;
        weight_scale_atoms<128, kAtom>(smem + T::RAW_OFF + s * kRawBytes, smem + T::SCALE_OFF + s * (4 * kAtom));
        ptx::fence_proxy_async_smem();  // (also for the rows' atoms, which the wait has seen)
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(full_bar(s));
      }
    }
    if (!ok && lane == 0) set_device_status(p.status, MOE_ERR_DEVICE_TIMEOUT);
  } else if (warp == 3) {
    // ---------------------------------------------------- the rows' scales
    const bool ok = row_scales<ROWS, ROWS / 32, T::STAGES>(p, offs, prefix, u_first, u_step, units, 0,
                                                           smem + T::SCALE_OFF + 2 * kAtom, 4 * kAtom, empty_bar, raw_bar,
                                                           deadline, abort_flag);
    if (!ok && lane == 0) set_device_status(p.status, MOE_ERR_DEVICE_TIMEOUT);
  } else if (warp >= 4) {
    // ------------------------------------------------------------ results
    const int q = warp & 3;
    const uint32_t at = tmem_base + ((uint32_t)(q * 32) << 16);
    uint32_t n = 0;
    bool ok = true;
    for (int u = u_first; u < units; u += u_step, ++n) {
      const Place x = places.at(u);
      const uint32_t b = n & 1u;
      ok = warp_wait(accf_bar(b), (n >> 1) & 1u, deadline, abort_flag);
      if (!ok) break;
      ptx::tc_fence_after();
      const int ch = x.mt * 128 + q * 32 + lane;
      const bool live = ch < p.N;
      for (int c = 0; c < x.n_valid; c += 32) {
        uint32_t d[32];
        __syncwarp();
        ptx::tmem_ld32(at + kAccCols * b + c, d);
        ptx::tmem_ld_wait();
        if (c + 32 >= x.n_valid) {  // everything is in registers: the accumulator can fill again
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(acce_bar(b));
        }
        if (p.out_f32) {
          float* out = static_cast<float*>(p.out) + (size_t)(x.row0 + c) * p.ld_out + ch;
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (live && c + j < x.n_valid) out[(size_t)j * p.ld_out] = __uint_as_float(d[j]);
        } else {
          // neighbouring lanes swap, so that each writes two channels of every second row
          __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + (size_t)(x.row0 + c + (lane & 1)) * p.ld_out + (ch & ~1);
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const uint32_t other = __shfl_xor_sync(0xffffffffu, (lane & 1) ? d[j] : d[j + 1], 1);
            const float lo = __uint_as_float((lane & 1) ? other : d[j]), hi = __uint_as_float((lane & 1) ? d[j + 1] : other);
            if (live && c + j + (lane & 1) < x.n_valid)
              *reinterpret_cast<__nv_bfloat162*>(out + (size_t)j * p.ld_out) = __floats2bfloat162_rn(lo, hi);
          }
        }
      }
    }
    if (!ok && lane == 0) set_device_status(p.status, MOE_ERR_DEVICE_TIMEOUT);
  }

  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc<false>(tmem_base, 512);
  }
}

template <int ROWS>
moe_status launch(const Params& p, const Maps& maps, int num_sms, cudaStream_t s) {
  using T = Tile<ROWS>;
  const long long tiles = (long long)p.R / ROWS + (p.R < p.E ? p.R : p.E);
  const long long units = tiles * p.MT;  // no more can exist: whole row tiles, and one per group
  MOE_TRY_CUDA(cudaFuncSetAttribute(mxfp4_gemm_kernel<ROWS>, cudaFuncAttributeMaxDynamicSharedMemorySize, T::SMEM_BYTES));
  MOE_TRY_CUDA(launch_k(mxfp4_gemm_kernel<ROWS>, dim3((unsigned)(units < num_sms ? units : num_sms)), dim3(kThreads),
                        T::SMEM_BYTES, s, p, maps));
  return MOE_OK;
}

}  // namespace

// From kMxManyRows rows an expert on average the product runs on
// mxfp4_gemm_many.cu, up to kMxFewRows in tiles of 64 rows here, between in
// tiles of 128.  64 experts, us in tiles of 64, of 128 and there:
//   rows              16            32            64            96            128           192
//   7168 -> 4096  152 154 172   154 156 173   157 160 176   242 173 182   213 185 189   295 324 189
//   2048 -> 4096   50  50  56    51  51  57    54  54  59    80  62  62    79  77  66   116 143  69
//    768 -> 2048   16  18  21    16  18  19    24  25  19    41  32  21    41  40  22    57  74  24
// (512 rows on 256 experts of 2048 x 7168: 288, 315, 346; 7168 -> 4096 spread as
// rank^-0.6 with 64 rows on average: 179, 170, 181, with 128: 277, 210, 192.)  The
// limit fits long reductions; with short ones the pair's kernel is ahead from some
// 48 rows on (768 -> 2048: 22.7, 23.9, 21.0), which the rule leaves out.  The average
// counts experts without rows, which the host cannot see: 16384 rows on 8 of 256
// experts of 7168 -> 4096 take 261 us, on 8 of 8 147.
constexpr long long kMxManyRows = 112, kMxFewRows = 32;

moe_status mxfp4_gemm_launch(const MxGemmArgs& a, cudaStream_t s) {
  Params p{};
  p.R = a.R;
  p.K = a.K;
  p.N = a.N;
  p.E = a.E;
  p.MT = ceil_div(a.N, 128);
  p.KS = ceil_div(a.K, kStep);
  p.KB = a.K / kMxBlock;
  p.out_f32 = a.out_f32;
  p.a_scales = a.a_scales;
  p.w_scales = a.w_scales;
  p.offsets = a.offsets;
  p.out = a.out;
  p.ld_out = a.ld_out;
  p.status = a.status;
  p.timeout_ns = a.timeout_ns;
  if (((long long)a.R / 64 + a.E) * p.MT > 0x7fff0000ll) return MOE_ERR_UNSUPPORTED;
  Maps maps;
  MOE_TRY(make_tmap_3d(&maps.w, a.w, a.E, a.N, a.K / 2, a.K / 2, 1, 128, 128, 128));
  MOE_TRY(make_tmap_3d(&maps.ws, a.w_scales, a.E, p.KB, a.N, a.N, 1, 8, 128, 0));
  for (int i = 0; i < 5; ++i) MOE_TRY(make_tmap_2d(&maps.a[i], a.a, a.R, a.K / 2, 1, 8u << i, 128, 128));
  if ((long long)a.R >= kMxManyRows * a.E) {
    const int es = a.out_f32 ? 4 : 2;
    MOE_TRY(make_tmap_3d(&maps.out, a.out, 1, a.R, a.N, a.ld_out * es, es, 32, 64 / es, 64));
    p.MT = ceil_div(a.N, 256);
    MOE_TRY(make_tmap_3d(&maps.ws, a.w_scales, a.E, p.KB, a.N, a.N, 1, 8, 256, 0));
    return mxfp4_gemm_many_launch(p, maps, a.num_sms, s);
  }
  // Few rows on average: more, smaller slots in flight.
  const bool few = a.R <= 64 || (long long)a.R <= kMxFewRows * a.E;
  return few ? launch<64>(p, maps, a.num_sms, s) : launch<128>(p, maps, a.num_sms, s);
}

}  // namespace moe
