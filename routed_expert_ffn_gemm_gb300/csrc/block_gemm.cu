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
// A unit is 256 channels x up to 256 rows of one expert on a cluster of two
// CTAs.  With many rows the CTAs split the rows, 128 on the MMA's M side each,
// and share the weights (N side); an accumulator lane is then a row, whose
// scale is one value for all of a lane's columns.  With few rows they split
// the channels (M side) and share the rows (N side, a multiple of 32), so
// that few rows cost few columns; the scales then come per column.  Each CTA
// copies all that it needs by itself, so that nothing passes between them:
// what both share comes from memory once and from L2 twice.  The MMAs are
// each CTA's own (cta_group::1): a block's sum goes from the tensor cores to
// the registers and the buffer back within the CTA; with one MMA of 256
// columns for both CTAs that round trip crosses them and bounds the loop.
// Units run row tiles first inside bands of 16, so that a weight tile is read
// from memory once while the band's rows stay in L2.  (From kManyRows rows an
// expert on average the product is block_gemm_many.cu's.)
//
// Roles: warp 0 copies (TMA), warp 1 issues the MMAs, warp 2 brings the
// scales to shared memory (cp.async), warps 4..11 hold the accumulators:
// a quarter of the lanes each, alternate chunks of 32 columns.  Tensor memory
// holds two buffers of 256 columns, one filling while the other is read: one
// block's sums with rows on M, two or four blocks' side by side with rows on N
// (a hand-over costs some 500 cycles whatever it hands over).
//
// Bound by HBM with few rows an expert (512 rows on 230 of 256 experts of 2048
// -> 7168: 479 us, 7.1 TB/s of weights; 8 rows on 8 experts of 7168 -> 4096:
// 43 us, 5.5 TB/s with launch and pipeline fill), by the hand-over of sums with
// more.
//
// Transposed weights ([E, K, N]: the data gradient with the forward's
// arrays) are the same tiles read MN-major by the MMA.
#include "block_gemm.cuh"

namespace moe {
namespace {

using namespace block_gemm;

constexpr int kThreads = 384;
constexpr int kOwnBytes = 128 * 128;          // the CTA's own operand (M side): 128 rows of 128 codes
constexpr int kGroup = 4, kScaleRing = 2;     // blocks of a step; steps' scales in flight
constexpr int kEpiWarps = 8;
constexpr int kChunks = 4;                    // chunks of 32 columns of an accumulating warp
constexpr int kOutPitch = 36;                 // words of a staged pair of rows (32 channels), padded against conflicts
static_assert(8 * 4 * kOutPitch <= kOutBytes, "staged pairs of rows");

// Tiles of up to 256 rows, or (FEW) 64: with few rows an expert, weights are
// all that moves, and slots of 24 KB instead of 48 keep twice as many of them
// in flight (8 rows of one token, 7168 x 4096: 53 -> 46 us; 512 rows of 230
// experts of 2048 x 7168: 565 -> 477).
template <bool FEW>
struct Tile {
  static constexpr int ROWS = FEW ? 64 : 256;
  static constexpr int BOX0 = FEW ? 0 : 2, BOXES = FEW ? 4 : 5;  // row boxes in use: Maps::a[BOX0] to [BOXES - 1]
  static constexpr int STEPS = FEW ? 2 : 1;               // steps in flight: block j of step i takes slot 4 (i % STEPS) + j
  static constexpr int STAGES = kGroup * STEPS;
  static constexpr int STAGE_BYTES = kOwnBytes + ROWS * 128;  // and the shared operand (N side)
  static constexpr int OUT_OFF = STAGES * STAGE_BYTES;
  static constexpr int SCALE_OFF = OUT_OFF + kEpiWarps * kOutBytes;
  static constexpr int WSCALE_OFF = SCALE_OFF + kScaleRing * kGroup * ROWS * 4;  // [ring][block][channel half]
  static constexpr int BAR_OFF = WSCALE_OFF + kScaleRing * kGroup * 8;
  // full[S], empty[S], acc_full[2], acc_empty[2], scale_full[2], scale_empty[2], drain
  static constexpr int NUM_BARS = 2 * STAGES + 4 + 2 * kScaleRing + 1;
  static constexpr int SLOT_OFF = BAR_OFF + 8 * NUM_BARS;
  static constexpr int ABORT_OFF = SLOT_OFF + 8;
  static constexpr int OFFS_OFF = ABORT_OFF + 8;
  static constexpr int PREFIX_OFF = OFFS_OFF + 4 * (kMaxGroups + 4);
  static constexpr int SMEM_BYTES = PREFIX_OFF + 4 * (kMaxGroups + 4) + 1024;
  static_assert(SMEM_BYTES <= 232448, "shared memory budget");
  // every CTA holds all of its SM's tensor memory: never two on one SM
  static_assert(2 * (SMEM_BYTES + 1024) > 232448 + 1024, "one CTA per SM");
};
// From this many rows on a unit's rows are the MMA's M side (always 256 of
// them), below it the N side (a multiple of 32): see the head of the file.  64
// experts of 7168 x 4096 with 120 rows each took 397 us on N and 503 on M;
// 80 rows 360 and 488.
constexpr int kRowsOnM = 129;
static_assert(kRowsOnM <= 129, "a batch of two blocks has 128 columns each");
// Registers: 384 x 168 at launch; the accumulating warps take what the
// other warpgroup gives back.
constexpr int kRegsLow = 72, kRegsHigh = 216;
static_assert(128 * kRegsLow + 256 * kRegsHigh <= kThreads * 168, "register split");

struct Unit {
  int g, row0, n_valid, n_mma, mt, tiles;
  int batch;  // blocks whose sums share an accumulator buffer, 256 / batch columns each
  bool rows_m;
};

template <bool FEW>
__device__ __forceinline__ Unit unit_of(int u, const int* offs, const int* prefix, int E, int MT) {
  const Place t = place_of<Tile<FEW>::ROWS>(u, offs, prefix, E, MT);
  Unit x;
  x.g = t.g;
  x.tiles = t.tiles;
  x.mt = t.mt;
  x.row0 = t.row0;
  x.n_valid = t.n_valid;
  x.rows_m = !FEW && x.n_valid >= kRowsOnM;
  x.n_mma = x.rows_m ? Tile<FEW>::ROWS : (x.n_valid + 31) / 32 * 32;
  x.batch = x.rows_m ? 1 : FEW || x.n_mma <= 64 ? 4 : 2;
  return x;
}

// Adds one accumulator buffer to a warp's registers, acc += scale * D.  The
// warp's pieces of the buffer are 32 columns at 64 t + first; once the last
// has arrived `release` hands the buffer back.  (Scalar adds: the registers that tcgen05.ld fills
// would have to be moved into pairs for packed ones.)
struct Accumulate {
  uint32_t at;  // tensor memory: the warp's lanes, its first column
  int first;    // its first column in the buffer
  int row;      // this lane's row of the CTA's 128 (rows on M)

  // Rows on M: one block, its scale f0 for channels 0..127, f1 for the rest.
  template <typename Release>
  __device__ __forceinline__ void rows_m(float (&acc)[kChunks][32], uint32_t buf, float f0, float f1,
                                         Release release) const {
    uint32_t d[2][32];
    const uint32_t from = at + 256u * buf;
    ptx::tmem_ld32(from, d[0]);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      ptx::tmem_ld_wait();
      if (t < 3)
        ptx::tmem_ld32(from + 64u * (t + 1), d[(t + 1) & 1]);
      else
        release();
      const float f = t < 2 ? f0 : f1;
#pragma unroll
      for (int j = 0; j < 32; ++j) acc[t][j] = fmaf(__uint_as_float(d[t & 1][j]), f, acc[t][j]);
    }
  }

  // Rows on N: n of BATCH blocks of 256 / BATCH columns; a column's scale is
  // its row's times the block's for the CTA's channels.
  template <int BATCH, int ROWS>
  __device__ __forceinline__ void rows_n(float (&acc)[kChunks][32], uint32_t buf, int n, int n_mma, const float* sc,
                                         const float* ws) const {
    constexpr int PER = 4 / BATCH;  // chunks of this warp in a block
    auto live = [&](int t) { return t / PER < n && (t % PER) * 64 + first < n_mma; };
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      if (live(t)) {
        uint32_t d[32];
        ptx::tmem_ld32(at + 256u * buf + 64u * t, d);
        ptx::tmem_ld_wait();
        const float w = ws[2 * (t / PER)];
        const float* s = sc + (t / PER) * ROWS + (t % PER) * 64 + first;
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          const float4 s4 = *reinterpret_cast<const float4*>(s + j);
          float* a = acc[t % PER] + j;
          a[0] = fmaf(__uint_as_float(d[j]), s4.x * w, a[0]);
          a[1] = fmaf(__uint_as_float(d[j + 1]), s4.y * w, a[1]);
          a[2] = fmaf(__uint_as_float(d[j + 2]), s4.z * w, a[2]);
          a[3] = fmaf(__uint_as_float(d[j + 3]), s4.w * w, a[3]);
        }
      }
    }
  }
};

// One warp's accumulators to memory.  Both ways go through the warp's piece
// of shared memory, so that neighbouring lanes store 16 bytes each of one
// row; fp32 results of rows on N are 128-byte rows as they lie.

// Rows on N: the lane's channel is ch0 + lane, acc[i][j] row c0 + 64 i + j of
// the unit.
__device__ __forceinline__ void store_rows_n(const Params& p, const Unit& x, const float (&acc)[kChunks][32],
                                             int ch0, int c_first, uint8_t* outb) {
  const int lane = threadIdx.x & 31;
  if (ch0 >= p.N) return;
  if (lane == 0) ptx::bulk_wait_read<0>();  // (a store of rows on M)
  __syncwarp();
  uint32_t* st = reinterpret_cast<uint32_t*>(outb);
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const int c0 = c_first + 64 * i;
    if (c0 >= x.n_valid) return;
    if (p.out_f32) {
      float* out = static_cast<float*>(p.out) + (size_t)(x.row0 + c0) * p.N + ch0 + lane;
      if (ch0 + lane < p.N)
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (c0 + j < x.n_valid) out[(size_t)j * p.N] = acc[i][j];
      continue;
    }
    const int ch = ch0 + (lane & 3) * 8;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + (size_t)(x.row0 + c0) * p.N + ch;
#pragma unroll
    for (int k = 0; k < 2; ++k) {  // 16 rows: words (pair of rows, channel) in, 8 channels of two rows out
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(acc[i][16 * k + 2 * j], acc[i][16 * k + 2 * j + 1]);
        st[j * kOutPitch + lane] = *reinterpret_cast<const uint32_t*>(&b);
      }
      __syncwarp();
      const uint32_t* src = st + (lane >> 2) * kOutPitch + (lane & 3) * 8;
      const uint4 a = *reinterpret_cast<const uint4*>(src), b = *reinterpret_cast<const uint4*>(src + 4);
      const int c = 16 * k + 2 * (lane >> 2);
      if (ch < p.N && c0 + c < x.n_valid)
        *reinterpret_cast<uint4*>(out + (size_t)c * p.N) =
            make_uint4(__byte_perm(a.x, a.y, 0x5410), __byte_perm(a.z, a.w, 0x5410), __byte_perm(b.x, b.y, 0x5410),
                       __byte_perm(b.z, b.w, 0x5410));
      if (ch < p.N && c0 + c + 1 < x.n_valid)
        *reinterpret_cast<uint4*>(out + (size_t)(c + 1) * p.N) =
            make_uint4(__byte_perm(a.x, a.y, 0x7632), __byte_perm(a.z, a.w, 0x7632), __byte_perm(b.x, b.y, 0x7632),
                       __byte_perm(b.z, b.w, 0x7632));
      __syncwarp();
    }
  }
}

template <bool TRANS, bool FEW>
__global__ void __launch_bounds__(kThreads, 1) block_gemm_kernel(const Params p, const __grid_constant__ Maps maps) {
  using T = Tile<FEW>;
  constexpr int kBN = T::ROWS, kStages = T::STAGES, kStageBytes = T::STAGE_BYTES;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_s = ptx::smem_u32(smem_raw);
  const uint32_t pad = (1024u - (raw_s & 1023u)) & 1023u;
  uint8_t* smem = smem_raw + pad;
  const uint32_t sbase = raw_s + pad, bars = sbase + T::BAR_OFF;
  auto full_bar = [&](int s) { return bars + 8u * s; };
  auto empty_bar = [&](int s) { return bars + 8u * (kStages + s); };
  auto accf_bar = [&](int b) { return bars + 8u * (2 * kStages + b); };
  auto acce_bar = [&](int b) { return bars + 8u * (2 * kStages + 2 + b); };
  auto sfull_bar = [&](int i) { return bars + 8u * (2 * kStages + 4 + i); };
  auto sempty_bar = [&](int i) { return bars + 8u * (2 * kStages + 4 + kScaleRing + i); };
  const uint32_t drain_bar = bars + 8u * (2 * kStages + 4 + 2 * kScaleRing);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + T::SLOT_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + T::ABORT_OFF);
  int* offs = reinterpret_cast<int*>(smem + T::OFFS_OFF);
  int* prefix = reinterpret_cast<int*>(smem + T::PREFIX_OFF);
  float* scales = reinterpret_cast<float*>(smem + T::SCALE_OFF);
  float* wscales = reinterpret_cast<float*>(smem + T::WSCALE_OFF);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = ptx::cluster_ctarank();
  const int u_first = (int)(blockIdx.x >> 1), u_step = (int)(gridDim.x >> 1);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(full_bar(s), 1);
      ptx::mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(accf_bar(b), 1);
      ptx::mbar_init(acce_bar(b), kEpiWarps);
    }
    for (int i = 0; i < kScaleRing; ++i) {
      ptx::mbar_init(sfull_bar(i), 32);  // each lane's copies
      ptx::mbar_init(sempty_bar(i), kEpiWarps);
    }
    ptx::mbar_init(drain_bar, 1);
    *abort_flag = 0;
    ptx::fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    ptx::prefetch_tmap(&maps.w);
    for (int i = T::BOX0; i < T::BOXES; ++i) ptx::prefetch_tmap(&maps.a[i]);
  }
  if (warp == 1) {
    ptx::tmem_alloc<false>(ptx::smem_u32(tmem_slot), 512);
    ptx::tmem_relinquish<false>();
  }
  griddep_wait();
  griddep_launch_dependents();

  row_tiles<kBN>(p, offs, prefix, kThreads);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int units = prefix[p.E] * p.MT;
  const uint64_t deadline = ptx::globaltimer_ns() + (uint64_t)p.timeout_ns;

  if (warp < 4) {
    ptx::regs_dec<kRegsLow>();
    if (warp == 0 && lane == 0) {
      // ---------------------------------------------------------- copies
      const uint64_t once = ptx::policy_evict_first(), keep = ptx::policy_evict_normal();
      uint32_t used = 0;  // bit j: parity of slot j's uses
      int base = 0;       // the step's first slot
      bool ok = true;
      for (int u = u_first; u < units && ok; u += u_step) {
        const Unit x = unit_of<FEW>(u, offs, prefix, p.E, p.MT);
        // rows on M: this CTA's 128 rows, both halves of the channels; rows on N:
        // all rows, this CTA's 128 channels.  The box holds the rows and few
        // more (one row on each of 8 experts of 7168 x 4096: 63 us with 32,
        // 48 with 16, 46 with 8); what the MMA reads past it is any earlier
        // block's, in columns that nobody stores.
        int box = T::BOX0;
        while (box < 4 && x.n_valid > 8 << box) ++box;
        const CUtensorMap* am = &maps.a[box];
        const uint32_t bytes = kOwnBytes + (x.rows_m ? 256u : 8u << box) * 128u;
        const int ch = x.mt * 256 + (x.rows_m ? 0 : (int)rank * 128), row = x.row0 + (x.rows_m ? (int)rank * 128 : 0);
        // (weights that the pair reads twice, or another unit again, stay in L2)
        const uint64_t pol = x.rows_m || x.tiles > 1 ? keep : once;
        for (int kb = 0; kb < p.KB; ++kb) {
          const int stage = base + kb % kGroup;
          if (!ptx::mbar_wait_bounded(empty_bar(stage), ((used >> stage) & 1u) ^ 1u, deadline, abort_flag)) {
            ok = false;
            break;
          }
          const uint32_t sa = sbase + stage * kStageBytes, fb = full_bar(stage);
          ptx::mbar_arrive_expect_tx(fb, bytes);
          ptx::tma_load_2d(x.rows_m ? sa : sa + kOwnBytes, am, fb, kb * 128, row, keep);
          const uint32_t wa = x.rows_m ? sa + kOwnBytes : sa;
          ptx::tma_load_box3(wa, &maps.w, fb, TRANS ? ch : kb * 128, TRANS ? kb * 128 : ch, x.g, pol);
          if (x.rows_m)
            ptx::tma_load_box3(wa + kOwnBytes, &maps.w, fb, TRANS ? ch + 128 : kb * 128, TRANS ? kb * 128 : ch + 128, x.g,
                               pol);
          used ^= 1u << stage;
          if (kb % kGroup == kGroup - 1 || kb == p.KB - 1) base = (base + kGroup) % kStages;
        }
      }
      // every slot's last arrival, too, before the CTA may leave
      for (int j = 0; j < kStages && ok; ++j)
        ok = ptx::mbar_wait_bounded(empty_bar(j), ((used >> j) & 1u) ^ 1u, deadline, abort_flag);
      if (!ok) {
        set_device_status(p.status, MOE_ERR_DEVICE_TIMEOUT);
        // let issued copies land before shared memory is released
        const uint64_t grace = ptx::globaltimer_ns() + 100000000ull;
        for (int j = 0; j < kStages; ++j)
          while (!ptx::mbar_try_wait(full_bar(j), ((used >> j) & 1u) ^ 1u) && ptx::globaltimer_ns() < grace) {
          }
      }
    } else if (warp == 1) {
      // ------------------------------------------------------------ MMAs
      // (the whole warp walks the loop and one elected lane issues: operands
      // stay in uniform registers, and four MMAs take 100 cycles to issue
      // instead of 400)
      const uint32_t one = ptx::elect_one() ? 1u : 0u;
      uint32_t slots = 0, bufs = 0;  // bit j: parity of the uses of slot j, of buffer j
      uint32_t next = 0;             // the buffer of a step of four blocks that share one
      int base = 0;                  // the step's first slot
      bool ok = true, any = false;
      for (int u = u_first; u < units && ok; u += u_step) {
        const Unit x = unit_of<FEW>(u, offs, prefix, p.E, p.MT);
        const int n_mma = __shfl_sync(0xffffffffu, x.n_mma, 0), batch = __shfl_sync(0xffffffffu, x.batch, 0);
        const bool rows_m = batch == 1;
        const uint32_t idesc =
            ptx::idesc_f16_f32(128, n_mma) | (!TRANS ? 0u : rows_m ? ptx::kIdescBMn : ptx::kIdescAMn);
        const uint64_t da0 = TRANS && !rows_m ? ptx::sdesc_mn_sw128(sbase, 16384) : ptx::sdesc_k_sw128(sbase);
        const uint64_t db0 = TRANS && rows_m ? ptx::sdesc_mn_sw128(sbase + kOwnBytes, 16384)
                                             : ptx::sdesc_k_sw128(sbase + kOwnBytes);
        const uint32_t astep = TRANS && !rows_m ? 4096 >> 4 : 2, bstep = TRANS && rows_m ? 4096 >> 4 : 2;
        // Block j of a step: slot j; buffer j % 2, one for blocks 0, 1 and one
        // for 2, 3, or one for all four.  A poll takes some 70 cycles, so the
        // next block's barriers are asked while this block's MMAs run.
        auto buffer = [&](int j) { return batch == 1 ? (uint32_t)(j & 1) : batch == 2 ? (uint32_t)(j >> 1) : next; };
        auto polled = [&](int from, int j) {
          const bool f = ptx::mbar_test_wait(full_bar(from + j), (slots >> (from + j)) & 1u);
          if (j & (batch - 1)) return f;
          const uint32_t b = buffer(j);
          return ptx::mbar_test_wait(acce_bar(b), ((bufs >> b) & 1u) ^ 1u) && f;
        };
        const int cols = 256 / batch;
        bool seen = false;
        for (int kb0 = 0; kb0 < p.KB && ok; kb0 += kGroup) {
          const int n = min(kGroup, p.KB - kb0);
#pragma unroll
          for (int j = 0; j < kGroup; ++j) {
            if (j >= n || !ok) break;
            const uint32_t b = buffer(j);
            const int slot = base + j;
            if (!seen) {
              ok = ptx::mbar_wait_bounded(full_bar(slot), (slots >> slot) & 1u, deadline, abort_flag) &&
                   ((j & (batch - 1)) != 0 ||
                    ptx::mbar_wait_bounded(acce_bar(b), ((bufs >> b) & 1u) ^ 1u, deadline, abort_flag));
            }
            ok = __all_sync(0xffffffffu, ok) != 0;
            if (!ok) break;
            ptx::tc_fence_after();
            slots ^= 1u << slot;
            const bool last = (j & (batch - 1)) == batch - 1 || j == n - 1;
            if (last) {
              bufs ^= 1u << b;
              next ^= batch == 4 ? 1u : 0u;
            }
            const uint32_t d = tmem_base + 256u * b + (uint32_t)((j & (batch - 1)) * cols);
            const uint64_t da = da0 + (uint32_t)(slot * (kStageBytes >> 4)),
                           db = db0 + (uint32_t)(slot * (kStageBytes >> 4));
            ptx::mma_f8_one<false>(one, d, da, db, idesc);  // 32 of the block's 128 per instruction
            ptx::mma_f8_one<true>(one, d, da + astep, db + bstep, idesc);
            ptx::mma_f8_one<true>(one, d, da + 2 * astep, db + 2 * bstep, idesc);
            ptx::mma_f8_one<true>(one, d, da + 3 * astep, db + 3 * bstep, idesc);
            if (last) ptx::mma_commit_one(one, accf_bar(b));
            ptx::mma_commit_one(one, empty_bar(slot));
            // (only within the unit: the next one may use the buffers in another way)
            seen = j + 1 < n ? polled(base, j + 1) : kb0 + kGroup < p.KB && polled((base + kGroup) % kStages, 0);
            any = true;
          }
          base = (base + kGroup) % kStages;
        }
      }
      if (!ok && one) {
        set_device_status(p.status, MOE_ERR_DEVICE_TIMEOUT);
        if (any) {  // MMAs in flight end before tensor memory is freed
          ptx::mma_commit(drain_bar);
          const uint64_t grace = ptx::globaltimer_ns() + 100000000ull;
          while (!ptx::mbar_try_wait(drain_bar, 0u) && ptx::globaltimer_ns() < grace) {
          }
        }
      }
    } else if (warp == 2) {
      // ------------------------------------------------- scales, by cp.async
      // (asynchronous, so that their latency never holds a block back)
      uint32_t it = 0;
      bool ok = true;
      for (int u = u_first; u < units && ok; u += u_step) {
        const Unit x = unit_of<FEW>(u, offs, prefix, p.E, p.MT);
        // rows on N: all rows, this CTA's 128 channels; rows on M: this CTA's
        // 128 rows, both halves of the channels.  (Channels past N: zero
        // weights, never stored.)
        const int first = x.rows_m ? (int)rank * 128 : 0;
        const int rows = x.rows_m ? min(128, x.n_valid - first) : x.n_valid;
        const int nb = min(x.mt * 2 + (x.rows_m ? lane & 1 : (int)rank), p.NB - 1);
        const float* wp = p.w_scales + (size_t)x.g * p.KB * p.NB + (TRANS ? (size_t)nb : (size_t)nb * p.KB);
        const float* ap = p.a_scales + (size_t)(x.row0 + first + lane) * p.KB;
        for (int kb = 0; kb < p.KB; kb += kGroup, ++it) {
          const uint32_t slot = it % kScaleRing;
          if (!warp_wait(sempty_bar(slot), ((it / kScaleRing) & 1u) ^ 1u, deadline, abort_flag)) {
            ok = false;
            break;
          }
          const uint32_t to = sbase + T::SCALE_OFF + slot * (kGroup * kBN * 4) + lane * 4;
          const int n = min(kGroup, p.KB - kb);
          for (int r = lane; r < rows; r += 32)
#pragma unroll
            for (int j = 0; j < kGroup; ++j)
              if (j < n) ptx::cp_async4(to + (uint32_t)(j * kBN + r - lane) * 4, ap + (size_t)(r - lane) * p.KB + kb + j);
          if ((lane >> 1) < n)  // lane: block lane / 2, channel half lane & 1
            ptx::cp_async4(sbase + T::WSCALE_OFF + slot * (kGroup * 8) + lane * 4,
                           wp + (size_t)(kb + (lane >> 1)) * (TRANS ? p.NB : 1));
          ptx::cp_async_arrive_noinc(sfull_bar(slot));
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      if (!ok && lane == 0) set_device_status(p.status, MOE_ERR_DEVICE_TIMEOUT);
    }
  } else {
    // ------------------------------------------------------- accumulation
    ptx::regs_inc<kRegsHigh>();
    const int q = warp & 3, eg = (warp - 4) >> 2;
    uint8_t* outb = smem + T::OUT_OFF + (warp - 4) * kOutBytes;
    const uint32_t tlane = tmem_base + ((uint32_t)(q * 32) << 16);
    const Accumulate step{tlane + eg * 32, eg * 32, q * 32 + lane};
    uint32_t sit = 0, bufs = 0, next = 0;  // (bufs, next: as the MMA warp has them)
    bool ok = true;
    for (int u = u_first; u < units; u += u_step) {
      int n_mma, batch;
      {
        const Unit x = unit_of<FEW>(u, offs, prefix, p.E, p.MT);
        n_mma = x.n_mma;
        batch = x.batch;
      }
      float acc[kChunks][32];
#pragma unroll
      for (int i = 0; i < kChunks; ++i)
#pragma unroll
        for (int j = 0; j < 32; ++j) acc[i][j] = 0.f;
      for (int kb0 = 0; kb0 < p.KB && ok; kb0 += kGroup, ++sit) {
        const uint32_t group = sit % kScaleRing;
        ok = warp_wait(sfull_bar(group), (sit / kScaleRing) & 1u, deadline, abort_flag);
        if (!ok) break;
        const float* sc = scales + group * kGroup * kBN;
        const float* ws = wscales + group * kGroup * 2;
        const int n = min(kGroup, p.KB - kb0);
        auto arrived = [&](uint32_t b) { return ptx::mbar_test_wait(accf_bar(b), (bufs >> b) & 1u); };
        auto acquire = [&](uint32_t b, bool seen) {  // buffer b is full
          seen = __all_sync(0xffffffffu, seen) || warp_wait(accf_bar(b), (bufs >> b) & 1u, deadline, abort_flag);
          ptx::tc_fence_after();
          return seen;
        };
        auto release = [&](uint32_t b) {
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(acce_bar(b));
          bufs ^= 1u << b;
        };
        if (!FEW && batch == 1) {
          bool seen = arrived(0);
#pragma unroll 1
          for (int j = 0; j < n; ++j) {
            const float f = sc[j * kBN + step.row], f0 = f * ws[2 * j], f1 = f * ws[2 * j + 1];
            const uint32_t b = j & 1;
            ok = acquire(b, seen);
            if (!ok) break;
            step.rows_m(acc, b, f0, f1, [&] {
              release(b);
              seen = arrived(b ^ 1u);  // (the answer comes while the last columns are added)
            });
          }
        } else if (!FEW && batch == 2) {
          for (int j = 0; j < n; j += 2) {
            const uint32_t b = j >> 1;
            ok = acquire(b, arrived(b));
            if (!ok) break;
            step.template rows_n<2, kBN>(acc, b, min(2, n - j), n_mma, sc + j * kBN, ws + 2 * j);
            release(b);
          }
        } else {
          ok = acquire(next, arrived(next));
          if (ok) {
            step.template rows_n<4, kBN>(acc, next, n, n_mma, sc, ws);
            release(next);
            next ^= 1u;
          }
        }
        if (!ok) break;
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(sempty_bar(group));
      }
      if (!ok) break;
      // (worked out again: the registers hold sums during the loop)
      const Unit x = unit_of<FEW>(u, offs, prefix, p.E, p.MT);
      if (!FEW && x.rows_m)
        store_rows_m<1, kChunks, 64>(p, &maps.out, x.row0, x.n_valid, acc, (int)rank * 128 + q * 32, x.mt * 256 + eg * 32, outb);
      else
        store_rows_n(p, x, acc, x.mt * 256 + (int)rank * 128 + q * 32, eg * 32, outb);
    }
    if (lane == 0) ptx::bulk_wait_all();
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

template <bool TRANS, bool FEW>
moe_status launch(const Params& p, const Maps& maps, int num_sms, cudaStream_t s) {
  static std::atomic<int> known[64];
  // no more pairs than units can exist: whole row tiles, and one per group
  const long long tiles = (long long)p.R / Tile<FEW>::ROWS + (p.R < p.E ? p.R : p.E);
  return launch_clusters<2>(block_gemm_kernel<TRANS, FEW>, known, Tile<FEW>::SMEM_BYTES, tiles * p.MT, num_sms, s, p, maps);
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
  if (((long long)a.R / Tile<true>::ROWS + a.E) * p.MT > 0x7fffffffll) return MOE_ERR_UNSUPPORTED;
  const bool many = (long long)a.R >= kManyRows * a.E;
  // Few rows an expert on average (a group of more than 64 rows then takes
  // several tiles, whose weights come from L2 again).  64 experts of 7168 x
  // 4096 with about 40 rows each: 297 us in tiles of 64, 329 in tiles of 256.
  // The average does not see how the rows lie: 45 on average with half of the
  // experts empty 266 and 185, 40 with most of them on one expert 220 and 162.
  const bool few = !many && (a.R <= 64 || (long long)a.R <= 48ll * a.E);
  const int channels = many ? 64 : 128;  // of a weight box
  Maps maps;
  if (a.transposed)
    MOE_TRY(make_tmap_3d(&maps.w, a.w, a.E, a.K, a.N, a.N, 1, 128, channels, channels));
  else
    MOE_TRY(make_tmap_3d(&maps.w, a.w, a.E, a.N, a.K, a.K, 1, channels, 128, 128));
  const int box0 = many ? 4 : few ? Tile<true>::BOX0 : Tile<false>::BOX0;
  const int boxes = few ? Tile<true>::BOXES : Tile<false>::BOXES;
  for (int i = box0; i < boxes; ++i) MOE_TRY(make_tmap_2d(&maps.a[i], a.a, a.R, a.K, 1, 8u << i, 128, 128));
  const int es = a.out_f32 ? 4 : 2;
  MOE_TRY(make_tmap_2d(&maps.out, a.out, a.R, a.N, es, 32, 64 / es, 64));
  if (many) return block_gemm_many_launch(p, maps, a.transposed, a.num_sms, s);
  if (few) return a.transposed ? launch<true, true>(p, maps, a.num_sms, s) : launch<false, true>(p, maps, a.num_sms, s);
  return a.transposed ? launch<true, false>(p, maps, a.num_sms, s) : launch<false, false>(p, maps, a.num_sms, s);
}

}  // namespace moe
