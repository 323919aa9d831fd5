// Dispatch: tokens to rows grouped by expert, dropped assignments without a
// row, rows as they are or as MXFP4.
//
// A row's place is its expert's offset plus the number of earlier assignments
// to the same expert: counts of 32 assignments at a time by match_any, prefix
// sums over warps, chunks and experts, no atomics whose order shows.
//
//   few assignments (kSmallRows): one launch.  Every CTA works the maps out for
//     itself in shared memory (they are a few KB) and then moves its share of
//     the rows; CTA 0 writes the maps.
//   many: counts of each chunk; prefix sums over the chunks, a CTA for each 32
//     experts; then CTAs rank a chunk's assignments and move its tokens.
//
// A token is read once and written to its k rows, so that x comes from memory
// once; as MXFP4 it is quantised once.  Memory's writes bound the large calls
// (16384 tokens of 2048 in bf16, eight of 128 experts each, 8.5 % dropped: 96 us,
// 5.8 TB/s, of which the maps take 8.5; 4096 of 7168 as MXFP4: 36 us, 5.1 TB/s,
// the maps 6.5), launch and the chain of prefix sums the small ones (64 tokens of
// 7168, eight of 256: 4.7 us).
#include "mxfp4.cuh"

namespace moe {
namespace {

// Assignments up to which one launch does it all.  One launch and three: 256
// tokens of 7168, eight of 256 experts each, 9.9 and 10.7 us, 384 13.5 and 14.8,
// 512 16.8 and 15.0 (as MXFP4 7.6 and 8.1, 10.6 and 9.7, 12.3 and 9.9); 256 of 2048
// 7.0 and 7.6, 512 11.2 and 9.4; 1024 of 4096, two of 8, 8.0 and 8.6, 2048 13.3 and
// 11.6.
constexpr int kSmallRows = 2048;
constexpr int kSmallThreads = 512;
constexpr int kChunkRows = 256;  // assignments of a chunk at most (whole tokens)
constexpr int kThreads = 256;
constexpr int kMoveWarps = 4;    // items an SM from which on a warp holds several pieces

enum Move { kNone, kCopy, kMxBf16, kMxF32 };

// Assignments of a chunk: whole tokens, kChunkRows at most.
__host__ __device__ inline int chunk_of(int k) { return kChunkRows / k * k; }

__device__ __forceinline__ uint32_t lanes_below() {
  uint32_t m;
  asm("mov.u32 %0, %%lanemask_lt;" : "=r"(m));
  return m;
}

// The expert of assignment a, -1 where it takes no row.
__device__ __forceinline__ int expert_of(const DispatchArgs& p, int a) {
  const int e = p.idx[a];
  if (e < p.E) return e < 0 ? -1 : e;
  set_device_status(p.status, MOE_ERR_DEVICE_BOUNDS);
  return -1;
}

// Rank of the lane's assignment among the warp's earlier ones of its expert;
// cnt[E] of the warp counts them.
__device__ __forceinline__ int rank_in_warp(int e, int* cnt) {
  const uint32_t peers = __match_any_sync(0xffffffffu, e);
  const int before = e >= 0 ? cnt[e] : 0;
  __syncwarp();
  if (e >= 0 && (peers & lanes_below()) == 0u) cnt[e] = before + __popc(peers);
  __syncwarp();
  return before + __popc(peers & lanes_below());
}

// Exclusive prefix sums of tot[0..E) into base[0..E], by the whole CTA
// (THREADS threads, E <= 1024); tot and base may be the same.
template <int THREADS>
__device__ __forceinline__ void expert_bases(const int* tot, int* base, int E, int* warp_tot) {
  constexpr int EACH = 1024 / THREADS;  // consecutive experts of a thread
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int v[EACH], sum = 0;
#pragma unroll
  for (int i = 0; i < EACH; ++i) {
    const int e = threadIdx.x * EACH + i;
    v[i] = e < E ? tot[e] : 0;
    sum += v[i];
  }
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int n = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += n;
  }
  if (lane == 31) warp_tot[warp] = incl;
  __syncthreads();
  int run = incl - sum;
  for (int w = 0; w < warp; ++w) run += warp_tot[w];
#pragma unroll
  for (int i = 0; i < EACH; ++i) {
    const int e = threadIdx.x * EACH + i;
    if (e <= E) base[e] = run;
    run += v[i];
  }
  if (E == 1024 && threadIdx.x == THREADS - 1) base[E] = run;
  __syncthreads();
}

// 16-byte vectors of a row (its bytes may pass 2^31).
__host__ __device__ __forceinline__ int vecs_of(const DispatchArgs& p) { return p.d / (p.f32 ? 4 : 8); }

// Pieces of a token's row that a warp moves at a time: 32 lanes of 16 bytes
// (kCopy) or of a block of 32 columns.
template <Move M>
__host__ __device__ __forceinline__ int pieces_of(const DispatchArgs& p) {
  return M == kNone ? 0 : ((M == kCopy ? vecs_of(p) : p.d / kMxBlock) + 31) / 32;
}

// One warp: pieces c .. c + N - 1 (those below `pieces`) of token t to the rows in
// `rows` (k of them, -1: none): all of them are read, then written a row at a
// time, so that a row gets N x 512 bytes in a go.
template <Move M, bool WIDE, int N>
__device__ __forceinline__ void move_pieces(const DispatchArgs& p, int t, int c, const int* rows) {
  const int lane = threadIdx.x & 31;
  if constexpr (M == kCopy) {
    const int vecs = vecs_of(p);
    const uint4* x = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.x) + (size_t)t * p.ldx * (p.f32 ? 4 : 2));
    uint4 v[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
      if ((c + i) * 32 + lane < vecs) v[i] = __ldg(x + (c + i) * 32 + lane);
    for (int j = 0; j < p.k; ++j) {
      if (rows[j] < 0) continue;
      uint4* to = static_cast<uint4*>(p.rows) + (size_t)rows[j] * vecs + c * 32 + lane;
#pragma unroll
      for (int i = 0; i < N; ++i)
        if ((c + i) * 32 + lane < vecs) to[i * 32] = v[i];
    }
  } else {
    constexpr bool F32 = M == kMxF32;
    const int nb = p.d / kMxBlock;
    uint4 codes[N];
    uint32_t scale[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int at = (c + i) * 32 + lane;
      if (at >= nb) continue;
      MxBlock<F32> b;
      load_words<MxBlock<F32>::WORDS, WIDE>(
          static_cast<const uint8_t*>(p.x) + ((size_t)t * p.ldx + (size_t)at * kMxBlock) * (F32 ? 4 : 2), b.w);
      scale[i] = b.codes(p.fit, codes[i]);
    }
    for (int j = 0; j < p.k; ++j) {
      if (rows[j] < 0) continue;
      const size_t to = (size_t)rows[j] * nb + c * 32 + lane;
#pragma unroll
      for (int i = 0; i < N; ++i)
        if ((c + i) * 32 + lane < nb) {
          static_cast<uint4*>(p.rows)[to + i * 32] = codes[i];
          p.row_scales[to + i * 32] = (uint8_t)scale[i];
        }
    }
  }
}

// ------------------------------------------------------------ few assignments
// smem: cnt[16][E], base[E + 1], row_of[R]
template <Move M, bool WIDE>
__global__ void __launch_bounds__(kSmallThreads) dispatch_small_kernel(const DispatchArgs p) {
  griddep_begin();
  constexpr int WARPS = kSmallThreads / 32;
  extern __shared__ int sm[];
  __shared__ int warp_tot[WARPS];
  const int R = p.T * p.k, E = p.E, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int* cnt = sm;
  int* base = cnt + WARPS * E;
  int* row_of = base + E + 1;
  for (int i = threadIdx.x; i < WARPS * E; i += kSmallThreads) cnt[i] = 0;
  __syncthreads();
  // a warp's assignments are consecutive, so that warps are in order; the rank
  // and the expert of each wait packed in row_of (R <= 2^11, E <= 2^10)
  const int seg = (R + WARPS * 32 - 1) / (WARPS * 32) * 32, a0 = min(R, warp * seg), a1 = min(R, a0 + seg);
  for (int s = a0; s < a1; s += 32) {
    const int a = s + lane, e = a < a1 ? expert_of(p, a) : -1;
    const int rank = rank_in_warp(e, cnt + warp * E);
    if (a < a1) row_of[a] = e < 0 ? -1 : e << 16 | rank;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kSmallThreads) {
    int run = 0;
    for (int w = 0; w < WARPS; ++w) {
      const int c = cnt[w * E + e];
      cnt[w * E + e] = run;
      run += c;
    }
    base[e] = run;
  }
  __syncthreads();
  const bool maps = blockIdx.x == 0;
  if (maps)
    for (int e = threadIdx.x; e < E; e += kSmallThreads) p.counts[e] = base[e];
  expert_bases<kSmallThreads>(base, base, E, warp_tot);
  for (int a = threadIdx.x; a < R; a += kSmallThreads) {
    const int v = row_of[a], e = v >> 16;
    const int row = v < 0 ? -1 : base[e] + cnt[a / seg * E + e] + (v & 0xffff);
    row_of[a] = row;
    if (maps) {
      p.inv_row[a] = row;
      if (row >= 0) p.row_token[row] = a / p.k;
    }
  }
  if (maps) {
    for (int e = threadIdx.x; e <= E; e += kSmallThreads) p.offsets[e] = base[e];
    for (int r = base[E] + threadIdx.x; r < R; r += kSmallThreads) p.row_token[r] = -1;
  }
  if constexpr (M != kNone) {
    __syncthreads();
    const int pieces = pieces_of<M>(p);
    // (the pieces go to the CTAs first, then to their warps)
    for (long long i = blockIdx.x + (long long)gridDim.x * warp; i < (long long)p.T * pieces;
         i += (long long)gridDim.x * WARPS) {
      const int t = (int)(i / pieces);
      move_pieces<M, WIDE, 1>(p, t, (int)(i - (long long)t * pieces), row_of + t * p.k);
    }
  }
}

// ----------------------------------------------------------- many assignments
// chunks[c][e]: assignments of chunk c to expert e
__global__ void __launch_bounds__(kThreads) dispatch_count_kernel(const DispatchArgs p, int chunk) {
  griddep_begin();
  extern __shared__ int sm[];
  for (int e = threadIdx.x; e < p.E; e += kThreads) sm[e] = 0;
  __syncthreads();
  const long long a = (long long)blockIdx.x * chunk + threadIdx.x;
  if ((int)threadIdx.x < chunk && a < (long long)p.T * p.k) {
    const int e = expert_of(p, (int)a);
    if (e >= 0) atomicAdd(&sm[e], 1);  // (a count: the order does not show)
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += kThreads) p.chunks[(size_t)blockIdx.x * p.E + e] = sm[e];
}

// Each chunk's counts become the sums over the chunks before it; counts[e] the
// total.  A CTA takes 32 experts (the lanes), a warp a slice of the chunks, of
// which the first kHeld stay in registers between the two passes.
__global__ void __launch_bounds__(1024) dispatch_scan_kernel(int n_chunks, int E, int32_t* __restrict__ chunks,
                                                             int32_t* __restrict__ counts) {
  griddep_begin();
  constexpr int kHeld = 16;
  __shared__ int part[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e = blockIdx.x * 32 + lane;
  const int per = (n_chunks + 31) / 32, c0 = min(n_chunks, warp * per), c1 = min(n_chunks, c0 + per);
  int32_t* at = chunks + (size_t)c0 * E + e;
  int held[kHeld], sum = 0;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) held[i] = e < E && c0 + i < c1 ? at[(size_t)i * E] : 0;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) sum += held[i];
  if (e < E)
#pragma unroll 8
    for (int c = c0 + kHeld; c < c1; ++c) sum += chunks[(size_t)c * E + e];
  part[warp][lane] = sum;
  __syncthreads();
  {  // warp: expert `warp` of the 32, lane: slice
    const int v = part[lane][warp];
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int n = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += n;
    }
    part[lane][warp] = incl - v;
    if (lane == 31 && blockIdx.x * 32 + warp < E) counts[blockIdx.x * 32 + warp] = incl;
  }
  __syncthreads();
  if (e >= E) return;
  int run = part[warp][lane];
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if (c0 + i < c1) {
      at[(size_t)i * E] = run;
      run += held[i];
    }
#pragma unroll 8
  for (int c = c0 + kHeld; c < c1; ++c) {
    const int v = chunks[(size_t)c * E + e];
    chunks[(size_t)c * E + e] = run;
    run += v;
  }
}

// smem: cnt[8][E], base[E + 1], row_of[kChunkRows].  N: pieces of a token that a
// warp holds at a time.
template <Move M, bool WIDE, int N>
__global__ void __launch_bounds__(kThreads) dispatch_move_kernel(const DispatchArgs p, int chunk) {
  griddep_begin();
  constexpr int WARPS = kThreads / 32;
  extern __shared__ int sm[];
  __shared__ int warp_tot[WARPS];
  const int R = p.T * p.k, E = p.E, warp = threadIdx.x >> 5;
  int* cnt = sm;
  int* base = cnt + WARPS * E;
  int* row_of = base + E + 1;
  for (int i = threadIdx.x; i < WARPS * E; i += kThreads) cnt[i] = 0;
  __syncthreads();
  const int first = blockIdx.x * chunk, n = min(chunk, R - first);
  const int a = first + threadIdx.x;
  const int e = (int)threadIdx.x < n ? expert_of(p, a) : -1;
  const int rank = rank_in_warp(e, cnt + warp * E);
  expert_bases<kThreads>(p.counts, base, E, warp_tot);
  for (int x = threadIdx.x; x < E; x += kThreads) {
    int run = base[x] + p.chunks[(size_t)blockIdx.x * E + x];
    for (int w = 0; w < WARPS; ++w) {
      const int c = cnt[w * E + x];
      cnt[w * E + x] = run;
      run += c;
    }
  }
  __syncthreads();
  if ((int)threadIdx.x < n) {
    const int row = e < 0 ? -1 : cnt[warp * E + e] + rank;
    row_of[threadIdx.x] = row;
    if (blockIdx.y == 0) {
      p.inv_row[a] = row;
      if (row >= 0) p.row_token[row] = a / p.k;
      if (a >= base[E]) p.row_token[a] = -1;
    }
  }
  if (blockIdx.x == 0 && blockIdx.y == 0)
    for (int x = threadIdx.x; x <= E; x += kThreads) p.offsets[x] = base[x];
  if constexpr (M != kNone) {
    __syncthreads();
    // (consecutive warps, consecutive N pieces of a token)
    const int per = (pieces_of<M>(p) + N - 1) / N, tokens = n / p.k, t0 = first / p.k;
    const int i = blockIdx.y * WARPS + warp, step = gridDim.y * WARPS;
    int t = i / per, c = i - t * per;
    const int step_t = step / per, step_c = step - step_t * per;
    while (t < tokens) {
      move_pieces<M, WIDE, N>(p, t0 + t, c * N, row_of + t * p.k);
      t += step_t;
      c += step_c;
      if (c >= per) {
        c -= per;
        ++t;
      }
    }
  }
}

template <Move M, bool WIDE>
moe_status launch(const DispatchArgs& a, cudaStream_t s) {
  const int R = a.T * a.k;
  if (R <= kSmallRows) {
    constexpr int WARPS = kSmallThreads / 32;
    const size_t smem = sizeof(int) * ((size_t)WARPS * a.E + a.E + 1 + R);
    if (smem > 40 * 1024)  // (48 KB, the static part among them, need no asking)
      MOE_TRY_CUDA(cudaFuncSetAttribute(dispatch_small_kernel<M, WIDE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        (int)(sizeof(int) * ((size_t)WARPS * 1024 + 1025 + kSmallRows))));
    const long long pieces = (long long)a.T * pieces_of<M>(a);
    const int grid = M == kNone ? 1 : (int)(pieces < a.num_sms ? pieces : a.num_sms);
    MOE_TRY_CUDA(launch_k(dispatch_small_kernel<M, WIDE>, dim3(grid), dim3(kSmallThreads), smem, s, a));
    return MOE_OK;
  }
  const int chunk = chunk_of(a.k), n = ceil_div(R, chunk);
  MOE_TRY_CUDA(launch_k(dispatch_count_kernel, dim3(n), dim3(kThreads), sizeof(int) * a.E, s, a, chunk));
  MOE_TRY_CUDA(launch_k(dispatch_scan_kernel, dim3(ceil_div(a.E, 32)), dim3(1024), 0, s, n, a.E, a.chunks, a.counts));
  const size_t smem = sizeof(int) * ((size_t)(kThreads / 32) * a.E + a.E + 1 + kChunkRows);
  // Pieces of a token that a warp holds: several where that still leaves items for
  // the SMs (16384 x 2048 to eight rows each: 102 us with one, 98 with four, 97
  // with eight; MXFP4 of 4096 x 7168: 43 with two, 40 with four; 2049 x 4096 to one
  // row: 13.7 with one, 9.1 with eight), one where there are few tokens (128 x
  // 7168 to 32 rows: 16.5 with one, 20.6 with eight; 342 x 2048 to six: 7.8, 9.3).
  constexpr int WARPS = kThreads / 32, MANY = M == kNone ? 1 : M == kCopy ? 8 : 4;
  const int pieces = pieces_of<M>(a);
  const bool many = (long long)a.T * ceil_div(pieces, MANY) >= (long long)kMoveWarps * a.num_sms;
  // Few chunks an SM end unevenly: up to eight CTAs rank a chunk then, and each
  // moves its share of what the chunk's tokens have (512 chunks: 112 us with one,
  // 102 with four; 128 of two assignments a token 81 with four, 68 with eight).
  // Chunks that leave SMs idle are shared among more, four CTAs an SM (65 tokens of
  // 7168 to 32 rows, nine chunks: 63 us where a warp took whole tokens, which gave
  // nine CTAs work, 11.3 here; 257 to eight rows 21 and 10.7; 40 chunks of 512: 9.5
  // with sixteen each, 8.4 here).
  const long long items = (long long)(chunk / a.k) * ceil_div(pieces, many ? MANY : 1);
  const int most = max(max(1, min(8, 16 * a.num_sms / n)), 4 * a.num_sms / n);
  const int shares = M == kNone ? 1 : (int)max(1ll, min((long long)most, (items + WARPS - 1) / WARPS));
  auto kern = many ? dispatch_move_kernel<M, WIDE, MANY> : dispatch_move_kernel<M, WIDE, 1>;
  MOE_TRY_CUDA(launch_k(kern, dim3(n, shares), dim3(kThreads), smem, s, a, chunk));
  return MOE_OK;
}

}  // namespace

// Counts of each chunk (nothing with few assignments).
size_t dispatch_workspace(int T, int E, int k) {
  const int R = T * k;
  return R <= kSmallRows ? 0 : (size_t)ceil_div(R, chunk_of(k)) * E * sizeof(int32_t);
}

moe_status dispatch_launch(const DispatchArgs& a, cudaStream_t s) {
  if (a.rows == nullptr) return launch<kNone, false>(a, s);
  if (!a.to_mx) return launch<kCopy, false>(a, s);
  const bool wide = ((reinterpret_cast<uintptr_t>(a.x) | (uintptr_t)(a.ldx * (a.f32 ? 4 : 2))) & 31u) == 0;
  if (a.f32) return wide ? launch<kMxF32, true>(a, s) : launch<kMxF32, false>(a, s);
  return wide ? launch<kMxBf16, true>(a, s) : launch<kMxBf16, false>(a, s);
}

}  // namespace moe
