// The router's balance loss and z loss with the per-expert counts, and the
// gradient of the logits.
//
//   p = softmax(l[t,:]), f_e = counts_e / (n k), P_e = mean of p[t,e] over
//   the n unmasked tokens;  balance = alpha E sum_e f_e P_e,
//   z = beta mean lse_t^2.  f holds counts and has no gradient, so
//   dl[t,e] = (alpha E / n) p (f_e - sum_j f_j p_j) + (2 beta / n) lse p,
//   plus the gradient through the kept weights (a softmax over the kept
//   slots): w_j (dw_j - sum_i w_i dw_i) at expert idx[t,j].
//
// Both directions read the logits once, a row by a group of LG lanes that
// keep it in registers; they are bound by that read (and the gradient's
// write), or by launch latency when there are few tokens: 32768 x 256 takes
// 12 us forward, 6 for the sum over CTAs and 20 for the gradient (a row's
// loads and reductions, not bandwidth, set that pace: the logits stay in L2),
// 64 x 8 both directions 9 us.  Sums over tokens
// go lane -> warp -> CTA -> fixed-order sum over CTAs without floating-point
// atomics, and the gradient's kept weights are added in shared memory once for
// each of a row's distinct experts: every run gives the same bits.
// Probabilities take __expf: with expf the error against 64 bits is the same
// (5.0e-8 of the 32768 x 256 gradient's norm, as of the plain form's) and the
// step takes 45.0 us instead of 43.7.
#include <math.h>

#include <atomic>

#include "ptx.cuh"
#include "train.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;       // gradient
constexpr int kWarps = kThreads / 32;
constexpr int kSumThreads = 1024;   // sum over the CTAs' parts: clusters of
constexpr int kSumCtas = 8;         // this many CTAs share the experts

// Lanes LG hold a row: lane l has columns (i * LG + l) * VEC + c.
template <int LG, int VEC, int NI>
struct Row {
  float v[NI * VEC];
  __device__ __forceinline__ static int col(int i, int l) { return (i * LG + l) * VEC; }
  __device__ __forceinline__ void load(const float* row, int E, int l) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int e = col(i, l);
      if constexpr (VEC == 4) {
        float4 q = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        if (e < E) q = __ldg(reinterpret_cast<const float4*>(row + e));
        v[4 * i] = q.x; v[4 * i + 1] = q.y; v[4 * i + 2] = q.z; v[4 * i + 3] = q.w;
      } else {
        v[i] = e < E ? __ldg(row + e) : -INFINITY;
      }
    }
  }
};

template <int LG>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = LG / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// (fmaxf drops NaN: a NaN logit shows in the sum of exponentials instead)
template <int LG>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int o = LG / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Workspace of one CTA: prob sums [E] (float), counts [E] (int), sum of
// lse^2 (float), unmasked tokens (int).
__host__ __device__ inline size_t part_words(int E) { return 2 * (size_t)E + 2; }

// Losses from the sums over tokens.
__device__ __forceinline__ void write_losses(const RouterLossArgs& a, float dot, float zs, int n) {
  const float fn = (float)n;
  a.counts[a.E] = n;
  a.loss[0] = n > 0 ? a.balance * (float)a.E * (dot / (fn * (float)a.k)) / fn : 0.f;
  a.loss[1] = n > 0 ? a.z * (zs / fn) : 0.f;
}

template <typename T>
__device__ __forceinline__ T warp_sum(T v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// Sum over the block in a fixed order, known to every thread.
template <typename T>
__device__ __forceinline__ T block_sum(T v, T* red) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  T s = 0;
  for (int w = 0; w < (int)(blockDim.x >> 5); ++w) s += red[w];
  return s;
}

// THREADS: many warps on each SM (rows wait for memory), as registers allow.
template <int LG, int VEC, int NI, int THREADS>
__global__ void __launch_bounds__(THREADS) router_losses_kernel(const RouterLossArgs a) {
  griddep_begin();
  constexpr int WARPS = THREADS / 32;
  extern __shared__ uint32_t sm[];
  float* psum = reinterpret_cast<float*>(sm);                 // [WARPS][E]
  int* hist = reinterpret_cast<int*>(sm + WARPS * a.E);       // [E]
  __shared__ float red_f[WARPS];
  __shared__ int red_n[WARPS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane & (LG - 1);
  constexpr int RPW = 32 / LG;  // rows of a warp at a time
  for (int e = threadIdx.x; e < a.E; e += THREADS) hist[e] = 0;
  __syncthreads();
  float P[NI * VEC], zs = 0.f;
  int n = 0;
#pragma unroll
  for (int i = 0; i < NI * VEC; ++i) P[i] = 0.f;
  const int step = gridDim.x * WARPS * RPW;
  int t = (blockIdx.x * WARPS + warp) * RPW + lane / LG;
  Row<LG, VEC, NI> ahead;
  if (t < a.T) ahead.load(a.logits + (size_t)t * a.E, a.E, l);
  // (all rows of the warp take the same number of steps)
  for (int t0 = t - lane / LG; t0 < a.T; t0 += step, t += step) {
    const bool here = t < a.T, live = here && (a.mask == nullptr || a.mask[t] != 0);
    Row<LG, VEC, NI> r = ahead;  // the next row is on its way during this one
    if (t + step < a.T) ahead.load(a.logits + (size_t)(t + step) * a.E, a.E, l);
    if (live)
      for (int j = l; j < a.k; j += LG) {
        const int e = a.idx[(size_t)t * a.k + j];
        if (e >= 0 && e < a.E)
          atomicAdd(hist + e, 1);
        else
          set_device_status(a.status, MOE_ERR_DEVICE_BOUNDS);
      }
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NI * VEC; ++i) {
      if (!here) r.v[i] = -INFINITY;
      m = fmaxf(m, r.v[i]);
    }
    m = group_max<LG>(m);
    const float m0 = m == -INFINITY ? 0.f : m;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NI * VEC; ++i) {
      r.v[i] = __expf(r.v[i] - m0);
      sum += r.v[i];
    }
    sum = group_sum<LG>(sum);
    // a row without any logit above -inf has no probabilities: it adds
    // nothing to P and z, and its lse of -inf gives it no gradient
    const float lse = sum == 0.f ? -INFINITY : m0 + logf(sum), inv = live && sum != 0.f ? 1.f / sum : 0.f;
    if (here && l == 0) a.lse[t] = lse;
    if (live && sum != 0.f) {
#pragma unroll
      for (int i = 0; i < NI * VEC; ++i) P[i] = fmaf(r.v[i], inv, P[i]);
      if (l == 0) zs = fmaf(lse, lse, zs);
    }
    if (live && l == 0) ++n;
  }
#pragma unroll
  for (int i = 0; i < NI * VEC; ++i) {
#pragma unroll
    for (int o = 16; o >= LG; o >>= 1) P[i] += __shfl_xor_sync(0xffffffffu, P[i], o);
    const int e = Row<LG, VEC, NI>::col(i / VEC, l) + i % VEC;
    if (lane < LG && e < a.E) psum[warp * a.E + e] = P[i];
  }
  zs = block_sum(zs, red_f);  // (its barriers: the sums and counts of all warps are written)
  n = block_sum(n, red_n);
  uint32_t* part = static_cast<uint32_t*>(a.workspace) + blockIdx.x * part_words(a.E);
  const bool alone = gridDim.x == 1;
  float dot = 0.f;
  for (int e = threadIdx.x; e < a.E; e += THREADS) {
    float s = 0.f;
    for (int w = 0; w < WARPS; ++w) s += psum[w * a.E + e];
    if (alone) {
      a.counts[e] = hist[e];
      dot += (float)hist[e] * s;
    } else {
      part[e] = __float_as_uint(s);
      part[a.E + e] = (uint32_t)hist[e];
    }
  }
  if (alone) {
    dot = block_sum(dot, red_f);
    if (threadIdx.x == 0) write_losses(a, dot, zs, n);
  } else if (threadIdx.x == 0) {
    part[2 * a.E] = __float_as_uint(zs);
    part[2 * a.E + 1] = (uint32_t)n;
  }
}

// Sums the parts in a fixed order: one cluster, its CTAs taking 32 experts at
// a time, a warp every 32nd part of them; the first CTA adds the CTAs' shares
// of sum_e c_e P_e through distributed shared memory.
__global__ void __launch_bounds__(kSumThreads) __cluster_dims__(kSumCtas, 1, 1)
    router_losses_sum_kernel(const RouterLossArgs a, int nparts) {
  ptx::cluster_arrive();  // (waited for in front of the first access to another CTA's memory)
  griddep_begin();
  constexpr int WARPS = kSumThreads / 32;
  __shared__ float sum_p[WARPS][32], red[WARPS];
  __shared__ int sum_c[WARPS][32], red_n[WARPS];
  __shared__ float shares[kSumCtas];
  const uint32_t* parts = static_cast<const uint32_t*>(a.workspace);
  const size_t pw = part_words(a.E);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rank = blockIdx.x;
  float dot = 0.f;
  for (int e0 = rank * 32; e0 < a.E; e0 += kSumCtas * 32) {
    const int e = e0 + lane;
    float P = 0.f;
    int c = 0;
    if (e < a.E)
#pragma unroll 5
      for (int b = warp; b < nparts; b += WARPS) {
        P += __uint_as_float(__ldcg(parts + b * pw + e));
        c += (int)__ldcg(parts + b * pw + a.E + e);
      }
    sum_p[warp][lane] = P;
    sum_c[warp][lane] = c;
    __syncthreads();
    if (warp == 0 && e < a.E) {
      P = 0.f;
      c = 0;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        P += sum_p[w][lane];
        c += sum_c[w][lane];
      }
      a.counts[e] = c;
      dot += (float)c * P;
    }
    __syncthreads();
  }
  dot = warp_sum(dot);  // (warp 0 has them all)
  float zs = 0.f;
  int n = 0;
  if (rank == 0) {
    for (int b = threadIdx.x; b < nparts; b += kSumThreads) {
      zs += __uint_as_float(__ldcg(parts + b * pw + 2 * a.E));
      n += (int)__ldcg(parts + b * pw + 2 * a.E + 1);
    }
    zs = block_sum(zs, red);
    n = block_sum(n, red_n);
  }
  ptx::cluster_wait();  // every CTA of the cluster has started
  if (threadIdx.x == 0) {
    const uint32_t to = ptx::mapa_shared(ptx::smem_u32(&shares[rank]), 0u);
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to), "f"(dot) : "memory");
  }
  ptx::cluster_sync();
  if (rank == 0 && threadIdx.x == 0) {
    float s = 0.f;
    for (int r = 0; r < kSumCtas; ++r) s += shares[r];
    write_losses(a, s, zs, n);
  }
}

template <int LG, int VEC, int NI>
__global__ void __launch_bounds__(kThreads) router_losses_backward_kernel(const RouterLossGradArgs a) {
  griddep_begin();
  extern __shared__ uint32_t sm[];
  float* f = reinterpret_cast<float*>(sm);                    // [E] counts / (n k)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane & (LG - 1);
  constexpr int RPW = 32 / LG;
  // what the kept weights add, at their experts' columns: one row per group
  float* add = f + a.E + (warp * RPW + lane / LG) * a.E;
  const int n = a.counts[a.E];
  const float inv_n = n > 0 ? 1.f / (float)n : 0.f, inv_nk = inv_n / (float)a.k;
  for (int e = threadIdx.x; e < a.E; e += kThreads) f[e] = (float)a.counts[e] * inv_nk;
  if (a.w != nullptr)
    for (int e = l; e < a.E; e += LG) add[e] = 0.f;
  __syncthreads();
  const float up = (a.grad != nullptr ? *a.grad : 1.f) * inv_n;
  const float cb = a.balance * (float)a.E, cz = 2.f * a.z;
  const int step = gridDim.x * kWarps * RPW;
  int t = (blockIdx.x * kWarps + warp) * RPW + lane / LG;
  constexpr int KI = 32 / LG;  // most kept slots of a lane
  struct Ahead {
    Row<LG, VEC, NI> r;
    float lse, w[KI], dw[KI];
    int e[KI];
  } ahead;
  auto load = [&](int t) {
    if (t >= a.T) return;
    ahead.r.load(a.logits + (size_t)t * a.E, a.E, l);
    ahead.lse = a.lse[t];
    if (a.w != nullptr)
#pragma unroll
      for (int i = 0; i < KI; ++i) {
        const int j = l + i * LG;
        const size_t at = (size_t)t * a.k + j;
        ahead.w[i] = j < a.k ? a.w[at] : 0.f;
        ahead.dw[i] = j < a.k ? a.dw[at] : 0.f;
        ahead.e[i] = j < a.k ? a.idx[at] : -1;
      }
  };
  load(t);
  for (int t0 = t - lane / LG; t0 < a.T; t0 += step, t += step) {
    const bool here = t < a.T, live = here && (a.mask == nullptr || a.mask[t] != 0);
    Ahead now = ahead;  // the next row is on its way during this one
    load(t + step);
    Row<LG, VEC, NI>& r = now.r;
    const float lse = here ? now.lse : -INFINITY;
    if (a.w != nullptr) {
      float dot = 0.f;
#pragma unroll
      for (int i = 0; i < KI; ++i)
        if (here) dot = fmaf(now.w[i], now.dw[i], dot);
      dot = group_sum<LG>(dot);
#pragma unroll
      for (int i = 0; i < KI; ++i) {
        const int e = here ? now.e[i] : -1;
        if (e >= 0 && e < a.E)
          atomicAdd(add + e, now.w[i] * (now.dw[i] - dot));  // (distinct experts: one add each)
        else if (here && l + i * LG < a.k)
          set_device_status(a.status, MOE_ERR_DEVICE_BOUNDS);
      }
      __syncwarp();
    }
    // Probabilities are the terms over their own sum: lse is rounded to fp32,
    // by 2^-25 of its magnitude, and exp(l - lse) alone would be off by that
    // (by 5e-4 where the logits are about 8000).
    const bool some = live && lse != -INFINITY;
    float fp = 0.f, sum = 0.f;
#pragma unroll
    for (int i = 0; i < NI * VEC; ++i) {
      const int e = Row<LG, VEC, NI>::col(i / VEC, l) + i % VEC;
      r.v[i] = some ? __expf(r.v[i] - lse) : 0.f;
      sum += r.v[i];
      if (e < a.E) fp = fmaf(f[e], r.v[i], fp);
    }
    fp = group_sum<LG>(fp);
    sum = group_sum<LG>(sum);
    const float inv = 1.f / sum, scale = up * inv;  // (sum 0 where nothing uses them)
    fp *= inv;
    const float zt = some ? cz * lse : 0.f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int e0 = Row<LG, VEC, NI>::col(i, l);
      if (!here || e0 >= a.E) continue;
      float d[VEC];
#pragma unroll
      for (int c = 0; c < VEC; ++c) {
        d[c] = some ? scale * (r.v[i * VEC + c] * fmaf(cb, f[e0 + c] - fp, zt)) : 0.f;
        if (a.w != nullptr) d[c] += add[e0 + c];
      }
      float* to = a.dlogits + (size_t)t * a.E + e0;
      if constexpr (VEC == 4)
        *reinterpret_cast<float4*>(to) = make_float4(d[0], d[1], d[2], d[3]);
      else
        *to = d[0];
    }
    if (a.w != nullptr) {
      __syncwarp();
#pragma unroll
      for (int i = 0; i < KI; ++i)
        if (here && now.e[i] >= 0 && now.e[i] < a.E) add[now.e[i]] = 0.f;
      __syncwarp();
    }
  }
}

// One of the row layouts: vectors of four when the rows are 16-byte aligned
// (E % 4 == 0), fewer lanes a row when it is short.
template <template <int, int, int> class Launch, typename Args>
moe_status dispatch(int E, const Args& a, int blocks, cudaStream_t s) {
  if (E % 4 == 0) {
    if (E <= 32) return Launch<8, 4, 1>::run(a, blocks, s);
    if (E <= 64) return Launch<16, 4, 1>::run(a, blocks, s);
    if (E <= 128) return Launch<32, 4, 1>::run(a, blocks, s);
    if (E <= 256) return Launch<32, 4, 2>::run(a, blocks, s);
    if (E <= 512) return Launch<32, 4, 4>::run(a, blocks, s);
    return Launch<32, 4, 8>::run(a, blocks, s);
  }
  if (E <= 32) return Launch<8, 1, 4>::run(a, blocks, s);
  if (E <= 128) return Launch<32, 1, 4>::run(a, blocks, s);
  if (E <= 512) return Launch<32, 1, 16>::run(a, blocks, s);
  return Launch<32, 1, 32>::run(a, blocks, s);
}
// Lanes that hold a row under dispatch()'s layouts.
int lanes_of_row(int E) { return E <= 32 ? 8 : E % 4 == 0 && E <= 64 ? 16 : 32; }
// Threads of the forward's CTAs: 64 registers a thread hold rows of up to 512
// logits beside their sums.
constexpr int forward_threads(int per_lane) { return per_lane <= 16 ? 1024 : 512; }
int forward_threads_of(int E) { return E > 512 ? 512 : 1024; }

template <int LG, int VEC, int NI>
struct Forward {
  static moe_status run(const RouterLossArgs& a, int blocks, cudaStream_t s) {
    constexpr int THREADS = forward_threads(NI * VEC);
    constexpr int MOST = LG * VEC * NI;  // experts of this layout
    const size_t smem = 4 * (size_t)(THREADS / 32 + 1) * a.E;
    auto kern = router_losses_kernel<LG, VEC, NI, THREADS>;
    // The limit belongs to the function, not to the launch: it is raised once
    // to what the layout's widest rows take, since a call that set its own
    // size could take it from another thread's between its setting and launch.
    static std::atomic<bool> raised[64];
    int dev = 0;
    MOE_TRY_CUDA(cudaGetDevice(&dev));
    if (dev < 0 || dev >= 64) return MOE_ERR_UNSUPPORTED;
    if (!raised[dev].load(std::memory_order_relaxed)) {
      MOE_TRY_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 4 * (THREADS / 32 + 1) * MOST));
      raised[dev].store(true, std::memory_order_relaxed);
    }
    MOE_TRY_CUDA(launch_k(kern, dim3(blocks), dim3(THREADS), smem, s, a));
    return MOE_OK;
  }
};
template <int LG, int VEC, int NI>
struct Backward {
  static moe_status run(const RouterLossGradArgs& a, int blocks, cudaStream_t s) {
    const size_t smem = 4 * (size_t)(1 + (a.w != nullptr ? kThreads / LG : 0)) * a.E;
    MOE_TRY_CUDA(launch_k(router_losses_backward_kernel<LG, VEC, NI>, dim3(blocks), dim3(kThreads), smem, s, a));
    return MOE_OK;
  }
};

int forward_blocks(int T, int E, int num_sms) {
  const int want = ceil_div(T, forward_threads_of(E) / lanes_of_row(E));
  return want < num_sms ? want : num_sms;
}

}  // namespace

size_t router_losses_workspace(int T, int E, int num_sms) {
  return 4 * part_words(E) * (size_t)forward_blocks(T > 0 ? T : 1, E, num_sms);
}

moe_status router_losses_launch(const RouterLossArgs& a, cudaStream_t s) {
  const int blocks = forward_blocks(a.T > 0 ? a.T : 1, a.E, a.num_sms);
  MOE_TRY((dispatch<Forward, RouterLossArgs>(a.E, a, blocks, s)));
  if (blocks > 1)
    MOE_TRY_CUDA(launch_k(router_losses_sum_kernel, dim3(kSumCtas), dim3(kSumThreads), 0, s, a, blocks));
  return MOE_OK;
}

moe_status router_losses_backward_launch(const RouterLossGradArgs& a, cudaStream_t s) {
  const int want = ceil_div(a.T, kThreads / lanes_of_row(a.E)), most = 4 * a.num_sms;
  return dispatch<Backward, RouterLossGradArgs>(a.E, a, want < most ? want : most, s);
}

}  // namespace moe
