// Combine over rows with dropped assignments, and its gradients.
//
//   out[t,:] = sum_j w[t,j] y[inv[t,j],:] (+ add[t,:])
//   dy[inv[t,j],:] = w[t,j] dout[t,:],   dw[t,j] = <dout[t,:], y[inv[t,j],:]>
//
// Token by token, so that dout is read once for its k rows and nothing is
// added atomically.  Forward: a warp takes a piece of 32 x 16 bytes of a token
// and has the loads of eight rows in flight.  Backward: a CTA takes a token,
// each thread 16 bytes of dout and of eight rows at a time; eight dot products
// stay in registers and are summed over lanes, then warps.  Both are bound by
// memory.
#include "mxfp4.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kGradThreads = 128;
constexpr int kSlots = 8;  // rows of a token in flight

// 16 bytes: 8 values of bf16 or 4 of fp32.
template <bool F32>
struct Vec {
  static constexpr int N = F32 ? 4 : 8;
  static __device__ __forceinline__ void values(uint4 q, float (&v)[N]) {
    if constexpr (F32) {
      v[0] = __uint_as_float(q.x);
      v[1] = __uint_as_float(q.y);
      v[2] = __uint_as_float(q.z);
      v[3] = __uint_as_float(q.w);
    } else {
      bf16_values(q, v);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&v)[N]) {
    if constexpr (F32)
      return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    else
      return bf16_pack(v);
  }
};

// The row of an assignment, -1 where it has none.
__device__ __forceinline__ int row_at(const int32_t* inv, size_t a, int R, int* status) {
  const int r = inv[a];
  if (r < R) return r < 0 ? -1 : r;
  set_device_status(status, MOE_ERR_DEVICE_BOUNDS);
  return -1;
}

template <bool F32>
__global__ void __launch_bounds__(kThreads) combine_rows_kernel(const CombineRowsArgs p, long long pieces_all, int pieces) {
  griddep_begin();
  using V = Vec<F32>;
  const int lane = threadIdx.x & 31, vecs = p.d / V::N;
  const uint4* rows = static_cast<const uint4*>(p.rows);
  for (long long i = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); i < pieces_all;
       i += (long long)gridDim.x * (kThreads / 32)) {
    const int t = (int)(i / pieces), at = (int)(i - (long long)t * pieces) * 32 + lane;
    int r = -1;
    float w = 1.f;
    if (lane < p.k) {
      r = row_at(p.inv_row, (size_t)t * p.k + lane, p.R, p.status);
      if (p.w != nullptr && r >= 0) w = p.w[(size_t)t * p.k + lane];
    }
    const bool live = at < vecs;
    float acc[V::N];
#pragma unroll
    for (int c = 0; c < V::N; ++c) acc[c] = 0.f;
    for (int j0 = 0; j0 < p.k; j0 += kSlots) {
      uint4 q[kSlots];
      int rj[kSlots];
#pragma unroll
      for (int j = 0; j < kSlots; ++j) {
        rj[j] = j0 + j < p.k ? __shfl_sync(0xffffffffu, r, j0 + j) : -1;
        if (live && rj[j] >= 0) q[j] = __ldg(rows + (size_t)rj[j] * vecs + at);
      }
#pragma unroll
      for (int j = 0; j < kSlots; ++j) {
        const float wj = __shfl_sync(0xffffffffu, w, (j0 + j) & 31);
        if (live && rj[j] >= 0) {
          float v[V::N];
          V::values(q[j], v);
#pragma unroll
          for (int c = 0; c < V::N; ++c) acc[c] = fmaf(wj, v[c], acc[c]);
        }
      }
    }
    if (!live) continue;
    const size_t o = (size_t)t * vecs + at;
    if (p.add != nullptr) {
      float v[V::N];
      V::values(static_cast<const uint4*>(p.add)[o], v);  // (add may be out)
#pragma unroll
      for (int c = 0; c < V::N; ++c) acc[c] += v[c];
    }
    static_cast<uint4*>(p.out)[o] = V::pack(acc);
  }
}

template <bool F32, bool DROWS, bool DW>
__global__ void __launch_bounds__(kGradThreads) combine_rows_backward_kernel(const CombineRowsGradArgs p) {
  griddep_begin();
  using V = Vec<F32>;
  constexpr int WARPS = kGradThreads / 32;
  __shared__ float part[WARPS][kSlots];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, vecs = p.d / V::N;
  const uint4* rows = static_cast<const uint4*>(p.rows);
  for (int t = blockIdx.x; t < p.T; t += gridDim.x) {
    const uint4* dout = static_cast<const uint4*>(p.d_out) + (size_t)t * vecs;
    for (int j0 = 0; j0 < p.k; j0 += kSlots) {
      int r[kSlots];
      float w[kSlots], dot[kSlots];
#pragma unroll
      for (int j = 0; j < kSlots; ++j) {
        const size_t a = (size_t)t * p.k + j0 + j;
        r[j] = j0 + j < p.k ? row_at(p.inv_row, a, p.R, p.status) : -1;
        w[j] = DROWS && r[j] >= 0 && p.w != nullptr ? p.w[a] : 1.f;
        dot[j] = 0.f;
      }
      for (int at = threadIdx.x; at < vecs; at += kGradThreads) {
        float d[V::N];
        const uint4 qd = dout[at];
        uint4 q[kSlots];
        if constexpr (DW) {
#pragma unroll
          for (int j = 0; j < kSlots; ++j)
            if (r[j] >= 0) q[j] = __ldg(rows + (size_t)r[j] * vecs + at);
        }
        V::values(qd, d);
#pragma unroll
        for (int j = 0; j < kSlots; ++j) {
          if (r[j] < 0) continue;
          if constexpr (DW) {
            float v[V::N];
            V::values(q[j], v);
#pragma unroll
            for (int c = 0; c < V::N; ++c) dot[j] = fmaf(d[c], v[c], dot[j]);
          }
          if constexpr (DROWS) {
            float v[V::N];
#pragma unroll
            for (int c = 0; c < V::N; ++c) v[c] = w[j] * d[c];
            static_cast<uint4*>(p.d_rows)[(size_t)r[j] * vecs + at] = V::pack(v);
          }
        }
      }
      if constexpr (DW) {
#pragma unroll
        for (int j = 0; j < kSlots; ++j) {
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], o);
          if (lane == 0) part[warp][j] = dot[j];
        }
        __syncthreads();
        const int j = (int)threadIdx.x;
        if (j < kSlots && j0 + j < p.k) {
          float sum = 0.f;
#pragma unroll
          for (int v = 0; v < WARPS; ++v) sum += part[v][j];
          p.dw[(size_t)t * p.k + j0 + j] = sum;
        }
        __syncthreads();
      }
    }
  }
}

}  // namespace

moe_status combine_rows_launch(const CombineRowsArgs& a, cudaStream_t s) {
  const int pieces = ceil_div(a.d / (a.f32 ? 4 : 8), 32);
  const long long all = (long long)a.T * pieces, want = (all + kThreads / 32 - 1) / (kThreads / 32);
  const int grid = (int)(want < 16ll * a.num_sms ? want : 16ll * a.num_sms);
  auto kern = a.f32 ? combine_rows_kernel<true> : combine_rows_kernel<false>;
  MOE_TRY_CUDA(launch_k(kern, dim3(grid), dim3(kThreads), 0, s, a, all, pieces));
  return MOE_OK;
}

moe_status combine_rows_backward_launch(const CombineRowsGradArgs& a, cudaStream_t s) {
  const int grid = a.T < 32 * a.num_sms ? a.T : 32 * a.num_sms;
  const bool dr = a.d_rows != nullptr, dw = a.dw != nullptr;
  if (!dr && !dw) return MOE_OK;
  auto kern = a.f32 ? (dr ? (dw ? combine_rows_backward_kernel<true, true, true> : combine_rows_backward_kernel<true, true, false>)
                          : combine_rows_backward_kernel<true, false, true>)
                    : (dr ? (dw ? combine_rows_backward_kernel<false, true, true> : combine_rows_backward_kernel<false, true, false>)
                          : combine_rows_backward_kernel<false, false, true>);
  MOE_TRY_CUDA(launch_k(kern, dim3(grid), dim3(kGradThreads), 0, s, a));
  return MOE_OK;
}

}  // namespace moe
