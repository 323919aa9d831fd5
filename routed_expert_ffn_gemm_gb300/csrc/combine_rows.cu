// Combine over rows with dropped assignments, and its gradients.
//
//   out[t,:] = sum_j w[t,j] y[inv[t,j],:] (+ add[t,:])
//   dy[inv[t,j],:] = w[t,j] dout[t,:],   dw[t,j] = <dout[t,:], y[inv[t,j],:]>
//
// Token by token, so that dout is read once for its k rows and nothing is
// added atomically.  A warp takes a token (forward: a token's pieces go to
// several warps, backward: a CTA takes it, where tokens are few) and keeps eight
// to twelve loads of 16 bytes in flight a lane: up to eight rows, or several
// pieces of fewer; the dot products of the weights' gradient stay in registers
// and are summed over lanes, then warps.  Bound by memory: 16384 tokens of 4096
// in bf16 with two rows each 77 us forward and 99 backward (79 and 99 at the rate
// of a copy), 16384 of 2048 with eight 108 and 180 (99 and 169); 64 tokens of 7168
// with eight rows 3.4 us forward.
#include "mxfp4.cuh"

namespace moe {
namespace {

constexpr int kThreads = 128;
constexpr int kGradThreads = 128;
// Forward: warps an SM for which a token's columns are shared out (2048 tokens of
// 7168 with eight rows each: 58 us with 16, 62 with 32, 54 with 64, 51 with 128, 52
// with 256; 2048 of 4096 with two 8.8 with 16, 7.3 with each of the others).
constexpr int kItems = 64;
constexpr long long kMaxGrid = 1 << 20;
// Backward: from this many tokens an SM on a warp takes a token, below a CTA.  A
// warp and a CTA each: 2048 tokens of 7168 with eight rows 99 and 79 us, 4096 of
// 4096 with two 27.4 and 28.8, 8192 of it 52 and 54; with eight rows of 2048 the
// CTA leads further on (4096 tokens: 52 and 48, 8192: 95 and 91).
constexpr int kTokenWarps = 16;

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

// An item is a token's columns [part * span, (part + 1) * span) of 16 bytes, taken
// by a warp: SLOTS rows and UNROLL pieces of each in flight.  ALL: k <= SLOTS,
// the sums of a piece are done at once; else a piece at a time takes its rows in
// groups of SLOTS.
template <bool F32, int SLOTS, int UNROLL, bool ALL>
__global__ void __launch_bounds__(kThreads) combine_rows_kernel(const CombineRowsArgs p, long long items, int parts,
                                                                int span) {
  static_assert(ALL || UNROLL == 1, "one piece's sums");
  constexpr bool EARLY = SLOTS <= 4;  // add's loads go with the rows' (with eight rows they would cost occupancy)
  griddep_begin();
  using V = Vec<F32>;
  const int lane = threadIdx.x & 31, vecs = p.d / V::N;
  const uint4* rows = static_cast<const uint4*>(p.rows);
  const uint4* add = static_cast<const uint4*>(p.add);  // (may be out)
  const long long step = (long long)gridDim.x * (kThreads / 32);
  for (long long item = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); item < items; item += step) {
    const int t = (int)(item / parts), part = (int)(item - (long long)t * parts);
    int r[SLOTS];
    float w[SLOTS];
    auto slots = [&](int j0) {
#pragma unroll
      for (int j = 0; j < SLOTS; ++j) {
        const size_t a = (size_t)t * p.k + j0 + j;
        r[j] = j0 + j < p.k ? row_at(p.inv_row, a, p.R, p.status) : -1;
        w[j] = r[j] >= 0 && p.w != nullptr ? p.w[a] : 1.f;
      }
    };
    if (ALL) slots(0);
    const int end = min(vecs, (part + 1) * span);
    for (int c0 = part * span + lane; c0 < end; c0 += 32 * UNROLL) {
      uint4 q[UNROLL][SLOTS], more[UNROLL];
      float acc[V::N];
      auto load = [&] {
#pragma unroll
        for (int i = 0; i < UNROLL; ++i) {
          const int at = c0 + 32 * i;
          if (at >= end) continue;
#pragma unroll
          for (int j = 0; j < SLOTS; ++j)
            if (r[j] >= 0) q[i][j] = __ldg(rows + (size_t)r[j] * vecs + at);
          if (EARLY && add != nullptr) more[i] = add[(size_t)t * vecs + at];
        }
      };
      auto sum = [&](int i) {
#pragma unroll
        for (int j = 0; j < SLOTS; ++j) {
          if (r[j] < 0) continue;
          float v[V::N];
          V::values(q[i][j], v);
#pragma unroll
          for (int c = 0; c < V::N; ++c) acc[c] = fmaf(w[j], v[c], acc[c]);
        }
      };
      auto store = [&](int i) {
        const size_t o = (size_t)t * vecs + c0 + 32 * i;
        if (add != nullptr) {
          float v[V::N];
          V::values(EARLY ? more[i] : add[o], v);
#pragma unroll
          for (int c = 0; c < V::N; ++c) acc[c] += v[c];
        }
        static_cast<uint4*>(p.out)[o] = V::pack(acc);
      };
      if constexpr (ALL) {
        load();
#pragma unroll
        for (int i = 0; i < UNROLL; ++i) {
          if (c0 + 32 * i >= end) continue;
#pragma unroll
          for (int c = 0; c < V::N; ++c) acc[c] = 0.f;
          sum(i);
          store(i);
        }
      } else {
#pragma unroll
        for (int c = 0; c < V::N; ++c) acc[c] = 0.f;
        for (int j0 = 0; j0 < p.k; j0 += SLOTS) {
          slots(j0);
          load();
          sum(0);
        }
        store(0);
      }
    }
  }
}

// SLOTS rows of a token at a time, UNROLL pieces of each in flight; WARPS warps
// of the CTA share a token (1 or all of them).
template <bool F32, bool DROWS, bool DW, int SLOTS, int UNROLL, int WARPS>
__global__ void __launch_bounds__(kGradThreads) combine_rows_backward_kernel(const CombineRowsGradArgs p) {
  griddep_begin();
  using V = Vec<F32>;
  constexpr int GROUP = 32 * WARPS, TOKENS = kGradThreads / GROUP;
  __shared__ float part[kGradThreads / 32][SLOTS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, me = threadIdx.x % GROUP, vecs = p.d / V::N;
  const uint4* rows = static_cast<const uint4*>(p.rows);
  for (int t = blockIdx.x * TOKENS + threadIdx.x / GROUP; t < p.T; t += gridDim.x * TOKENS) {
    const uint4* dout = static_cast<const uint4*>(p.d_out) + (size_t)t * vecs;
    for (int j0 = 0; j0 < p.k; j0 += SLOTS) {
      int r[SLOTS];
      float w[SLOTS], dot[SLOTS];
#pragma unroll
      for (int j = 0; j < SLOTS; ++j) {
        const size_t a = (size_t)t * p.k + j0 + j;
        r[j] = j0 + j < p.k ? row_at(p.inv_row, a, p.R, p.status) : -1;
        w[j] = DROWS && r[j] >= 0 && p.w != nullptr ? p.w[a] : 1.f;
        dot[j] = 0.f;
      }
      for (int at0 = me; at0 < vecs; at0 += GROUP * UNROLL) {
        uint4 qd[UNROLL], q[UNROLL][SLOTS];
#pragma unroll
        for (int i = 0; i < UNROLL; ++i) {
          const int at = at0 + GROUP * i;
          if (at >= vecs) continue;
          qd[i] = dout[at];
          if constexpr (DW) {
#pragma unroll
            for (int j = 0; j < SLOTS; ++j)
              if (r[j] >= 0) q[i][j] = __ldg(rows + (size_t)r[j] * vecs + at);
          }
        }
#pragma unroll
        for (int i = 0; i < UNROLL; ++i) {
          const int at = at0 + GROUP * i;
          if (at >= vecs) continue;
          float d[V::N];
          V::values(qd[i], d);
#pragma unroll
          for (int j = 0; j < SLOTS; ++j) {
            if (r[j] < 0) continue;
            float v[V::N];
            if constexpr (DW) {
              V::values(q[i][j], v);
#pragma unroll
              for (int c = 0; c < V::N; ++c) dot[j] = fmaf(d[c], v[c], dot[j]);
            }
            if constexpr (DROWS) {
#pragma unroll
              for (int c = 0; c < V::N; ++c) v[c] = w[j] * d[c];
              static_cast<uint4*>(p.d_rows)[(size_t)r[j] * vecs + at] = V::pack(v);
            }
          }
        }
      }
      if constexpr (DW) {
#pragma unroll
        for (int j = 0; j < SLOTS; ++j) {
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], o);
        }
        if constexpr (WARPS == 1) {
#pragma unroll
          for (int j = 0; j < SLOTS; ++j)
            if (lane == j && j0 + j < p.k) p.dw[(size_t)t * p.k + j0 + j] = dot[j];
        } else {
#pragma unroll
          for (int j = 0; j < SLOTS; ++j)
            if (lane == 0) part[warp][j] = dot[j];
          __syncthreads();
          const int j = (int)threadIdx.x;
          if (j < SLOTS && j0 + j < p.k) {
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
}

template <bool F32, bool DROWS, bool DW>
moe_status launch_backward(const CombineRowsGradArgs& a, cudaStream_t s) {
  constexpr int ALL = kGradThreads / 32;
  const bool wide = a.T < kTokenWarps * a.num_sms;  // few tokens: a CTA each
  const int ctas = wide ? a.T : ceil_div(a.T, ALL), most = 64 * a.num_sms;
  auto few = a.k <= 2   ? combine_rows_backward_kernel<F32, DROWS, DW, 2, 4, ALL>
             : a.k <= 4 ? combine_rows_backward_kernel<F32, DROWS, DW, 4, 2, ALL>
                        : combine_rows_backward_kernel<F32, DROWS, DW, 8, 1, ALL>;
  auto many = a.k <= 2   ? combine_rows_backward_kernel<F32, DROWS, DW, 2, 4, 1>
              : a.k <= 4 ? combine_rows_backward_kernel<F32, DROWS, DW, 4, 2, 1>
                         : combine_rows_backward_kernel<F32, DROWS, DW, 8, 1, 1>;
  auto kern = wide ? few : many;
  MOE_TRY_CUDA(launch_k(kern, dim3(ctas < most ? ctas : most), dim3(kGradThreads), 0, s, a));
  return MOE_OK;
}

}  // namespace

namespace {

template <bool F32, int SLOTS, int UNROLL, bool ALL>
moe_status launch_forward(const CombineRowsArgs& a, cudaStream_t s) {
  // a warp a token, or a token's pieces over several warps where tokens are few
  const int vecs = a.d / Vec<F32>::N, pieces = ceil_div(vecs, 32 * UNROLL);
  const int parts = max(1, min(pieces, kItems * a.num_sms / a.T));
  const int span = ceil_div(pieces, parts) * 32 * UNROLL;
  const long long items = (long long)a.T * ceil_div(vecs, span);
  const long long want = (items + kThreads / 32 - 1) / (kThreads / 32);
  MOE_TRY_CUDA(launch_k(combine_rows_kernel<F32, SLOTS, UNROLL, ALL>, dim3((unsigned)(want < kMaxGrid ? want : kMaxGrid)),
                        dim3(kThreads), 0, s, a, items, ceil_div(vecs, span), span));
  return MOE_OK;
}

template <bool F32>
moe_status launch_forward(const CombineRowsArgs& a, cudaStream_t s) {
  if (a.k <= 1) return launch_forward<F32, 1, 4, true>(a, s);
  if (a.k <= 2) return launch_forward<F32, 2, 4, true>(a, s);
  if (a.k <= 4) return launch_forward<F32, 4, 2, true>(a, s);
  return a.k <= 8 ? launch_forward<F32, 8, 1, true>(a, s) : launch_forward<F32, 8, 1, false>(a, s);
}

}  // namespace

moe_status combine_rows_launch(const CombineRowsArgs& a, cudaStream_t s) {
  return a.f32 ? launch_forward<true>(a, s) : launch_forward<false>(a, s);
}

moe_status combine_rows_backward_launch(const CombineRowsGradArgs& a, cudaStream_t s) {
  const bool dr = a.d_rows != nullptr, dw = a.dw != nullptr;
  if (!dr && !dw) return MOE_OK;
  if (!dr) return a.f32 ? launch_backward<true, false, true>(a, s) : launch_backward<false, false, true>(a, s);
  if (!dw) return a.f32 ? launch_backward<true, true, false>(a, s) : launch_backward<false, true, false>(a, s);
  return a.f32 ? launch_backward<true, true, true>(a, s) : launch_backward<false, true, true>(a, s);
}

}  // namespace moe
