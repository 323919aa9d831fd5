// C-ABI entry points of the expert-training operators: host-side checks,
// then one launcher each (include/moe.h states the operations).
#include <stdlib.h>

#include "train.cuh"

namespace moe {
namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

cudaStream_t stream_of(moe_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

constexpr int kMaxExperts = 1024;
constexpr int kMaxRows = 1 << 24;  // as T * k of the layer

// How long the waits inside a launch may take, counted from its start: the
// limit for a launch that gets stuck, and on top of it a long time for what a
// large one has to do (2 R N K operations at 1e14 a second, the experts'
// matrices at 5e11 elements; kernels take a tenth of it or less), so that it
// is not cut off for its size alone.
long long wait_limit_ns(int R, int N, int K, int E) {
  static long long v = [] {
    const char* s = getenv("MOE_WAIT_LIMIT_NS");
    const long long x = s ? atoll(s) : 0;
    return x > 0 ? x : kDefaultWaitNs;
  }();
  const double nk = (double)N * K;
  return v + (long long)(2e-5 * R * nk + 2e-3 * E * nk);
}

moe_status check_router_losses(int32_t T, int32_t E, int32_t k) {
  if (T < 0 || E <= 0 || k <= 0 || k > E) return MOE_ERR_INVALID_ARG;
  if (E > kMaxExperts || k > 32 || (int64_t)T * k > kMaxRows) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_quantize_blocks_e4m3(int32_t rows, int32_t cols, int32_t x_dtype, int32_t scale_kind, const void* x,
                                    int64_t ld_x, uint8_t* codes, float* scales, moe_stream_t stream) {
  if (rows < 0) return MOE_ERR_INVALID_ARG;
  if (cols <= 0 || cols % 8 != 0 || rows > kMaxRows) return MOE_ERR_UNSUPPORTED;
  if (x_dtype != MOE_F32 && x_dtype != MOE_BF16) return MOE_ERR_UNSUPPORTED;
  if (scale_kind != MOE_SCALE_AMAX && scale_kind != MOE_SCALE_POW2) return MOE_ERR_INVALID_ARG;
  if (ld_x < cols || ld_x % (x_dtype == MOE_F32 ? 4 : 8) != 0) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if (x == nullptr || codes == nullptr || scales == nullptr) return MOE_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(codes) || !aligned16(scales)) return MOE_ERR_INVALID_ARG;
  DeviceCtx ctx;
  MOE_TRY(device_ctx(&ctx));
  return quantize_blocks_launch(x, x_dtype == MOE_F32, scale_kind == MOE_SCALE_POW2, rows, cols, ld_x, codes, scales,
                                ctx.num_sms, stream_of(stream));
}

moe_status moe_grouped_block_gemm(int32_t R, int32_t K, int32_t N, int32_t E, int32_t transposed, int32_t out_dtype,
                                  const uint8_t* a_codes, const float* a_scales, const int32_t* offsets,
                                  const uint8_t* w_codes, const float* w_scales, void* out, moe_stream_t stream) {
  if (R < 0 || K <= 0 || N <= 0 || E <= 0) return MOE_ERR_INVALID_ARG;
  if (K % 16 != 0 || N % 16 != 0 || E > kMaxExperts || R > kMaxRows) return MOE_ERR_UNSUPPORTED;
  if (out_dtype != MOE_F32 && out_dtype != MOE_BF16) return MOE_ERR_UNSUPPORTED;
  if (R == 0) return MOE_OK;
  if (!a_codes || !a_scales || !offsets || !w_codes || !w_scales || !out) return MOE_ERR_INVALID_ARG;
  if (!aligned16(a_codes) || !aligned16(a_scales) || !aligned16(offsets) || !aligned16(w_codes) ||
      !aligned16(w_scales) || !aligned16(out))
    return MOE_ERR_INVALID_ARG;
  DeviceCtx ctx;
  MOE_TRY(device_ctx(&ctx));
  BlockGemmArgs a{R,       K,       N,        E,   transposed != 0, out_dtype == MOE_F32, a_codes,        a_scales,
                  offsets, w_codes, w_scales, out, ctx.num_sms,     ctx.status,           wait_limit_ns(R, N, K, E)};
  return block_gemm_launch(a, stream_of(stream));
}

moe_status moe_swiglu_save_e4m3(int32_t R, int32_t ffn, const void* g, const void* u, int64_t ld, void* h,
                                uint8_t* h_codes, float* h_scales, uint8_t* saved_codes, float* saved_scales,
                                moe_stream_t stream) {
  if (R < 0) return MOE_ERR_INVALID_ARG;
  if (ffn <= 0 || ffn % 16 != 0 || R > kMaxRows) return MOE_ERR_UNSUPPORTED;
  if (ld < ffn || ld % 8 != 0 || (h_codes == nullptr) != (h_scales == nullptr)) return MOE_ERR_INVALID_ARG;
  if (R == 0) return MOE_OK;
  if (g == nullptr || u == nullptr || saved_codes == nullptr || saved_scales == nullptr) return MOE_ERR_INVALID_ARG;
  if (!aligned16(g) || !aligned16(u) || !aligned16(h) || !aligned16(h_codes) || !aligned16(h_scales) ||
      !aligned16(saved_codes) || !aligned16(saved_scales))
    return MOE_ERR_INVALID_ARG;
  DeviceCtx ctx;
  MOE_TRY(device_ctx(&ctx));
  SwigluSaveArgs a{R, ffn, g, u, ld, h, h_codes, h_scales, saved_codes, saved_scales};
  return swiglu_save_launch(a, ctx.num_sms, stream_of(stream));
}

moe_status moe_swiglu_backward_e4m3(int32_t R, int32_t ffn, const uint8_t* saved_codes, const float* saved_scales,
                                    const void* dh, void* dg, void* du, int64_t ld, void* h, uint8_t* d_codes,
                                    float* d_scales, moe_stream_t stream) {
  if (R < 0) return MOE_ERR_INVALID_ARG;
  if (ffn <= 0 || ffn % 16 != 0 || R > kMaxRows) return MOE_ERR_UNSUPPORTED;
  if (d_codes != nullptr && ffn % kQBlock != 0) return MOE_ERR_UNSUPPORTED;
  if (ld < ffn || ld % 8 != 0 || (d_codes == nullptr) != (d_scales == nullptr)) return MOE_ERR_INVALID_ARG;
  if (R == 0) return MOE_OK;
  if (!saved_codes || !saved_scales || !dh || !dg || !du) return MOE_ERR_INVALID_ARG;
  if (!aligned16(saved_codes) || !aligned16(saved_scales) || !aligned16(dh) || !aligned16(dg) || !aligned16(du) ||
      !aligned16(h) || !aligned16(d_codes) || !aligned16(d_scales))
    return MOE_ERR_INVALID_ARG;
  DeviceCtx ctx;
  MOE_TRY(device_ctx(&ctx));
  SwigluBackwardArgs a{R, ffn, saved_codes, saved_scales, dh, dg, du, ld, h, d_codes, d_scales};
  return swiglu_backward_launch(a, ctx.num_sms, stream_of(stream));
}

moe_status moe_grouped_wgrad(int32_t R, int32_t N, int32_t K, int32_t E, int32_t x_dtype, int32_t dw_dtype,
                             int32_t accumulate, const void* dy, int64_t ld_dy, const void* x, const float* x_scales,
                             const int32_t* offsets, void* dw, moe_stream_t stream) {
  if (R < 0 || N <= 0 || K <= 0 || E <= 0) return MOE_ERR_INVALID_ARG;
  if (N % 16 != 0 || K % 16 != 0 || E > kMaxExperts || R > kMaxRows) return MOE_ERR_UNSUPPORTED;
  if (x_dtype != MOE_BF16 && x_dtype != MOE_FP8_E4M3) return MOE_ERR_UNSUPPORTED;
  if (dw_dtype != MOE_F32 && dw_dtype != MOE_BF16) return MOE_ERR_UNSUPPORTED;
  if (ld_dy < N || ld_dy % 8 != 0) return MOE_ERR_INVALID_ARG;
  if (dw == nullptr || !aligned16(dw)) return MOE_ERR_INVALID_ARG;
  if (R == 0) {  // every expert is empty: zero gradients
    if (accumulate) return MOE_OK;
    MOE_TRY_CUDA(cudaMemsetAsync(dw, 0, (size_t)E * N * K * (dw_dtype == MOE_F32 ? 4 : 2), stream_of(stream)));
    return MOE_OK;
  }
  if (!dy || !x || !offsets || (x_dtype == MOE_FP8_E4M3) != (x_scales != nullptr)) return MOE_ERR_INVALID_ARG;
  if (!aligned16(dy) || !aligned16(x) || !aligned16(x_scales) || !aligned16(offsets)) return MOE_ERR_INVALID_ARG;
  DeviceCtx ctx;
  MOE_TRY(device_ctx(&ctx));
  WgradArgs a{R,  N,       K,  E, dy, ld_dy, x, x_scales, offsets, dw, dw_dtype == MOE_F32, accumulate != 0,
              ctx.num_sms, ctx.status, wait_limit_ns(R, N, K, E)};
  return grouped_wgrad_launch(a, stream_of(stream));
}

moe_status moe_router_losses_workspace_size_for(int32_t T, int32_t E, int32_t num_sms, size_t* bytes) {
  if (bytes == nullptr || num_sms < 1 || num_sms > 4096) return MOE_ERR_INVALID_ARG;
  MOE_TRY(check_router_losses(T, E, 1));
  *bytes = router_losses_workspace(T, E, num_sms);
  return MOE_OK;
}

moe_status moe_router_losses_workspace_size(int32_t T, int32_t E, size_t* bytes) {
  if (bytes == nullptr) return MOE_ERR_INVALID_ARG;
  DeviceCtx ctx;
  MOE_TRY(device_ctx(&ctx));
  return moe_router_losses_workspace_size_for(T, E, ctx.num_sms, bytes);
}

moe_status moe_router_losses(int32_t T, int32_t E, int32_t k, const float* logits, const int32_t* topk_idx,
                             const uint8_t* mask, float balance_coef, float z_coef, float* loss, int32_t* counts,
                             float* lse, void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  MOE_TRY(check_router_losses(T, E, k));
  if (loss == nullptr || counts == nullptr) return MOE_ERR_INVALID_ARG;
  if (T > 0 && (logits == nullptr || topk_idx == nullptr || lse == nullptr)) return MOE_ERR_INVALID_ARG;
  if (!aligned16(logits)) return MOE_ERR_INVALID_ARG;
  DeviceCtx ctx;
  MOE_TRY(device_ctx(&ctx));
  if (workspace == nullptr || workspace_bytes < router_losses_workspace(T, E, ctx.num_sms)) return MOE_ERR_WORKSPACE;
  if (!aligned16(workspace)) return MOE_ERR_INVALID_ARG;
  RouterLossArgs a{T,    E,      k,   logits,    topk_idx,    mask,      balance_coef, z_coef,
                   loss, counts, lse, workspace, ctx.num_sms, ctx.status};
  return router_losses_launch(a, stream_of(stream));
}

moe_status moe_router_losses_backward(int32_t T, int32_t E, int32_t k, const float* logits, const int32_t* topk_idx,
                                      const uint8_t* mask, float balance_coef, float z_coef, const int32_t* counts,
                                      const float* lse, const float* grad_loss, const float* topk_w,
                                      const float* d_topk_w, float* d_logits, moe_stream_t stream) {
  MOE_TRY(check_router_losses(T, E, k));
  if ((topk_w == nullptr) != (d_topk_w == nullptr)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!logits || !counts || !lse || !d_logits || (topk_w != nullptr && topk_idx == nullptr))
    return MOE_ERR_INVALID_ARG;
  if (!aligned16(logits) || !aligned16(d_logits)) return MOE_ERR_INVALID_ARG;
  DeviceCtx ctx;
  MOE_TRY(device_ctx(&ctx));
  RouterLossGradArgs a{T,   E,         k,      logits,   topk_idx, mask,        balance_coef, z_coef, counts,
                       lse, grad_loss, topk_w, d_topk_w, d_logits, ctx.num_sms, ctx.status};
  return router_losses_backward_launch(a, stream_of(stream));
}

}  // extern "C"
