// C-ABI entry points of the 4-bit operators and the token movement: host-side
// checks, then one launcher each (include/moe.h states the operations).
#include "mxfp4.cuh"

namespace moe {
namespace {

bool aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

cudaStream_t stream_of(moe_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

constexpr int kMaxExperts = 1024;
constexpr int kMaxSlots = 32;
constexpr int kMaxRows = 1 << 24;

bool plain_type(int t) { return t == MOE_F32 || t == MOE_BF16; }

// Tokens, slots and, for the movement of rows, columns.
moe_status check_tokens(int32_t T, int32_t d, int32_t k) {
  if (T < 0 || d <= 0 || k <= 0) return MOE_ERR_INVALID_ARG;
  if (k > kMaxSlots || (int64_t)T * k > kMaxRows || d % 8 != 0) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe_status check_mx_rows(int32_t rows, int32_t cols, int32_t dtype, int32_t matrix_rows) {
  if (rows < 0 || matrix_rows < 0) return MOE_ERR_INVALID_ARG;
  if (cols <= 0 || cols % kMxBlock != 0 || rows > kMaxRows || !plain_type(dtype)) return MOE_ERR_UNSUPPORTED;
  if (matrix_rows > 0 && rows % matrix_rows != 0) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

bool mx_scale_kind(int32_t k) { return k == MOE_MX_FLOOR || k == MOE_MX_FIT; }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_dispatch_workspace_size(int32_t T, int32_t E, int32_t k, size_t* bytes) {
  if (bytes == nullptr || E <= 0) return MOE_ERR_INVALID_ARG;
  MOE_TRY(check_tokens(T, 8, k));
  if (E > kMaxExperts) return MOE_ERR_UNSUPPORTED;
  *bytes = dispatch_workspace(T, E, k);
  return MOE_OK;
}

moe_status moe_dispatch(int32_t T, int32_t d, int32_t E, int32_t k, int32_t x_dtype, int32_t rows_dtype,
                        int32_t scale_kind, const void* x, int64_t ld_x, const int32_t* topk_idx, int32_t* counts,
                        int32_t* offsets, int32_t* row_token, int32_t* inv_row, void* rows, uint8_t* row_scales,
                        void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  MOE_TRY(check_tokens(T, d, k));
  if (E <= 0 || !mx_scale_kind(scale_kind)) return MOE_ERR_INVALID_ARG;
  if (E > kMaxExperts || !plain_type(x_dtype)) return MOE_ERR_UNSUPPORTED;
  const bool to_mx = rows_dtype == MOE_MXFP4;
  if ((!to_mx && rows_dtype != x_dtype) || (to_mx && d % kMxBlock != 0)) return MOE_ERR_UNSUPPORTED;
  if (counts == nullptr || offsets == nullptr || !aligned(counts) || !aligned(offsets)) return MOE_ERR_INVALID_ARG;
  if (T == 0) {
    MOE_TRY_CUDA(cudaMemsetAsync(counts, 0, sizeof(int32_t) * E, stream_of(stream)));
    MOE_TRY_CUDA(cudaMemsetAsync(offsets, 0, sizeof(int32_t) * (E + 1), stream_of(stream)));
    return MOE_OK;
  }
  if (topk_idx == nullptr || row_token == nullptr || inv_row == nullptr) return MOE_ERR_INVALID_ARG;
  if (!aligned(topk_idx) || !aligned(row_token) || !aligned(inv_row)) return MOE_ERR_INVALID_ARG;
  if (rows != nullptr) {
    if (x == nullptr || (to_mx && row_scales == nullptr)) return MOE_ERR_INVALID_ARG;
    if (ld_x < d || ld_x % (x_dtype == MOE_F32 ? 4 : 8) != 0) return MOE_ERR_INVALID_ARG;
    if (!aligned(x) || !aligned(rows) || !aligned(row_scales)) return MOE_ERR_INVALID_ARG;
  }
  const size_t need = dispatch_workspace(T, E, k);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return MOE_ERR_WORKSPACE;
  if (!aligned(workspace)) return MOE_ERR_INVALID_ARG;
  DeviceCtx ctx;
  MOE_TRY(device_ctx(&ctx));
  DispatchArgs a{T,      d,       E,         k,       x_dtype == MOE_F32, to_mx, scale_kind == MOE_MX_FIT, x, ld_x, topk_idx,
                 counts, offsets, row_token, inv_row, rows, row_scales, static_cast<int32_t*>(workspace), ctx.num_sms,
                 ctx.status};
  return dispatch_launch(a, stream_of(stream));
}

moe_status moe_combine_rows(int32_t T, int32_t d, int32_t k, int32_t R, int32_t dtype, const void* rows,
                            const int32_t* inv_row, const float* topk_w, const void* add, void* out,
                            moe_stream_t stream) {
  MOE_TRY(check_tokens(T, d, k));
  if (R < 0) return MOE_ERR_INVALID_ARG;
  if (!plain_type(dtype) || R > kMaxRows) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if ((rows == nullptr && R > 0) || inv_row == nullptr || out == nullptr) return MOE_ERR_INVALID_ARG;
  if (!aligned(rows) || !aligned(inv_row) || !aligned(topk_w) || !aligned(add) || !aligned(out))
    return MOE_ERR_INVALID_ARG;
  DeviceCtx ctx;
  MOE_TRY(device_ctx(&ctx));
  CombineRowsArgs a{T, d, k, R, dtype == MOE_F32, rows, inv_row, topk_w, add, out, ctx.num_sms, ctx.status};
  return combine_rows_launch(a, stream_of(stream));
}

moe_status moe_combine_rows_backward(int32_t T, int32_t d, int32_t k, int32_t R, int32_t dtype, const void* d_out,
                                     const void* rows, const int32_t* inv_row, const float* topk_w, void* d_rows,
                                     float* d_topk_w, moe_stream_t stream) {
  MOE_TRY(check_tokens(T, d, k));
  if (R < 0) return MOE_ERR_INVALID_ARG;
  if (!plain_type(dtype) || R > kMaxRows) return MOE_ERR_UNSUPPORTED;
  if (T == 0 || (d_rows == nullptr && d_topk_w == nullptr)) return MOE_OK;
  if (d_out == nullptr || inv_row == nullptr || (d_topk_w != nullptr && rows == nullptr && R > 0))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(d_out) || !aligned(rows) || !aligned(inv_row) || !aligned(topk_w) || !aligned(d_rows) ||
      !aligned(d_topk_w))
    return MOE_ERR_INVALID_ARG;
  DeviceCtx ctx;
  MOE_TRY(device_ctx(&ctx));
  CombineRowsGradArgs a{T,      d,      k,        R,           dtype == MOE_F32, d_out, rows, inv_row,
                        topk_w, d_rows, d_topk_w, ctx.num_sms, ctx.status};
  return combine_rows_backward_launch(a, stream_of(stream));
}

moe_status moe_quantize_mxfp4(int32_t rows, int32_t cols, int32_t x_dtype, int32_t scale_kind, int32_t matrix_rows,
                              const void* x, int64_t ld_x, uint8_t* codes, uint8_t* scales, moe_stream_t stream) {
  MOE_TRY(check_mx_rows(rows, cols, x_dtype, matrix_rows));
  if (!mx_scale_kind(scale_kind)) return MOE_ERR_INVALID_ARG;
  if (ld_x < cols || ld_x % (x_dtype == MOE_F32 ? 4 : 8) != 0) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if (x == nullptr || codes == nullptr || scales == nullptr) return MOE_ERR_INVALID_ARG;
  if (!aligned(x) || !aligned(codes) || !aligned(scales)) return MOE_ERR_INVALID_ARG;
  return quantize_mxfp4_launch(x, x_dtype == MOE_F32, scale_kind == MOE_MX_FIT, rows, cols, matrix_rows, ld_x, codes,
                               scales, stream_of(stream));
}

moe_status moe_mxfp4_values(int32_t rows, int32_t cols, int32_t dtype, int32_t matrix_rows, const uint8_t* codes,
                            const uint8_t* scales, void* out, moe_stream_t stream) {
  MOE_TRY(check_mx_rows(rows, cols, dtype, matrix_rows));
  if (rows == 0) return MOE_OK;
  if (codes == nullptr || scales == nullptr || out == nullptr) return MOE_ERR_INVALID_ARG;
  if (!aligned(codes) || !aligned(scales) || !aligned(out)) return MOE_ERR_INVALID_ARG;
  return mxfp4_values_launch(codes, scales, dtype == MOE_F32, rows, cols, matrix_rows, out,
                             stream_of(stream));
}

moe_status moe_swiglu_mxfp4(int32_t R, int32_t ffn, int32_t scale_kind, const void* g, const void* u, int64_t ld,
                            uint8_t* codes, uint8_t* scales, void* h, moe_stream_t stream) {
  if (R < 0 || !mx_scale_kind(scale_kind)) return MOE_ERR_INVALID_ARG;
  if (ffn <= 0 || ffn % kMxBlock != 0 || R > kMaxRows) return MOE_ERR_UNSUPPORTED;
  if (ld < ffn || ld % 8 != 0) return MOE_ERR_INVALID_ARG;
  if (R == 0) return MOE_OK;
  if (g == nullptr || u == nullptr || codes == nullptr || scales == nullptr) return MOE_ERR_INVALID_ARG;
  if (!aligned(g) || !aligned(u) || !aligned(codes) || !aligned(scales) || !aligned(h)) return MOE_ERR_INVALID_ARG;
  SwigluMxArgs a{R, ffn, scale_kind == MOE_MX_FIT, g, u, ld, codes, scales, h};
  return swiglu_mxfp4_launch(a, stream_of(stream));
}

moe_status moe_grouped_mxfp4_gemm(int32_t R, int32_t K, int32_t N, int32_t E, int32_t out_dtype,
                                  const uint8_t* a_codes, const uint8_t* a_scales, const int32_t* offsets,
                                  const uint8_t* w_codes, const uint8_t* w_scales, void* out, int64_t ld_out,
                                  moe_stream_t stream) {
  if (R < 0 || K <= 0 || N <= 0 || E <= 0) return MOE_ERR_INVALID_ARG;
  if (K % kMxBlock != 0 || N % 16 != 0 || E > kMaxExperts || R > kMaxRows || !plain_type(out_dtype))
    return MOE_ERR_UNSUPPORTED;
  if (ld_out < N || ld_out % (out_dtype == MOE_F32 ? 4 : 8) != 0) return MOE_ERR_INVALID_ARG;
  if (R == 0) return MOE_OK;
  if (!a_codes || !a_scales || !offsets || !w_codes || !w_scales || !out) return MOE_ERR_INVALID_ARG;
  if (!aligned(a_codes) || !aligned(a_scales) || !aligned(offsets) || !aligned(w_codes) || !aligned(w_scales) ||
      !aligned(out))
    return MOE_ERR_INVALID_ARG;
  DeviceCtx ctx;
  MOE_TRY(device_ctx(&ctx));
  MxGemmArgs a{R,        K,   N,      E,           out_dtype == MOE_F32, a_codes, a_scales, offsets, w_codes,
               w_scales, out, ld_out, ctx.num_sms, ctx.status,           wait_limit_ns(R, N, K, E)};
  return mxfp4_gemm_launch(a, stream_of(stream));
}

}  // extern "C"
