// ck_fp4_api.cu -- the extern "C" boundary of the microscaled fp4 operators declared in
// include/ck.h: argument validation and workspace layout.
#include <cuda_runtime_api.h>
#include <stdint.h>

#include "ck.h"
#include "ck_internal.h"

namespace ck {

static constexpr int kMaxExperts = 1024;
static constexpr int64_t kTileRows = 128, kTileBytes = 512;

static bool fp4_float(ck_dtype d) { return d == CK_F32 || d == CK_F16 || d == CK_BF16; }
static bool fp4_format(ck_fp4_format f) { return f == CK_MXFP4 || f == CK_NVFP4; }
// On an address that the type's elements can have (NULL is one).
static bool fp4_at(const void* p, ck_dtype d) { return aligned(p, d == CK_F32 ? 4 : d == CK_FP4 ? 1 : 2); }
static int64_t up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }
static int64_t fp4_block_of(ck_fp4_format f) { return f == CK_NVFP4 ? 16 : 32; }
// Sizes beyond these are refused before any of them is multiplied.
static bool fp4_sizes(int64_t M, int64_t K, ck_fp4_format f) {
    return fp4_format(f) && M >= 0 && M < (1LL << 31) && K > 0 && K < (1LL << 31) &&
           K % fp4_block_of(f) == 0;
}
static int64_t scale_bytes(int64_t M, int64_t K, ck_fp4_format f, int n_experts) {
    const int64_t blocks = n_experts > 0 ? M / kTileRows + n_experts : up(M, kTileRows) / kTileRows;
    return blocks * (up(K, 4 * fp4_block_of(f)) / (4 * fp4_block_of(f))) * kTileBytes;
}

static ck_status product(const void* x, ck_dtype x_dtype, int64_t M, int64_t K, int64_t stride_m,
                         int64_t stride_k, ck_fp4_format format, const uint8_t* x_scales,
                         const float* x_ts, const int32_t* offsets, int n_experts, const uint8_t* w,
                         int64_t N, int64_t w_ld, int64_t w_stride, const uint8_t* w_scales,
                         const float* w_ts, const void* bias, ck_dtype bias_dtype, void* out,
                         ck_dtype out_dtype, int64_t ldo, void* workspace, size_t workspace_bytes,
                         int* dev_status, cudaStream_t stream) {
    const bool codes_in = x_dtype == CK_FP4;
    if (!(codes_in || fp4_float(x_dtype)) || !fp4_float(out_dtype) || !fp4_format(format) ||
        (bias && !fp4_float(bias_dtype)))
        return CK_ERR_INVALID_ARG;
    if (M < 0 || N < 0 || K <= 0 || K % fp4_block_of(format) != 0) return CK_ERR_INVALID_ARG;
    if (w_ld < K / 2 || w_ld % 16 != 0 || ldo < N) return CK_ERR_INVALID_ARG;
    if (format == CK_MXFP4 && (x_ts || w_ts)) return CK_ERR_INVALID_ARG;
    if (codes_in && (stride_k != 1 || stride_m < K / 2 || stride_m % 16 != 0)) return CK_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return CK_OK;
    if (!x || !w || !w_scales || !out || (codes_in && !x_scales)) return CK_ERR_INVALID_ARG;
    if (!aligned(w, 16) || !aligned(w_scales, 16)) return CK_ERR_INVALID_ARG;
    if (codes_in && (!aligned(x, 16) || !aligned(x_scales, 16))) return CK_ERR_INVALID_ARG;
    if (!fp4_at(x, x_dtype) || !fp4_at(out, out_dtype) || (bias && !fp4_at(bias, bias_dtype)) ||
        !aligned(x_ts, 4) || !aligned(w_ts, 4) || !aligned(offsets, 4) || !aligned(dev_status, 4))
        return CK_ERR_INVALID_ARG;
    if (M >= (1LL << 31) || N >= (1LL << 31) || K >= (1LL << 31)) return CK_ERR_UNSUPPORTED;

    Fp4Product a = {};
    a.M = M;
    a.K = K;
    a.nv = format == CK_NVFP4;
    a.x_ts = x_ts;
    a.offsets = offsets;
    a.n_experts = n_experts;
    a.w = w;
    a.N = N;
    a.w_ld = w_ld;
    a.w_stride = w_stride;
    a.w_scales = w_scales;
    a.w_ts = w_ts;
    a.bias = bias;
    a.bias_dt = bias_dtype;
    a.out = out;
    a.out_dt = out_dtype;
    a.ldo = ldo;
    a.dev_status = dev_status;
    const bool ragged = out_dtype != CK_F32 && (ldo % 8 != 0 || !aligned(out, 16));
    const bool few = !offsets && fp4_few_takes(M, N, K, a.nv, ragged);
    if (codes_in) {
        a.codes = static_cast<const uint8_t*>(x);
        a.ldq = stride_m;
        a.scales = x_scales;
        return few ? launch_fp4_few(a, nullptr, x_dtype, 0, 0, stream) : launch_fp4_gemm(a, stream);
    }
    if (!offsets && fp4_few_fuses(M, K)) return launch_fp4_few(a, x, x_dtype, stride_m, stride_k, stream);
    const size_t need = ck_fp4_linear_workspace_bytes(M, K, format, offsets ? n_experts : 0);
    if (!workspace || workspace_bytes < need || !aligned(workspace, 256)) return CK_ERR_WORKSPACE;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const int64_t pitch = up(K / 2, 16);
    uint8_t* scales = ws + up(M * pitch, 256);
    const ck_status st = launch_quant_fp4(x, x_dtype, M, K, stride_m, stride_k, a.nv, x_ts, offsets,
                                          n_experts, ws, pitch, scales, stream);
    if (st != CK_OK) return st;
    a.codes = ws;
    a.ldq = pitch;
    a.scales = scales;
    a.dependent = true;
    return few ? launch_fp4_few(a, nullptr, x_dtype, 0, 0, stream) : launch_fp4_gemm(a, stream);
}

}  // namespace ck

using namespace ck;

extern "C" {

size_t ck_fp4_scales_bytes(int64_t M, int64_t K, ck_fp4_format format, int n_experts) {
    if (!fp4_sizes(M, K, format) || n_experts < 0 || n_experts > kMaxExperts) return 0;
    return (size_t)scale_bytes(M, K, format, n_experts);
}

size_t ck_fp4_linear_workspace_bytes(int64_t M, int64_t K, ck_fp4_format format, int n_experts) {
    if (!fp4_sizes(M, K, format) || n_experts < 0 || n_experts > kMaxExperts) return 0;
    if (n_experts == 0 && fp4_few_fuses(M, K)) return 0;   // one launch, nothing to keep
    return (size_t)up(M * up(K / 2, 16), 256) + (size_t)scale_bytes(M, K, format, n_experts);
}

ck_status ck_quant_fp4(const void* x, ck_dtype x_dtype, int64_t M, int64_t K, int64_t stride_m,
                       int64_t stride_k, ck_fp4_format format, const float* tensor_scale,
                       const int32_t* offsets, int n_experts, uint8_t* codes, int64_t ldq,
                       uint8_t* scales, cudaStream_t stream) {
    if (!fp4_float(x_dtype) || !fp4_format(format) || M < 0 || K <= 0 ||
        K % fp4_block_of(format) != 0 || ldq < K / 2 || (format == CK_MXFP4 && tensor_scale) ||
        (offsets && (n_experts < 1 || n_experts > kMaxExperts)))
        return CK_ERR_INVALID_ARG;
    if (M == 0) return CK_OK;
    if (!x || !codes || !scales || !aligned(scales, 16) || !fp4_at(x, x_dtype) ||
        !aligned(tensor_scale, 4) || !aligned(offsets, 4))
        return CK_ERR_INVALID_ARG;
    if (!fp4_sizes(M, K, format)) return CK_ERR_UNSUPPORTED;
    return launch_quant_fp4(x, x_dtype, M, K, stride_m, stride_k, format == CK_NVFP4, tensor_scale,
                            offsets, n_experts, codes, ldq, scales, stream);
}

ck_status ck_dequant_fp4(const uint8_t* codes, int64_t ldq, const uint8_t* scales, int64_t M, int64_t K,
                         ck_fp4_format format, const float* tensor_scale, const int32_t* offsets,
                         int n_experts, void* out, ck_dtype out_dtype, int64_t ldo,
                         cudaStream_t stream) {
    if (!fp4_float(out_dtype) || !fp4_format(format) || M < 0 || K <= 0 ||
        K % fp4_block_of(format) != 0 || ldq < K / 2 || ldo < K ||
        (format == CK_MXFP4 && tensor_scale) ||
        (offsets && (n_experts < 1 || n_experts > kMaxExperts)))
        return CK_ERR_INVALID_ARG;
    if (M == 0) return CK_OK;
    if (!codes || !scales || !out || !aligned(scales, 16) || !fp4_at(out, out_dtype) ||
        !aligned(tensor_scale, 4) || !aligned(offsets, 4))
        return CK_ERR_INVALID_ARG;
    if (!fp4_sizes(M, K, format)) return CK_ERR_UNSUPPORTED;
    return launch_dequant_fp4(codes, ldq, scales, M, K, format == CK_NVFP4, tensor_scale, offsets,
                              n_experts, out, out_dtype, ldo, stream);
}

ck_status ck_fp4_linear(const void* x, ck_dtype x_dtype, int64_t M, int64_t K, int64_t stride_m,
                        int64_t stride_k, ck_fp4_format format, const uint8_t* x_scales,
                        const float* x_tensor_scale, const uint8_t* w, int64_t N, int64_t w_ld,
                        const uint8_t* w_scales, const float* w_tensor_scale, const void* bias,
                        ck_dtype bias_dtype, void* out, ck_dtype out_dtype, int64_t ldo,
                        void* workspace, size_t workspace_bytes, int* dev_status,
                        cudaStream_t stream) {
    return product(x, x_dtype, M, K, stride_m, stride_k, format, x_scales, x_tensor_scale, nullptr, 0, w,
                   N, w_ld, 0, w_scales, w_tensor_scale, bias, bias_dtype, out, out_dtype, ldo, workspace,
                   workspace_bytes, dev_status, stream);
}

ck_status ck_fp4_expert_linear(const void* x, ck_dtype x_dtype, int64_t M, int64_t K, int64_t stride_m,
                               int64_t stride_k, ck_fp4_format format, const uint8_t* x_scales,
                               const float* x_tensor_scale, const int32_t* offsets, int n_experts,
                               const uint8_t* w, int64_t N, int64_t w_ld, int64_t w_stride,
                               const uint8_t* w_scales, const float* w_tensor_scale, const void* bias,
                               ck_dtype bias_dtype, void* out, ck_dtype out_dtype, int64_t ldo,
                               void* workspace, size_t workspace_bytes, int* dev_status,
                               cudaStream_t stream) {
    if (n_experts < 1 || n_experts > kMaxExperts) return CK_ERR_INVALID_ARG;
    if (n_experts > 1 && (w_stride % 16 != 0 || w_stride < 0 || (N > 0 && w_stride / N < w_ld)))
        return CK_ERR_INVALID_ARG;
    if (M > 0 && N > 0 && !offsets) return CK_ERR_INVALID_ARG;
    return product(x, x_dtype, M, K, stride_m, stride_k, format, x_scales, x_tensor_scale, offsets,
                   n_experts, w, N, w_ld, w_stride, w_scales, w_tensor_scale, bias, bias_dtype, out,
                   out_dtype, ldo, workspace, workspace_bytes, dev_status, stream);
}

void ck_internal_fp4_tile(int64_t M, int64_t N, int64_t K, ck_fp4_format format, int n_experts, int ragged,
                          int* ctas, int* rows) {
    const Fp4Shape s = fp4_gemm_shape(M, N, K, n_experts > 0 ? n_experts : 1);
    *ctas = n_experts == 0 && fp4_few_takes(M, N, K, format == CK_NVFP4, ragged != 0) ? 0 : s.cg;
    *rows = s.bn;
}

}  // extern "C"
