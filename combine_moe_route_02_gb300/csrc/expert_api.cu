// expert_api.cu -- the C ABI of the experts: argument checks on the host (before
// any CUDA call), then the launch.
#include <climits>

#include "expert_internal.cuh"

using namespace moe;

namespace {

inline bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline bool format_ok(int f) { return f == MOE_SCALE_FP32 || f == MOE_SCALE_UE8M0; }
// scales: floats are 4-byte aligned, bytes need nothing
inline bool scale_aligned(const void *p, int f) { return f == MOE_SCALE_UE8M0 || aligned(p, 4); }
inline bool rows_ok(int64_t R) { return R >= 0 && R < INT_MAX; }
// sides of a weight: what the kernels' 32-bit tile numbers hold with 256 experts
inline bool sides_ok(int rows, int cols) { return rows >= 1 && cols >= 1 && rows <= (1 << 18) && cols <= (1 << 18); }
// blocks of 128 columns in all rows, and a grid of one CTA for 32 of them
inline bool blocks_ok(int64_t R, int I) { return R * (I / 128) < (int64_t(1) << 36); }

// The status of a launch; a device that cannot run these kernels is not a CUDA failure.
moe_status launched(cudaError_t e) { return e == cudaErrorNotSupported ? MOE_ERR_UNSUPPORTED : from_cuda(e); }

}  // namespace

extern "C" {

moe_status moe_quantize_weight(const void *W, int E, int rows, int cols, void *W_fp8, void *W_scale, int scale_format,
                               moe_stream_t stream)
{
    NvtxRange nvtx_range("moe_quantize_weight");
    if (E < 1 || E > 256 || rows < 1 || rows > (1 << 22) || cols < 1 || !format_ok(scale_format))
        return MOE_ERR_INVALID_ARG;
    if (!W || !W_fp8 || !W_scale) return MOE_ERR_INVALID_ARG;
    if (cols % 8 != 0) return MOE_ERR_MISALIGNED;
    if (!aligned(W, 16) || !aligned(W_fp8, 16) || !scale_aligned(W_scale, scale_format)) return MOE_ERR_MISALIGNED;
    return launched(launch_quantize_weight(W, E, rows, cols, W_fp8, W_scale, scale_format,
                                           reinterpret_cast<cudaStream_t>(stream)));
}

moe_status moe_expert_gemm(const void *X_fp8, const void *X_scale, int x_scale_format, const void *W_fp8,
                           const void *W_scale, int w_scale_format, const int32_t *expert_offsets, int64_t R, int E,
                           int rows, int cols, int transpose, void *Y, int32_t *status_word, moe_stream_t stream)
{
    NvtxRange nvtx_range("moe_expert_gemm");
    if (E < 1 || E > 256 || !rows_ok(R) || !sides_ok(rows, cols)) return MOE_ERR_INVALID_ARG;
    if ((R / 224 + 256) * ((rows > cols ? rows : cols) / 256 + 1) > INT_MAX) return MOE_ERR_INVALID_ARG;  // tiles
    if (!format_ok(x_scale_format) || !format_ok(w_scale_format)) return MOE_ERR_INVALID_ARG;
    const int red = transpose ? rows : cols, out = transpose ? cols : rows;
    if (red % 128 != 0 || out % 16 != 0) return MOE_ERR_INVALID_ARG;
    if (!expert_offsets && E != 1) return MOE_ERR_INVALID_ARG;
    if (R == 0) return MOE_OK;
    if (!X_fp8 || !X_scale || !W_fp8 || !W_scale || !Y) return MOE_ERR_INVALID_ARG;
    if (!aligned(X_fp8, 16) || !aligned(W_fp8, 16) || !aligned(Y, 16) || !scale_aligned(X_scale, x_scale_format) ||
        !scale_aligned(W_scale, w_scale_format) || !aligned(expert_offsets, 4) || !aligned(status_word, 4))
        return MOE_ERR_MISALIGNED;
    ExpertGemmArgs a{X_fp8, X_scale, W_fp8, W_scale, expert_offsets, R, E, rows, cols, transpose ? 1 : 0,
                     x_scale_format, w_scale_format, Y, status_word};
    return launched(launch_expert_gemm(a, reinterpret_cast<cudaStream_t>(stream)));
}

moe_status moe_expert_wgrad(const void *dY, const void *X_fp8, const void *X_scale, int x_scale_format,
                            const int32_t *expert_offsets, int64_t R, int E, int rows, int cols, const float *add,
                            void *dW, int dw_bf16, int32_t *status_word, moe_stream_t stream)
{
    NvtxRange nvtx_range("moe_expert_wgrad");
    if (E < 1 || E > 256 || !rows_ok(R) || !sides_ok(rows, cols) || !format_ok(x_scale_format))
        return MOE_ERR_INVALID_ARG;
    if (rows % 8 != 0 || cols % 128 != 0) return MOE_ERR_INVALID_ARG;
    if (!expert_offsets && E != 1) return MOE_ERR_INVALID_ARG;
    if (!dW || (R > 0 && (!dY || !X_fp8 || !X_scale))) return MOE_ERR_INVALID_ARG;
    if (dw_bf16 && add == dW) return MOE_ERR_INVALID_ARG;   // two formats in one buffer
    if (!aligned(dY, 16) || !aligned(X_fp8, 16) || !aligned(dW, 16) || !aligned(add, 16) ||
        !scale_aligned(X_scale, x_scale_format) || !aligned(expert_offsets, 4) || !aligned(status_word, 4))
        return MOE_ERR_MISALIGNED;
    ExpertWgradArgs a{dY, X_fp8, X_scale, expert_offsets, R, E, rows, cols, x_scale_format, dw_bf16 ? 1 : 0,
                      add, dW, status_word};
    return launched(launch_expert_wgrad(a, reinterpret_cast<cudaStream_t>(stream)));
}

moe_status moe_swiglu(const void *GU, int64_t R, int I, void *A_fp8, void *A_scale, void *GU_fp8, void *GU_scale,
                      int scale_format, moe_stream_t stream)
{
    NvtxRange nvtx_range("moe_swiglu");
    if (!rows_ok(R) || I < 1 || I > (1 << 20) || I % 128 != 0 || !blocks_ok(R, I) || !format_ok(scale_format))
        return MOE_ERR_INVALID_ARG;
    if ((GU_fp8 == nullptr) != (GU_scale == nullptr)) return MOE_ERR_INVALID_ARG;
    if (R == 0) return MOE_OK;
    if (!GU || !A_fp8 || !A_scale) return MOE_ERR_INVALID_ARG;
    if (!aligned(GU, 16) || !aligned(A_fp8, 16) || !aligned(GU_fp8, 16) || !scale_aligned(A_scale, scale_format) ||
        !scale_aligned(GU_scale, scale_format))
        return MOE_ERR_MISALIGNED;
    return launched(launch_swiglu(GU, R, I, A_fp8, A_scale, GU_fp8, GU_scale, scale_format,
                                  reinterpret_cast<cudaStream_t>(stream)));
}

moe_status moe_swiglu_backward(const void *dA, const void *GU_fp8, const void *GU_scale, int gu_scale_format, int64_t R,
                               int I, void *dGU, void *dGU_fp8, void *dGU_scale, int scale_format,
                               int32_t *status_word, moe_stream_t stream)
{
    NvtxRange nvtx_range("moe_swiglu_backward");
    if (!rows_ok(R) || I < 1 || I > (1 << 20) || I % 128 != 0 || !blocks_ok(R, I)) return MOE_ERR_INVALID_ARG;
    if (!format_ok(gu_scale_format) || !format_ok(scale_format)) return MOE_ERR_INVALID_ARG;
    if ((dGU_fp8 == nullptr) != (dGU_scale == nullptr)) return MOE_ERR_INVALID_ARG;
    if (R == 0) return MOE_OK;
    if (!dA || !GU_fp8 || !GU_scale || (!dGU && !dGU_fp8)) return MOE_ERR_INVALID_ARG;
    if (!aligned(dA, 16) || !aligned(GU_fp8, 16) || !aligned(dGU, 16) || !aligned(dGU_fp8, 16) ||
        !scale_aligned(GU_scale, gu_scale_format) || !scale_aligned(dGU_scale, scale_format) || !aligned(status_word, 4))
        return MOE_ERR_MISALIGNED;
    return launched(launch_swiglu_backward(dA, GU_fp8, GU_scale, gu_scale_format, R, I, dGU, dGU_fp8, dGU_scale,
                                           scale_format, status_word, reinterpret_cast<cudaStream_t>(stream)));
}

namespace {
bool layer_sizes_ok(int H, int I, int E, int K)
{
    return H >= 128 && H % 128 == 0 && H <= 65536 && I >= 128 && I % 128 == 0 && I <= 65536 && E >= 1 && E <= 256 &&
           K >= 1 && K <= 16 && K <= E;
}
}  // namespace

size_t moe_layer_workspace_size(int N, int H, int I, int E, int K)
{
    if (N < 1 || N > 64 || !layer_sizes_ok(H, I, E, K)) return 0;
    return layer_workspace_bytes(N, H, I, E, K);
}

moe_status moe_layer(const void *X, const void *W_gate, const float *bias, const void *W1_fp8, const void *W1_scale,
                     const void *W2_fp8, const void *W2_scale, int scale_format, const void *residual, int N, int H,
                     int I, int E, int K, int renorm, int32_t *topk_idx, float *topk_w, void *out,
                     int32_t *status_word, void *workspace, size_t workspace_bytes, moe_stream_t stream)
{
    NvtxRange nvtx_range("moe_layer");
    if (N < 0 || !layer_sizes_ok(H, I, E, K) || !format_ok(scale_format)) return MOE_ERR_INVALID_ARG;
    if (N == 0) return MOE_OK;
    if (N > 64) return MOE_ERR_UNSUPPORTED;
    if (!X || !W_gate || !W1_fp8 || !W1_scale || !W2_fp8 || !W2_scale || !topk_idx || !topk_w || !out)
        return MOE_ERR_INVALID_ARG;
    if (!aligned(X, 16) || !aligned(W_gate, 16) || !aligned(W1_fp8, 16) || !aligned(W2_fp8, 16) ||
        !aligned(residual, 16) || !aligned(out, 16) || !scale_aligned(W1_scale, scale_format) ||
        !scale_aligned(W2_scale, scale_format) || !aligned(bias, 4) || !aligned(topk_idx, 4) || !aligned(topk_w, 4) ||
        !aligned(status_word, 4))
        return MOE_ERR_MISALIGNED;
    if (!workspace || workspace_bytes < layer_workspace_bytes(N, H, I, E, K)) return MOE_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return MOE_ERR_MISALIGNED;
    LayerArgs a{X, W_gate, bias, W1_fp8, W1_scale, W2_fp8, W2_scale, residual, N, H, I, E, K, renorm ? 1 : 0,
                scale_format, topk_idx, topk_w, out, status_word, workspace};
    return launched(launch_layer(a, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
