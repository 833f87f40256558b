// norm_api.cu -- the C ABI of the norms around the experts: argument checks on the host (before any CUDA call), then
// the launches.
#include "expert_internal.cuh"

using namespace moe;

namespace {

inline bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline bool sizes_ok(int64_t N, int H) { return N >= 0 && N < (int64_t(1) << 31) && H >= 8 && H <= 16384 && H % 8 == 0; }
inline bool type_ok(int t) { return t == MOE_GRAD_FP32 || t == MOE_GRAD_BF16; }

// The status of a launch; a device that cannot run these kernels is not a CUDA failure.
moe_status launched(cudaError_t e) { return e == cudaErrorNotSupported ? MOE_ERR_UNSUPPORTED : from_cuda(e); }

}  // namespace

extern "C" {

moe_status moe_rms_norm(const void *X, const void *residual, const void *weight, int weight_type, float eps, int64_t N,
                        int H, void *S, void *Y, void *Y_fp8, void *Y_scale, int scale_format, float *rstd,
                        moe_stream_t stream)
{
    NvtxRange nvtx_range("moe_rms_norm");
    if (!sizes_ok(N, H) || !type_ok(weight_type) || !(eps > 0.f && eps <= 1.f)) return MOE_ERR_INVALID_ARG;
    if (scale_format != MOE_SCALE_FP32 && scale_format != MOE_SCALE_UE8M0) return MOE_ERR_INVALID_ARG;
    if ((Y_fp8 == nullptr) != (Y_scale == nullptr) || (Y_fp8 && H % 128 != 0)) return MOE_ERR_INVALID_ARG;
    if ((residual == nullptr) != (S == nullptr) && N > 0) return MOE_ERR_INVALID_ARG;
    if (N == 0) return MOE_OK;
    if (!X || !weight || (!Y && !Y_fp8)) return MOE_ERR_INVALID_ARG;
    if (S && S == Y) return MOE_ERR_INVALID_ARG;       // (both may be X, but not at once)
    if (!aligned(X, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(S, 16) || !aligned(Y, 16) ||
        !aligned(Y_fp8, 16) || !aligned(rstd, 4) || (scale_format == MOE_SCALE_FP32 && !aligned(Y_scale, 4)))
        return MOE_ERR_MISALIGNED;
    RmsNormArgs a{X, residual, weight, N, H, weight_type == MOE_GRAD_BF16, scale_format, eps, S, Y, Y_fp8, Y_scale, rstd};
    return launched(launch_rms_norm(a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t moe_rms_norm_backward_workspace_size(int64_t N, int H)
{
    return sizes_ok(N, H) ? static_cast<size_t>(rms_norm_table_rows(N, H)) * H * sizeof(float) : 0;
}

moe_status moe_rms_norm_backward(const void *dY, const void *S, const void *weight, int weight_type, const float *rstd,
                                 const void *dS, const float *add, int64_t N, int H, void *dX, float *dweight,
                                 int32_t *status_word, void *workspace, size_t workspace_bytes, moe_stream_t stream)
{
    NvtxRange nvtx_range("moe_rms_norm_backward");
    if (!sizes_ok(N, H) || !type_ok(weight_type)) return MOE_ERR_INVALID_ARG;
    if (!dweight || (N > 0 && (!dY || !S || !weight || !rstd || !dX))) return MOE_ERR_INVALID_ARG;
    if (!aligned(dY, 16) || !aligned(S, 16) || !aligned(weight, 16) || !aligned(dS, 16) || !aligned(dX, 16) ||
        !aligned(rstd, 4) || !aligned(add, 4) || !aligned(dweight, 4) || !aligned(status_word, 4))
        return MOE_ERR_MISALIGNED;
    if (N > 0 && (!workspace || workspace_bytes < moe_rms_norm_backward_workspace_size(N, H))) return MOE_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return MOE_ERR_MISALIGNED;
    RmsNormBackwardArgs a{dY, S, dS, weight, rstd, add, N, H, weight_type == MOE_GRAD_BF16, dX, dweight, workspace, status_word};
    return launched(launch_rms_norm_backward(a, reinterpret_cast<cudaStream_t>(stream)));
}

namespace {
// every tensor of the list, and what they are together
moe_status check_list(const void *const *grads, void *const *out, const int64_t *sizes, const int *types, int n)
{
    if (n < 0 || (n > 0 && (!grads || !sizes || !types))) return MOE_ERR_INVALID_ARG;
    int64_t bytes = 0;
    for (int i = 0; i < n; ++i) {
        if (!type_ok(types[i]) || sizes[i] < 0 || sizes[i] > (int64_t(1) << 42)) return MOE_ERR_INVALID_ARG;
        bytes += sizes[i] * 4;
        if (bytes > int64_t(1) << 44 || (sizes[i] > 0 && (!grads[i] || (out && !out[i])))) return MOE_ERR_INVALID_ARG;
    }
    for (int i = 0; i < n; ++i) {
        if (sizes[i] == 0) continue;
        const uintptr_t by = types[i] == MOE_GRAD_BF16 ? 2 : 4;
        if (!aligned(grads[i], by) || (out && !aligned(out[i], by))) return MOE_ERR_MISALIGNED;
    }
    return MOE_OK;
}

moe_status grad_norm(const GradArgs &a, size_t workspace_bytes, moe_stream_t stream)
{
    const moe_status s = check_list(a.grads, a.out, a.sizes, a.types, a.n);
    if (s != MOE_OK) return s;
    if (!a.norm) return MOE_ERR_INVALID_ARG;
    if (!aligned(a.norm, 4)) return MOE_ERR_MISALIGNED;
    if (!a.workspace || workspace_bytes < grad_norm_workspace_bytes(a.n)) return MOE_ERR_WORKSPACE;
    if (!aligned(a.workspace, 16)) return MOE_ERR_MISALIGNED;
    return launched(launch_grad_norm(a, reinterpret_cast<cudaStream_t>(stream)));
}
}  // namespace

size_t moe_grad_norm_workspace_size(int n) { return n < 0 ? 0 : grad_norm_workspace_bytes(n); }

moe_status moe_grad_norm(const void *const *grads, const int64_t *sizes, const int *types, int n, float *norm,
                         void *workspace, size_t workspace_bytes, moe_stream_t stream)
{
    NvtxRange nvtx_range("moe_grad_norm");
    return grad_norm(GradArgs{grads, nullptr, sizes, types, n, 0, 0.0, norm, workspace}, workspace_bytes, stream);
}

moe_status moe_clip_grad_norm(const void *const *grads, void *const *out, const int64_t *sizes, const int *types, int n,
                              double max_norm, float *norm, void *workspace, size_t workspace_bytes, moe_stream_t stream)
{
    NvtxRange nvtx_range("moe_clip_grad_norm");
    if (!(max_norm >= 0)) return MOE_ERR_INVALID_ARG;
    return grad_norm(GradArgs{grads, out, sizes, types, n, 1, max_norm, norm, workspace}, workspace_bytes, stream);
}

}  // extern "C"
