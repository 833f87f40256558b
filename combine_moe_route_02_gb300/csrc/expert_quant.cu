// expert_quant.cu -- the memory-bound steps around the expert products: E4M3
// weights with 128x128 scales, and the gated activation between the two products
// with its gradient, reading and writing E4M3 rows with 1x128 scales.
#include "expert_internal.cuh"

namespace moe {
namespace {

constexpr uint32_t kFull = 0xffffffffu;

__device__ __forceinline__ void bf16x8_to_f32(const uint4 &x, float (&f)[8])
{
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint4 f32_to_bf16x8(const float (&f)[8])
{
    uint4 v;
    __nv_bfloat162 *h = reinterpret_cast<__nv_bfloat162 *>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    return v;
}

__device__ __forceinline__ float amax8(const float (&f)[8])
{
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(f[i]));
    return m;
}

// 16 values of a 1x128 block held by 8 lanes: their codes, and the block's scale byte.
__device__ __forceinline__ uint4 quant_block(const float (&f)[16], uint32_t &byte)
{
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(f[i]));
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
    byte = block_scale_byte(m);
    const float inv = scale_reciprocal(byte);
    uint32_t q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        q[i] = f32x4_to_e4m3x4(f[4 * i] * inv, f[4 * i + 1] * inv, f[4 * i + 2] * inv, f[4 * i + 3] * inv);
    return make_uint4(q[0], q[1], q[2], q[3]);
}

__device__ __forceinline__ void codes_to_f32(const uint4 &q, float s, float (&f)[16])
{
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 lo = e4m3x2_to_f32x2(w[i] & 0xFFFFu), hi = e4m3x2_to_f32x2(w[i] >> 16);
        f[4 * i] = lo.x * s;
        f[4 * i + 1] = lo.y * s;
        f[4 * i + 2] = hi.x * s;
        f[4 * i + 3] = hi.y * s;
    }
}

__device__ __forceinline__ void bf16x16_to_f32(const uint4 &a, const uint4 &b, float (&f)[16])
{
    bf16x8_to_f32(a, *reinterpret_cast<float (*)[8]>(&f[0]));
    bf16x8_to_f32(b, *reinterpret_cast<float (*)[8]>(&f[8]));
}

// ---------------------------------------------------------------------------
// Weights: one CTA per 128x128 block, the block in registers between the maximum and the codes.  One read and
// one write, HBM-bound: 64 x 2048 x 2048 in 124 us, 6.5 TB/s.
// ---------------------------------------------------------------------------
constexpr int kQwThreads = 256;

__global__ void __launch_bounds__(kQwThreads)
    quantize_weight_kernel(const uint4 *__restrict__ W, int rows, int cols, uint8_t *__restrict__ q, void *scale, int ue8m0)
{
    __shared__ float part[kQwThreads / 32];
    const int r0 = blockIdx.y * 128, c0 = blockIdx.x * 128;
    const int chunk = threadIdx.x & 15, row = threadIdx.x >> 4;
    const int64_t base = static_cast<int64_t>(blockIdx.z) * rows;
    const bool col_ok = c0 + chunk * 8 < cols;
    uint4 x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = r0 + row + 16 * i;
        x[i] = make_uint4(0, 0, 0, 0);
        if (r < rows && col_ok) x[i] = __ldcs(W + ((base + r) * cols + c0) / 8 + chunk);
    }
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float f[8];
        bf16x8_to_f32(x[i], f);
        m = fmaxf(m, amax8(f));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kQwThreads / 32; ++i) m = fmaxf(m, part[i]);
    const uint32_t byte = block_scale_byte(m);
    const float inv = scale_reciprocal(byte);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = r0 + row + 16 * i;
        if (r >= rows || !col_ok) continue;
        float f[8];
        bf16x8_to_f32(x[i], f);
        *reinterpret_cast<uint2 *>(q + (base + r) * cols + c0 + chunk * 8) =
            make_uint2(f32x4_to_e4m3x4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv),
                       f32x4_to_e4m3x4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv));
    }
    if (threadIdx.x == 0)
        store_scale(scale, ue8m0, (static_cast<int64_t>(blockIdx.z) * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x, byte);
}

// ---------------------------------------------------------------------------
// Gated activation.  A unit is one row's block of 128 columns of A, held by 8 lanes
// of 16 columns; unit u lies in row u / nb (nb = I / 128), its columns of A start at
// 128 u, those of the gate at 128 u + row * I, of the up half I further.  The bound is
// the memory's, but not by much (60% of the issue slots): a lane of 16 columns instead
// of 8 halves the share of the scales and shuffles.  131072 x 1024 with the checkpoint:
// 147 us, 6.4 TB/s (184 us with 8); the gradient of 32761 x 1024: 55 us, 6.2 TB/s.
// ---------------------------------------------------------------------------
constexpr int kActThreads = 256;
constexpr int kLanes = 8;

struct Rows {
    int64_t units;
    int nb, I;
    __device__ __forceinline__ int64_t row(int64_t u) const
    {
        return units <= 0xFFFFFFFFll ? static_cast<uint32_t>(u) / static_cast<uint32_t>(nb) : u / nb;
    }
};

template <bool kKeep>
__global__ void __launch_bounds__(kActThreads)
    swiglu_kernel(const __nv_bfloat16 *__restrict__ GU, const Rows d, uint8_t *__restrict__ A, void *A_scale,
                  uint8_t *__restrict__ K, void *K_scale, int ue8m0)
{
    const int l = threadIdx.x & (kLanes - 1);
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * (kActThreads / kLanes) + threadIdx.x / kLanes;
    const bool there = unit < d.units;
    const int64_t u = there ? unit : d.units - 1, row = d.row(u);
    const uint4 *src = reinterpret_cast<const uint4 *>(GU + u * 128 + row * d.I + l * 16);
    const uint4 g0 = __ldcs(src), g1 = __ldcs(src + 1), u0 = __ldcs(src + d.I / 8), u1 = __ldcs(src + d.I / 8 + 1);
    float fg[16], fu[16], a[16];
    bf16x16_to_f32(g0, g1, fg);
    bf16x16_to_f32(u0, u1, fu);
#pragma unroll
    for (int x = 0; x < 16; ++x) a[x] = fg[x] * sigmoid(fg[x]) * fu[x];
    uint32_t sa, sg, su;
    const uint4 qa = quant_block(a, sa);
    uint4 qg, qu;
    if (kKeep) {
        qg = quant_block(fg, sg);
        qu = quant_block(fu, su);
    }
    if (!there) return;
    *reinterpret_cast<uint4 *>(A + u * 128 + l * 16) = qa;
    if (l == 0) store_scale(A_scale, ue8m0, u, sa);
    if (kKeep) {
        uint8_t *dst = K + u * 128 + row * d.I + l * 16;
        *reinterpret_cast<uint4 *>(dst) = qg;
        *reinterpret_cast<uint4 *>(dst + d.I) = qu;
        if (l == 0) {
            store_scale(K_scale, ue8m0, u + row * d.nb, sg);
            store_scale(K_scale, ue8m0, u + row * d.nb + d.nb, su);
        }
    }
}

__global__ void __launch_bounds__(kActThreads)
    swiglu_backward_kernel(const __nv_bfloat16 *__restrict__ dA, const uint8_t *__restrict__ K, const void *K_scale,
                           int k_ue8m0, const Rows d, __nv_bfloat16 *__restrict__ dGU, uint8_t *__restrict__ Q,
                           void *Q_scale, int ue8m0, int32_t *status)
{
    const int l = threadIdx.x & (kLanes - 1);
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * (kActThreads / kLanes) + threadIdx.x / kLanes;
    const bool there = unit < d.units;
    const int64_t u = there ? unit : d.units - 1, row = d.row(u), at = u * 128 + row * d.I + l * 16;
    const uint4 *da = reinterpret_cast<const uint4 *>(dA + u * 128 + l * 16);
    const uint4 a0 = __ldcs(da), a1 = __ldcs(da + 1);
    const uint4 qg = __ldcs(reinterpret_cast<const uint4 *>(K + at));
    const uint4 qu = __ldcs(reinterpret_cast<const uint4 *>(K + at + d.I));
    bool bad = false;
    const uint32_t sg = load_scale_byte(K_scale, k_ue8m0, u + row * d.nb, bad);
    const uint32_t su = load_scale_byte(K_scale, k_ue8m0, u + row * d.nb + d.nb, bad);
    if (bad) report_status(status, MOE_ERR_BAD_SCALE);
    float fa[16], dg[16], du[16];
    bf16x16_to_f32(a0, a1, fa);
    codes_to_f32(qg, scale_value(sg), dg);
    codes_to_f32(qu, scale_value(su), du);
#pragma unroll
    for (int x = 0; x < 16; ++x) {
        const float g = dg[x], up = du[x], s = sigmoid(g), as = fa[x] * s;
        du[x] = as * g;
        dg[x] = as * up * (1.f + g * (1.f - s));
    }
    if (dGU && there) {
        uint4 *dst = reinterpret_cast<uint4 *>(dGU + at);
        dst[0] = f32_to_bf16x8(*reinterpret_cast<float (*)[8]>(&dg[0]));
        dst[1] = f32_to_bf16x8(*reinterpret_cast<float (*)[8]>(&dg[8]));
        dst += d.I / 8;
        dst[0] = f32_to_bf16x8(*reinterpret_cast<float (*)[8]>(&du[0]));
        dst[1] = f32_to_bf16x8(*reinterpret_cast<float (*)[8]>(&du[8]));
    }
    if (Q) {
        uint32_t bg, bu;
        const uint4 cg = quant_block(dg, bg), cu = quant_block(du, bu);
        if (there) {
            *reinterpret_cast<uint4 *>(Q + at) = cg;
            *reinterpret_cast<uint4 *>(Q + at + d.I) = cu;
            if (l == 0) {
                store_scale(Q_scale, ue8m0, u + row * d.nb, bg);
                store_scale(Q_scale, ue8m0, u + row * d.nb + d.nb, bu);
            }
        }
    }
}

Rows make_rows(int64_t R, int I) { return Rows{R * (I / 128), I / 128, I}; }

unsigned act_grid(const Rows &d)
{
    const int64_t per = kActThreads / kLanes;
    return static_cast<unsigned>((d.units + per - 1) / per);
}

}  // namespace

cudaError_t launch_quantize_weight(const void *W, int E, int rows, int cols, void *q, void *scale, int ue8m0,
                                   cudaStream_t stream)
{
    int dev = 0;
    const cudaError_t err = expert_device(&dev);
    if (err != cudaSuccess) return err;
    const dim3 grid((cols - 1) / 128 + 1, (rows - 1) / 128 + 1, E);   // (cols may be within 127 of 2^31)
    quantize_weight_kernel<<<grid, kQwThreads, 0, stream>>>(static_cast<const uint4 *>(W), rows, cols,
                                                            static_cast<uint8_t *>(q), scale, ue8m0);
    return cudaGetLastError();
}

cudaError_t launch_swiglu(const void *GU, int64_t R, int I, void *A_fp8, void *A_scale, void *GU_fp8, void *GU_scale,
                          int ue8m0, cudaStream_t stream)
{
    int dev = 0;
    const cudaError_t err = expert_device(&dev);
    if (err != cudaSuccess) return err;
    const Rows d = make_rows(R, I);
    const auto kernel = GU_fp8 ? swiglu_kernel<true> : swiglu_kernel<false>;
    kernel<<<act_grid(d), kActThreads, 0, stream>>>(static_cast<const __nv_bfloat16 *>(GU), d, static_cast<uint8_t *>(A_fp8),
                                                    A_scale, static_cast<uint8_t *>(GU_fp8), GU_scale, ue8m0);
    return cudaGetLastError();
}

cudaError_t launch_swiglu_backward(const void *dA, const void *GU_fp8, const void *GU_scale, int gu_ue8m0, int64_t R,
                                   int I, void *dGU, void *dGU_fp8, void *dGU_scale, int ue8m0, int32_t *status,
                                   cudaStream_t stream)
{
    int dev = 0;
    const cudaError_t err = expert_device(&dev);
    if (err != cudaSuccess) return err;
    const Rows d = make_rows(R, I);
    swiglu_backward_kernel<<<act_grid(d), kActThreads, 0, stream>>>(
        static_cast<const __nv_bfloat16 *>(dA), static_cast<const uint8_t *>(GU_fp8), GU_scale, gu_ue8m0, d,
        static_cast<__nv_bfloat16 *>(dGU), static_cast<uint8_t *>(dGU_fp8), dGU_scale, ue8m0, status);
    return cudaGetLastError();
}

}  // namespace moe
