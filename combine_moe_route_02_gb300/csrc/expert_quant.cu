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

// Eight values of a 1x128 block held by 16 lanes: their codes, and the block's scale byte.
__device__ __forceinline__ uint2 quant_block(const float (&f)[8], uint32_t &byte)
{
    float m = amax8(f);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
    byte = block_scale_byte(m);
    const float inv = scale_reciprocal(byte);
    return make_uint2(f32x4_to_e4m3x4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv),
                      f32x4_to_e4m3x4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv));
}

__device__ __forceinline__ void codes8_to_f32(const uint2 &q, float s, float (&f)[8])
{
    const uint32_t w[4] = {q.x & 0xFFFFu, q.x >> 16, q.y & 0xFFFFu, q.y >> 16};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = e4m3x2_to_f32x2(w[i]);
        f[2 * i] = v.x * s;
        f[2 * i + 1] = v.y * s;
    }
}

// ---------------------------------------------------------------------------
// Weights: one CTA per 128x128 block, the block in registers between the maximum and the codes.
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
// Gated activation.  A unit is one row's block of 128 columns of A, held by 16
// lanes of 8 columns; unit u lies in row u / nb (nb = I / 128), its columns of A
// start at 128 u, those of the gate at 128 u + row * I, of the up half I further.
// ---------------------------------------------------------------------------
constexpr int kActThreads = 256;
constexpr int kUnits = 2;   // units per half warp, all loaded before the first is used

struct Rows {
    int64_t units;
    int nb, I;
    __device__ __forceinline__ int64_t row(int64_t u) const
    {
        return units <= 0xFFFFFFFFll ? static_cast<uint32_t>(u) / static_cast<uint32_t>(nb) : u / nb;
    }
};

__global__ void __launch_bounds__(kActThreads)
    swiglu_kernel(const __nv_bfloat16 *__restrict__ GU, const Rows d, uint8_t *__restrict__ A, void *A_scale,
                  uint8_t *__restrict__ K, void *K_scale, int ue8m0)
{
    const int l = threadIdx.x & 15;
    const int64_t u0 = (static_cast<int64_t>(blockIdx.x) * (kActThreads / 16)) * kUnits + (threadIdx.x >> 4);
    uint4 g[kUnits], u[kUnits];
    int64_t row[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const int64_t unit = u0 + i * (kActThreads / 16);
        g[i] = u[i] = make_uint4(0, 0, 0, 0);
        row[i] = 0;
        if (unit < d.units) {
            row[i] = d.row(unit);
            const __nv_bfloat16 *src = GU + unit * 128 + row[i] * d.I + l * 8;
            g[i] = __ldcs(reinterpret_cast<const uint4 *>(src));
            u[i] = __ldcs(reinterpret_cast<const uint4 *>(src + d.I));
        }
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const int64_t unit = u0 + i * (kActThreads / 16);
        float fg[8], fu[8], a[8];
        bf16x8_to_f32(g[i], fg);
        bf16x8_to_f32(u[i], fu);
#pragma unroll
        for (int x = 0; x < 8; ++x) a[x] = __fdividef(fg[x], 1.f + __expf(-fg[x])) * fu[x];
        uint32_t sa, sg, su;
        const uint2 qa = quant_block(a, sa);
        uint2 qg = make_uint2(0, 0), qu = make_uint2(0, 0);
        if (K) {
            qg = quant_block(fg, sg);
            qu = quant_block(fu, su);
        }
        if (unit >= d.units) continue;
        *reinterpret_cast<uint2 *>(A + unit * 128 + l * 8) = qa;
        if (l == 0) store_scale(A_scale, ue8m0, unit, sa);
        if (K) {
            uint8_t *dst = K + unit * 128 + row[i] * d.I + l * 8;
            *reinterpret_cast<uint2 *>(dst) = qg;
            *reinterpret_cast<uint2 *>(dst + d.I) = qu;
            if (l == 0) {
                store_scale(K_scale, ue8m0, unit + row[i] * d.nb, sg);
                store_scale(K_scale, ue8m0, unit + row[i] * d.nb + d.nb, su);
            }
        }
    }
}

__global__ void __launch_bounds__(kActThreads)
    swiglu_backward_kernel(const __nv_bfloat16 *__restrict__ dA, const uint8_t *__restrict__ K, const void *K_scale,
                           int k_ue8m0, const Rows d, __nv_bfloat16 *__restrict__ dGU, uint8_t *__restrict__ Q,
                           void *Q_scale, int ue8m0, int32_t *status)
{
    const int l = threadIdx.x & 15;
    const int64_t u0 = (static_cast<int64_t>(blockIdx.x) * (kActThreads / 16)) * kUnits + (threadIdx.x >> 4);
    uint4 da[kUnits];
    uint2 g[kUnits], u[kUnits];
    uint32_t sg[kUnits], su[kUnits];
    int64_t row[kUnits];
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const int64_t unit = u0 + i * (kActThreads / 16);
        da[i] = make_uint4(0, 0, 0, 0);
        g[i] = u[i] = make_uint2(0, 0);
        sg[i] = su[i] = 127;
        row[i] = 0;
        if (unit < d.units) {
            row[i] = d.row(unit);
            const uint8_t *src = K + unit * 128 + row[i] * d.I + l * 8;
            da[i] = __ldcs(reinterpret_cast<const uint4 *>(dA + unit * 128 + l * 8));
            g[i] = __ldcs(reinterpret_cast<const uint2 *>(src));
            u[i] = __ldcs(reinterpret_cast<const uint2 *>(src + d.I));
            sg[i] = load_scale_byte(K_scale, k_ue8m0, unit + row[i] * d.nb, bad);
            su[i] = load_scale_byte(K_scale, k_ue8m0, unit + row[i] * d.nb + d.nb, bad);
        }
    }
    if (bad) report_status(status, MOE_ERR_BAD_SCALE);
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const int64_t unit = u0 + i * (kActThreads / 16);
        float fa[8], fg[8], fu[8], dg[8], du[8];
        bf16x8_to_f32(da[i], fa);
        codes8_to_f32(g[i], scale_value(sg[i]), fg);
        codes8_to_f32(u[i], scale_value(su[i]), fu);
#pragma unroll
        for (int x = 0; x < 8; ++x) {
            const float s = __fdividef(1.f, 1.f + __expf(-fg[x]));
            const float as = fa[x] * s;
            du[x] = as * fg[x];
            dg[x] = as * fu[x] * (1.f + fg[x] * (1.f - s));
        }
        uint32_t bg = 0, bu = 0;
        uint2 qg = make_uint2(0, 0), qu = make_uint2(0, 0);
        if (Q) {
            qg = quant_block(dg, bg);
            qu = quant_block(du, bu);
        }
        if (unit >= d.units) continue;
        const int64_t at = unit * 128 + row[i] * d.I + l * 8;
        if (dGU) {
            *reinterpret_cast<uint4 *>(dGU + at) = f32_to_bf16x8(dg);
            *reinterpret_cast<uint4 *>(dGU + at + d.I) = f32_to_bf16x8(du);
        }
        if (Q) {
            *reinterpret_cast<uint2 *>(Q + at) = qg;
            *reinterpret_cast<uint2 *>(Q + at + d.I) = qu;
            if (l == 0) {
                store_scale(Q_scale, ue8m0, unit + row[i] * d.nb, bg);
                store_scale(Q_scale, ue8m0, unit + row[i] * d.nb + d.nb, bu);
            }
        }
    }
}

Rows make_rows(int64_t R, int I) { return Rows{R * (I / 128), I / 128, I}; }

unsigned act_grid(const Rows &d)
{
    const int64_t per = static_cast<int64_t>(kActThreads / 16) * kUnits;
    return static_cast<unsigned>((d.units + per - 1) / per);
}

}  // namespace

cudaError_t launch_quantize_weight(const void *W, int E, int rows, int cols, void *q, void *scale, int ue8m0,
                                   cudaStream_t stream)
{
    const dim3 grid((cols + 127) / 128, (rows + 127) / 128, E);
    quantize_weight_kernel<<<grid, kQwThreads, 0, stream>>>(static_cast<const uint4 *>(W), rows, cols,
                                                            static_cast<uint8_t *>(q), scale, ue8m0);
    return cudaGetLastError();
}

cudaError_t launch_swiglu(const void *GU, int64_t R, int I, void *A_fp8, void *A_scale, void *GU_fp8, void *GU_scale,
                          int ue8m0, cudaStream_t stream)
{
    const Rows d = make_rows(R, I);
    swiglu_kernel<<<act_grid(d), kActThreads, 0, stream>>>(static_cast<const __nv_bfloat16 *>(GU), d,
                                                           static_cast<uint8_t *>(A_fp8), A_scale,
                                                           static_cast<uint8_t *>(GU_fp8), GU_scale, ue8m0);
    return cudaGetLastError();
}

cudaError_t launch_swiglu_backward(const void *dA, const void *GU_fp8, const void *GU_scale, int gu_ue8m0, int64_t R,
                                   int I, void *dGU, void *dGU_fp8, void *dGU_scale, int ue8m0, int32_t *status,
                                   cudaStream_t stream)
{
    const Rows d = make_rows(R, I);
    swiglu_backward_kernel<<<act_grid(d), kActThreads, 0, stream>>>(
        static_cast<const __nv_bfloat16 *>(dA), static_cast<const uint8_t *>(GU_fp8), GU_scale, gu_ue8m0, d,
        static_cast<__nv_bfloat16 *>(dGU), static_cast<uint8_t *>(dGU_fp8), dGU_scale, ue8m0, status);
    return cudaGetLastError();
}

}  // namespace moe
