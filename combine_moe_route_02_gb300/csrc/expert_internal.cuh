// expert_internal.cuh -- what the kernels behind the dispatch (expert products,
// gated activation, few-token layer) share: power-of-two block scales, the E4M3
// quantiser, the walk over ragged groups of rows, and their launchers.
#pragma once

#include "moe_internal.cuh"

namespace moe {

// ---------------------------------------------------------------------------
// Power-of-two scales.  A scale travels as its UE8M0 byte b (s = 2^(b - 127)),
// whichever of the two formats it is stored in.
// ---------------------------------------------------------------------------
constexpr uint32_t kRcp448F32Bits = 0x3B124925u;  // fl32(1/448)

// The byte of the block scale of a 128-block with this largest magnitude:
// t = fl32(max(amax, 1e-4) * fl32(1/448)), rounded up to a power of two.
__device__ __forceinline__ uint32_t block_scale_byte(float amax)
{
    const float t = __fmul_rn(fmaxf(amax, 1e-4f), __uint_as_float(kRcp448F32Bits));
    uint16_t e;
    asm("cvt.rp.satfinite.ue8m0x2.f32 %0, %1, %2;" : "=h"(e) : "f"(0.0f), "f"(t));
    return e & 0xFFu;
}

// 2^(127 - b): the exact reciprocal of the scale with byte b in 1..253.
__device__ __forceinline__ float scale_reciprocal(uint32_t b) { return __uint_as_float((254u - b) << 23); }
__device__ __forceinline__ float scale_value(uint32_t b)
{
    // byte 0 is 2^-127, a subnormal; byte 255 a NaN
    return __uint_as_float(b == 0 ? 0x00400000u : b == 255 ? 0x7FFFFFFFu : b << 23);
}

// Four fp32 values to four E4M3 codes (round to nearest even, saturating), the first in the low byte.
__device__ __forceinline__ uint32_t f32x4_to_e4m3x4(float a, float b, float c, float d)
{
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

// Two E4M3 codes (low 16 bits of `q`) to fp32, exactly.
__device__ __forceinline__ float2 e4m3x2_to_f32x2(uint32_t q)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(q)));
    float2 f;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(f.x), "=f"(f.y)
        : "r"(h));
    return f;
}

// Scale `at` of an array in either format, as stored; and its byte.  `bad` is raised where a float is
// not a positive normal power of two.
__device__ __forceinline__ uint32_t load_scale_bits(const void *p, int ue8m0, int64_t at)
{
    return ue8m0 ? __ldg(static_cast<const uint8_t *>(p) + at) : __ldg(static_cast<const uint32_t *>(p) + at);
}
__device__ __forceinline__ uint32_t scale_bits_byte(uint32_t w, int ue8m0, bool &bad)
{
    if (ue8m0) return w;
    bad |= (w & 0x807FFFFFu) != 0 || w - 1u >= 0x7F7FFFFFu;   // (not 0, below infinity)
    return (w >> 23) & 0xFFu;
}
__device__ __forceinline__ uint32_t load_scale_byte(const void *p, int ue8m0, int64_t at, bool &bad)
{
    return scale_bits_byte(load_scale_bits(p, ue8m0, at), ue8m0, bad);
}

__device__ __forceinline__ void store_scale(void *p, int ue8m0, int64_t at, uint32_t byte)
{
    if (ue8m0)
        static_cast<uint8_t *>(p)[at] = static_cast<uint8_t>(byte);
    else
        static_cast<float *>(p)[at] = __uint_as_float(byte << 23);
}

// ---------------------------------------------------------------------------
// CTA pairs (clusters of two): TMEM and MMAs of cta_group::2, arrivals on the
// leader's barriers
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Arrive on the barrier at this shared-memory offset in CTA `rank` of the cluster.  For what the pair's
// tensor cores read from their own CTA's memory, or have read from TMEM, and is already ordered before the
// async proxy: with .release.cluster an arrival took ~1100 cycles, this one ~100.
__device__ __forceinline__ void mbar_arrive_at(uint64_t *bar, uint32_t rank)
{
    asm volatile(
        "{\n\t.reg .b32 a;\n\t"
        "mapa.shared::cluster.u32 a, %0, %1;\n\t"
        "mbarrier.arrive.shared::cluster.b64 _, [a];\n\t}" ::"r"(smem_u32(bar)),
        "r"(rank)
        : "memory");
}

// A warp's waits, all lanes together: the warp's control flow stays uniform, which keeps the operands
// of the TMA and tcgen05 instructions that follow in uniform registers (a single-lane branch around
// the expert products' loops cost 70 cycles for each MMA issued).  The polling loop is out of line.
static __device__ __noinline__ bool warp_wait_slow(uint64_t *bar, uint32_t parity, volatile int *abort)
{
    return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, abort));
}
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort)
{
    if (__all_sync(0xffffffffu, mbar_try_wait(smem_u32(bar), parity))) return true;
    return warp_wait_slow(bar, parity, abort);
}
// TMA load of a box with the default cache policy.
__device__ __forceinline__ void tma_load_3d_plain(void *smem_dst, const CUtensorMap *map, uint64_t *bar, int32_t c0, int32_t c1,
                                                  int32_t c2)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            smem_u32(smem_dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
        : "memory");
}

// TMA store of a box (what lies outside the tensor is left out), in this thread's bulk async-group.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap *map, const void *smem_src, int32_t c0, int32_t c1, int32_t c2)
{
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(smem_src))
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

// Until all but the last N of this thread's bulk stores have read their shared memory / all are complete.
template <int N>
__device__ __forceinline__ void bulk_wait_read()
{
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
template <int N>
__device__ __forceinline__ void bulk_wait()
{
    asm volatile("cp.async.bulk.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void fence_proxy_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r != 0;
}

__device__ __forceinline__ void tmem_alloc_pair(uint32_t *dst, uint32_t ncols)
{
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols)
{
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

// 32 lanes x 8 consecutive 32-bit columns to TMEM: thread t of the warp gives lane (base lane + t).
__device__ __forceinline__ void tmem_st_32x32b_x8(uint32_t taddr, const float (&v)[8])
{
    uint32_t r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = __float_as_uint(v[i]);
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Arrive, in both CTAs, on the barrier at this offset once the pair's tcgen05 operations issued so far are done.
__device__ __forceinline__ void tc_commit_pair(uint64_t *bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}

// ---------------------------------------------------------------------------
// Launchers (validated arguments, the launch's cudaError_t)
// ---------------------------------------------------------------------------
// The current device, if it is one that these kernels are for; cudaErrorNotSupported otherwise.
inline cudaError_t expert_device(int *dev)
{
    const cudaError_t err = cudaGetDevice(dev);
    if (err != cudaSuccess) return err;
    return device_cc_major(*dev) == 10 ? cudaSuccess : cudaErrorNotSupported;
}

struct ExpertGemmArgs {
    const void *X, *X_scale;
    const void *W, *W_scale;
    const int32_t *offsets;  // [E + 1], or nullptr: one group of all R rows
    int64_t R;
    int E, rows, cols, transpose, x_ue8m0, w_ue8m0;
    void *Y;
    int32_t *status;
};
cudaError_t launch_expert_gemm(const ExpertGemmArgs &a, cudaStream_t stream);

struct ExpertWgradArgs {
    const void *dY;
    const void *X, *X_scale;
    const int32_t *offsets;
    int64_t R;
    int E, rows, cols, x_ue8m0, bf16_out;
    const float *add;
    void *dW;
    int32_t *status;
};
cudaError_t launch_expert_wgrad(const ExpertWgradArgs &a, cudaStream_t stream);

cudaError_t launch_quantize_weight(const void *W, int E, int rows, int cols, void *q, void *scale, int ue8m0,
                                   cudaStream_t stream);
cudaError_t launch_swiglu(const void *GU, int64_t R, int I, void *A_fp8, void *A_scale, void *GU_fp8, void *GU_scale,
                          int ue8m0, cudaStream_t stream);
cudaError_t launch_swiglu_backward(const void *dA, const void *GU_fp8, const void *GU_scale, int gu_ue8m0, int64_t R,
                                   int I, void *dGU, void *dGU_fp8, void *dGU_scale, int ue8m0, int32_t *status,
                                   cudaStream_t stream);

struct LayerArgs {
    const void *X, *W_gate;
    const float *bias;
    const void *W1, *W1_scale, *W2, *W2_scale;
    const void *residual;
    int N, H, I, E, K, renorm, ue8m0;
    int32_t *topk_idx;
    float *topk_w;
    void *out;
    int32_t *status;
    void *workspace;
};
size_t layer_workspace_bytes(int N, int H, int I, int E, int K);
cudaError_t launch_layer(const LayerArgs &a, cudaStream_t stream);

// A tiled tensor map, 128-byte swizzle unless told otherwise; false if the driver refuses it.
bool encode_map(CUtensorMap *map, CUtensorMapDataType type, int elem_bytes, const void *base, int rank,
                const uint64_t *dims, const uint32_t *box, CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B);

}  // namespace moe
