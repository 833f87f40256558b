// expert_wgrad.cu -- weight gradients of the expert products, from the E4M3
// checkpoint of the rows that went into them.
//
//   dW[e, n, k] = add[e, n, k] + sum_{r in group e} dY[r, n] * x[r, k] sx[r, k/128]
//
// The reduction runs over rows, so the rows' scales cannot leave the sum; but a
// scale is a power of two, so x * sx is a bf16 number exactly, and the product is a
// bf16 one with fp32 accumulation.  The E4M3 rows are read as they are (half the
// bytes of bf16) and become bf16 on their way through shared memory.
//
// Both operands have the reduction on their slow axis (MN-major).  Persistent
// CTAs; a tile is 128 weight rows x 256 weight columns of one expert, a ring
// stage 64 rows of the group.  Warp roles:
//   warp 0       TMA producer (dY 64 x 128 bf16, x 64 x 256 E4M3)
//   warp 1       MMA issuer (one thread)
//   warp 3       allocates TMEM
//   warps 4..7   epilogue
//   warps 8..15  converters E4M3 -> bf16; in a group's last stage they also clear
//                the rows behind its end (the next group's, or none)
#include "expert_internal.cuh"

namespace moe {
namespace {

constexpr int kTileM = 128, kTileN = 256, kRows = 64, kStages = 3;
constexpr int kABytes = kRows * kTileM * 2;       // two boxes of 64 columns
constexpr int kRawBytes = kRows * kTileN;         // two boxes of 128 columns
constexpr int kBBytes = kRows * kTileN * 2;       // four boxes of 64 columns
constexpr int kBox = kRows * 128;                 // bytes of a box
constexpr int kStageBytes = kABytes + kRawBytes + kBBytes;
constexpr int kEpiBytes = 4 * 32 * 128;
constexpr int kThreads = 512;
constexpr int kConvWarps = 8;
constexpr uint32_t kTmemCols = 512;
constexpr int kMaxE = 256;

struct Tail {
    uint64_t full[kStages], conv[kStages], empty[kStages];
    uint64_t acc_full[2], acc_empty[2], drain;
    uint32_t tmem_base;
    int abort, bad_index, bad_scale;
    int begin[kMaxE], count[kMaxE];
};
constexpr size_t kSmemBytes = 1024 + kStages * kStageBytes + kEpiBytes + sizeof(Tail);
static_assert(kSmemBytes <= 227 * 1024, "shared memory");

struct Params {
    const void *X_scale;
    const int32_t *offsets;
    const float *add;
    void *dW;
    int64_t R;
    int E, rows, cols, x_ue8m0, bf16_out;
    int m_tiles, n_tiles;
    int32_t *status;
};

// Two bf16 products per call; exact here (the factors are powers of two).
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Four E4M3 codes -> four bf16, times f (and f2 where it is not 1).  A code's bits
// s eeee mmm, moved to s 0000 eeee mmm 0000, are the bf16 number code * 2^-120
// (its subnormals included), so that 2^120 goes into f.
__device__ __forceinline__ uint2 codes_to_bf16(uint32_t w, uint32_t f)
{
    uint32_t lo, hi;   // each code in the low byte of a half, its sign spread over the high byte
    asm("prmt.b32 %0, %1, 0, 0x9180;" : "=r"(lo) : "r"(w));
    asm("prmt.b32 %0, %1, 0, 0xB3A2;" : "=r"(hi) : "r"(w));
    return make_uint2(mul_bf16x2((lo << 4) & 0x87F087F0u, f), mul_bf16x2((hi << 4) & 0x87F087F0u, f));
}

// Whether one of four codes is a NaN (s 1111 111).
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }

__device__ __forceinline__ uint32_t set_nan(uint32_t v, uint32_t w, int i)
{
    if (((w >> (8 * i)) & 0x7F) == 0x7F) v = (v & 0xFFFF0000u) | 0x7FFFu;
    if (((w >> (8 * i + 8)) & 0x7F) == 0x7F) v = (v & 0x0000FFFFu) | 0x7FFF0000u;
    return v;
}

__global__ void __launch_bounds__(kThreads, 1)
    expert_wgrad_kernel(const __grid_constant__ CUtensorMap tmY, const __grid_constant__ CUtensorMap tmX, const Params p)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *epi = ring + kStages * kStageBytes;
    Tail &tail = *reinterpret_cast<Tail *>(epi + kEpiBytes);
    volatile int *abort_flag = &tail.abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&tail.full[s], 1);
            mbar_init(&tail.conv[s], kConvWarps);
            mbar_init(&tail.empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tail.acc_full[b], 1);
            mbar_init(&tail.acc_empty[b], 4);
        }
        mbar_init(&tail.drain, 1);
        tail.abort = tail.bad_index = tail.bad_scale = 0;
        fence_mbarrier_init();
        tma_prefetch_desc(&tmY);
        tma_prefetch_desc(&tmX);
    }
    if (warp == 3) {
        tmem_alloc(&tail.tmem_base, kTmemCols);
        tmem_relinquish();
    }
    __syncthreads();
    if (static_cast<int>(threadIdx.x) < p.E) {
        const int e = threadIdx.x;
        int64_t a = p.offsets ? p.offsets[e] : 0, b = p.offsets ? p.offsets[e + 1] : p.R;
        if (a < 0 || b < a || b > p.R) {
            tail.bad_index = 1;
            a = b = 0;
        }
        tail.begin[e] = static_cast<int>(a);
        tail.count[e] = static_cast<int>(b - a);
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = tail.tmem_base;
    const int per = p.m_tiles * p.n_tiles;
    const int tiles = p.E * per;

    if (warp == 0) {
        if (lane == 0) {
            const uint64_t keep = l2_policy_evict_normal();
            uint32_t s = 0, ph = 0, issued = 0;
            for (int tile = blockIdx.x; tile < tiles && !*abort_flag; tile += gridDim.x) {
                const int e = tile / per, i = tile - e * per, m0 = (i / p.n_tiles) * kTileM, n0 = (i % p.n_tiles) * kTileN;
                const int count = tail.count[e], begin = tail.begin[e];
                const int boxes = p.cols - n0 > 128 ? 2 : 1;
                for (int r = 0; r < count; r += kRows) {
                    if (!mbar_wait_bounded(&tail.empty[s], ph ^ 1u, abort_flag)) break;
                    uint8_t *a = ring + s * kStageBytes, *raw = a + kABytes;
                    mbar_arrive_expect_tx(&tail.full[s], kABytes + boxes * kBox);
                    tma_load_2d(a, &tmY, &tail.full[s], m0, begin + r, keep);
                    tma_load_2d(a + kBox, &tmY, &tail.full[s], m0 + 64, begin + r, keep);
                    tma_load_2d(raw, &tmX, &tail.full[s], n0, begin + r, keep);
                    if (boxes > 1) tma_load_2d(raw + kBox, &tmX, &tail.full[s], n0 + 128, begin + r, keep);
                    ++issued;
                    if (++s == kStages) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
            if (*abort_flag) {
                const uint32_t from = issued > kStages ? issued - kStages : 0u;
                for (uint32_t x = from; x < issued; ++x) {
                    volatile int no_abort = 0;
                    mbar_wait_bounded(&tail.full[x % kStages], (x / kStages) & 1u, &no_abort);
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            const uint64_t a0 = make_smem_desc_sw128(smem_u32(ring), kBox, 1024);
            const uint64_t b0 = make_smem_desc_sw128(smem_u32(ring + kABytes + kRawBytes), kBox, 1024);
            uint32_t s = 0, ph = 0;
            int j = 0;
            bool stop = false;
            for (int tile = blockIdx.x; tile < tiles && !stop; tile += gridDim.x) {
                const int e = tile / per, i = tile - e * per, n0 = (i % p.n_tiles) * kTileN;
                const int count = tail.count[e];
                if (count == 0) continue;
                const uint32_t idesc = make_idesc_bf16_f32(kTileM, p.cols - n0 > 128 ? 256 : 128, 1, 1);
                const int b = j & 1;
                if (!mbar_wait_bounded(&tail.acc_empty[b], ((j >> 1) & 1) ^ 1, abort_flag)) break;
                tc_fence_after_sync();
                const uint32_t d = tmem + b * kTileN;
                for (int r = 0; r < count; r += kRows) {
                    if (!mbar_wait_bounded(&tail.conv[s], ph, abort_flag)) {
                        stop = true;
                        break;
                    }
                    tc_fence_after_sync();
                    const uint64_t at = (s * kStageBytes) >> 4;
#pragma unroll
                    for (int k = 0; k < kRows / 16; ++k)
                        tc_mma_f16(d, a0 + at + k * 128, b0 + at + k * 128, idesc, (r | k) != 0);
                    tc_commit(&tail.empty[s]);
                    if (++s == kStages) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
                if (stop) break;
                tc_commit(&tail.acc_full[b]);
                ++j;
            }
            tc_commit(&tail.drain);
            volatile int no_abort = 0;
            mbar_wait_bounded(&tail.drain, 0, &no_abort);
        }
    } else if (warp >= 8) {
        const int t = threadIdx.x - 256, c = t & 7, r0 = t >> 3;   // 16-byte chunk of a row, first row
        const int kblocks = p.cols >> 7;
        uint32_t s = 0, ph = 0;
        bool bad = false;
        for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
            const int e = tile / per, i = tile - e * per, n0 = (i % p.n_tiles) * kTileN;
            const int count = tail.count[e];
            const int64_t begin = tail.begin[e];
            const int boxes = p.cols - n0 > 128 ? 2 : 1;
            bool ok = true;
            for (int r = 0; r < count; r += kRows) {
                const int valid = count - r;
                uint32_t sb[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int row = r0 + 32 * (x & 1), kb = x >> 1;
                    sb[x] = 127;
                    if (row < valid && kb < boxes)
                        sb[x] = load_scale_byte(p.X_scale, p.x_ue8m0, (begin + r + row) * kblocks + (n0 >> 7) + kb, bad);
                }
                ok = __all_sync(0xffffffffu, mbar_wait_bounded(&tail.full[s], ph, abort_flag, 32));
                if (!ok) break;
                uint8_t *a = ring + s * kStageBytes, *raw = a + kABytes, *b = raw + kRawBytes;
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int row = r0 + 32 * (x & 1), kb = x >> 1;
                    if (kb >= boxes) continue;
                    uint4 w = make_uint4(0, 0, 0, 0);
                    if (row < valid) w = *reinterpret_cast<const uint4 *>(raw + kb * kBox + row * 128 + ((c ^ (row & 7)) << 4));
                    // 2^120 * s as a bf16; beyond its range the rest goes into a second factor
                    const uint32_t ex = 120u + sb[x];
                    const uint32_t f = (ex < 254u ? ex : 254u) * 0x00800080u;
                    uint2 v[4] = {codes_to_bf16(w.x, f), codes_to_bf16(w.y, f), codes_to_bf16(w.z, f),
                                  codes_to_bf16(w.w, f)};
                    if (ex > 254u) {
                        const uint32_t f2 = (127u + ex - 254u) * 0x00800080u;
#pragma unroll
                        for (int y = 0; y < 4; ++y) v[y] = make_uint2(mul_bf16x2(v[y].x, f2), mul_bf16x2(v[y].y, f2));
                    }
                    if (nan_codes(w.x) | nan_codes(w.y) | nan_codes(w.z) | nan_codes(w.w)) {
                        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            v[y] = make_uint2(set_nan(v[y].x, ww[y], 0), set_nan(v[y].y, ww[y], 2));
                    }
                    // chunk c is bf16 columns 16 c .. 16 c + 15: two 16-byte chunks of box c / 4.  Half of
                    // the lanes store the second one first, so that a row's eight stores meet eight banks
                    uint8_t *dst = b + (kb * 2 + (c >> 2)) * kBox + row * 128;
                    const int ch = (c & 3) * 2, first = c >> 2;
                    const uint4 lo = make_uint4(v[0].x, v[0].y, v[1].x, v[1].y);
                    const uint4 hi = make_uint4(v[2].x, v[2].y, v[3].x, v[3].y);
                    *reinterpret_cast<uint4 *>(dst + (((ch + first) ^ (row & 7)) << 4)) = first ? hi : lo;
                    *reinterpret_cast<uint4 *>(dst + (((ch + 1 - first) ^ (row & 7)) << 4)) = first ? lo : hi;
                }
                if (valid < kRows) {
                    // rows behind the group's end: whatever dY holds there must not meet the zeros of x
                    for (int x = t; x < (kRows - valid) * 16; x += kConvWarps * 32)
                        *reinterpret_cast<uint4 *>(a + (x & 8 ? kBox : 0) + (valid + (x >> 4)) * 128 + ((x & 7) << 4)) =
                            make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&tail.conv[s]);
                if (++s == kStages) {
                    s = 0;
                    ph ^= 1u;
                }
            }
            if (!ok) break;
        }
        if (bad) tail.bad_scale = 1;
    } else if (warp >= 4) {
        const int w = warp - 4;
        uint8_t *buf = epi + w * 32 * 128;
        const uint32_t lane_addr = tmem + (static_cast<uint32_t>(w * 32) << 16);
        int j = 0;
        for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
            const int e = tile / per, i = tile - e * per, m0 = (i / p.n_tiles) * kTileM, n0 = (i % p.n_tiles) * kTileN;
            const bool some = tail.count[e] != 0;
            const int b = j & 1;
            if (some) {
                if (!__all_sync(0xffffffffu, mbar_wait_bounded(&tail.acc_full[b], (j >> 1) & 1, abort_flag, 64))) break;
                tc_fence_after_sync();
                ++j;
            }
            const int width = p.cols - n0 > 128 ? 256 : 128;
            const int64_t base = (static_cast<int64_t>(e) * p.rows + m0 + w * 32) * p.cols + n0;
            for (int c = 0; c < width; c += 32) {
                float v[32];
                if (some) {
                    tmem_ld_32x32b_x32(lane_addr + b * kTileN + c, v);
                    tmem_ld_wait();
                } else {
#pragma unroll
                    for (int x = 0; x < 32; ++x) v[x] = 0.f;
                }
                // a row of 32 fp32 is eight 16-byte chunks, chunk x of row l at place x ^ (l & 7)
#pragma unroll
                for (int x = 0; x < 8; ++x)
                    *reinterpret_cast<float4 *>(buf + lane * 128 + ((x ^ (lane & 7)) << 4)) =
                        make_float4(v[4 * x], v[4 * x + 1], v[4 * x + 2], v[4 * x + 3]);
                __syncwarp();
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    const int row = x * 4 + (lane >> 3), ch = lane & 7;
                    float4 y = *reinterpret_cast<const float4 *>(buf + row * 128 + ((ch ^ (row & 7)) << 4));
                    if (m0 + w * 32 + row < p.rows) {
                        const int64_t at = base + static_cast<int64_t>(row) * p.cols + c + ch * 4;
                        if (p.add) {
                            const float4 z = __ldcs(reinterpret_cast<const float4 *>(p.add + at));
                            y.x += z.x;
                            y.y += z.y;
                            y.z += z.z;
                            y.w += z.w;
                        }
                        if (p.bf16_out) {
                            __nv_bfloat162 h[2] = {__floats2bfloat162_rn(y.x, y.y), __floats2bfloat162_rn(y.z, y.w)};
                            __stcs(reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.dW) + at),
                                   *reinterpret_cast<uint2 *>(h));
                        } else {
                            __stcs(reinterpret_cast<float4 *>(static_cast<float *>(p.dW) + at), y);
                        }
                    }
                }
                __syncwarp();
            }
            if (some) {
                tc_fence_before_sync();
                if (lane == 0) mbar_arrive(&tail.acc_empty[b]);
            }
        }
    }

    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == 3) tmem_dealloc(tmem, kTmemCols);
    if (threadIdx.x == 0) {
        if (tail.abort) report_status(p.status, MOE_ERR_TIMEOUT);
        if (tail.bad_index) report_status(p.status, MOE_ERR_BAD_INDEX);
        if (tail.bad_scale) report_status(p.status, MOE_ERR_BAD_SCALE);
    }
}

}  // namespace

cudaError_t launch_expert_wgrad(const ExpertWgradArgs &a, cudaStream_t stream)
{
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (device_cc_major(dev) != 10) return cudaErrorNotSupported;
    CUtensorMap tmY, tmX;
    const uint64_t R = a.R > 0 ? a.R : 1;   // (no rows: the maps are not used)
    const uint64_t yd[2] = {static_cast<uint64_t>(a.rows), R};
    const uint32_t yb[2] = {64, kRows};
    const uint64_t xd[2] = {static_cast<uint64_t>(a.cols), R};
    const uint32_t xb[2] = {128, kRows};
    if (!encode_map_sw128(&tmY, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.R > 0 ? a.dY : a.dW, 2, yd, yb) ||
        !encode_map_sw128(&tmX, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.R > 0 ? a.X : a.dW, 2, xd, xb))
        return cudaErrorInvalidValue;
    static std::atomic<uint64_t> done{0};
    const uint64_t bit = 1ull << (dev & 63);
    if (!(done.load(std::memory_order_relaxed) & bit)) {
        err = cudaFuncSetAttribute(expert_wgrad_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   static_cast<int>(kSmemBytes));
        if (err != cudaSuccess) return err;
        done.fetch_or(bit, std::memory_order_relaxed);
    }
    Params p;
    p.X_scale = a.X_scale;
    p.offsets = a.offsets;
    p.add = a.add;
    p.dW = a.dW;
    p.R = a.R;
    p.E = a.E;
    p.rows = a.rows;
    p.cols = a.cols;
    p.x_ue8m0 = a.x_ue8m0;
    p.bf16_out = a.bf16_out;
    p.m_tiles = (a.rows + kTileM - 1) / kTileM;
    p.n_tiles = (a.cols + kTileN - 1) / kTileN;
    p.status = a.status;
    const int64_t tiles = static_cast<int64_t>(a.E) * p.m_tiles * p.n_tiles;
    const int sms = device_sm_count(dev);
    expert_wgrad_kernel<<<static_cast<int>(tiles < sms ? tiles : sms), kThreads, kSmemBytes, stream>>>(tmY, tmX, p);
    return cudaGetLastError();
}

}  // namespace moe
