// norm.cu -- the norm in front of the router, with the residual stream's addition and E4M3 rows, and its gradient.
//
//   s = bf16(x + residual);  rstd = 1 / sqrt(mean s^2 + eps);  y = s rstd w
//   dx = rstd (d - xh mean(d xh)) + dS,  d = dy w,  xh = s rstd;   dw = sum over the rows of dy xh (+ add)
//
// One pass over the rows: a row stays in the registers of its threads (a warp's for short rows, else a CTA's; kV
// chunks of 16 bytes each, neighbouring threads neighbouring chunks) between its sum and what is written.  The sums
// are held in 32 bits.
#include "expert_internal.cuh"

namespace moe {
namespace {

constexpr uint32_t kFull = 0xffffffffu;

__device__ __forceinline__ void unpack(const uint4 &x, float (&f)[8])
{
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint4 pack(const float (&f)[8])
{
    uint4 v;
    __nv_bfloat162 *h = reinterpret_cast<__nv_bfloat162 *>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    return v;
}

// Chunk c of the weight.
__device__ __forceinline__ void load_weight(const void *w, int bf16, int c, float (&f)[8])
{
    if (bf16) {
        unpack(__ldg(static_cast<const uint4 *>(w) + c), f);
    } else {
        const float4 a = __ldg(static_cast<const float4 *>(w) + 2 * c), b = __ldg(static_cast<const float4 *>(w) + 2 * c + 1);
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    }
}

constexpr int kWarpRows = 4;      // rows of a CTA where a row is a warp's
constexpr int kMostThreads = 512;
constexpr int kTwoThreads = 384;  // the most with two chunks each

// The sum over the threads of a row, the same in each of them.  `part`: a float for each warp; a second call takes
// another array.
template <bool kWarp>
__device__ __forceinline__ float row_sum(float v, float *part)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    if constexpr (!kWarp) {
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
        __syncthreads();
        // every warp adds them up in the same order
        const int warps = blockDim.x >> 5, i = threadIdx.x & 15;
        v = i < warps ? part[i] : 0.f;
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    }
    return v;
}

struct Forward {
    const uint4 *X, *residual;
    const void *w;
    int64_t N;
    int H, w_bf16, ue8m0;
    float eps;
    uint4 *S, *Y;
    uint2 *Q;
    void *Q_scale;
    float *rstd;
};

template <bool kWarp, int kV>
__global__ void __launch_bounds__(kMostThreads) rms_norm_kernel(const Forward p)
{
    __shared__ float part[kMostThreads / 32];
    const int T = kWarp ? 32 : blockDim.x, t = kWarp ? threadIdx.x & 31 : threadIdx.x, chunks = p.H >> 3;
    const int64_t row = kWarp ? static_cast<int64_t>(blockIdx.x) * kWarpRows + (threadIdx.x >> 5) : blockIdx.x;
    if (kWarp && row >= p.N) return;
    const int64_t base = row * chunks;
    uint4 x[kV], r[kV];
#pragma unroll
    for (int j = 0; j < kV; ++j) {
        const int c = t + T * j;
        x[j] = r[j] = make_uint4(0, 0, 0, 0);
        if (c < chunks) x[j] = __ldcs(p.X + base + c);
        if (p.residual && c < chunks) r[j] = __ldcs(p.residual + base + c);
    }
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < kV; ++j) {
        if (p.residual) {
            // (two bf16 numbers added in 32 bits and rounded once more are the sum rounded once: where 32 bits do not
            // hold it the smaller number is below 2^-16 of the larger, which is far from the middle of two bf16)
            float a[8], b[8];
            unpack(x[j], a);
            unpack(r[j], b);
#pragma unroll
            for (int i = 0; i < 8; ++i) a[i] += b[i];
            x[j] = pack(a);
            if (p.S && t + T * j < chunks) p.S[base + t + T * j] = x[j];
        }
        float a[8];
        unpack(x[j], a);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = fmaf(a[i], a[i], sum);
    }
    const float rstd = 1.f / sqrtf(row_sum<kWarp>(sum, part) / static_cast<float>(p.H) + p.eps);
    if (p.rstd && t == 0) p.rstd[row] = rstd;
#pragma unroll
    for (int j = 0; j < kV; ++j) {
        const int c = t + T * j;
        if (T * j >= chunks) break;
        float y[8], w[8];
        const bool there = c < chunks;
        load_weight(p.w, p.w_bf16, there ? c : chunks - 1, w);
        unpack(x[j], y);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = y[i] * rstd * w[i];
        if (p.Y && there) p.Y[base + c] = pack(y);
        if (p.Q) {
            // a block of 128 columns is 16 neighbouring lanes
            float m = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(y[i]));
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
            const uint32_t byte = block_scale_byte(m);
            const float inv = scale_reciprocal(byte);
            if (there) {
                p.Q[base + c] = make_uint2(f32x4_to_e4m3x4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv),
                                           f32x4_to_e4m3x4(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv));
                if ((t & 15) == 0) store_scale(p.Q_scale, p.ue8m0, (base + c) >> 4, byte);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Gradient.  A CTA takes rows blockIdx.x, + gridDim.x, ... (a warp's rows: kWarpRows at a time): its threads keep to
// their columns and sum dy xh for them.  kFlush rows at a time are summed in registers, those sums in shared memory,
// and the CTA's own row of the workspace's table is their sum; a second launch adds the table's rows up.  The order
// is the same in every call.
// ---------------------------------------------------------------------------
constexpr int kFlush = 64;

struct Backward {
    const uint4 *dY, *S, *dS;
    const void *w;
    const float *rstd;
    int64_t N;
    int H, w_bf16;
    uint4 *dX;
    float *table;                 // [gridDim.x][H]
};

template <bool kWarp, int kV>
__global__ void __launch_bounds__(kV <= 2 ? kTwoThreads : kMostThreads, kV <= 2 ? 2 : 1) rms_norm_backward_kernel(const Backward p)
{
    __shared__ float part[2][kMostThreads / 32];
    extern __shared__ float sums[];       // [kV][8][threads], so that neighbouring threads are neighbours
    const int T = kWarp ? 32 : blockDim.x, t = kWarp ? threadIdx.x & 31 : threadIdx.x, chunks = p.H >> 3;
    const int rows = kWarp ? kWarpRows : 1;
    const float of_H = static_cast<float>(p.H);
    float acc[kV][8];
#pragma unroll
    for (int j = 0; j < kV; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            acc[j][i] = 0.f;
            sums[(j * 8 + i) * blockDim.x + threadIdx.x] = 0.f;
        }
    int n = 0;
    for (int64_t r = static_cast<int64_t>(blockIdx.x) * rows; r < p.N; r += static_cast<int64_t>(gridDim.x) * rows, ++n) {
        const int64_t row = kWarp ? r + (threadIdx.x >> 5) : r;
        const bool row_ok = row < p.N;
        const int64_t base = (row_ok ? row : p.N - 1) * chunks;
        uint4 dy[kV], s[kV], ds[kV];
#pragma unroll
        for (int j = 0; j < kV; ++j) {
            const int c = t + T * j;
            dy[j] = s[j] = ds[j] = make_uint4(0, 0, 0, 0);
            if (c < chunks) {
                dy[j] = __ldcs(p.dY + base + c);
                s[j] = __ldcs(p.S + base + c);
                if (p.dS) ds[j] = __ldcs(p.dS + base + c);
            }
        }
        const float rstd = p.rstd[row_ok ? row : p.N - 1];
        if (n == kFlush) {
            n = 0;
#pragma unroll
            for (int j = 0; j < kV; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    sums[(j * 8 + i) * blockDim.x + threadIdx.x] += acc[j][i];
                    acc[j][i] = 0.f;
                }
        }
        float dot = 0.f;
#pragma unroll
        for (int j = 0; j < kV; ++j) {
            const int c = t + T * j;
            float a[8], b[8], w[8];
            unpack(dy[j], a);
            unpack(s[j], b);
            load_weight(p.w, p.w_bf16, c < chunks ? c : chunks - 1, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float v = a[i] * (b[i] * rstd);
                dot = fmaf(v, w[i], dot);
                if (row_ok) acc[j][i] += v;
            }
        }
        const float mean = row_sum<kWarp>(dot, part[n & 1]) / of_H;
#pragma unroll
        for (int j = 0; j < kV; ++j) {
            const int c = t + T * j;
            if (c >= chunks) break;
            float a[8], b[8], e[8], w[8];
            unpack(dy[j], a);
            unpack(s[j], b);
            unpack(ds[j], e);
            load_weight(p.w, p.w_bf16, c, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) a[i] = fmaf(rstd, a[i] * w[i] - b[i] * rstd * mean, e[i]);
            if (row_ok) p.dX[base + c] = pack(a);
        }
    }
    pdl_launch_dependents();
#pragma unroll
    for (int j = 0; j < kV; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[j][i] += sums[(j * 8 + i) * blockDim.x + threadIdx.x];
    if constexpr (kWarp) {
        // the warps' sums, added by the first
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kV; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) sums[(j * 8 + i) * blockDim.x + threadIdx.x] = acc[j][i];
        __syncthreads();
        if (threadIdx.x >= 32) return;
#pragma unroll
        for (int j = 0; j < kV; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                acc[j][i] = 0.f;
#pragma unroll
                for (int k = 0; k < kWarpRows; ++k) acc[j][i] += sums[(j * 8 + i) * blockDim.x + threadIdx.x + 32 * k];
            }
    }
#pragma unroll
    for (int j = 0; j < kV; ++j) {
        const int c = t + T * j;
        if (c >= chunks) break;
        float4 *dst = reinterpret_cast<float4 *>(p.table + static_cast<int64_t>(blockIdx.x) * p.H) + 2 * c;
        dst[0] = make_float4(acc[j][0], acc[j][1], acc[j][2], acc[j][3]);
        dst[1] = make_float4(acc[j][4], acc[j][5], acc[j][6], acc[j][7]);
    }
}

// dw = the sum of the table's rows (+ add): 32 columns a CTA, 16 threads for the rows of each, four sums a thread.
constexpr int kSumThreads = 512;

__global__ void __launch_bounds__(kSumThreads) rms_norm_dweight_kernel(const float *__restrict__ table, int rows, int H, const float *add, float *dw)
{
    __shared__ float part[kSumThreads / 32][32];
    constexpr int kStep = kSumThreads / 32;
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), k = threadIdx.x >> 5;
    pdl_wait_prior_grids();
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (c < H) {
        const float *at = table + c;
        int r = k;
        for (; r + 3 * kStep < rows; r += 4 * kStep)
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] += at[static_cast<int64_t>(r + i * kStep) * H];
        for (int i = 0; r < rows; r += kStep, ++i) v[i & 3] += at[static_cast<int64_t>(r) * H];
    }
    part[k][threadIdx.x & 31] = (v[0] + v[1]) + (v[2] + v[3]);
    __syncthreads();
    if (k == 0 && c < H) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < kStep; ++i) sum += part[i][threadIdx.x];
        dw[c] = add ? add[c] + sum : sum;
    }
}

// How a row of H columns is held: a warp of one or two chunks a lane up to 512 columns, else as many threads, whole
// warps, as two chunks each (beyond 6144 columns four) make of it.
struct Shape {
    bool warp;
    int per, threads;
};
Shape shape_of(int H)
{
    const int chunks = H / 8;
    if (chunks <= 64) return Shape{true, chunks <= 32 ? 1 : 2, 32 * kWarpRows};
    const int per = chunks <= 2 * kTwoThreads ? 2 : 4;
    return Shape{false, per, ((chunks + per - 1) / per + 31) / 32 * 32};
}

}  // namespace

cudaError_t launch_rms_norm(const RmsNormArgs &a, cudaStream_t stream)
{
    int dev = 0;
    const cudaError_t err = expert_device(&dev);
    if (err != cudaSuccess) return err;
    Forward p;
    p.X = static_cast<const uint4 *>(a.X);
    p.residual = static_cast<const uint4 *>(a.residual);
    p.w = a.weight;
    p.N = a.N;
    p.H = a.H;
    p.w_bf16 = a.w_bf16;
    p.ue8m0 = a.ue8m0;
    p.eps = a.eps;
    p.S = static_cast<uint4 *>(a.S);
    p.Y = static_cast<uint4 *>(a.Y);
    p.Q = static_cast<uint2 *>(a.Y_fp8);
    p.Q_scale = a.Y_scale;
    p.rstd = a.rstd;
    const Shape f = shape_of(a.H);
    const unsigned grid = static_cast<unsigned>(f.warp ? (a.N + kWarpRows - 1) / kWarpRows : a.N);
    const auto kernel = f.warp ? (f.per == 1 ? rms_norm_kernel<true, 1> : rms_norm_kernel<true, 2>)
                               : (f.per == 2 ? rms_norm_kernel<false, 2> : rms_norm_kernel<false, 4>);
    kernel<<<grid, f.threads, 0, stream>>>(p);
    return cudaGetLastError();
}

int rms_norm_table_rows(int64_t N, int H)
{
    // as many CTAs as the 152 SMs of a GB300 hold at 80 registers a thread (128 where a thread has four chunks), eight
    // an SM at most, and no more than there are rows for.  (Of 65536 x 4096 and 16381 x 1032, bursts: 351 and 39 us; with
    // 64 registers, 4/3 of the threads and some spills 368 and 42; with 96 registers 415 and 42.)
    const Shape f = shape_of(H);
    const int fit = (f.per <= 2 ? 2 * kTwoThreads : 512) / f.threads, most = 152 * (fit < 8 ? fit : 8);
    const int64_t n = f.warp ? (N + kWarpRows - 1) / kWarpRows : N;
    return static_cast<int>(n < most ? n : most);
}

cudaError_t launch_rms_norm_backward(const RmsNormBackwardArgs &a, cudaStream_t stream)
{
    int dev = 0;
    const cudaError_t err = expert_device(&dev);
    if (err != cudaSuccess) return err;
    Backward p;
    p.dY = static_cast<const uint4 *>(a.dY);
    p.S = static_cast<const uint4 *>(a.S);
    p.dS = static_cast<const uint4 *>(a.dS);
    p.w = a.weight;
    p.rstd = a.rstd;
    p.N = a.N;
    p.H = a.H;
    p.w_bf16 = a.w_bf16;
    p.dX = static_cast<uint4 *>(a.dX);
    p.table = static_cast<float *>(a.workspace);
    const int grid = rms_norm_table_rows(a.N, a.H);
    cudaLaunchConfig_t cfg = {};
    cfg.stream = stream;
    if (grid > 0) {
        const Shape f = shape_of(a.H);
        const auto kernel = f.warp ? (f.per == 1 ? rms_norm_backward_kernel<true, 1> : rms_norm_backward_kernel<true, 2>)
                                   : (f.per == 2 ? rms_norm_backward_kernel<false, 2> : rms_norm_backward_kernel<false, 4>);
        cfg.gridDim = dim3(grid);
        cfg.blockDim = dim3(f.threads);
        cfg.dynamicSmemBytes = f.per * 8 * f.threads * sizeof(float);
        if (cfg.dynamicSmemBytes > 48 * 1024) {
            static std::atomic<uint64_t> done{0};
            const uint64_t bit = 1ull << (dev & 63);
            if (!(done.load(std::memory_order_relaxed) & bit)) {
                const cudaError_t e = cudaFuncSetAttribute(rms_norm_backward_kernel<false, 4>, cudaFuncAttributeMaxDynamicSharedMemorySize, 64 * 1024);
                if (e != cudaSuccess) return e;
                done.fetch_or(bit, std::memory_order_relaxed);
            }
        }
        const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
        if (e != cudaSuccess) return e;
    }
    cfg.gridDim = dim3((a.H + 31) / 32);
    cfg.blockDim = dim3(kSumThreads);
    cfg.dynamicSmemBytes = 0;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, rms_norm_dweight_kernel, static_cast<const float *>(p.table), grid, a.H, a.add, a.dweight);
}

}  // namespace moe
