// norm.cu -- the norm in front of the router, with the residual stream's addition and E4M3 rows, and its gradient.
//
//   s = bf16(x + residual);  rstd = 1 / sqrt(mean s^2 + eps);  y = s rstd w
//   dx = rstd (d - xh mean(d xh)) + dS,  d = dy w,  xh = s rstd;   dw = sum over the rows of dy xh (+ add)
//
// One pass over the rows: a row stays in the registers of its threads (a warp's for short rows, else a CTA's; kV
// chunks of 16 bytes each, neighbouring threads neighbouring chunks) between its sum and what is written.  The sums
// are held in 32 bits.  HBM's bound: 65536 x 4096 with the residual and E4M3 rows 349 us (6.9 TB/s), the gradient of
// the same 334 (6.4 TB/s); one row 2.4 us in a graph.  Rows of a warp: 65536 x 1024 with the residual and E4M3 rows 91 us
// (6.6 TB/s), 262144 x 128 69 (4.4: a lane has one chunk or none, and what is under way is little).  The gradient of
// 16381 x 1032 takes 27 us in a graph where its bytes take 15: two launches and the ring's start are 7 of it, and a row's
// 129 chunks are five to a lane, the last nearly empty (H = 1024: 24; three warps to a row: 29; a condition on each
// chunk's loads: 30).
#include "bulk_ring.cuh"
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

// In pairs, for the packed arithmetic.
__device__ __forceinline__ void unpack2(const uint4 &x, float2 (&f)[4])
{
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}
__device__ __forceinline__ uint4 pack2(const float2 (&f)[4])
{
    uint4 v;
    __nv_bfloat162 *h = reinterpret_cast<__nv_bfloat162 *>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[i].x, f[i].y);
    return v;
}
__device__ __forceinline__ float2 twice(float x) { return make_float2(x, x); }

// Chunk c of the weight.
__device__ __forceinline__ void load_weight2(const void *w, int bf16, int c, float2 (&f)[4])
{
    if (bf16) {
        unpack2(__ldg(static_cast<const uint4 *>(w) + c), f);
    } else {
        const float4 a = __ldg(static_cast<const float4 *>(w) + 2 * c), b = __ldg(static_cast<const float4 *>(w) + 2 * c + 1);
        f[0] = make_float2(a.x, a.y), f[1] = make_float2(a.z, a.w), f[2] = make_float2(b.x, b.y), f[3] = make_float2(b.z, b.w);
    }
}
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
constexpr int warp_ctas(int per) { return per <= 2 ? 6 : 4; }      // of the gradient's on an SM then
constexpr int kMostThreads = 512;

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
// Gradient.  A CTA takes groups of rows blockIdx.x, + gridDim.x, ... (a group is a row, or kWarpRows rows of a warp
// each): its threads keep to their columns and sum dy xh for them.  The rows come through a ring in shared memory, each
// input's as one bulk copy, so that what all CTAs of an SM have under way is most of its shared memory whatever the
// registers hold.  kFlush groups at a time are summed in registers, those sums in the CTA's own row of the workspace's
// table (by one warp after the other where a row is a warp's); a second launch adds the table's rows up.  The order is
// the same in every call.
// ---------------------------------------------------------------------------
constexpr int kFlush = 64;
constexpr int kSlots = 8;

struct Backward {
    const uint8_t *dY, *S, *dS;
    const void *w;
    const float *rstd;
    int64_t N;
    int H, w_bf16, slots;
    uint4 *dX;
    float *table;                 // [gridDim.x][H]
    int32_t *status;
};

// (out of line, for the loop's sake)
__device__ __noinline__ void wait_slow(uint64_t *bar, uint32_t phase, volatile int *abort) { mbar_wait_bounded(bar, phase, abort); }

template <bool kWarp, int kV>
__global__ void __launch_bounds__(kWarp ? 32 * kWarpRows : kMostThreads, kWarp ? warp_ctas(kV) : kV <= 2 ? 2 : 1) rms_norm_backward_kernel(const Backward p)
{
    __shared__ float part[2][kMostThreads / 32];
    __shared__ uint64_t full[kSlots];
    __shared__ volatile int abort;
    __shared__ uint32_t issued;   // groups asked for (thread 0's)
    extern __shared__ __align__(128) uint8_t ring[];
    const int T = kWarp ? 32 : blockDim.x, t = kWarp ? threadIdx.x & 31 : threadIdx.x, chunks = p.H >> 3;
    constexpr int rows = kWarp ? kWarpRows : 1;
    const uint32_t array = rows * p.H * 2, inputs = p.dS ? 3 : 2, stage = array * inputs;
    const int64_t groups = (p.N + rows - 1) / rows, mine = (groups - blockIdx.x + gridDim.x - 1) / gridDim.x;
    const float per_H = 1.f / static_cast<float>(p.H);
    float *table = p.table + static_cast<int64_t>(blockIdx.x) * p.H;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kSlots; ++i) mbar_init(&full[i], 1);
        abort = 0;
        fence_mbarrier_init();
    }
    __syncthreads();
    const auto issue = [&](int64_t i, int slot) {
        const int64_t r = (blockIdx.x + i * gridDim.x) * rows, left = p.N - r;
        const uint32_t bytes = static_cast<uint32_t>(left < rows ? left : rows) * p.H * 2;
        const int64_t at = r * p.H * 2;
        uint8_t *to = ring + slot * stage;
        mbar_arrive_expect_tx(&full[slot], bytes * inputs);
        bulk_load(to, p.dY + at, bytes, &full[slot]);
        bulk_load(to + array, p.S + at, bytes, &full[slot]);
        if (p.dS) bulk_load(to + 2 * array, p.dS + at, bytes, &full[slot]);
        issued = static_cast<uint32_t>(i) + 1;
    };
    if (threadIdx.x == 0)
        for (int i = 0; i < p.slots && i < mine; ++i) issue(i, i);

    float2 acc[kV][4];
#pragma unroll
    for (int j = 0; j < kV; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[j][i] = twice(0.f);
    const auto add_to_table = [&](bool first) {
#pragma unroll
        for (int j = 0; j < kV; ++j) {
            const int c = t + T * j;
            if (c < chunks) {
                float4 *dst = reinterpret_cast<float4 *>(table) + 2 * c;
                float4 a = make_float4(acc[j][0].x, acc[j][0].y, acc[j][1].x, acc[j][1].y), b = make_float4(acc[j][2].x, acc[j][2].y, acc[j][3].x, acc[j][3].y);
                if (!first) {
                    const float4 x = dst[0], y = dst[1];
                    a.x += x.x, a.y += x.y, a.z += x.z, a.w += x.w;
                    b.x += y.x, b.y += y.y, b.z += y.z, b.w += y.w;
                }
                dst[0] = a;
                dst[1] = b;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[j][i] = twice(0.f);
        }
    };
    const auto flush = [&](bool first) {
        if constexpr (kWarp) {
            for (int w = 0; w < kWarpRows; ++w) {
                if (static_cast<int>(threadIdx.x >> 5) == w) add_to_table(first && w == 0);
                __syncthreads();
            }
        } else {
            add_to_table(first);
        }
    };
    int slot = 0, before = 0, n = 0;
    uint32_t phase = 0;
    bool first = true;
    int64_t row = static_cast<int64_t>(blockIdx.x) * rows + (kWarp ? threadIdx.x >> 5 : 0);
    const int64_t step = static_cast<int64_t>(gridDim.x) * rows;
    uint4 *dx = p.dX + row * chunks + t;
    const uint8_t *own = ring + (kWarp ? (threadIdx.x >> 5) * p.H * 2 : 0) + t * 16;
    float rstd_next = __ldg(p.rstd + (row < p.N ? row : p.N - 1));       // a group ahead
    for (int64_t g = 0; g < mine; ++g, ++n, row += step, dx += step * chunks) {
        const bool row_ok = !kWarp || row < p.N;
        const float rstd = rstd_next;
        rstd_next = __ldg(p.rstd + (row + step < p.N ? row + step : p.N - 1));
        if (n == kFlush) {
            flush(first);
            first = false;
            n = 0;
        }
        // (a wait that ran out sets `abort`: the loop goes on without copies and without waiting, in step)
        if (!mbar_try_wait(smem_u32(&full[slot]), phase)) wait_slow(&full[slot], phase, &abort);
        const uint8_t *at = own + slot * stage;
        const uint4 *dy = reinterpret_cast<const uint4 *>(at), *s = reinterpret_cast<const uint4 *>(at + array),
                    *ds = reinterpret_cast<const uint4 *>(at + 2 * array);
        // d = dy w times xh = s rstd, and the weight's sum.  (s rstd comes first: dy s may be beyond 32 bits where rstd is 0, and
        // that row's part of the sums would be a NaN.)
        // (only the last chunk of a thread may not be there: the loads of the others carry no condition, which would make
        // them wait for one another)
        float2 dot = twice(0.f);
        if (row_ok) {
#pragma unroll
            for (int j = 0; j < kV; ++j) {
                const int c = t + T * j;
                if (j + 1 == kV && c >= chunks) break;
                float2 a[4], b[4], w[4];
                unpack2(dy[T * j], a);
                unpack2(s[T * j], b);
                load_weight2(p.w, p.w_bf16, c, w);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 xh = __fmul2_rn(b[i], twice(rstd));
                    dot = __ffma2_rn(__fmul2_rn(a[i], w[i]), xh, dot);
                    acc[j][i] = __ffma2_rn(a[i], xh, acc[j][i]);
                }
            }
        }
        if (kWarp) __syncthreads();
        const float minus_mean = -(row_sum<kWarp>(dot.x + dot.y, part[n & 1]) * per_H);
        // every thread is past that barrier, so none reads the group before any more: its place is filled again
        if (threadIdx.x == 0 && g > 0 && g - 1 + p.slots < mine && !abort) issue(g - 1 + p.slots, before);
        if (row_ok) {
#pragma unroll
            for (int j = 0; j < kV; ++j) {
                const int c = t + T * j;
                if (j + 1 == kV && c >= chunks) break;
                float2 a[4], b[4], e[4], w[4];
                unpack2(dy[T * j], a);
                unpack2(s[T * j], b);
                unpack2(p.dS ? ds[T * j] : make_uint4(0, 0, 0, 0), e);
                load_weight2(p.w, p.w_bf16, c, w);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 d = __ffma2_rn(__fmul2_rn(b[i], twice(rstd)), twice(minus_mean), __fmul2_rn(a[i], w[i]));
                    a[i] = __ffma2_rn(d, twice(rstd), e[i]);
                }
                dx[T * j] = pack2(a);
            }
        }
        before = slot;
        if (++slot == p.slots) {
            slot = 0;
            phase ^= 1u;
        }
    }
    pdl_launch_dependents();
    flush(first);
    __syncthreads();              // (a thread may have given up at the last group)
    if (threadIdx.x == 0 && abort) {
        report_status(p.status, MOE_ERR_TIMEOUT);
        // what may still be under way lands before this CTA's memory is another's
        for (uint32_t x = ring_first_open(issued, p.slots); x < issued; ++x) {
            volatile int no_abort = 0;
            mbar_wait_bounded(&full[ring_place(x, p.slots)], ring_parity(x, p.slots), &no_abort);
        }
    }
}

// dw = the sum of the table's rows (+ add): 8 columns a CTA (a sector of each row), 128 threads for the rows of each,
// eight sums a thread, so that the whole table is asked for in a round or two by a CTA on most SMs.
constexpr int kSumThreads = 1024;

__global__ void __launch_bounds__(kSumThreads) rms_norm_dweight_kernel(const float *__restrict__ table, int rows, int H, const float *add, float *dw)
{
    constexpr int kStep = kSumThreads / 8, kEach = 8;
    __shared__ float part[kSumThreads / 32][8];
    const int c = blockIdx.x * 8 + (threadIdx.x & 7), k = threadIdx.x >> 3;      // (H is whole in 8)
    pdl_wait_prior_grids();
    float v[kEach] = {};
    const float *at = table + c;
    for (int r = k; r < rows; r += kEach * kStep) {
        // (no condition on the loads, which would make them wait for one another)
        float x[kEach];
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int of = r + i * kStep;
            x[i] = at[static_cast<int64_t>(of < rows ? of : r) * H];
        }
#pragma unroll
        for (int i = 0; i < kEach; ++i) v[i] += r + i * kStep < rows ? x[i] : 0.f;
    }
    float sum = ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
    sum += __shfl_xor_sync(kFull, sum, 8);
    sum += __shfl_xor_sync(kFull, sum, 16);
    if ((threadIdx.x & 31) < 8) part[threadIdx.x >> 5][threadIdx.x & 7] = sum;
    __syncthreads();
    if (threadIdx.x < 8) {
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < kSumThreads / 32; ++i) sum += part[i][threadIdx.x];
        dw[c] = add ? add[c] + sum : sum;
    }
}

// How a row of H columns is held: by a warp of up to five chunks a lane up to 1184 columns (the gradient's ring then still
// has two places for four rows of three inputs in a quarter of an SM), else by as many threads, whole warps, as two chunks
// each (beyond 8192 columns four) make of it.
struct Shape {
    bool warp;
    int per, threads;
};
Shape shape_of(int H)
{
    const int chunks = H / 8;
    if (chunks <= 148) return Shape{true, (chunks + 31) / 32, 32 * kWarpRows};
    const int per = chunks <= 2 * kMostThreads ? 2 : 4;
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
    constexpr decltype(&rms_norm_kernel<true, 1>) of_warps[5] = {rms_norm_kernel<true, 1>, rms_norm_kernel<true, 2>, rms_norm_kernel<true, 3>,
                                                                 rms_norm_kernel<true, 4>, rms_norm_kernel<true, 5>};
    const auto kernel = f.warp ? of_warps[f.per - 1] : f.per == 2 ? rms_norm_kernel<false, 2> : rms_norm_kernel<false, 4>;
    kernel<<<grid, f.threads, 0, stream>>>(p);
    return cudaGetLastError();
}

namespace {
// CTAs of the gradient on an SM: 64 registers a thread (128 where a thread has four chunks), eight at most; a warp's rows: by
// warp_ctas().
int resident(const Shape &f)
{
    const int fit = (f.per <= 2 ? 1024 : 512) / f.threads;
    return f.warp ? warp_ctas(f.per) : fit < 8 ? fit : 8;
}

template <bool kWarp, int kV>
cudaError_t launch_gradient(Backward &p, const Shape &f, int grid, int dev, cudaStream_t stream)
{
    // an SM's shared memory but for what the CTAs hold besides (1 KiB of the system's, the kernel's own), in equal parts
    const int ctas = resident(f), own = 1024 + 512;
    const int stage = (kWarp ? kWarpRows : 1) * p.H * 2 * (p.dS ? 3 : 2);
    const int part = ((ctas == 1 ? 227 * 1024 : 228 * 1024 / ctas) - own) / stage;
    p.slots = part < kSlots ? part : kSlots;          // two at least, whatever H is
    static std::atomic<uint64_t> done{0};
    const uint64_t bit = 1ull << (dev & 63);
    if (!(done.load(std::memory_order_relaxed) & bit)) {
        const cudaError_t err = cudaFuncSetAttribute(rms_norm_backward_kernel<kWarp, kV>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                     227 * 1024 - own);
        if (err != cudaSuccess) return err;
        done.fetch_or(bit, std::memory_order_relaxed);
    }
    rms_norm_backward_kernel<kWarp, kV><<<grid, f.threads, p.slots * stage, stream>>>(p);
    return cudaGetLastError();
}
}  // namespace

int rms_norm_table_rows(int64_t N, int H)
{
    // as many CTAs as the 152 SMs of a GB300 hold, and no more than there are rows for
    const Shape f = shape_of(H);
    const int most = 152 * resident(f);
    const int64_t n = f.warp ? (N + kWarpRows - 1) / kWarpRows : N;
    return static_cast<int>(n < most ? n : most);
}

cudaError_t launch_rms_norm_backward(const RmsNormBackwardArgs &a, cudaStream_t stream)
{
    int dev = 0;
    cudaError_t err = expert_device(&dev);
    if (err != cudaSuccess) return err;
    Backward p;
    p.dY = static_cast<const uint8_t *>(a.dY);
    p.S = static_cast<const uint8_t *>(a.S);
    p.dS = static_cast<const uint8_t *>(a.dS);
    p.w = a.weight;
    p.rstd = a.rstd;
    p.N = a.N;
    p.H = a.H;
    p.w_bf16 = a.w_bf16;
    p.dX = static_cast<uint4 *>(a.dX);
    p.table = static_cast<float *>(a.workspace);
    p.status = a.status;
    const int grid = rms_norm_table_rows(a.N, a.H);
    if (grid > 0) {
        const Shape f = shape_of(a.H);
        constexpr decltype(&launch_gradient<true, 1>) of_warps[5] = {launch_gradient<true, 1>, launch_gradient<true, 2>, launch_gradient<true, 3>,
                                                                     launch_gradient<true, 4>, launch_gradient<true, 5>};
        const auto launch = f.warp ? of_warps[f.per - 1] : f.per == 2 ? launch_gradient<false, 2> : launch_gradient<false, 4>;
        err = launch(p, f, grid, dev, stream);
        if (err != cudaSuccess) return err;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.stream = stream;
    cfg.gridDim = dim3(a.H / 8);
    cfg.blockDim = dim3(kSumThreads);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, rms_norm_dweight_kernel, static_cast<const float *>(p.table), grid, a.H, a.add, a.dweight);
}

}  // namespace moe
