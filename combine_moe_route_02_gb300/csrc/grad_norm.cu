// grad_norm.cu -- the 2-norm of many tensors together, and the tensors scaled down to a largest norm.
//
//   norm = sqrt(sum g^2);  c = min(1, max_norm / (norm + 1e-6));  out = g c
//
// Tensors of any size and type are cut into chunks of 32 KiB, which a grid of resident CTAs takes in turn; a chunk's
// tensor is found in a table that travels with the launch.  A thread sums the squares of its part of a chunk (32 or 64
// values) in 32 bits, and those sums in 64, so that the result is right to the last bits of 32 however many there
// are; the order is the same in every call.  Where the largest value of a part is so large or small that its square
// leaves 32 bits, the part is summed in 64 bits instead.
//
// The clipping is a second launch: every CTA adds up the first one's sums (some 600) by itself, then takes the chunks
// in the opposite order, since the last ones are what is left in L2 (24 blocks of 152 MB in bf16: 78 us against 81).
// HBM's bound: 402M fp32 gradients (1.6 GB) read twice and written once in 731 us, 6.6 TB/s.  Chunks of 16 KiB and twice
// the CTAs 747, a CTA for each chunk in the second launch 869, five CTAs an SM there 753, stores that stay in L2 737.
// 1024 tensors of 65536 fp32 values 132 us in a graph, one of as many values 128; 2500 of 26840 (three launches of either
// kernel) 160.  An output whose address differs from the input's modulo 16 is written by single values: 67M bf16 values
// 230 us against 64, fp32 278 against 128.
#include "expert_internal.cuh"

namespace moe {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kThreads = 256;
constexpr int kChunkBytes = 32 * 1024;
constexpr int kVectors = kChunkBytes / 16 / kThreads;     // 16-byte loads of a thread in a whole chunk
constexpr int kFew = 128, kMany = 1024;                   // tensors of a launch: less than 4 or 32 KB of arguments

template <int kN>
struct Table {
    int n;
    int first[kN + 1];            // first chunk of each tensor
    const uint8_t *src[kN];
    uint8_t *dst[kN];
    int64_t bytes[kN];            // twice the tensor's bytes, plus 1 where it is bf16
};

struct Chunk {
    const uint8_t *src;
    uint8_t *dst;
    int bytes;
    bool bf16;
};

template <int kN>
__device__ __forceinline__ Chunk find(const Table<kN> &t, int chunk)
{
    int lo = 0, hi = t.n;         // first[lo] <= chunk < first[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (t.first[mid] <= chunk)
            lo = mid;
        else
            hi = mid;
    }
    const int64_t at = static_cast<int64_t>(chunk - t.first[lo]) * kChunkBytes, left = (t.bytes[lo] >> 1) - at;
    Chunk c;
    c.src = t.src[lo] + at;
    c.dst = t.dst[lo] + at;
    c.bytes = left < kChunkBytes ? static_cast<int>(left) : kChunkBytes;
    c.bf16 = t.bytes[lo] & 1;
    return c;
}

__device__ __forceinline__ float load_one(const uint8_t *p, bool bf16)
{
    return bf16 ? __uint_as_float(static_cast<uint32_t>(*reinterpret_cast<const uint16_t *>(p)) << 16)
                : *reinterpret_cast<const float *>(p);
}

// A chunk is `head` bytes up to the first 16-byte boundary, whole vectors, and the rest.
struct Cut {
    int head, vectors, tail;      // bytes, 16 bytes, bytes
    __device__ __forceinline__ explicit Cut(const Chunk &c)
    {
        head = static_cast<int>(-reinterpret_cast<uintptr_t>(c.src) & 15);
        head = head < c.bytes ? head : c.bytes;
        vectors = (c.bytes - head) >> 4;
        tail = c.bytes - head - vectors * 16;
    }
};

// Squares of up to eight values a vector: their 32-bit sum, and the largest magnitude (NaNs left out of it).
__device__ __forceinline__ void squares(const uint4 &v, bool bf16, float &sum, float &most)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = __uint_as_float(bf16 ? w[i] << 16 : w[i]);
        sum = fmaf(a, a, sum);
        most = fmaxf(most, fabsf(a));
        if (bf16) {
            const float b = __uint_as_float(w[i] & 0xFFFF0000u);
            sum = fmaf(b, b, sum);
            most = fmaxf(most, fabsf(b));
        }
    }
}
__device__ __forceinline__ double squares64(const uint4 &v, bool bf16)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    double sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const double a = __uint_as_float(bf16 ? w[i] << 16 : w[i]);
        sum += a * a;
        if (bf16) {
            const double b = __uint_as_float(w[i] & 0xFFFF0000u);
            sum += b * b;
        }
    }
    return sum;
}

// The sum over the CTA, in thread 0.
__device__ __forceinline__ double block_sum(double v, double *part)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0;
    if (threadIdx.x == 0)
        for (int i = 0; i < kThreads / 32; ++i) v += part[i];
    return v;
}

template <int kN>
__global__ void __launch_bounds__(kThreads) grad_squares_kernel(const __grid_constant__ Table<kN> t, double *sums)
{
    __shared__ double part[kThreads / 32];
    pdl_launch_dependents();
    double total = 0;
    for (int i = blockIdx.x; i < t.first[t.n]; i += gridDim.x) {
        const Chunk c = find(t, i);
        const Cut cut(c);
        const uint4 *src = reinterpret_cast<const uint4 *>(c.src + cut.head);
        uint4 v[kVectors];
#pragma unroll
        for (int k = 0; k < kVectors; ++k) {
            const int at = threadIdx.x + k * kThreads;
            v[k] = at < cut.vectors ? __ldg(src + at) : make_uint4(0, 0, 0, 0);
        }
        float sum = 0.f, most = 0.f;
        // the ends, one value a thread
        const int shift = c.bf16 ? 1 : 2, before = cut.head >> shift, ends = before + (cut.tail >> shift);
        float one = 0.f;
        if (static_cast<int>(threadIdx.x) < ends) {
            const int at = threadIdx.x << shift;
            one = load_one(c.src + (at < cut.head ? at : at + cut.vectors * 16), c.bf16);
            sum = one * one;
            most = fabsf(one);
            if (one != one) most = 0.f;
        }
#pragma unroll
        for (int k = 0; k < kVectors; ++k) squares(v[k], c.bf16, sum, most);
        // 2^60 squared 64 times stays below 2^127; 64 squares next to one of 2^-100, each off by at most the 2^-150 of
        // the smallest subnormal's half, are off by 2^-44 of it
        if ((most < 0x1p60f && most > 0x1p-50f) || most == 0.f) {
            total += sum;
        } else {
            total += static_cast<double>(one) * one;
#pragma unroll 1
            for (int k = 0; k < kVectors; ++k) {
                const int at = threadIdx.x + k * kThreads;
                if (at < cut.vectors) total += squares64(__ldg(src + at), c.bf16);
            }
        }
    }
    total = block_sum(total, part);
    if (threadIdx.x == 0) sums[blockIdx.x] = total;
}

// The norm of the sums, in thread 0.
__device__ __forceinline__ double norm_of(const double *sums, int n, double *part)
{
    double v = 0;
    for (int i = threadIdx.x; i < n; i += kThreads) v += sums[i];
    return sqrt(block_sum(v, part));
}

__global__ void __launch_bounds__(kThreads) grad_norm_kernel(const double *sums, int n, float *norm)
{
    __shared__ double part[kThreads / 32];
    pdl_wait_prior_grids();
    const double v = norm_of(sums, n, part);
    if (threadIdx.x == 0) *norm = static_cast<float>(v);
}

__device__ __forceinline__ uint4 scaled(const uint4 &v, bool bf16, float c)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (bf16) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(w[i] << 16) * c, __uint_as_float(w[i] & 0xFFFF0000u) * c);
            r[i] = *reinterpret_cast<const uint32_t *>(&h);
        } else {
            r[i] = __float_as_uint(__uint_as_float(w[i]) * c);
        }
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

__device__ __forceinline__ void store_one(uint8_t *p, bool bf16, float v)
{
    if (bf16)
        *reinterpret_cast<__nv_bfloat16 *>(p) = __float2bfloat16_rn(v);
    else
        *reinterpret_cast<float *>(p) = v;
}

// (No pointer is declared restrict: a tensor may be scaled in place.)
template <int kN>
__global__ void __launch_bounds__(kThreads)
    grad_scale_kernel(const __grid_constant__ Table<kN> t, const double *sums, int n, double max_norm, float *norm)
{
    __shared__ double part[kThreads / 32];
    __shared__ float by;
    pdl_wait_prior_grids();
    const double v = norm_of(sums, n, part);
    if (threadIdx.x == 0) {
        const double c = max_norm / (v + 1e-6);
        // a norm that is no finite number leaves the tensors as they are, and what decides is the norm that the caller sees
        const float seen = static_cast<float>(v);
        by = c < 1 && seen <= 3.402823466e38f ? static_cast<float>(c) : 1.f;
        if (norm && blockIdx.x == 0) *norm = seen;
    }
    __syncthreads();
    const float c = by;
    for (int i = t.first[t.n] - 1 - static_cast<int>(blockIdx.x); i >= 0; i -= gridDim.x) {
        const Chunk k = find(t, i);
        if (c == 1.f && k.src == k.dst) continue;
        const int shift = k.bf16 ? 1 : 2;
        if ((reinterpret_cast<uintptr_t>(k.src) ^ reinterpret_cast<uintptr_t>(k.dst)) & 15) {
            for (int at = threadIdx.x << shift; at < k.bytes; at += kThreads << shift)
                store_one(k.dst + at, k.bf16, load_one(k.src + at, k.bf16) * c);
            continue;
        }
        const Cut cut(k);
        const uint4 *src = reinterpret_cast<const uint4 *>(k.src + cut.head);
        uint4 *dst = reinterpret_cast<uint4 *>(k.dst + cut.head);
        uint4 x[kVectors];
#pragma unroll
        for (int j = 0; j < kVectors; ++j) {
            const int at = threadIdx.x + j * kThreads;
            if (at < cut.vectors) x[j] = __ldcs(src + at);
        }
        const int ends = (cut.head + cut.tail) >> shift;
        if (static_cast<int>(threadIdx.x) < ends) {
            int at = threadIdx.x << shift;
            if (at >= cut.head) at += cut.vectors * 16;
            store_one(k.dst + at, k.bf16, load_one(k.src + at, k.bf16) * c);
        }
#pragma unroll
        for (int j = 0; j < kVectors; ++j) {
            const int at = threadIdx.x + j * kThreads;
            if (at < cut.vectors) __stcs(dst + at, scaled(x[j], k.bf16, c));
        }
    }
}

int resident(int dev) { return device_sm_count(dev) * 4 < kGradNormCtas ? device_sm_count(dev) * 4 : kGradNormCtas; }

// Part of the list that fits a launch, from tensor `from`: its chunks (below 2^30, as all tensors together are at
// most 2^44 bytes), and where the next part begins.
template <int kN>
int fill(Table<kN> &t, const GradArgs &a, int from, int &next)
{
    int64_t chunks = 0;
    int n = 0, i = from;
    for (; i < a.n && n < kN; ++i) {
        const int64_t bytes = a.sizes[i] * (a.types[i] == MOE_GRAD_BF16 ? 2 : 4);
        const int64_t more = (bytes + kChunkBytes - 1) / kChunkBytes;
        if (more == 0) continue;
        t.first[n] = static_cast<int>(chunks);
        t.src[n] = static_cast<const uint8_t *>(a.grads[i]);
        t.dst[n] = a.out ? static_cast<uint8_t *>(a.out[i]) : const_cast<uint8_t *>(t.src[n]);
        t.bytes[n] = 2 * bytes + (a.types[i] == MOE_GRAD_BF16);
        chunks += more;
        ++n;
    }
    t.n = n;
    t.first[n] = static_cast<int>(chunks);
    next = i;
    return static_cast<int>(chunks);
}

template <int kN>
cudaError_t run(const GradArgs &a, int dev, cudaStream_t stream)
{
    Table<kN> t;
    const int most = resident(dev);
    double *sums = static_cast<double *>(a.workspace);
    int total = 0;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaError_t err;
    int chunks = 0;
    for (int from = 0; from < a.n;) {
        chunks = fill(t, a, from, from);
        if (chunks == 0) continue;
        const int grid = chunks < most ? chunks : most;
        // (not a programmatic launch: what is before it in the stream may write the gradients)
        cfg.gridDim = dim3(grid);
        err = cudaLaunchKernelEx(&cfg, grad_squares_kernel<kN>, t, sums + total);
        if (err != cudaSuccess) return err;
        total += grid;
    }
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (!a.clip || total == 0) {
        cfg.gridDim = dim3(1);
        return cudaLaunchKernelEx(&cfg, grad_norm_kernel, static_cast<const double *>(sums), total, a.norm);
    }
    float *norm = a.norm;
    for (int from = 0; from < a.n;) {
        if (a.n <= kN)
            from = a.n;                    // the one part is still in the table
        else
            chunks = fill(t, a, from, from);
        if (chunks == 0) continue;
        cfg.gridDim = dim3(chunks < most ? chunks : most);
        err = cudaLaunchKernelEx(&cfg, grad_scale_kernel<kN>, t, static_cast<const double *>(sums), total, a.max_norm, norm);
        if (err != cudaSuccess) return err;
        norm = nullptr;
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_grad_norm(const GradArgs &a, cudaStream_t stream)
{
    int dev = 0;
    const cudaError_t err = expert_device(&dev);
    if (err != cudaSuccess) return err;
    return a.n <= kFew ? run<kFew>(a, dev, stream) : run<kMany>(a, dev, stream);
}

size_t grad_norm_workspace_bytes(int n)
{
    // a sum for each CTA of each launch
    return static_cast<size_t>(n <= kFew ? 1 : (n - 1) / kMany + 1) * kGradNormCtas * sizeof(double);
}

}  // namespace moe
