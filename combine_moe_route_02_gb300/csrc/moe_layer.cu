// moe_layer.cu -- a whole mixture-of-experts layer for a few tokens in one
// cooperative launch: router, both products of the chosen experts, combine.
//
//   idx, w = top-K of softmax(X W_gate + bias)          as moe_route
//   g, u   = rows of W1[e] times q(x);  a = silu(g) u   q: E4M3, 1x128 power-of-two scales
//   y      = W2[e] q(a);   out = sum_k w_k y_k (+ residual)
//
// With N <= 64 tokens the time is the weights of the experts that are touched, read
// once; everything else is arranged around that stream.  One CTA per SM.  A unit of
// work is 16 weight rows of one expert (8 gate and 8 up rows of W1, or 16 rows of
// W2); the units of all touched experts are split evenly and in order over the CTAs,
// and a CTA's over its eight streaming warps.  Each of those is on its own: it copies
// its units in pieces of 16 rows x 512 bytes to a ring of three in shared memory (bulk
// copies, W1's and then W2's without a pause between: they need only the routing, so
// that W2 is in flight while the CTAs wait for each other between the products),
// multiplies a piece by the tokens of its expert (mma.sync, 16 rows x 8 tokens x 32:
// the tensor work is far below the stream's time, so the registers' path costs
// nothing), applies each 128-block's scales in fp32, and holds a unit's whole
// reduction in its registers: no sum crosses warps, and none depends on an order.
//
// Phases, with grid barriers where marked:
//   logits of row slices of W_gate, x to E4M3 | top-K, one CTA per token | lists of
//   each expert's tokens; W1 units, the activation in fp32, and by whoever completes
//   a 128-block its E4M3 form | W2 units | weighted sum.
#include "expert_internal.cuh"

namespace moe {
namespace {

constexpr int kMaxN = 64, kMaxE = 256, kMaxK = 16;
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kStreams = 8;                   // streaming warps
constexpr int kWide = 512;                    // reduction bytes of a row in one ring stage: four 128-blocks
constexpr int kRowBytes = kWide + 64;         // 64: eight rows at one offset meet different banks
constexpr int kStages = 3;                    // of each streaming warp
constexpr int kStageBytes = 16 * kRowBytes;
constexpr int kRingBytes = kStreams * kStages * kStageBytes;
constexpr int kMostBlocks = 256;              // 128-blocks of the activation that a CTA counts for itself

struct Header {                               // zero before the first call, left zero by every call
    unsigned barrier[4], done, aborted;
};

struct Smem {
    uint64_t full[kStreams][kStages];
    int abort;
    int active;                               // touched experts
    uint32_t mask[kMaxE][2];                  // tokens of each expert
    int16_t expert[kMaxE];                    // the touched ones, ascending
    int16_t first[kMaxE + 1];                 // where each touched expert's slots start
    int16_t slot[kMaxN * kMaxK];              // slots n * K + k by expert, then token
    int16_t token[kMaxN * kMaxK];             // their n
    float logit[kMaxE];
    int done[kMostBlocks];                    // units that this CTA has done of its 128-blocks
};
constexpr size_t kSmemBytes = 1024 + kRingBytes + sizeof(Smem);
static_assert(kSmemBytes <= 227 * 1024, "shared memory");

struct Layout {                               // byte offsets into the workspace
    size_t counters, x8, xs, part, a, a8, as, y, total;
};

__host__ __device__ inline size_t up256(size_t v) { return (v + 255) & ~size_t(255); }

// Rows of a slice of W_gate: at most 128 slices.
__host__ __device__ inline int slice_rows(int H) { return (((H + 127) / 128) + 7) & ~7; }

// Bytes of a row's scales in the workspace: whole words, one for each ring stage.
__host__ __device__ inline int scale_stride(int n) { return ((n / 128) + 3) & ~3; }

Layout make_layout(int N, int H, int I, int E, int K)
{
    const size_t S = (H + slice_rows(H) - 1) / slice_rows(H), slots = static_cast<size_t>(N) * K;
    Layout l;
    l.counters = 256;
    l.x8 = up256(l.counters + static_cast<size_t>(E) * (I / 128) * 4);
    l.xs = up256(l.x8 + static_cast<size_t>(N) * H);
    l.part = up256(l.xs + static_cast<size_t>(N) * scale_stride(H));
    l.a = up256(l.part + S * N * E * 4);
    l.a8 = up256(l.a + slots * I * 4);
    l.as = up256(l.a8 + slots * I);
    l.y = up256(l.as + slots * scale_stride(I));
    l.total = up256(l.y + slots * H * 4);
    return l;
}

struct Params {
    LayerArgs a;
    Layout l;
};

// Which units of `total` this CTA takes.
__device__ __forceinline__ void my_units(int total, int &from, int &to)
{
    from = static_cast<int>(static_cast<int64_t>(total) * blockIdx.x / gridDim.x);
    to = static_cast<int>(static_cast<int64_t>(total) * (blockIdx.x + 1) / gridDim.x);
}

// All CTAs' threads; what they wrote before is visible to all after.  A CTA that gives up
// goes on through the remaining phases (each wait then ends at once), so that every thread meets
// every barrier and the counters always end complete; its results are then worthless, and the
// status word says so.
__device__ void grid_barrier(Header *h, int which, Smem &sm)
{
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        red_add_release_gpu(&h->barrier[which], 1);
        const uint64_t t0 = globaltimer_ns();
        for (uint32_t it = 1; !*const_cast<volatile int *>(&sm.abort) && ld_acquire_gpu(&h->barrier[which]) < gridDim.x; ++it) {
            if ((it & 63u) == 0 && (ld_acquire_gpu(&h->aborted) || globaltimer_ns() - t0 > kWaitLimitNs)) {
                atomicExch(&h->aborted, 1u);
                sm.abort = 1;
                break;
            }
        }
        __threadfence();
    }
    __syncthreads();
}

__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four values of a 128-block per lane of a warp -> codes; the block's scale byte in every lane.
__device__ __forceinline__ uint32_t quant_warp_block(const float (&f)[4], uint32_t &byte)
{
    float m = fmaxf(fmaxf(fabsf(f[0]), fabsf(f[1])), fmaxf(fabsf(f[2]), fabsf(f[3])));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    byte = block_scale_byte(m);
    const float inv = scale_reciprocal(byte);
    return f32x4_to_e4m3x4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv);
}

// ---------------------------------------------------------------------------
// Router
// ---------------------------------------------------------------------------
__device__ void partial_logits(const Params &p, float *xs)
{
    const int H = p.a.H, E = p.a.E, N = p.a.N, t = threadIdx.x;
    const int hc = slice_rows(H);
    const int slices = (H + hc - 1) / hc;
    float *part = reinterpret_cast<float *>(static_cast<uint8_t *>(p.a.workspace) + p.l.part);
    const int Er = (E + 31) & ~31, groups = kThreads / Er;
    const int e = t % Er, tg = t / Er;
    for (int s = blockIdx.x; s < slices; s += gridDim.x) {
        const int from = s * hc, rows = H - from < hc ? H - from : hc;   // a multiple of 8
        __syncthreads();
        for (int i = t; i < N * rows; i += kThreads) {
            const int n = i / rows, h = i - n * rows;
            xs[n * hc + h] = __bfloat162float(static_cast<const __nv_bfloat16 *>(p.a.X)[static_cast<int64_t>(n) * H + from + h]);
        }
        __syncthreads();
        if (e >= E || tg >= groups) continue;
        float acc[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) acc[i] = 0.f;
        for (int h = 0; h < rows; h += 8) {
            float w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                w[i] = __bfloat162float(static_cast<const __nv_bfloat16 *>(p.a.W_gate)[static_cast<int64_t>(from + h + i) * E + e]);
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const int n = tg + i * groups;
                if (n >= N) break;
                const float4 x0 = *reinterpret_cast<const float4 *>(xs + n * hc + h);
                const float4 x1 = *reinterpret_cast<const float4 *>(xs + n * hc + h + 4);
                float v = acc[i];
                v = fmaf(x0.x, w[0], v);
                v = fmaf(x0.y, w[1], v);
                v = fmaf(x0.z, w[2], v);
                v = fmaf(x0.w, w[3], v);
                v = fmaf(x1.x, w[4], v);
                v = fmaf(x1.y, w[5], v);
                v = fmaf(x1.z, w[6], v);
                acc[i] = fmaf(x1.w, w[7], v);
            }
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const int n = tg + i * groups;
            if (n >= N) break;
            part[(static_cast<int64_t>(s) * N + n) * E + e] = acc[i];
        }
    }
}

// x to E4M3, by the CTAs from the last on (the first ones hold the slices of W_gate).
__device__ void quantise_x(const Params &p)
{
    const int H = p.a.H, blocks = H / 128, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint8_t *x8 = static_cast<uint8_t *>(p.a.workspace) + p.l.x8, *xs = static_cast<uint8_t *>(p.a.workspace) + p.l.xs;
    const int me = gridDim.x - 1 - blockIdx.x;
    const int stride = scale_stride(H);
    for (int i = me * kWarps + warp; i < p.a.N * blocks; i += gridDim.x * kWarps) {
        const uint2 v = *reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(p.a.X) +
                                                         static_cast<int64_t>(i) * 128 + lane * 4);
        const float f[4] = {__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u), __uint_as_float(v.y << 16),
                            __uint_as_float(v.y & 0xFFFF0000u)};
        uint32_t byte;
        const uint32_t q = quant_warp_block(f, byte);
        reinterpret_cast<uint32_t *>(x8)[static_cast<int64_t>(i) * 32 + lane] = q;
        if (lane == 0) xs[(i / blocks) * stride + i % blocks] = static_cast<uint8_t>(byte);
    }
}

__device__ __forceinline__ bool above(float v, int e, float b, int be) { return v > b || (v == b && e < be); }

// Top-K of token n from the slices' partial logits.
__device__ void select(const Params &p, int n, Smem &sm, float *scratch)
{
    const int E = p.a.E, N = p.a.N, K = p.a.K, t = threadIdx.x, lane = t & 31;
    const int hc = slice_rows(p.a.H), slices = (p.a.H + hc - 1) / hc;
    const float *part = reinterpret_cast<const float *>(static_cast<const uint8_t *>(p.a.workspace) + p.l.part);
    const int Er = (E + 31) & ~31, groups = kThreads / Er;
    const int e = t % Er, tg = t / Er;
    if (e < E && tg < groups) {
        float s = 0.f;
#pragma unroll 8
        for (int i = tg; i < slices; i += groups) s += __ldcg(part + (static_cast<int64_t>(i) * N + n) * E + e);
        scratch[tg * Er + e] = s;
    }
    __syncthreads();
    if (t < E) {
        float s = 0.f;
        for (int g = 0; g < groups; ++g) s += scratch[g * Er + t];
        if (p.a.bias) s += p.a.bias[t];
        sm.logit[t] = isnan(s) ? -INFINITY : s;
    }
    __syncthreads();
    if (t < 32) {
        float v[kMaxE / 32];
#pragma unroll
        for (int i = 0; i < kMaxE / 32; ++i) v[i] = lane + 32 * i < E ? sm.logit[lane + 32 * i] : -INFINITY;
        uint32_t taken = 0;
        float first = 0.f, sum = 0.f, my_p = 0.f;
        int my_i = 0;
        for (int k = 0; k < K; ++k) {
            float bv = -INFINITY;
            int bi = 0x7fffffff;
#pragma unroll
            for (int i = 0; i < kMaxE / 32; ++i) {
                const int c = lane + 32 * i;
                if (c < E && !((taken >> i) & 1u) && above(v[i], c, bv, bi)) {
                    bv = v[i];
                    bi = c;
                }
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                const float ov = __shfl_xor_sync(0xffffffffu, bv, o);
                const int oi = __shfl_xor_sync(0xffffffffu, bi, o);
                if (above(ov, oi, bv, bi)) {
                    bv = ov;
                    bi = oi;
                }
            }
            if ((bi & 31) == lane) taken |= 1u << (bi >> 5);
            if (k == 0) first = bv;
            const float pr = expf(bv - first);
            sum += pr;
            if (lane == k) {
                my_p = pr;
                my_i = bi;
            }
        }
        if (!p.a.renorm) {
            sum = 0.f;
#pragma unroll
            for (int i = 0; i < kMaxE / 32; ++i)
                if (v[i] != -INFINITY) sum += expf(v[i] - first);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        }
        if (lane < K) {
            p.a.topk_idx[n * K + lane] = my_i;
            p.a.topk_w[n * K + lane] = my_p / sum;
        }
    }
}

// Each expert's slots, ascending by token (K different experts per token: a bit per token).
__device__ void make_lists(const Params &p, Smem &sm)
{
    const int t = threadIdx.x, lane = t & 31, E = p.a.E, K = p.a.K, slots = p.a.N * K;
    for (int i = t; i < 2 * E; i += kThreads) sm.mask[i >> 1][i & 1] = 0;
    __syncthreads();
    int e[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int s = t + i * kThreads;
        e[i] = s < slots ? __ldcg(p.a.topk_idx + s) : -1;
        if (e[i] < 0 || e[i] >= E) {
            e[i] = -1;   // (ids that are not there: only after a barrier that gave up)
            continue;
        }
        const int n = s / K;
        atomicOr(&sm.mask[e[i]][n >> 5], 1u << (n & 31));
    }
    __syncthreads();
    if (t < 32) {
        int active = 0, before = 0;
        for (int b = 0; b < E; b += 32) {
            const int x = b + lane;
            const int c = x < E ? __popc(sm.mask[x][0]) + __popc(sm.mask[x][1]) : 0;
            const uint32_t some = __ballot_sync(0xffffffffu, c > 0);
            int sum = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += y;
            }
            if (c > 0) {
                const int at = active + __popc(some & ((1u << lane) - 1u));
                sm.expert[at] = static_cast<int16_t>(x);
                sm.first[at] = static_cast<int16_t>(before + sum - c);
            }
            if (x < E) sm.logit[x] = __int_as_float(before + sum - c);   // where this expert's slots start
            active += __popc(some);
            before += __shfl_sync(0xffffffffu, sum, 31);
        }
        if (lane == 0) {
            sm.active = active;
            sm.first[active] = static_cast<int16_t>(before);
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (e[i] < 0) continue;
        const int s = t + i * kThreads, n = s / K;
        const uint32_t m0 = sm.mask[e[i]][0], m1 = sm.mask[e[i]][1];
        const uint32_t below = (1u << (n & 31)) - 1u;
        const int rank = n < 32 ? __popc(m0 & below) : __popc(m0) + __popc(m1 & below);
        const int at = __float_as_int(sm.logit[e[i]]) + rank;
        sm.slot[at] = static_cast<int16_t>(s);
        sm.token[at] = static_cast<int16_t>(n);
    }
    __syncthreads();
}

// ---------------------------------------------------------------------------
// The products.  FIRST: units of 8 gate + 8 up rows of W1, tokens from x8; else 16
// rows of W2, slots from a8.
// ---------------------------------------------------------------------------
// A streaming warp's walk over the pieces of its units, first W1's, then W2's.
struct Pieces {
    int product, u, to, k;        // (product 2: the end)

    __device__ __forceinline__ void enter(const Params &p, const Smem &sm, int warp)
    {
        for (; product < 2; ++product) {
            int from;
            my_units(sm.active * (product == 0 ? p.a.I / 8 : p.a.H / 16), from, to);
            u = from + warp;
            k = 0;
            if (u < to) break;
        }
    }
    __device__ __forceinline__ void next(const Params &p, const Smem &sm, int warp)
    {
        k += kWide;
        if (k < (product == 0 ? p.a.H : p.a.I)) return;
        k = 0;
        u += kStreams;
        if (u < to) return;
        ++product;
        enter(p, sm, warp);
    }
    // Asks for the piece: lane r < 16 its row r.
    __device__ __forceinline__ void copy(const Params &p, const Smem &sm, uint8_t *stage, uint64_t *full, int lane) const
    {
        const LayerArgs &a = p.a;
        const int red = product == 0 ? a.H : a.I, per = product == 0 ? a.I / 8 : a.H / 16;
        const int ai = u / per, i = u - ai * per;
        const int64_t e = sm.expert[ai];
        const int width = red - k < kWide ? red - k : kWide;
        if (lane == 0) mbar_arrive_expect_tx(full, 16 * width);
        __syncwarp();
        if (lane < 16) {
            const uint8_t *row =
                product == 0 ? static_cast<const uint8_t *>(a.W1) + (e * 2 * a.I + (lane & 8 ? a.I : 0) + i * 8 + (lane & 7)) * a.H
                             : static_cast<const uint8_t *>(a.W2) + (e * a.H + i * 16 + lane) * a.I;
            bulk_load(stage + lane * kRowBytes, row + k, width, full);
        }
    }
};

struct Stream {
    uint8_t *ring;
    uint64_t *full;
    Pieces ahead;                 // the next piece to ask for
    uint32_t asked, done;

    __device__ __forceinline__ void ask(const Params &p, const Smem &sm, int warp, int lane)
    {
        if (ahead.product == 2) return;
        const uint32_t s = asked % kStages;
        ahead.copy(p, sm, ring + s * kStageBytes, full + s, lane);
        ahead.next(p, sm, warp);
        ++asked;
    }
};

template <bool FIRST>
__device__ void product(const Params &p, Smem &sm, Stream &st)
{
    const LayerArgs &a = p.a;
    uint8_t *ws = static_cast<uint8_t *>(a.workspace);
    const int red = FIRST ? a.H : a.I, rblocks = red / 128, stride = scale_stride(red);
    const int per = FIRST ? a.I / 8 : a.H / 16;      // units of an expert
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    const uint8_t *src = ws + (FIRST ? p.l.x8 : p.l.a8), *src_scale = ws + (FIRST ? p.l.xs : p.l.as);
    const void *W_scale = FIRST ? a.W1_scale : a.W2_scale;
    float *act = reinterpret_cast<float *>(ws + p.l.a);
    float *y = reinterpret_cast<float *>(ws + p.l.y);
    int from, to;
    my_units(sm.active * per, from, to);
    bool bad = false;
    for (int u = from + warp; u < to; u += kStreams) {
        const int ai = u / per, i = u - ai * per, e = sm.expert[ai];
        const int s0 = sm.first[ai], T = sm.first[ai + 1] - s0, groups = (T + 7) >> 3;
        const int16_t *who = (FIRST ? sm.token : sm.slot) + s0;
        // where the scales of the unit's rows start; gate and up rows lie in different blocks
        const int64_t sc0 = FIRST ? (static_cast<int64_t>(e) * (2 * a.I / 128) + i / 16) * rblocks
                                  : (static_cast<int64_t>(e) * (a.H / 128) + i / 8) * rblocks;
        const int64_t sc1 = FIRST ? sc0 + static_cast<int64_t>(a.I / 128) * rblocks : sc0;
        float acc[8][4];
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int x = 0; x < 4; ++x) acc[j][x] = 0.f;
        float sw0 = 0.f, sw1 = 0.f;                  // of block (32 at a time) + lane
        for (int k0 = 0; k0 < rblocks; k0 += kWide / 128) {
            if ((k0 & 31) == 0) {
                const int b = k0 + lane < rblocks ? k0 + lane : rblocks - 1;
                sw0 = scale_value(load_scale_byte(W_scale, a.ue8m0, sc0 + b, bad));
                sw1 = FIRST ? scale_value(load_scale_byte(W_scale, a.ue8m0, sc1 + b, bad)) : sw0;
            }
            const uint32_t s = st.done % kStages;
            warp_wait(st.full + s, (st.done / kStages) & 1u, &sm.abort);
            const uint8_t *row = st.ring + s * kStageBytes + g * kRowBytes + t4 * 16;
            const int nb = rblocks - k0 < 4 ? rblocks - k0 : 4;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (j >= groups) break;
                // the tokens' side: eight of them, one a lane group; the scales of the two whose sums this
                // lane holds
                const bool mine = j * 8 + g < T;
                const uint8_t *tok = src + static_cast<int64_t>(mine ? who[j * 8 + g] : who[0]) * red + k0 * 128 + t4 * 16;
                uint4 b0[4], b1[4];
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    b0[b] = b1[b] = make_uint4(0, 0, 0, 0);
                    if (mine && b < nb) {
                        b0[b] = *reinterpret_cast<const uint4 *>(tok + b * 128);
                        b1[b] = *reinterpret_cast<const uint4 *>(tok + b * 128 + 64);
                    }
                }
                uint32_t st0 = 0, st1 = 0;
                if (j * 8 + t4 * 2 < T)
                    st0 = *reinterpret_cast<const uint32_t *>(src_scale + who[j * 8 + t4 * 2] * stride + k0);
                if (j * 8 + t4 * 2 + 1 < T)
                    st1 = *reinterpret_cast<const uint32_t *>(src_scale + who[j * 8 + t4 * 2 + 1] * stride + k0);
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    if (b >= nb) break;
                    const uint4 lo0 = *reinterpret_cast<const uint4 *>(row + b * 128);
                    const uint4 lo1 = *reinterpret_cast<const uint4 *>(row + b * 128 + 64);
                    const uint4 hi0 = *reinterpret_cast<const uint4 *>(row + 8 * kRowBytes + b * 128);
                    const uint4 hi1 = *reinterpret_cast<const uint4 *>(row + 8 * kRowBytes + b * 128 + 64);
                    float d[4] = {0.f, 0.f, 0.f, 0.f};
                    // four K = 32 steps; which k a lane's bytes stand for is the same on both sides
                    mma_e4m3(d, lo0.x, hi0.x, lo0.y, hi0.y, b0[b].x, b0[b].y);
                    mma_e4m3(d, lo0.z, hi0.z, lo0.w, hi0.w, b0[b].z, b0[b].w);
                    mma_e4m3(d, lo1.x, hi1.x, lo1.y, hi1.y, b1[b].x, b1[b].y);
                    mma_e4m3(d, lo1.z, hi1.z, lo1.w, hi1.w, b1[b].z, b1[b].w);
                    const float w0 = __shfl_sync(0xffffffffu, sw0, (k0 + b) & 31);
                    const float w1 = FIRST ? __shfl_sync(0xffffffffu, sw1, (k0 + b) & 31) : w0;
                    const float x0 = scale_value((st0 >> (8 * b)) & 0xFFu), x1 = scale_value((st1 >> (8 * b)) & 0xFFu);
                    acc[j][0] = fmaf(d[0], w0 * x0, acc[j][0]);
                    acc[j][1] = fmaf(d[1], w0 * x1, acc[j][1]);
                    acc[j][2] = fmaf(d[2], w1 * x0, acc[j][2]);
                    acc[j][3] = fmaf(d[3], w1 * x1, acc[j][3]);
                }
            }
            __syncwarp();                            // all lanes have read the stage
            ++st.done;
            st.ask(p, sm, warp, lane);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (j >= groups) break;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int col = j * 8 + t4 * 2 + x;
                if (col >= T) continue;
                const int64_t slot = sm.slot[s0 + col];
                if (FIRST) {
                    const float gate = acc[j][x], up = acc[j][2 + x];
                    __stcg(act + slot * a.I + i * 8 + g, gate / (1.f + __expf(-gate)) * up);
                } else {
                    __stcg(y + slot * a.H + i * 16 + g, acc[j][x]);
                    __stcg(y + slot * a.H + i * 16 + 8 + g, acc[j][2 + x]);
                }
            }
        }
        if (FIRST) {
            // Whoever completes the sixteen units of a 128-block of the activation turns it into E4M3.  The
            // units that this CTA has of it are counted here, CTAs that share one meet in the workspace.
            const int b0 = u & ~15, b1 = b0 + 16;    // (an expert's units are whole blocks)
            const int ours = (b1 < to ? b1 : to) - (b0 > from ? b0 : from);
            const int at = (u >> 4) - (from >> 4);
            const bool count_here = ((to - 1) >> 4) - (from >> 4) < kMostBlocks;
            int last = 0;
            __threadfence_block();
            __syncwarp();
            if (lane == 0) {
                const int n = count_here ? ours : 1;
                last = !count_here || atomicAdd(&sm.done[at], 1) == ours - 1;
                if (last && n != 16) {
                    unsigned *counter = reinterpret_cast<unsigned *>(ws + p.l.counters) + (u >> 4);
                    __threadfence();
                    last = atomicAdd(counter, n) + n == 16;
                    if (last) *counter = 0;
                    __threadfence();
                }
                __threadfence_block();
            }
            __syncwarp();
            if (__shfl_sync(0xffffffffu, last, 0)) {
                const int b = i >> 4;
                for (int n = 0; n < T; ++n) {
                    const int64_t slot = sm.slot[s0 + n];
                    const float4 v = __ldcg(reinterpret_cast<const float4 *>(act + slot * a.I + b * 128) + lane);
                    const float f[4] = {v.x, v.y, v.z, v.w};
                    uint32_t byte;
                    const uint32_t q = quant_warp_block(f, byte);
                    __stcg(reinterpret_cast<uint32_t *>(ws + p.l.a8 + slot * a.I + b * 128) + lane, q);
                    if (lane == 0) ws[p.l.as + slot * scale_stride(a.I) + b] = static_cast<uint8_t>(byte);
                }
            }
        }
    }
    if (bad) report_status(a.status, MOE_ERR_BAD_SCALE);
}

__device__ void combine(const Params &p)
{
    const LayerArgs &a = p.a;
    const float *y = reinterpret_cast<const float *>(static_cast<const uint8_t *>(a.workspace) + p.l.y);
    const int quads = a.H / 4;
    const int total = a.N * quads;
    for (int i = blockIdx.x * kThreads + threadIdx.x; i < total; i += gridDim.x * kThreads) {
        const int n = i / quads, h = (i - n * quads) * 4;
        float s[4] = {0.f, 0.f, 0.f, 0.f};
        for (int k = 0; k < a.K; ++k) {
            const float w = __ldcg(a.topk_w + n * a.K + k);
            const float4 v = __ldcg(reinterpret_cast<const float4 *>(y + static_cast<int64_t>(n * a.K + k) * a.H + h));
            s[0] = fmaf(w, v.x, s[0]);
            s[1] = fmaf(w, v.y, s[1]);
            s[2] = fmaf(w, v.z, s[2]);
            s[3] = fmaf(w, v.w, s[3]);
        }
        const int64_t at = static_cast<int64_t>(n) * a.H + h;
        if (a.residual) {
            const uint2 r = *reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(a.residual) + at);
            s[0] += __uint_as_float(r.x << 16);
            s[1] += __uint_as_float(r.x & 0xFFFF0000u);
            s[2] += __uint_as_float(r.y << 16);
            s[3] += __uint_as_float(r.y & 0xFFFF0000u);
        }
        __nv_bfloat162 o[2] = {__floats2bfloat162_rn(s[0], s[1]), __floats2bfloat162_rn(s[2], s[3])};
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) + at) = *reinterpret_cast<uint2 *>(o);
    }
}

__global__ void __launch_bounds__(kThreads, 1) moe_layer_kernel(const Params p)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Smem &sm = *reinterpret_cast<Smem *>(ring + kRingBytes);
    Header *hdr = static_cast<Header *>(p.a.workspace);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStreams * kStages; ++i) mbar_init(&sm.full[0][0] + i, 1);
        sm.abort = 0;
        fence_mbarrier_init();
    }
    for (int i = threadIdx.x; i < kMostBlocks; i += kThreads) sm.done[i] = 0;
    __syncthreads();

    float *scratch = reinterpret_cast<float *>(ring);   // the ring is not in use yet
    partial_logits(p, scratch);
    quantise_x(p);
    grid_barrier(hdr, 0, sm);
    for (int n = blockIdx.x; n < p.a.N; n += gridDim.x) {
        __syncthreads();
        select(p, n, sm, scratch);
    }
    grid_barrier(hdr, 1, sm);
    fence_proxy_async_smem();   // the ring's memory passes from these threads to the copies
    make_lists(p, sm);
    Stream st;
    st.asked = st.done = 0;
    if (warp < kStreams) {
        st.ring = ring + warp * kStages * kStageBytes;
        st.full = sm.full[warp];
        st.ahead.product = 0;
        st.ahead.enter(p, sm, warp);
        for (int i = 0; i < kStages; ++i) st.ask(p, sm, warp, lane);
        product<true>(p, sm, st);
    }
    grid_barrier(hdr, 2, sm);
    if (warp < kStreams) product<false>(p, sm, st);
    grid_barrier(hdr, 3, sm);
    combine(p);
    if (*const_cast<volatile int *>(&sm.abort) != 0 && warp < kStreams) {
        // let the copies in flight land before the CTA ends
        for (uint32_t x = st.asked > kStages ? st.asked - kStages : 0u; x < st.asked; ++x) {
            volatile int no_abort = 0;
            mbar_wait_bounded(st.full + x % kStages, (x / kStages) & 1u, &no_abort);
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        if (sm.abort) report_status(p.a.status, MOE_ERR_TIMEOUT);
        // the last CTA to get here leaves the counters at zero for the next call
        __threadfence();
        if (atomicAdd(&hdr->done, 1u) == gridDim.x - 1) {
            __threadfence();
            if (atomicExch(&hdr->aborted, 0u)) {
                unsigned *counters = reinterpret_cast<unsigned *>(static_cast<uint8_t *>(p.a.workspace) + p.l.counters);
                for (int i = 0; i < p.a.E * (p.a.I / 128); ++i) counters[i] = 0;
            }
            for (int i = 0; i < 4; ++i) hdr->barrier[i] = 0;
            hdr->done = 0;
        }
    }
}

}  // namespace

size_t layer_workspace_bytes(int N, int H, int I, int E, int K) { return make_layout(N, H, I, E, K).total; }

cudaError_t launch_layer(const LayerArgs &a, cudaStream_t stream)
{
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    static std::atomic<uint64_t> done{0};
    const uint64_t bit = 1ull << (dev & 63);
    if (!(done.load(std::memory_order_relaxed) & bit)) {
        err = cudaFuncSetAttribute(moe_layer_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   static_cast<int>(kSmemBytes));
        if (err != cudaSuccess) return err;
        done.fetch_or(bit, std::memory_order_relaxed);
    }
    Params p{a, make_layout(a.N, a.H, a.I, a.E, a.K)};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(device_sm_count(dev));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeCooperative;
    at[0].val.cooperative = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, moe_layer_kernel, p);
}

}  // namespace moe
