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
// W2); the units of all touched experts (but the last fifth, where there are many) are
// split evenly and in order over the CTAs, and a CTA's over its sixteen warps.  Each of those is on its own: it copies its
// units in pieces of 16 rows x 256 bytes to a ring of three in shared memory (TMA,
// W1's and then W2's without a pause between: they need only the routing, so that W2
// is in flight while the CTAs wait for each other between the products), multiplies a
// piece by the tokens of its expert (mma.sync, 16 rows x 8 tokens, the codes as f16:
// the tensor work is far below the stream's time), applies each 128-block's scales in
// fp32, and holds a unit's whole reduction in its registers: no sum crosses warps but
// those of shared units (two halves, added in order), none depends on timing.
//
// Phases, with grid barriers where marked:
//   logits of row slices of W_gate, x to E4M3 | top-K, one CTA per token | lists of
//   each expert's tokens; W1 units, the activation in fp32, and by whoever completes
//   a 128-block its E4M3 form | W2 units | weighted sum.
//
// Measured, H = 2048, I = 1024, 128 experts, top 8: 64 tokens 166 us (795 MB, 4.8 TB/s).  Without the tensor work
// it takes 6 us less: what bounds it is the stream (5.5 TB/s while it runs), 17 us before the
// first weight is asked for, and some 6 us at each product's end.  One token 35 us for 51 MB: the phases one after
// the other, each some microseconds of first-touch latency, 9.5 of them before the first weight.  (W1's first
// 32 to 96 MB asked into L2 at the start, before the routing is known: 2 to 6 us slower; the routing's own loads
// and barriers then wait behind them.)
#include "expert_internal.cuh"

namespace moe {
namespace {

constexpr int kMaxN = 64, kMaxE = 256, kMaxK = 16;
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kWide = 256;                    // reduction bytes of a row in one ring stage: two 128-blocks
constexpr int kPieceBlocks = kWide / 128;
constexpr int kStages = 3;                    // of each streaming warp
constexpr int kStageBytes = 16 * kWide;
constexpr int kTaken = 8;                     // units (and ends of products) that a warp may be ahead of its work
constexpr int kRingBytes = kWarps * kStages * kStageBytes;
constexpr int kMostBlocks = 256;              // 128-blocks of the activation that a CTA counts for itself
// An expert's tokens are taken 8 at a time, each lot as an entry of its own: a second one reads the expert's
// weights again, from L2.  (Lots of 16 made some units twice as long as others: 299 us where lots of 8 took 207,
// for 64 tokens on 128 experts, top 8.)
constexpr int kLot = 8;
constexpr int kMostLots = kMaxE + kMaxN * kMaxK / kLot;
// The last units of a product are common: a CTA that is done with its own takes one after the other, as some get
// a fifth less of the memory's rate than others (64 tokens as above: 169 us, 180 without, 173 with an eighth or
// a half common).  With fewer than four units for each warp it does not pay (10 tokens: 115 us, 111 without).
constexpr int kPoolRounds = 4, kPoolShare = 5;
constexpr int kRedundant = 2;                 // up to this many tokens every CTA finds their top-K itself

struct Header {                               // zero before the first call, left zero by every call
    unsigned barrier[4], done, aborted;
    unsigned pool[2];                         // how many of each product's common units are taken
};

struct Smem {
    uint64_t full[kWarps][kStages];
    int abort;
    int active;                               // lots of all touched experts
    int units[2];                             // of each product
    int pool_from[2];                         // those from here on are common to the CTAs
    int unit_from[2], unit_to[2];             // those that this CTA has of its own
    int shared[2];                            // whether two warps share each of them, a half of its reduction each
    int next[2];                              // the first of its own that no warp has taken
    int taken[kWarps][kTaken];                // each warp's, in order, `units` behind a product's last
    union {
        struct {
            uint32_t mask[kMaxE][2];          // tokens of each expert
            float logit[kMaxE];
        };
        float4 half[kWarps / 2][32];          // (once the lists stand) the second halves of shared units' sums
    };
    int16_t expert[kMostLots];                // of each lot, ascending
    int16_t first[kMostLots + 1];             // where its slots start
    int16_t idx[kRedundant * kMaxK];          // the top-K ids where every CTA has found them
    int16_t slot[kMaxN * kMaxK];              // slots n * K + k by expert, then token
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

// Bytes of a row's scales in the workspace: whole pairs, one for each ring stage.
__host__ __device__ inline int scale_stride(int n) { return ((n / 128) + 1) & ~1; }

Layout make_layout(int N, int H, int I, int E, int K)
{
    const size_t S = (H + slice_rows(H) - 1) / slice_rows(H), slots = static_cast<size_t>(N) * K;
    Layout l;
    l.counters = 256;
    l.x8 = up256(l.counters + static_cast<size_t>(E + kMaxN * kMaxK / kLot) * (I / 128) * 4);
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
struct Maps {
    CUtensorMap w1, w2;                       // boxes of 2 x 8 rows (gate, up) and of 16 rows, x 256 bytes
};

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

// d += 16 rows x 8 tokens over 64 of the reduction: a lane's 16 codes of rows g and g + 8 and of token g, as
// f16, which holds every E4M3 value, four at a time.  Which k a lane's codes stand for is the same on both
// sides.  (mma.sync on the codes themselves took 150 cycles for each 32 of k, three times as long.)
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t (&h)[2])
{
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(h[0]), "=r"(h[1])
        : "r"(w));
}
__device__ __forceinline__ void mma_codes(float (&d)[4], uint32_t lo, uint32_t hi, uint32_t tok)
{
    uint32_t a[2], b[2], t[2];
    codes_to_f16(lo, a);
    codes_to_f16(hi, b);
    codes_to_f16(tok, t);
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(b[0]), "r"(a[1]), "r"(b[1]), "r"(t[0]), "r"(t[1]));
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
    const int hx = (hc + 15) & ~15;              // of x in shared memory: whole sixteens
    const int slices = (H + hc - 1) / hc;
    float *part = reinterpret_cast<float *>(static_cast<uint8_t *>(p.a.workspace) + p.l.part);
    const int Er = (E + 31) & ~31, groups = kThreads / Er;
    const int e = t % Er, tg = t / Er;
    for (int s = blockIdx.x; s < slices; s += gridDim.x) {
        const int from = s * hc, rows = H - from < hc ? H - from : hc;   // a multiple of 8
        __syncthreads();
        for (int i = t; i < N * hx; i += kThreads) {
            const int n = i / hx, h = i - n * hx;
            xs[i] = h < rows ? __bfloat162float(static_cast<const __nv_bfloat16 *>(p.a.X)[static_cast<int64_t>(n) * H + from + h])
                             : 0.f;
        }
        __syncthreads();
        if (e >= E || tg >= groups) continue;
        float acc[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) acc[i] = 0.f;
        for (int h = 0; h < rows; h += 16) {
            // (rows come in eights: those that are not there read the last one, against zeros of x)
            float w[16];
#pragma unroll
            for (int i = 0; i < 16; ++i)
                w[i] = __bfloat162float(
                    static_cast<const __nv_bfloat16 *>(p.a.W_gate)[static_cast<int64_t>(from + (h + i < rows ? h + i : rows - 1)) * E + e]);
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const int n = tg + i * groups;
                if (n >= N) break;
#pragma unroll
                for (int j = 0; j < 16; j += 4) {
                    const float4 x = *reinterpret_cast<const float4 *>(xs + n * hx + h + j);
                    acc[i] = fmaf(x.x, w[j], acc[i]);
                    acc[i] = fmaf(x.y, w[j + 1], acc[i]);
                    acc[i] = fmaf(x.z, w[j + 2], acc[i]);
                    acc[i] = fmaf(x.w, w[j + 3], acc[i]);
                }
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

// Top-K of token n from the slices' partial logits.
__device__ void select(const Params &p, int n, Smem &sm, float *scratch)
{
    const int E = p.a.E, N = p.a.N, K = p.a.K, t = threadIdx.x, lane = t & 31;
    const int hc = slice_rows(p.a.H), slices = (p.a.H + hc - 1) / hc;
    const float *part = reinterpret_cast<const float *>(static_cast<const uint8_t *>(p.a.workspace) + p.l.part);
    const int Er = (E + 31) & ~31, groups = kThreads / Er;
    const int e = t % Er, tg = t / Er;
    if (e < E && tg < groups) {
        // sixteen loads in flight, added in order
        float s = 0.f;
        const float *src = part + static_cast<int64_t>(n) * E + e;
        for (int i = tg; i < slices; i += 16 * groups) {
            float v[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const int at = i + j * groups;
                v[j] = __ldcg(src + static_cast<int64_t>(at < slices ? at : slices - 1) * N * E);
            }
#pragma unroll
            for (int j = 0; j < 16; ++j) s += i + j * groups < slices ? v[j] : 0.f;
        }
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
        float first = 0.f, sum = 0.f, my_p = 0.f;
        int my_i = 0;
        // (the order of the values as unsigned numbers: + 0 makes one zero of two, a NaN is -inf already)
        uint32_t key[kMaxE / 32];
#pragma unroll
        for (int i = 0; i < kMaxE / 32; ++i) {
            const uint32_t w = __float_as_uint(v[i] + 0.f);
            key[i] = lane + 32 * i < E ? (w & 0x80000000u ? ~w : w | 0x80000000u) : 0u;
        }
        for (int k = 0; k < K; ++k) {
            uint32_t best = 0;
            int bi = 0x7fffffff;
#pragma unroll
            for (int i = 0; i < kMaxE / 32; ++i)
                if (key[i] > best) {          // (a taken one's key is 0, below that of -inf)
                    best = key[i];
                    bi = lane + 32 * i;
                }
            const uint32_t top = __reduce_max_sync(0xffffffffu, best);
            bi = __reduce_min_sync(0xffffffffu, best == top ? bi : 0x7fffffff);
#pragma unroll
            for (int i = 0; i < kMaxE / 32; ++i)
                if (bi == lane + 32 * i) key[i] = 0;
            const float value = __uint_as_float(top & 0x80000000u ? top & 0x7FFFFFFFu : ~top);
            if (k == 0) first = value;
            if (lane == k) {
                my_p = value;
                my_i = bi;
            }
        }
        my_p = lane < K ? expf(my_p - first) : 0.f;
        sum = my_p;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (!p.a.renorm) {
            sum = 0.f;
#pragma unroll
            for (int i = 0; i < kMaxE / 32; ++i)
                if (v[i] != -INFINITY) sum += expf(v[i] - first);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        }
        if (lane < K) {
            if (N <= kRedundant) sm.idx[n * K + lane] = static_cast<int16_t>(my_i);
            if (N > kRedundant || blockIdx.x == 0) {
                p.a.topk_idx[n * K + lane] = my_i;
                p.a.topk_w[n * K + lane] = my_p / sum;
            }
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
        e[i] = s >= slots ? -1 : p.a.N <= kRedundant ? sm.idx[s] : __ldcg(p.a.topk_idx + s);
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
            const int lots = (c + kLot - 1) / kLot;
            int sum = c | lots << 16;               // both scans in one
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += y;
            }
            const int start = before + (sum & 0xFFFF) - c, at = active + (sum >> 16) - lots;
            for (int i = 0; i < lots; ++i) {
                sm.expert[at + i] = static_cast<int16_t>(x);
                sm.first[at + i] = static_cast<int16_t>(start + i * kLot);
            }
            if (x < E) sm.logit[x] = __int_as_float(start);   // where this expert's slots start
            sum = __shfl_sync(0xffffffffu, sum, 31);
            active += sum >> 16;
            before += sum & 0xFFFF;
        }
        if (lane == 0) {
            sm.active = active;
            sm.first[active] = static_cast<int16_t>(before);
        }
        if (lane < 2) {
            // (below 2^31: at most 384 lots of 8192 units, and some hundreds of CTAs)
            const unsigned units = active * (lane == 0 ? p.a.I / 8 : p.a.H / 16), ctas = gridDim.x;
            const unsigned total = units < ctas * kWarps * kPoolRounds ? units : units - units / kPoolShare;
            sm.units[lane] = units;
            sm.pool_from[lane] = total;
            sm.next[lane] = sm.unit_from[lane] = total / ctas * blockIdx.x + total % ctas * blockIdx.x / ctas;
            sm.unit_to[lane] = total / ctas * (blockIdx.x + 1) + total % ctas * (blockIdx.x + 1) / ctas;
            // where no CTA has more than half as many units as warps (one token, top 8 of 128 experts of
            // 2048 x 1024: 33 us, 41 without)
            sm.shared[lane] = (total + ctas - 1) / ctas * 2 <= kWarps;
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
    }
    __syncthreads();
}

// ---------------------------------------------------------------------------
// The products.  The first: units of 8 gate + 8 up rows of W1, tokens from x8; the
// second: of 16 rows of W2, slots from a8.
// ---------------------------------------------------------------------------
// Where the second half of a shared unit starts: whole pieces.
__device__ __forceinline__ int middle(int red) { return ((red + kWide - 1) / kWide + 1) / 2 * kWide; }

// What the warp asks for next: first W1's pieces, then W2's.  A piece is one TMA box: 8 gate and 8 up rows, or
// 16 rows, of 256 bytes.
// (As one bulk copy per row, issued by sixteen lanes, asking took 1300 cycles a piece, as eight asynchronous
// 16-byte copies per lane 400 to 750: more than the work on the piece.)
struct Stream {
    uint8_t *ring;
    uint64_t *full;
    uint32_t asked, place;        // pieces asked for, and the ring's place for the next
    uint32_t done, phase;         // the place of the next piece to work on, and its phase
    bool ok;                      // no wait has run out; then nothing more is asked for
    int product, k, red, per;
    int from, to;                 // the part of a row that this warp takes
    int row, outer;               // the box's first row, and its expert (for W1: gate half)
    uint32_t taken, worked;       // units (and ends) taken, and worked on

    // The next unit: whichever of the CTA's no warp has taken yet (a fixed share for each warp left some
    // with a seventh unit where others had six).  Behind a product's last, its end is noted and the next
    // product entered; a half without pieces is only noted.
    __device__ __forceinline__ void take(const Params &p, Smem &sm, int warp, int lane, bool enter)
    {
        while (product < 2) {
            if (enter) {
                red = product == 0 ? p.a.H : p.a.I;
                per = product == 0 ? p.a.I / 8 : p.a.H / 16;
                const bool shared = sm.shared[product] != 0;
                from = shared && (warp & 1) ? middle(red) : 0;
                to = shared && !(warp & 1) && middle(red) < red ? middle(red) : red;
            }
            const int end = sm.units[product];
            int u = end;
            if (!sm.shared[product]) {
                if (lane == 0) {
                    u = atomicAdd(&sm.next[product], 1);
                    if (u >= sm.unit_to[product]) {
                        u = sm.pool_from[product];
                        if (u < end) u += atomicAdd(&static_cast<Header *>(p.a.workspace)->pool[product], 1u);
                        u = u < end ? u : end;
                    }
                }
                u = __shfl_sync(0xffffffffu, u, 0);
            } else if (enter && sm.unit_from[product] + (warp >> 1) < sm.unit_to[product]) {
                u = sm.unit_from[product] + (warp >> 1);    // (at most one)
            }
            if (lane == 0) sm.taken[warp][taken % kTaken] = u;
            ++taken;
            enter = u == end;
            if (enter) {
                ++product;
                continue;
            }
            if (from >= to) continue;
            const int lot = static_cast<unsigned>(u) / static_cast<unsigned>(per), i = u - lot * per, e = sm.expert[lot];
            row = product == 0 ? i * 8 : i * 16;
            outer = product == 0 ? 2 * e : e;
            break;
        }
        k = from;
        __syncwarp();
    }
    __device__ __forceinline__ void ask(const Params &p, const Maps &maps, Smem &sm, int warp, int lane)
    {
        if (product == 2) return;
        if (ok && elect_one()) {
            mbar_arrive_expect_tx(full + place, kStageBytes);
            tma_load_3d_plain(ring + place * kStageBytes, product == 0 ? &maps.w1 : &maps.w2, full + place, k, row, outer);
        }
        __syncwarp();
        asked += ok;
        place = place + 1 == kStages ? 0 : place + 1;
        k += kWide;
        if (k >= to) take(p, sm, warp, lane, false);
    }
};

// Eight tokens' side of a piece: a lane's bytes of one of them, the scales of the two whose sums it holds.
struct Tokens {
    uint4 b0[kPieceBlocks], b1[kPieceBlocks];
    uint32_t s0, s1;

    // (no condition on the loads: a block behind the last reads the one before it and is not used)
    __device__ __forceinline__ void load(const uint8_t *src, const uint8_t *sc0, const uint8_t *sc1, int k0, int nb)
    {
#pragma unroll
        for (int b = 0; b < kPieceBlocks; ++b) {
            const uint8_t *at = src + (k0 + (b < nb ? b : 0)) * 128;
            b0[b] = *reinterpret_cast<const uint4 *>(at);
            b1[b] = *reinterpret_cast<const uint4 *>(at + 64);
        }
        s0 = *reinterpret_cast<const uint16_t *>(sc0 + k0);
        s1 = *reinterpret_cast<const uint16_t *>(sc1 + k0);
    }
};

__device__ __forceinline__ void unit_sums(bool first, const LayerArgs &a, Smem &sm, volatile int *abort,
                                          const Maps &maps, Stream &st, const Params &p, int warp, int lane, const uint8_t *src,
                                          const uint8_t *src_scale, int lot, int T, int64_t sc0, int64_t sc1, int from,
                                          int rblocks, bool &bad, float (&acc)[4])
{
    const int red = first ? a.H : a.I, stride = scale_stride(red);
    const int g = lane >> 2, t4 = lane & 3;
    const void *W_scale = first ? a.W1_scale : a.W2_scale;
    const int16_t *slots = sm.slot + sm.first[lot];
    auto who = [&](int col) { return first ? slots[col] / a.K : slots[col]; };
    // (places without a token take the lot's first one's: no sum crosses columns, and theirs goes nowhere)
    const uint8_t *tok = src + static_cast<int64_t>(who(g < T ? g : 0)) * red + t4 * 16;
    const uint8_t *ts0 = src_scale + who(t4 * 2 < T ? t4 * 2 : 0) * stride;
    const uint8_t *ts1 = src_scale + who(t4 * 2 + 1 < T ? t4 * 2 + 1 : 0) * stride;
#pragma unroll
    for (int x = 0; x < 4; ++x) acc[x] = 0.f;
    float sw0 = 0.f, sw1 = 0.f;                      // scales of block (32 at a time) + lane
    const int lo_at = g * kWide + t4 * 16, hi_at = lo_at + 8 * kWide;
    // one piece, blocks k0 on, by the tokens `x`; those of the next piece are on their way meanwhile
    auto step = [&](const Tokens &x, Tokens &next, int k0) {
        const int nb = rblocks - k0;
        if (nb > kPieceBlocks) next.load(tok, ts0, ts1, k0 + kPieceBlocks, nb - kPieceBlocks);
        if ((k0 & 31) == 0 || k0 == from) {
            const int at = (k0 & ~31) + lane, b = at < rblocks ? at : rblocks - 1;
            sw0 = scale_value(load_scale_byte(W_scale, a.ue8m0, sc0 + b, bad));
            sw1 = first ? scale_value(load_scale_byte(W_scale, a.ue8m0, sc1 + b, bad)) : sw0;
        }
        st.ok = st.ok && warp_wait(st.full + st.done, st.phase, abort);
        const uint8_t *stage = st.ring + st.done * kStageBytes;
#pragma unroll
        for (int b = 0; b < kPieceBlocks; ++b) {
            if (b >= nb) break;
            const uint4 lo0 = *reinterpret_cast<const uint4 *>(stage + lo_at + b * 128);
            const uint4 lo1 = *reinterpret_cast<const uint4 *>(stage + lo_at + b * 128 + 64);
            const uint4 hi0 = *reinterpret_cast<const uint4 *>(stage + hi_at + b * 128);
            const uint4 hi1 = *reinterpret_cast<const uint4 *>(stage + hi_at + b * 128 + 64);
            const float w0 = __shfl_sync(0xffffffffu, sw0, (k0 + b) & 31), w1 = __shfl_sync(0xffffffffu, sw1, (k0 + b) & 31);
            // eight K = 16 steps in two chains
            float d[4] = {0.f, 0.f, 0.f, 0.f}, f[4] = {0.f, 0.f, 0.f, 0.f};
            mma_codes(d, lo0.x, hi0.x, x.b0[b].x);
            mma_codes(f, lo1.x, hi1.x, x.b1[b].x);
            mma_codes(d, lo0.y, hi0.y, x.b0[b].y);
            mma_codes(f, lo1.y, hi1.y, x.b1[b].y);
            mma_codes(d, lo0.z, hi0.z, x.b0[b].z);
            mma_codes(f, lo1.z, hi1.z, x.b1[b].z);
            mma_codes(d, lo0.w, hi0.w, x.b0[b].w);
            mma_codes(f, lo1.w, hi1.w, x.b1[b].w);
            // (the tokens' scales are this kernel's own: bytes 105 to 254)
            const float x0 = __uint_as_float((x.s0 >> (8 * b) & 0xFFu) << 23), x1 = __uint_as_float((x.s1 >> (8 * b) & 0xFFu) << 23);
            acc[0] = fmaf(d[0] + f[0], w0 * x0, acc[0]);
            acc[1] = fmaf(d[1] + f[1], w0 * x1, acc[1]);
            acc[2] = fmaf(d[2] + f[2], w1 * x0, acc[2]);
            acc[3] = fmaf(d[3] + f[3], w1 * x1, acc[3]);
        }
        __syncwarp();                                // all lanes have read the stage
        st.done = st.done + 1 == kStages ? 0 : st.done + 1;
        st.phase ^= st.done == 0;
        st.ask(p, maps, sm, warp, lane);
    };
    Tokens x, y;
    if (from < rblocks) x.load(tok, ts0, ts1, from, rblocks - from);
    for (int k0 = from; k0 < rblocks; k0 += 2 * kPieceBlocks) {
        step(x, y, k0);
        if (k0 + kPieceBlocks < rblocks) step(y, x, k0 + kPieceBlocks);
    }
}

// A unit's sums to where they go: the activation of its 8 features, or 16 elements of y.  (The approximate exponential
// is some |gate| 2^-24 off, as its argument is scaled in 32 bits; the activation is then rounded to E4M3.)
__device__ __forceinline__ void unit_out(bool first, const LayerArgs &a, const Smem &sm, float *dst, int lot, int i, int T, int lane,
                                         const float (&acc)[4])
{
    const int g = lane >> 2, t4 = lane & 3;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int col = t4 * 2 + x;
        if (col >= T) continue;
        const int64_t slot = sm.slot[sm.first[lot] + col];
        if (first) {
            const float gate = acc[x], up = acc[2 + x];
            __stcg(dst + slot * a.I + i * 8 + g, gate / (1.f + __expf(-gate)) * up);
        } else {
            __stcg(dst + slot * a.H + i * 16 + g, acc[x]);
            __stcg(dst + slot * a.H + i * 16 + 8 + g, acc[2 + x]);
        }
    }
}

// (One body for both products, so that the second finds its code in the instruction cache: with a few units
// for each warp, code that runs for the first time is what takes the time.)
__device__ __forceinline__ void product(bool first, const Params &p, const Maps &maps, Smem &sm, Stream &st)
{
    const LayerArgs &a = p.a;
    uint8_t *ws = static_cast<uint8_t *>(a.workspace);
    const int rblocks = (first ? a.H : a.I) / 128;
    const int per = first ? a.I / 8 : a.H / 16;      // units of a lot
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint8_t *src = ws + (first ? p.l.x8 : p.l.a8), *src_scale = ws + (first ? p.l.xs : p.l.as);
    float *act = reinterpret_cast<float *>(ws + p.l.a);
    float *dst = first ? act : reinterpret_cast<float *>(ws + p.l.y);
    const int from = sm.unit_from[first ? 0 : 1], to = sm.unit_to[first ? 0 : 1], end = sm.units[first ? 0 : 1];
    bool bad = false;
    const bool shared = sm.shared[first ? 0 : 1] != 0;
    const int mid = middle(rblocks * 128) / 128;
    const int k_from = shared && (warp & 1) ? mid : 0, k_to = shared && !(warp & 1) && mid < rblocks ? mid : rblocks;
    for (;;) {
        const int u = sm.taken[warp][st.worked % kTaken];
        ++st.worked;
        if (u == end) break;
        const int lot = static_cast<unsigned>(u) / static_cast<unsigned>(per), i = u - lot * per;
        const int e = sm.expert[lot], T = sm.first[lot + 1] - sm.first[lot];
        // where the scales of the unit's rows start; gate and up rows lie in different blocks
        const int64_t sc0 = first ? (static_cast<int64_t>(e) * (2 * a.I / 128) + i / 16) * rblocks
                                  : (static_cast<int64_t>(e) * (a.H / 128) + i / 8) * rblocks;
        const int64_t sc1 = first ? sc0 + static_cast<int64_t>(a.I / 128) * rblocks : sc0;
        float acc[4];
        unit_sums(first, a, sm, &sm.abort, maps, st, p, warp, lane, src, src_scale, lot, T, sc0, sc1, k_from, k_to,
                         bad, acc);
        if (shared) {
            // (a warp has at most one shared unit of a product)
            if (warp & 1) sm.half[warp >> 1][lane] = make_float4(acc[0], acc[1], acc[2], acc[3]);
            named_barrier_sync(1 + (warp >> 1), 64);
            if (warp & 1) continue;
            const float4 h = sm.half[warp >> 1][lane];
            acc[0] += h.x;
            acc[1] += h.y;
            acc[2] += h.z;
            acc[3] += h.w;
        }
        unit_out(first, a, sm, dst, lot, i, T, lane, acc);
        if (first) {
            // Whoever completes the sixteen units of a 128-block of the activation turns it into E4M3.  The
            // units that this CTA has of its own are counted here, CTAs that share a block meet in the workspace.
            const int b0 = u & ~15, b1 = b0 + 16;   // (a lot's units are whole blocks)
            const int ours = (b1 < to ? b1 : to) - (b0 > from ? b0 : from);
            const int at = (u >> 4) - (from >> 4);
            const bool count_here = u < to && ((to - 1) >> 4) - (from >> 4) < kMostBlocks;
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
                const int16_t *slots = sm.slot + sm.first[lot];
                float4 v[kLot];
#pragma unroll
                for (int n = 0; n < kLot; ++n)
                    v[n] = __ldcg(reinterpret_cast<const float4 *>(act + static_cast<int64_t>(slots[n < T ? n : 0]) * a.I + b * 128) + lane);
#pragma unroll
                for (int n = 0; n < kLot; ++n) {
                    if (n >= T) break;
                    const int64_t slot = slots[n];
                    const float f[4] = {v[n].x, v[n].y, v[n].z, v[n].w};
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

__global__ void __launch_bounds__(kThreads, 1)
    moe_layer_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Params p)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Smem &sm = *reinterpret_cast<Smem *>(ring + kRingBytes);
    Header *hdr = static_cast<Header *>(p.a.workspace);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kWarps * kStages; ++i) mbar_init(&sm.full[0][0] + i, 1);
        sm.abort = 0;
        fence_mbarrier_init();
        tma_prefetch_desc(&maps.w1);
        tma_prefetch_desc(&maps.w2);
    }
    for (int i = threadIdx.x; i < kMostBlocks; i += kThreads) sm.done[i] = 0;
    __syncthreads();

    float *scratch = reinterpret_cast<float *>(ring);   // the ring is not in use yet
    partial_logits(p, scratch);
    quantise_x(p);
    grid_barrier(hdr, 0, sm);
    // (with few tokens every CTA does what one would, and no barrier is needed behind it)
    const bool redundant = p.a.N <= kRedundant;
    for (int n = redundant ? 0 : blockIdx.x; n < p.a.N; n += redundant ? 1 : gridDim.x) {
        __syncthreads();
        select(p, n, sm, scratch);
    }
    if (redundant)
        __syncthreads();
    else
        grid_barrier(hdr, 1, sm);
    fence_proxy_async_smem();   // the ring's memory passes from these threads to the copies
    make_lists(p, sm);
    Stream st;
    st.asked = st.place = st.done = st.phase = 0;
    st.ring = ring + warp * kStages * kStageBytes;
    st.full = sm.full[warp];
    st.product = 0;
    st.taken = st.worked = 0;
    st.ok = true;
    st.take(p, sm, warp, lane, true);
    for (int i = 0; i < kStages; ++i) st.ask(p, maps, sm, warp, lane);
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
        product(i == 0, p, maps, sm, st);
        grid_barrier(hdr, 2 + i, sm);
    }
    combine(p);
    if (*const_cast<volatile int *>(&sm.abort) != 0) {
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
                for (int i = 0; i < (p.a.E + kMaxN * kMaxK / kLot) * (p.a.I / 128); ++i) counters[i] = 0;
            }
            for (int i = 0; i < 4; ++i) hdr->barrier[i] = 0;
            hdr->pool[0] = hdr->pool[1] = 0;
            hdr->done = 0;
        }
    }
}

}  // namespace

size_t layer_workspace_bytes(int N, int H, int I, int E, int K) { return make_layout(N, H, I, E, K).total; }

cudaError_t launch_layer(const LayerArgs &a, cudaStream_t stream)
{
    int dev = 0;
    cudaError_t err = expert_device(&dev);
    if (err != cudaSuccess) return err;
    static std::atomic<uint64_t> done{0};
    const uint64_t bit = 1ull << (dev & 63);
    if (!(done.load(std::memory_order_relaxed) & bit)) {
        err = cudaFuncSetAttribute(moe_layer_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   static_cast<int>(kSmemBytes));
        if (err != cudaSuccess) return err;
        done.fetch_or(bit, std::memory_order_relaxed);
    }
    Maps maps;
    const uint64_t d1[3] = {static_cast<uint64_t>(a.H), static_cast<uint64_t>(a.I), static_cast<uint64_t>(a.E) * 2};
    const uint64_t d2[3] = {static_cast<uint64_t>(a.I), static_cast<uint64_t>(a.H), static_cast<uint64_t>(a.E)};
    const uint32_t b1[3] = {kWide, 8, 2}, b2[3] = {kWide, 16, 1};
    if (!encode_map(&maps.w1, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.W1, 3, d1, b1, CU_TENSOR_MAP_SWIZZLE_NONE) ||
        !encode_map(&maps.w2, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.W2, 3, d2, b2, CU_TENSOR_MAP_SWIZZLE_NONE))
        return cudaErrorInvalidValue;
    const Params p{a, make_layout(a.N, a.H, a.I, a.E, a.K)};
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
    return cudaLaunchKernelEx(&cfg, moe_layer_kernel, maps, p);
}

}  // namespace moe
