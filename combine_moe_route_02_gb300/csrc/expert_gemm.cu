// expert_gemm.cu -- the experts' matrix products in E4M3 with power-of-two block
// scales, over the ragged row groups that the dispatch writes.
//
//   Y[r, m] = sum_k x[r, k] sx[r, k/128] * w[e(r), m, k] sw[e(r), m/128, k/128]
//
// (m over the weight's rows, k over its columns; `transpose` swaps the two, which
// is the product of the input gradient).  Every scale is a power of two, so the
// tensor cores apply them themselves (tcgen05.mma kind::mxf8f6f4.block_scale, one
// UE8M0 byte per row and K = 32 step): no partial sum leaves TMEM before the end
// of the reduction, and the accumulation is fp32 throughout.  (The tensor cores cut where they
// add: positive products came out 1.2e-5 / 5e-5 / 3.3e-4 of their sum too small at a reduction of 2^14 / 2^16 /
// 2^18, the most that is taken, against 3.9e-3 for the half step of the bf16 result.)
//
// The weights sit on the M side of the MMA and the tokens on the N side, whose size
// can be any multiple of 16: a group of c rows is cut into ceil(c / 224) tiles of
// equal size, so that a ragged group pays for at most 15 rows that it does not have.
//
// Persistent CTA pairs (cta_group::2): a tile is 256 output features x up to 224
// tokens, each CTA holds the accumulators of 128 of the features and brings their
// weights and half of the tokens, which halves the token bytes that an SM takes in.
// Warp roles, in each CTA:
//   warp 0      TMA producer (weights 128 x 128, the tokens in one box)
//   warp 1      leader: MMA issuer (one thread), copies the scales to TMEM
//               (tcgen05.cp); other CTA: tells the leader which stages have landed
//   warps 2, 3, 8, 9  scale producers: gather the bytes of 16 128-blocks per row; warp 3
//               allocates TMEM
//   warps 4..7  epilogue: TMEM -> registers -> bf16, transposed through shared memory
//
// Measured (burst, 1.94 GHz): 16384 tokens on 128 experts, top 8, 2048 x 2048: 354 us, 3.1 PFLOP/s, the
// tensor pipe 67% busy; the rest is the latency of a ring that 180 KiB in flight per SM do not quite cover
// (back to back the board's power limit makes it 417 us).  The input gradient of 16381 unevenly routed
// tokens, 64 experts of 1024 x 4096: 122 us against 85 for its bytes.
#include <mutex>

#include "expert_internal.cuh"

namespace moe {
namespace {

constexpr int kTileM = 256;        // output features per tile, half of them in each CTA
constexpr int kHalfM = 128;
constexpr int kTileN = 224;        // most tokens per tile: two accumulators and the scales fit TMEM
constexpr int kBlk = 128;          // reduction block of a scale, and of a ring stage
constexpr int kStages = 6;
constexpr int kScaleSlots = 2;
constexpr int kABytes = kHalfM * kBlk;
constexpr int kBBytes = kTileN / 2 * kBlk;      // half of the tokens
constexpr int kStageBytes = kABytes + kBBytes;
constexpr int kScaleQuadBytes = 512 + 1024;   // four blocks: 128 feature words, 256 token words
constexpr int kScaleSlotBytes = 4 * kScaleQuadBytes;
constexpr int kEpiBytes = 4 * 32 * 64;        // per epilogue warp 32 tokens x 32 features
constexpr int kThreads = 320;
constexpr uint32_t kTmemCols = 512;
// Scales lie behind the two accumulators: 4 + 8 columns for four blocks.  Five places in turn: when one is
// written again its MMAs have completed, those of the tile before the last by the wait for its accumulator,
// nearer ones because at least six blocks of the ring lie between.
constexpr uint32_t kSfCol = 2 * kTileN, kSfCols = 12, kSfPlaces = 5;
static_assert(kSfCol + kSfPlaces * kSfCols <= kTmemCols, "TMEM");
constexpr int kMaxE = 256;

struct Tail {
    uint64_t full[kStages], empty[kStages];
    uint64_t sf_full[kScaleSlots], sf_empty[kScaleSlots];
    uint64_t acc_full[2], acc_empty[2], drain;
    uint32_t tmem_base;
    int abort, bad_index, bad_scale;
    int tiles;                    // token tiles of all groups
    int first[kMaxE + 1];         // first token tile of each group
    int begin[kMaxE], count[kMaxE], size[kMaxE];   // its rows, and the rows of its tiles but the last
};

constexpr size_t kSmemBytes =
    1024 + kStages * kStageBytes + kScaleSlots * kScaleSlotBytes + kEpiBytes + sizeof(Tail);
static_assert(kSmemBytes <= 227 * 1024, "shared memory");

// Boxes of token rows: a tile takes the smallest that holds its half, so that a stage is two copies
// (issuing a copy took ~90 cycles: with one for every 32 rows the producer set the pace).
constexpr int kBoxes = 5;
__host__ __device__ constexpr int box_rows(int i) { return i == 0 ? 112 : i == 1 ? 96 : i == 2 ? 80 : i == 3 ? 64 : 32; }
struct TokenMaps {
    CUtensorMap map[kBoxes];
};

struct Params {
    const void *X_scale, *W_scale;
    const int32_t *offsets;
    int64_t R;
    int E, out, red;              // output features, reduction length
    int transpose, x_ue8m0, w_ue8m0;
    int x_vec;                    // 1: a row's four scales are one aligned vector; 2: sixteen are (bytes)
    int m_tiles;
    void *Y;
    int32_t *status;
};

// One tile of a group: its features, where its rows start, how many it holds.
struct Tile {
    int e, m0, rows;
    int64_t row0;
};

// A role's walk over its CTA pair's tiles (pair, pair + pairs, ...; the features of a token tile
// follow each other): the group only ever moves forward.
struct Walk {
    int tile, j, i, e;            // tile, its token tile and feature tile, the group reached

    __device__ __forceinline__ Walk(int pair, int m_tiles) : tile(pair), j(pair / m_tiles), i(pair - j * m_tiles), e(0) {}

    __device__ __forceinline__ void next(int pairs, int m_tiles)
    {
        tile += pairs;
        i += pairs;
        if (i >= m_tiles) {
            const int n = i / m_tiles;
            j += n;
            i -= n * m_tiles;
        }
    }

    __device__ __forceinline__ Tile get(const Tail &t)
    {
        while (t.first[e + 1] <= j) ++e;
        Tile r;
        r.e = e;
        r.m0 = i * kTileM;
        const int size = t.size[e], at = (j - t.first[e]) * size;
        r.row0 = static_cast<int64_t>(t.begin[e]) + at;
        const int left = t.count[e] - at;
        r.rows = left < size ? left : size;
        return r;
    }
};

// kind::mxf8f6f4, E4M3 x E4M3 -> fp32, UE8M0 scales; the scale byte of the word is `sf`.
__device__ __forceinline__ uint32_t make_idesc(uint32_t N, uint32_t a_mn_major, uint32_t sf)
{
    return (sf << 4) | (a_mn_major << 15) | ((N >> 3) << 17) | (1u << 23) | ((kTileM >> 4) << 24) | (sf << 29);
}

__device__ __forceinline__ void mma_scaled(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                           uint32_t sfb, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

// 32 rows of 16 bytes from shared memory to 4 TMEM columns, repeated in the four lane quarters; each
// CTA of the pair from its own memory to its own TMEM.
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint32_t saddr)
{
    const uint64_t desc = static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(128 >> 4) << 32) |
                          (1ull << 46);   // no swizzle, 8-row groups 128 B apart
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// 32 lanes x 32 columns of TMEM as fragments of 8x8: v[16 h + 4 c + 2 r + i] is row 16 h + 8 r + lane / 4,
// column 8 c + 2 (lane % 4) + i.
__device__ __forceinline__ void tmem_ld_fragments(uint32_t taddr, float (&v)[32])
{
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t r[16];
        asm volatile(
            "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
            "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
              "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
            : "r"(taddr + (static_cast<uint32_t>(16 * h) << 16))
            : "memory");
#pragma unroll
        for (int i = 0; i < 16; ++i) v[16 * h + i] = __uint_as_float(r[i]);
    }
}

// Those fragments (rows features, columns tokens) as bf16 to shared memory with the tokens as rows of 64
// bytes: stmatrix transposes each 8x8.  The 16-byte piece f of token t lies at place f ^ (t / 2 % 4).
__device__ __forceinline__ void store_transposed(uint32_t buf, int lane, const float (&v)[32])
{
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        // the four matrices: features 0..7, 8..15, 16..23, 24..31 of tokens 8 c .. 8 c + 7
        uint32_t m[4];
#pragma unroll
        for (int f = 0; f < 4; ++f) {
            const int at = 16 * (f >> 1) + 4 * c + 2 * (f & 1);
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[at], v[at + 1]);
            m[f] = *reinterpret_cast<const uint32_t *>(&h);
        }
        // lane l gives the address of row l % 8 of matrix l / 8
        const int tok = 8 * c + (lane & 7), f = lane >> 3;
        const uint32_t addr = buf + tok * 64 + ((f ^ ((tok >> 1) & 3)) << 4);
        asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(m[0]),
                     "r"(m[1]), "r"(m[2]), "r"(m[3])
                     : "memory");
    }
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    expert_gemm_kernel(const __grid_constant__ TokenMaps tmX, const __grid_constant__ CUtensorMap tmW, const Params p)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sf_ring = ring + kStages * kStageBytes;
    uint8_t *epi = sf_ring + kScaleSlots * kScaleSlotBytes;
    Tail &tail = *reinterpret_cast<Tail *>(epi + kEpiBytes);
    volatile int *abort_flag = &tail.abort;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&tail.full[s], rank == 0 ? 2 : 1);   // the leader's: its own stage and the other CTA's
            mbar_init(&tail.empty[s], 1);
        }
        for (int s = 0; s < kScaleSlots; ++s) {
            mbar_init(&tail.sf_full[s], 4);
            mbar_init(&tail.sf_empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tail.acc_full[b], 1);
            mbar_init(&tail.acc_empty[b], 8);
        }
        mbar_init(&tail.drain, 1);
        tail.abort = tail.bad_index = tail.bad_scale = 0;
        fence_mbarrier_init();
        tma_prefetch_desc(&tmX.map[0]);
        tma_prefetch_desc(&tmW);
    }
    if (warp == 3) {
        tmem_alloc_pair(&tail.tmem_base, kTmemCols);
    }
    // the groups: rows and token tiles of each (a group outside [0, R] holds none)
    __syncthreads();
    if (threadIdx.x < kMaxE) {
        const int e = threadIdx.x;
        int64_t a = 0, b = 0;
        if (e < p.E) {
            a = p.offsets ? p.offsets[e] : 0;
            b = p.offsets ? p.offsets[e + 1] : p.R;
            if (a < 0 || b < a || b > p.R) {
                tail.bad_index = 1;
                a = b = 0;
            }
            tail.begin[e] = static_cast<int>(a);
            tail.count[e] = static_cast<int>(b - a);
        }
        int v = static_cast<int>((b - a + kTileN - 1) / kTileN);
        // a group's tiles are equal parts, whole in 16 (size <= kTileN, so that none is empty); inclusive
        // scan of their number over the 256 threads
        if (v > 0) tail.size[e] = (static_cast<int>((b - a + v - 1) / v) + 15) & ~15;
        int x = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        int *part = reinterpret_cast<int *>(epi);
        if (lane == 31) part[warp] = x;
        named_barrier_sync(1, kMaxE);
        for (int w = 0; w < warp; ++w) x += part[w];
        if (e < p.E) tail.first[e + 1] = x;
        if (e == 0) tail.first[0] = 0;
    }
    tc_fence_before_sync();
    cluster_sync();               // both CTAs' barriers stand, both hold TMEM
    tc_fence_after_sync();
    const uint32_t tmem = tail.tmem_base;
    const int tiles = tail.first[p.E] * p.m_tiles;
    const int blocks = p.red / kBlk;

    if (warp == 0) {
        // weights of a group are read by several CTAs at about the same time, tokens too
        const uint64_t keep = l2_policy_evict_normal();
        uint32_t s = 0, ph = 0, issued = 0;
        bool ok = true;
        for (Walk walk(pair, p.m_tiles); walk.tile < tiles && ok; walk.next(pairs, p.m_tiles)) {
            const Tile t = walk.get(tail);
            const int half = ((t.rows + 15) & ~15) >> 1;        // tokens of each CTA
            int box = kBoxes - 1;
#pragma unroll
            for (int i = 0; i < kBoxes - 1; ++i)
                if (half > box_rows(i + 1)) {
                    box = i;
                    break;
                }
            const CUtensorMap *map = &tmX.map[box];
            const uint32_t bytes = kABytes + box_rows(box) * kBlk;
            const int m0 = t.m0 + rank * kHalfM;
            const int32_t row0 = static_cast<int32_t>(t.row0) + rank * half;
            for (int kb = 0; kb < blocks; ++kb) {
                ok = warp_wait(&tail.empty[s], ph ^ 1u, abort_flag);
                if (!ok) break;
                uint8_t *a = ring + s * kStageBytes, *b = a + kABytes;
                if (elect_one()) {
                    mbar_arrive_expect_tx(&tail.full[s], bytes);
                    tma_load_3d(a, &tmW, &tail.full[s], p.transpose ? m0 : kb * kBlk, p.transpose ? kb * kBlk : m0, t.e, keep);
                    tma_load_2d(b, map, &tail.full[s], kb * kBlk, row0, keep);
                }
                __syncwarp();
                ++issued;
                if (++s == kStages) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
        if (!ok) {
            // let the copies already issued land before the CTA ends
            const uint32_t from = issued > kStages ? issued - kStages : 0u;
            for (uint32_t x = from; x < issued; ++x) {
                volatile int no_abort = 0;
                mbar_wait_bounded(&tail.full[x % kStages], (x / kStages) & 1u, &no_abort);
            }
        }
    } else if (warp == 1 && rank != 0) {
        uint32_t s = 0, ph = 0;
        bool ok = true;
        for (Walk walk(pair, p.m_tiles); walk.tile < tiles && ok; walk.next(pairs, p.m_tiles)) {
            for (int kb = 0; kb < blocks; ++kb) {
                ok = warp_wait(&tail.full[s], ph, abort_flag);
                if (!ok) break;
                if (elect_one()) mbar_arrive_at(&tail.full[s], 0);
                __syncwarp();
                if (++s == kStages) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
    } else if (warp == 1) {
        // A: the weights, K-major (128-byte rows of k) or, transposed, MN-major (rows of m); 8-row
        // groups 1024 B apart either way.  A K = 32 step is 32 bytes of a row, or 32 rows.
        const uint64_t a0 = make_smem_desc_sw128(smem_u32(ring), 16, 1024);
        const uint64_t b0 = make_smem_desc_sw128(smem_u32(ring + kABytes), 16, 1024);
        const uint32_t a_step = p.transpose ? 32 * 128 / 16 : 2;
        uint32_t s = 0, ph = 0, q = 0, qph = 0, sf_place = 0;
        int j = 0;
        bool ok = true;
        for (Walk walk(pair, p.m_tiles); walk.tile < tiles; walk.next(pairs, p.m_tiles)) {
            const Tile t = walk.get(tail);
            const int b = j & 1;
            ok = warp_wait(&tail.acc_empty[b], ((j >> 1) & 1) ^ 1, abort_flag);
            if (!ok) break;
            tc_fence_after_sync();
            const uint32_t d = tmem + b * kTileN;
            const uint32_t idesc0 = make_idesc((t.rows + 15) & ~15, p.transpose, 0);
            for (int k0 = 0; k0 < blocks && ok; k0 += 4) {
                if ((k0 & 15) == 0) {
                    ok = warp_wait(&tail.sf_full[q], qph, abort_flag);
                    if (!ok) break;
                    tc_fence_after_sync();
                }
                const uint32_t src = smem_u32(sf_ring + q * kScaleSlotBytes) + ((k0 >> 2) & 3) * kScaleQuadBytes;
                const uint32_t sfa = tmem + kSfCol + sf_place * kSfCols, sfb = sfa + 4;
                sf_place = sf_place + 1 == kSfPlaces ? 0 : sf_place + 1;
                const bool last = (k0 & 15) == 12 || k0 + 4 >= blocks;    // of the slot
                if (elect_one()) {
                    copy_scales(sfa, src);
                    copy_scales(sfb, src + 512);
                    copy_scales(sfb + 4, src + 1024);
                    if (last) tc_commit_pair(&tail.sf_empty[q]);
                }
                __syncwarp();
                if (last) {
                    q ^= 1u;
                    qph ^= q ^ 1u;
                }
#pragma unroll
                for (uint32_t kk = 0; kk < 4; ++kk) {
                    if (k0 + static_cast<int>(kk) >= blocks) break;
                    ok = warp_wait(&tail.full[s], ph, abort_flag);
                    if (!ok) break;
                    tc_fence_after_sync();
                    const uint64_t at = (s * kStageBytes) >> 4;
                    const uint32_t idesc = idesc0 | (kk << 4) | (kk << 29);
                    if (elect_one()) {
#pragma unroll
                        for (int i = 0; i < kBlk / 32; ++i)
                            mma_scaled(d, a0 + at + i * a_step, b0 + at + i * 2, idesc, sfa, sfb, (k0 | kk | i) != 0);
                        tc_commit_pair(&tail.empty[s]);
                    }
                    __syncwarp();
                    if (++s == kStages) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
            if (!ok) break;
            if (elect_one()) tc_commit_pair(&tail.acc_full[b]);
            __syncwarp();
            ++j;
        }
        if (elect_one()) tc_commit_pair(&tail.drain);
        __syncwarp();
        volatile int no_abort = 0;
        mbar_wait_bounded(&tail.drain, 0, &no_abort);
    } else if (warp == 2 || warp == 3 || warp >= 8) {
        // Scale words: byte i of a row's word is the scale of 128-block 4 q + i.  Tokens: row r at
        // lane r % 32, word r / 32 of a 128-row atom; features: one word for the whole 128.  Two warps,
        // one for each atom, fill a slot with 16 blocks; two such teams take turns, so that a team has
        // two tiles' time (16 blocks each) for the loads' latency and the hand-over.
        const int team = warp >= 8, half = warp & 1;
        const int m_blocks = (p.out + kBlk - 1) / kBlk;
        uint32_t turn = 0, ph = 0;
        bool bad = false, ok = true;
        for (Walk walk(pair, p.m_tiles); walk.tile < tiles && ok; walk.next(pairs, p.m_tiles)) {
            Tile t;
            t.e = -1;
            for (int k0 = 0; k0 < blocks && ok; k0 += 16, turn ^= 1u) {
                if (turn != static_cast<uint32_t>(team)) continue;
                if (t.e < 0) t = walk.get(tail);
                // (blocks and rows that are not there read their neighbour's scale and are never used: the
                // loads carry no condition and are all in flight together)
                const int n = blocks - k0;
                uint32_t feat[4], tok[4][4];
                if (half == 0) {
                    const int mb = t.m0 / kBlk + rank < m_blocks ? t.m0 / kBlk + rank : m_blocks - 1;
                    const int step = p.transpose ? m_blocks : 1;
                    const int64_t at = p.transpose ? static_cast<int64_t>(t.e) * blocks * m_blocks + mb
                                                   : (static_cast<int64_t>(t.e) * m_blocks + mb) * blocks;
                    uint32_t v[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        v[i] = load_scale_bits(p.W_scale, p.w_ue8m0, at + (k0 + (i < n ? i : n - 1)) * step);
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[i] = scale_bits_byte(v[i], p.w_ue8m0, bad);
#pragma unroll
                    for (int i = 0; i < 4; ++i) feat[i] = v[4 * i] | v[4 * i + 1] << 8 | v[4 * i + 2] << 16 | v[4 * i + 3] << 24;
                }
                int64_t at[4];
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const int r = half * 128 + g * 32 + lane;
                    at[g] = (t.row0 + (r < t.rows ? r : t.rows - 1)) * blocks + k0;
                }
                if (p.x_vec == 2) {
                    const uint8_t *xs = static_cast<const uint8_t *>(p.X_scale);
                    uint4 v[4];
#pragma unroll
                    for (int g = 0; g < 4; ++g) v[g] = __ldg(reinterpret_cast<const uint4 *>(xs + at[g]));
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        tok[g][0] = v[g].x;
                        tok[g][1] = v[g].y;
                        tok[g][2] = v[g].z;
                        tok[g][3] = v[g].w;
                    }
                } else if (p.x_vec == 1 && p.x_ue8m0) {
                    const uint8_t *xs = static_cast<const uint8_t *>(p.X_scale);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int g = 0; g < 4; ++g)
                            tok[g][i] = __ldg(reinterpret_cast<const uint32_t *>(xs + at[g] + (4 * i < n ? 4 * i : 0)));
                } else if (p.x_vec == 1) {
                    const float *xs = static_cast<const float *>(p.X_scale);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (4 * i >= n) break;
                        uint4 v[4];
#pragma unroll
                        for (int g = 0; g < 4; ++g) v[g] = __ldg(reinterpret_cast<const uint4 *>(xs + at[g] + 4 * i));
#pragma unroll
                        for (int g = 0; g < 4; ++g)
                            tok[g][i] = scale_bits_byte(v[g].x, 0, bad) | scale_bits_byte(v[g].y, 0, bad) << 8 |
                                        scale_bits_byte(v[g].z, 0, bad) << 16 | scale_bits_byte(v[g].w, 0, bad) << 24;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (4 * i >= n) break;
                        uint32_t v[4][4];
#pragma unroll
                        for (int g = 0; g < 4; ++g)
#pragma unroll
                            for (int b = 0; b < 4; ++b)
                                v[g][b] = load_scale_bits(p.X_scale, p.x_ue8m0, at[g] + (4 * i + b < n ? 4 * i + b : n - 1));
#pragma unroll
                        for (int g = 0; g < 4; ++g) {
                            tok[g][i] = 0;
#pragma unroll
                            for (int b = 0; b < 4; ++b) tok[g][i] |= scale_bits_byte(v[g][b], p.x_ue8m0, bad) << (8 * b);
                        }
                    }
                }
                ok = __all_sync(0xffffffffu, mbar_wait_bounded(&tail.sf_empty[team], ph ^ 1u, abort_flag, 32));
                ph ^= 1u;
                uint4 *slot = reinterpret_cast<uint4 *>(sf_ring + team * kScaleSlotBytes);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint4 *quad = slot + i * (kScaleQuadBytes / 16);
                    if (half == 0) quad[lane] = make_uint4(feat[i], feat[i], feat[i], feat[i]);
                    quad[32 + half * 32 + lane] = make_uint4(tok[0][i], tok[1][i], tok[2][i], tok[3][i]);
                }
                // (each CTA's copy to TMEM reads these bytes from its own shared memory: once they are ordered
                // before the async proxy, the arrival at the leader has no other memory to order)
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive_at(&tail.sf_full[team], 0);
            }
        }
        if (bad) tail.bad_scale = 1;
    } else {
        const int w = warp - 4;
        uint8_t *buf = epi + w * 32 * 64;
        const uint32_t buf_addr = smem_u32(buf);
        const uint32_t lane_addr = tmem + (static_cast<uint32_t>(w * 32) << 16);
        int j = 0;
        for (Walk walk(pair, p.m_tiles); walk.tile < tiles; walk.next(pairs, p.m_tiles)) {
            const Tile t = walk.get(tail);
            const int b = j & 1;
            if (!__all_sync(0xffffffffu, mbar_wait_bounded(&tail.acc_full[b], (j >> 1) & 1, abort_flag, 64))) break;
            tc_fence_after_sync();
            const int m = t.m0 + rank * kHalfM + w * 32;  // this warp's features
            const int feats = p.out - m;                 // a multiple of 16, may be <= 0
            // a lane's four 16-byte pieces of a chunk: tokens lane / 4 + 8 i, features 8 (lane % 4) on
            const bool part_ok = (lane & 3) * 8 < feats;
            __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.Y) + (t.row0 + (lane >> 2)) * p.out + m + (lane & 3) * 8;
            float v[2][32];
            tmem_ld_fragments(lane_addr + b * kTileN, v[0]);
#pragma unroll 2
            for (int c = 0, x = 0; c < t.rows; c += 32, x ^= 1) {
                tmem_ld_wait();
                store_transposed(buf_addr, lane, v[x]);
                if (c + 32 < t.rows) tmem_ld_fragments(lane_addr + b * kTileN + c + 32, v[x ^ 1]);
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int tok = i * 8 + (lane >> 2);
                    const uint4 y = *reinterpret_cast<const uint4 *>(buf + tok * 64 + (((lane & 3) ^ ((tok >> 1) & 3)) << 4));
                    if (c + tok < t.rows && part_ok)
                        *reinterpret_cast<uint4 *>(dst + static_cast<int64_t>(c + 8 * i) * p.out) = y;
                }
                __syncwarp();
            }
            tc_fence_before_sync();
            if (lane == 0) mbar_arrive_at(&tail.acc_empty[b], 0);
            ++j;
        }
    }

    tc_fence_before_sync();
    cluster_sync();               // the leader's MMAs have read the other CTA's memory
    tc_fence_after_sync();
    if (warp == 3) tmem_dealloc_pair(tmem, kTmemCols);
    if (threadIdx.x == 0) {
        if (tail.abort) report_status(p.status, MOE_ERR_TIMEOUT);
        if (tail.bad_index) report_status(p.status, MOE_ERR_BAD_INDEX);
        if (tail.bad_scale) report_status(p.status, MOE_ERR_BAD_SCALE);
    }
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_tiled()
{
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(ptr);
    });
    return fn;
}

}  // namespace

bool encode_map(CUtensorMap *map, CUtensorMapDataType type, int elem_bytes, const void *base, int rank,
                const uint64_t *dims, const uint32_t *box, CUtensorMapSwizzle swizzle)
{
    EncodeTiledFn fn = encode_tiled();
    if (!fn) return false;
    cuuint64_t d[5], strides[4];
    cuuint32_t b[5], ones[5];
    uint64_t bytes = elem_bytes;
    for (int i = 0; i < rank; ++i) {
        d[i] = dims[i];
        b[i] = box[i];
        ones[i] = 1;
        bytes *= dims[i];
        if (i + 1 < rank) strides[i] = bytes;
    }
    return fn(map, type, rank, const_cast<void *>(base), d, strides, b, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
              swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_expert_gemm(const ExpertGemmArgs &a, cudaStream_t stream)
{
    int dev = 0;
    cudaError_t err = expert_device(&dev);
    if (err != cudaSuccess) return err;
    const int red = a.transpose ? a.rows : a.cols, out = a.transpose ? a.cols : a.rows;

    TokenMaps tmX;
    CUtensorMap tmW;
    const uint64_t xd[2] = {static_cast<uint64_t>(red), static_cast<uint64_t>(a.R)};
    const uint64_t wd[3] = {static_cast<uint64_t>(a.cols), static_cast<uint64_t>(a.rows), static_cast<uint64_t>(a.E)};
    const uint32_t wb[3] = {128, 128, 1};
    for (int i = 0; i < kBoxes; ++i) {
        const uint32_t xb[2] = {kBlk, static_cast<uint32_t>(box_rows(i))};
        if (!encode_map(&tmX.map[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.X, 2, xd, xb)) return cudaErrorInvalidValue;
    }
    if (!encode_map(&tmW, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.W, 3, wd, wb)) return cudaErrorInvalidValue;

    static std::atomic<uint64_t> done{0};
    const uint64_t bit = 1ull << (dev & 63);
    if (!(done.load(std::memory_order_relaxed) & bit)) {
        err = cudaFuncSetAttribute(expert_gemm_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   static_cast<int>(kSmemBytes));
        if (err != cudaSuccess) return err;
        done.fetch_or(bit, std::memory_order_relaxed);
    }
    Params p;
    p.X_scale = a.X_scale;
    p.W_scale = a.W_scale;
    p.offsets = a.offsets;
    p.R = a.R;
    p.E = a.E;
    p.out = out;
    p.red = red;
    p.transpose = a.transpose;
    p.x_ue8m0 = a.x_ue8m0;
    p.w_ue8m0 = a.w_ue8m0;
    const uintptr_t xs = reinterpret_cast<uintptr_t>(a.X_scale);
    p.x_vec = (red / kBlk) % 4 == 0 && xs % (a.x_ue8m0 ? 4 : 16) == 0;
    if (a.x_ue8m0 && (red / kBlk) % 16 == 0 && xs % 16 == 0) p.x_vec = 2;
    p.m_tiles = (out + kTileM - 1) / kTileM;
    p.Y = a.Y;
    p.status = a.status;
    // the most tiles that R rows in E groups can make; no more pairs than that
    const int64_t most = (a.R / kTileN + (a.R < a.E ? a.R : a.E) + 1) * p.m_tiles;
    const int pairs = device_sm_count(dev) / 2;
    const int grid = 2 * static_cast<int>(most < pairs ? most : pairs);
    expert_gemm_kernel<<<grid, kThreads, kSmemBytes, stream>>>(tmX, tmW, p);
    return cudaGetLastError();
}

}  // namespace moe
