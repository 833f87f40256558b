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
// The tensor cores cut where they add to an accumulator (measured: a sum of 16384 rows
// comes out 7e-6 of its size too small).  A 32-bit result is therefore summed in
// segments of 2048 rows, each in an accumulator of its own, and the segments are
// added to what is in dW already, rounding to nearest (2048 rows: 6e-7).  A result of bf16 type is off
// by 2^-9 anyway and takes segments of 16384 rows (2e-5); those of a longer group are added up, in 32 bits,
// in the other of the two accumulators (with one segment for any length, 2^20 rows of positive products
// came out 4e-3 of their sum too small, 2^22 rows 2e-2).
//
// Both operands have the reduction on their slow axis (MN-major).  Persistent CTA
// pairs (cta_group::2); a tile is 256 weight rows x 256 weight columns of one expert,
// a ring stage 64 rows of the group.  Each CTA holds the accumulators of 128 of the
// weight rows, and brings those columns of dY and half of the columns of x: it
// converts 128 columns, one scale for each row, in the time of a 256 x 256 x 64 MMA.
// Warp roles, in each CTA:
//   warp 0        TMA producer (dY 64 x 128 bf16, x 64 x 128 E4M3)
//   warp 1        MMA issuer (one thread of the leader)
//   warp 3        allocates TMEM
//   warps 4..11   epilogue, two warps to a quarter of the TMEM lanes
//   warps 12..23  three teams of converters E4M3 -> bf16, each with its own places of
//                 the ring; in a group's last stage they also clear the rows behind its end
//                 (the next group's, or none)
//
// Measured (burst): 16384 tokens on 128 experts, top 8, 2048 x 2048, bf16: 672 us, 1.64 PFLOP/s, the tensor
// pipe 69% busy beside converters that take 56% of the issue slots (back to back, at the power limit, 781 us).
// 1023 tokens on 64 experts of 512 x 1024, added to 32-bit gradients: 65 us for 273 MB (4.2 TB/s), bound by the
// latency of the boxes in and out of tiles that have 32 rows to reduce.
#include <climits>

#include "expert_internal.cuh"

namespace moe {
namespace {

constexpr int kTileM = 256, kTileN = 256, kRows = 64;
constexpr int kHalf = 128;                        // weight rows, and columns of x, of each CTA
constexpr int kBox = kRows * 128;                 // bytes of a box: 64 rows of 128 bytes
constexpr int kABytes = 2 * kBox;                 // two boxes of 64 columns
constexpr int kRawBytes = kBox;                   // 128 columns; a row lies where its second half will, of
constexpr int kBBytes = 2 * kBox;                 // two boxes of 64 columns
constexpr int kStageBytes = kABytes + kBBytes;
constexpr int kEpiWarps = 8, kTeams = 3, kTeamWarps = 4;
constexpr int kBufBytes = 32 * 64;                // a buffer of an epilogue warp: 32 rows x 16 fp32
// Shared memory goes to ring stages or to the epilogue's buffers.  With something to add, small groups are
// bound by its way in: four buffers keep three boxes of it in flight for each of the eight warps (64 experts
// of 512 x 1024 with 32 rows each: 65 us, 82 us with two thirds of that in flight).  Without, a sixth stage
// covers more of the ring's latency (128 experts of 2048 x 2048, 1024 rows each: 683 us, 724 us with five).
template <bool kLoads>
struct Split {
    static constexpr int kStages = kLoads ? 5 : 6, kBufs = kLoads ? 4 : 2;
};
constexpr int kSegment = 2048, kSegmentBf16 = 16384;   // rows, whole stages
constexpr int kMostStages = 6, kMostBufs = 4;
constexpr int kThreads = 32 * (4 + kEpiWarps + kTeams * kTeamWarps);
constexpr uint32_t kTmemCols = 512;
constexpr int kMaxE = 256;

struct Tail {
    uint64_t full[kMostStages], conv[kMostStages], empty[kMostStages];
    uint64_t acc_full[2], acc_empty[2], drain;
    uint64_t added[kEpiWarps][kMostBufs];
    uint32_t tmem_base;
    int abort, bad_index, bad_scale;
    uint32_t valid[kMaxE / 32];   // a bit for each group that lies inside [0, R]
    int off[kMaxE + 1];
};
template <bool kLoads>
constexpr size_t smem_bytes()
{
    return 1024 + Split<kLoads>::kStages * kStageBytes + Split<kLoads>::kBufs * kEpiWarps * kBufBytes + sizeof(Tail);
}
static_assert(smem_bytes<false>() <= 227 * 1024 && smem_bytes<true>() <= 227 * 1024, "shared memory");

struct Params {
    const void *X_scale;
    const int32_t *offsets;
    int64_t R;
    int E, rows, cols, x_ue8m0, bf16_out, has_add;
    int segment;                  // rows that are summed in one go
    int m_tiles, n_tiles;
    int32_t *status;
};

// Tile `tile` of the walk: expert-major, the columns of a row of tiles next to each other.
struct Tile {
    int e, m0, n0, count;
    int64_t begin;
};
__device__ __forceinline__ Tile get_tile(const Tail &t, const Params &p, int tile)
{
    const int per = p.m_tiles * p.n_tiles;
    Tile r;
    r.e = tile / per;
    const int i = tile - r.e * per, m = i / p.n_tiles;
    r.m0 = m * kTileM;
    r.n0 = (i - m * p.n_tiles) * kTileN;
    r.begin = t.off[r.e];
    r.count = (t.valid[r.e >> 5] >> (r.e & 31)) & 1u ? t.off[r.e + 1] - t.off[r.e] : 0;
    return r;
}

// The stages of a CTA pair's walk (groups without rows have none) that a team converts: those in its own
// places of the ring, place % kTeams == team.  (A place has to be one team's: a wait by parity is right only
// for who waits for every phase.)  Of each, how many rows of the group from its first on there are, and where
// their scales of this CTA's columns are.
template <int kStages>
struct Stages {
    int tile, i, count;           // the tile, the first row in its group, the group's rows
    int place, team;
    int64_t scales;               // of the group's first row

    __device__ __forceinline__ Stages(const Tail &t, const Params &p, int pair, int pairs, int tiles, int team, int rank)
        : tile(pair - pairs), i(team * kRows), count(0), place(team), team(team)
    {
        settle(t, p, pairs, tiles, rank);
    }
    // How many stages on the team's next place is.
    static __device__ __forceinline__ int step(int place, int team)
    {
        return place + kTeams < kStages ? kTeams : kStages - place + team;
    }
    __device__ __forceinline__ void next(const Tail &t, const Params &p, int pairs, int tiles, int rank)
    {
        const int n = step(place, team);
        i += n * kRows;
        place += n;
        if (place >= kStages) place -= kStages;
        if (i >= count) settle(t, p, pairs, tiles, rank);
    }
    __device__ __forceinline__ void settle(const Tail &t, const Params &p, int pairs, int tiles, int rank)
    {
        while (i >= count && tile < tiles) {
            i -= (count + kRows - 1) / kRows * kRows;
            count = 0;
            tile += pairs;
            if (tile < tiles) {
                const Tile w = get_tile(t, p, tile);
                const int kblocks = p.cols >> 7, kb = (w.n0 >> 7) + rank;
                // (columns behind the edge: any scale will do for their zeros)
                scales = w.begin * kblocks + (kb < kblocks ? kb : kblocks - 1);
                count = w.count;
            }
        }
    }
    __device__ __forceinline__ int valid() const { return count - i; }
};

__device__ __forceinline__ void mma_f16_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Two bf16 products per call; exact here (the factors are powers of two).
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Four E4M3 codes -> four bf16, times f.  A code's bits s eeee mmm, moved to
// s 0000 eeee mmm 0000, are the bf16 number code * 2^-120 (its subnormals included),
// so that 2^120 goes into f.
__device__ __forceinline__ uint2 codes_to_bf16(uint32_t w, uint32_t f)
{
    uint32_t lo, hi;   // each code in the low byte of a half, its sign spread over the high byte
    asm("prmt.b32 %0, %1, 0, 0x9180;" : "=r"(lo) : "r"(w));
    asm("prmt.b32 %0, %1, 0, 0xB3A2;" : "=r"(hi) : "r"(w));
    return make_uint2(mul_bf16x2((lo << 4) & 0x87F087F0u, f), mul_bf16x2((hi << 4) & 0x87F087F0u, f));
}

// Bits 0x80808080 of the result: which of four codes are NaNs (s 1111 111).
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) { return (w & 0x7F7F7F7Fu) + 0x01010101u; }

__device__ __forceinline__ uint32_t set_nan(uint32_t v, uint32_t w, int i)
{
    if (((w >> (8 * i)) & 0x7F) == 0x7F) v = (v & 0xFFFF0000u) | 0x7FFFu;
    if (((w >> (8 * i + 8)) & 0x7F) == 0x7F) v = (v & 0x0000FFFFu) | 0x7FFF0000u;
    return v;
}

// Eight codes of one row, none of them a NaN -> 16 bytes, times f = 2^120 * s.
__device__ __forceinline__ uint4 convert_codes(const uint2 &w, uint32_t f)
{
    const uint2 a = codes_to_bf16(w.x, f), b = codes_to_bf16(w.y, f);
    return make_uint4(a.x, a.y, b.x, b.y);
}

// The same with NaN codes, the NaN scale 255, and where 2^120 * s (s = 2^(byte - 127)) is beyond bf16's range.
__device__ __forceinline__ uint4 convert_codes_rare(const uint2 &w, uint32_t byte)
{
    const uint32_t ex = 120u + byte, ex1 = ex < 254u ? ex : 254u;
    const uint32_t f = ex1 * 0x00800080u, f2 = (127u + ex - ex1) * 0x00800080u;
    uint2 a = codes_to_bf16(w.x, f), b = codes_to_bf16(w.y, f);
    a = make_uint2(mul_bf16x2(a.x, f2), mul_bf16x2(a.y, f2));
    b = make_uint2(mul_bf16x2(b.x, f2), mul_bf16x2(b.y, f2));
    a = make_uint2(set_nan(a.x, w.x, 0), set_nan(a.y, w.x, 2));
    b = make_uint2(set_nan(b.x, w.y, 0), set_nan(b.y, w.y, 2));
    if (byte == 255) a = b = make_uint2(0x7FFF7FFFu, 0x7FFF7FFFu);
    return make_uint4(a.x, a.y, b.x, b.y);
}

// kLoads: boxes come in to the epilogue (something to add, or fp32 groups of several segments).  kHeld: a bf16 result
// whose groups may have several segments (a kernel of its own: together with the reading of fp32 segments it took
// more than the 80 registers that a thread has).
template <bool kLoads, bool kHeld>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    expert_wgrad_kernel(const __grid_constant__ CUtensorMap tmY, const __grid_constant__ CUtensorMap tmX,
                        const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmAdd, const Params p)
{
    constexpr int kStages = Split<kLoads>::kStages, kBufs = Split<kLoads>::kBufs;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *epi = ring + kStages * kStageBytes;
    Tail &tail = *reinterpret_cast<Tail *>(epi + kBufs * kEpiWarps * kBufBytes);
    volatile int *abort_flag = &tail.abort;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&tail.full[s], 1);
            mbar_init(&tail.conv[s], 2 * kTeamWarps);   // the leader's: both CTAs' converters
            mbar_init(&tail.empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tail.acc_full[b], 1);
            mbar_init(&tail.acc_empty[b], 2 * kEpiWarps);
        }
        mbar_init(&tail.drain, 1);
        for (int i = 0; i < kEpiWarps * kMostBufs; ++i) mbar_init(&tail.added[0][0] + i, 1);
        tail.abort = tail.bad_index = tail.bad_scale = 0;
        fence_mbarrier_init();
        tma_prefetch_desc(&tmY);
        tma_prefetch_desc(&tmX);
        tma_prefetch_desc(&tmW);
        if (kLoads) tma_prefetch_desc(&tmAdd);
    }
    if (warp == 3) tmem_alloc_pair(&tail.tmem_base, kTmemCols);
    __syncthreads();
    if (threadIdx.x < kMaxE) {
        const int e = threadIdx.x;
        int a = 0, b = 0;
        if (e < p.E) {
            a = p.offsets ? p.offsets[e] : 0;
            b = p.offsets ? p.offsets[e + 1] : static_cast<int>(p.R);
            tail.off[e] = a;
            if (e == p.E - 1) tail.off[p.E] = b;
        }
        const bool good = a >= 0 && a <= b && b <= p.R;
        const uint32_t mask = __ballot_sync(0xffffffffu, good);
        if (lane == 0) tail.valid[warp] = mask;
        if (!good) tail.bad_index = 1;
    }
    tc_fence_before_sync();
    cluster_sync();               // both CTAs' barriers stand, both hold TMEM
    tc_fence_after_sync();
    const uint32_t tmem = tail.tmem_base;
    const int tiles = p.E * p.m_tiles * p.n_tiles;

    if (warp == 0) {
        const uint64_t keep = l2_policy_evict_normal();
        uint32_t s = 0, ph = 0, issued = 0;
        bool ok = true;
        for (int tile = pair; tile < tiles && ok; tile += pairs) {
            const Tile t = get_tile(tail, p, tile);
            const int m = t.m0 + rank * kHalf, n = t.n0 + rank * kHalf;
            for (int r = 0; r < t.count; r += kRows) {
                ok = warp_wait(&tail.empty[s], ph ^ 1u, abort_flag);
                if (!ok) break;
                uint8_t *a = ring + s * kStageBytes;
                const int row = static_cast<int>(t.begin) + r;
                if (elect_one()) {
                    mbar_arrive_expect_tx(&tail.full[s], kABytes + kRawBytes);
                    tma_load_2d(a + kABytes + kBBytes - kRawBytes, &tmX, &tail.full[s], n, row, keep);
                    tma_load_2d(a, &tmY, &tail.full[s], m, row, keep);
                    tma_load_2d(a + kBox, &tmY, &tail.full[s], m + 64, row, keep);
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
    } else if (warp == 1 && rank == 0) {
        const uint64_t a0 = make_smem_desc_sw128(smem_u32(ring), kBox, 1024);
        const uint64_t b0 = make_smem_desc_sw128(smem_u32(ring + kABytes), kBox, 1024);
        const uint32_t idesc = make_idesc_bf16_f32(kTileM, kTileN, 1, 1);
        uint32_t s = 0, ph = 0;
        uint32_t b = 0, used = 0;     // the accumulator, and a phase bit for each
        bool ok = true;
        for (int tile = pair; tile < tiles; tile += pairs) {
            const int count = get_tile(tail, p, tile).count;
            // (such a tile's segments take turns in one accumulator, their sum is in the other; the next tile starts
            // in the same one, so that its wait covers both)
            const bool held = kHeld && count > p.segment;
            for (int r0 = 0; r0 < count && ok; r0 += p.segment) {
                const int end = count - r0 < p.segment ? count : r0 + p.segment;
                ok = warp_wait(&tail.acc_empty[b], (used >> b & 1u) ^ 1u, abort_flag);
                if (!ok) break;
                used ^= 1u << b;
                tc_fence_after_sync();
                const uint32_t d = tmem + b * kTileN;
                for (int r = r0; r < end; r += kRows) {
                    ok = warp_wait(&tail.conv[s], ph, abort_flag);
                    if (!ok) break;
                    tc_fence_after_sync();
                    const uint64_t at = (s * kStageBytes) >> 4;
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < kRows / 16; ++k)
                            mma_f16_pair(d, a0 + at + k * 128, b0 + at + k * 128, idesc, ((r - r0) | k) != 0);
                        tc_commit_pair(&tail.empty[s]);
                    }
                    __syncwarp();
                    if (++s == kStages) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
                if (!ok) break;
                if (elect_one()) tc_commit_pair(&tail.acc_full[b]);
                __syncwarp();
                if (!held) b ^= 1u;
            }
            if (!ok) break;
        }
        if (elect_one()) tc_commit_pair(&tail.drain);
        __syncwarp();
        volatile int no_abort = 0;
        mbar_wait_bounded(&tail.drain, 0, &no_abort);
    } else if (warp >= 4 + kEpiWarps) {
        const int team = (warp - 4 - kEpiWarps) / kTeamWarps;
        const int t = threadIdx.x - 32 * (4 + kEpiWarps + team * kTeamWarps);
        // eight codes of a row, and the first of eight rows, 8 apart: their places in the swizzled tiles
        // differ by whole groups of eight rows
        const int c = t & 15, r0 = t >> 4;
        const int raw_at = r0 * 128 + (((c >> 1) ^ r0) << 4) + (c & 1) * 8;
        const int dst_at = (c >> 3) * kBox + r0 * 128 + (((c & 7) ^ r0) << 4);
        const int kblocks = p.cols >> 7;
        bool bad = false, ok = true;
        uint32_t s = team, ph = 0;
        // A warp converts 16 rows of a stage, two at a time: lane l (and l + 16) loads the scale of the row
        // r0 of lanes 16 (l & 1) on, 8 (l / 2) further, and hands it out by shuffles
        const int srow = 2 * (t >> 5) + (lane & 1) + 8 * ((lane & 15) >> 1);
        using Walk = Stages<kStages>;
        auto fetch = [&](const Walk &g) {
            // (rows behind the group's end: any scale will do for their zeros)
            const int row = g.i + srow < g.count ? g.i + srow : g.count - 1;
            return load_scale_bits(p.X_scale, p.x_ue8m0, g.scales + static_cast<int64_t>(row) * kblocks);
        };
        // The scales of this team's next two stages are on their way while it converts one (with one, the
        // wait for them was a third of the team's time).  rows: of the stage; 0: there is none.
        Walk ahead(tail, p, pair, pairs, tiles, team, rank);
        auto take = [&](uint32_t &scale, int &rows) {
            rows = 0;
            if (ahead.tile < tiles) {
                scale = fetch(ahead);
                rows = ahead.valid();
                ahead.next(tail, p, pairs, tiles, rank);
            }
        };
        uint32_t sb = 0, sb1 = 0, sb2 = 0;
        int valid, valid1, valid2;
        take(sb, valid);
        take(sb1, valid1);
        take(sb2, valid2);
        while (valid > 0) {
            const uint32_t byte = scale_bits_byte(sb, p.x_ue8m0, bad);
            const uint32_t factor = (120u + byte) * 0x00800080u;      // 2^120 * s as a bf16, twice
            ok = warp_wait(&tail.full[s], ph, abort_flag);
            if (!ok) break;
            uint8_t *a = ring + s * kStageBytes, *b = a + kABytes, *raw = b + kBBytes - kRawBytes;
            // a warp's rows are in registers before their bf16 forms overwrite them
            uint2 v[8];
#pragma unroll
            for (int x = 0; x < 8; ++x) v[x] = *reinterpret_cast<const uint2 *>(raw + raw_at + x * 1024);
            if (valid < kRows) {
                // the group's last rows.  Behind them x is zero, and whatever dY holds there must not meet
                // those zeros
#pragma unroll
                for (int x = 0; x < 8; ++x)
                    if (r0 + 8 * x >= valid) v[x] = make_uint2(0, 0);
                for (int x = t; x < (kRows - valid) * 16; x += kTeamWarps * 32)
                    *reinterpret_cast<uint4 *>(a + (x & 8 ? kBox : 0) + (valid + (x >> 4)) * 128 + ((x & 7) << 4)) =
                        make_uint4(0, 0, 0, 0);
            }
            __syncwarp();
            uint32_t nan = 0;
#pragma unroll
            for (int x = 0; x < 8; ++x) nan |= nan_codes(v[x].x) | nan_codes(v[x].y);
            if (!__any_sync(0xffffffffu, (nan & 0x80808080u) != 0 || byte > 134u)) {
#pragma unroll
                for (int x = 0; x < 8; ++x)
                    *reinterpret_cast<uint4 *>(b + dst_at + x * 1024) =
                        convert_codes(v[x], __shfl_sync(0xffffffffu, factor, 2 * x + (r0 & 1)));
            } else {
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    const uint32_t y = __shfl_sync(0xffffffffu, byte, 2 * x + (r0 & 1));
                    *reinterpret_cast<uint4 *>(b + dst_at + x * 1024) =
                        r0 + 8 * x < valid ? convert_codes_rare(v[x], y) : make_uint4(0, 0, 0, 0);
                }
            }
            // (each CTA's tensor core reads these bytes from its own shared memory: once they are ordered
            // before the async proxy, the arrival at the leader has no other memory to order)
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive_at(&tail.conv[s], 0);
            s += Walk::step(s, team);
            if (s >= kStages) {
                s -= kStages;
                ph ^= 1u;
            }
            // (loads in flight are waited for by the fence above: they are issued right behind it)
            sb = sb1;
            valid = valid1;
            sb1 = sb2;
            valid1 = valid2;
            take(sb2, valid2);
        }
        if (bad) tail.bad_scale = 1;
    } else if (warp >= 4) {
        // 32 rows x 128 columns of a tile: 16 columns at a time from TMEM (a lane is a row), through one of
        // four buffers of shared memory, out as a TMA box.  What is added comes in the same way, up to
        // three boxes ahead (by loads to registers, 16 KiB in flight per SM, it took twice the time).
        const int w = warp - 4, quarter = w & 3, side = w >> 2;   // TMEM lanes, columns 128 side on
        uint8_t *bufs = epi + w * kBufs * kBufBytes;
        const uint32_t lane_addr = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + side * 128;
        const int dm = rank * kHalf + quarter * 32, dn = side * 128;
        // place of a lane's 16-byte piece x: its row's bytes, swizzled as the boxes are (64- or 32-byte rows)
        const int row64 = lane * 64, swz64 = (lane >> 1) & 3, row32 = lane * 32, swz32 = (lane >> 2) & 1;
        // The boxes to come: of which tile, segment and columns the next one is.  A first segment's is added
        // to `add`'s, if there is one, a later one's to what this warp has stored of the one before.
        int a_tile = pair, a_row = 0, a_c = 0;
        uint32_t asked = 0, q = 0, landed = 0;                    // q: boxes done; landed: a phase bit per buffer
        uint32_t wanted = 0;                                      // a bit per buffer: its box has been asked for
        const bool bf16_out = kHeld || p.bf16_out;
        auto ask = [&]() {
            Tile t;
            while (a_tile < tiles) {
                t = get_tile(tail, p, a_tile);
                if (t.m0 + dm < p.rows && t.n0 + dn < p.cols) break;
                a_tile += pairs;
            }
            if (a_tile >= tiles) return;
            const uint32_t b = asked % kBufs;
            if ((!kHeld && a_row > 0) || p.has_add) {
                if (lane == 0) {
                    uint64_t *bar = &tail.added[w][b];
                    // eight boxes lie between a segment's and the next one's, three of which are asked for ahead
                    if (!kHeld && a_row > 0) {
                        bulk_wait<4>();
                        fence_proxy_async_all();
                    }
                    mbar_arrive_expect_tx(bar, kBufBytes);
                    tma_load_3d(bufs + b * kBufBytes, !kHeld && a_row > 0 ? &tmW : &tmAdd, bar, t.n0 + dn + a_c, t.m0 + dm, t.e,
                                l2_policy_evict_first());
                }
                wanted |= 1u << b;
            }
            __syncwarp();
            ++asked;
            a_c += 16;
            if (a_c == kHalf) {
                a_c = 0;
                a_row += p.segment;
                if (bf16_out || t.count - a_row <= 0) {           // (a bf16 result is written once)
                    a_row = 0;
                    a_tile += pairs;
                }
            }
        };
        if (kLoads)
            for (int i = 0; i < kBufs - 1; ++i) ask();
        uint32_t acc = lane_addr, used = 0;                       // the accumulator, and a phase bit for each
        bool ok = true;
        for (int tile = pair; tile < tiles && ok; tile += pairs) {
            const Tile t = get_tile(tail, p, tile);
            const bool some = t.count != 0, held = kHeld && t.count > p.segment;
            const int m = t.m0 + dm, n = t.n0 + dn;
            const bool inside = n < p.cols && m < p.rows;         // (columns come in whole 128)
            for (int r0 = 0; (r0 < t.count || r0 == 0) && ok; r0 += p.segment) {
                if (some) {
                    const uint32_t b = acc / kTileN & 1u;
                    ok = __all_sync(0xffffffffu, mbar_wait_bounded(&tail.acc_full[b], used >> b & 1u, abort_flag, 64));
                    if (!ok) break;
                    tc_fence_after_sync();
                    used ^= 1u << b;
                }
                if (held && t.count - r0 > p.segment) {
                    // not the last segment: to the sum so far, which this warp alone reads and writes
                    for (int c = 0; c < kHalf && inside; c += 8) {
                        float v[8], z[8];
                        tmem_ld_32x32b_x8(acc + c, v);
                        if (r0 > 0) tmem_ld_32x32b_x8((acc ^ kTileN) + c, z);
                        tmem_ld_wait();
                        if (r0 > 0) {
    #pragma unroll
                            for (int x = 0; x < 8; ++x) v[x] += z[x];
                        }
                        tmem_st_32x32b_x8((acc ^ kTileN) + c, v);
                    }
                    tmem_st_wait();
                    tc_fence_before_sync();
                    if (lane == 0) mbar_arrive_at(&tail.acc_empty[acc / kTileN & 1u], 0);
                    continue;
                }
                for (int c = 0; c < kHalf && inside; c += 16, ++q) {
                    const uint32_t at = q % kBufs;
                    uint8_t *buf = bufs + at * kBufBytes;
                    if (kLoads) {
                        // the buffer of the box before this one is free again once it has been read
                        bulk_wait_read<0>();
                        __syncwarp();
                        ask();
                    } else {
                        bulk_wait_read<kBufs - 1>();
                        __syncwarp();
                    }
                    float v[16];
                    if (some) {
                        tmem_ld_32x32b_x16(acc + c, v);
                        tmem_ld_wait();
                        if (held) {
    #pragma unroll
                            for (int h = 0; h < 16; h += 8) {
                                float z[8];
                                tmem_ld_32x32b_x8((acc ^ kTileN) + c + h, z);
                                tmem_ld_wait();
    #pragma unroll
                                for (int x = 0; x < 8; ++x) v[h + x] += z[x];
                            }
                        }
                    } else {
    #pragma unroll
                        for (int x = 0; x < 16; ++x) v[x] = 0.f;
                    }
                    if (kLoads && (wanted >> at & 1u)) {
                        ok = warp_wait(&tail.added[w][at], landed >> at & 1u, abort_flag);
                        if (!ok) break;
                        landed ^= 1u << at;
                        wanted ^= 1u << at;
    #pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const float4 z = *reinterpret_cast<const float4 *>(buf + row64 + ((x ^ swz64) << 4));
                            v[4 * x] += z.x;
                            v[4 * x + 1] += z.y;
                            v[4 * x + 2] += z.z;
                            v[4 * x + 3] += z.w;
                        }
                        if (bf16_out) __syncwarp();                 // (other lanes' rows lie where this one writes)
                    }
                    if (bf16_out) {
    #pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            uint4 h;
                            __nv_bfloat162 *hp = reinterpret_cast<__nv_bfloat162 *>(&h);
    #pragma unroll
                            for (int i = 0; i < 4; ++i) hp[i] = __floats2bfloat162_rn(v[8 * x + 2 * i], v[8 * x + 2 * i + 1]);
                            *reinterpret_cast<uint4 *>(buf + row32 + ((x ^ swz32) << 4)) = h;
                        }
                    } else {
    #pragma unroll
                        for (int x = 0; x < 4; ++x)
                            *reinterpret_cast<float4 *>(buf + row64 + ((x ^ swz64) << 4)) =
                                make_float4(v[4 * x], v[4 * x + 1], v[4 * x + 2], v[4 * x + 3]);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) tma_store_3d(&tmW, buf, n + c, m, t.e);
                }
                if (!ok) break;
                if (some) {
                    tc_fence_before_sync();
                    if (lane == 0) mbar_arrive_at(&tail.acc_empty[acc / kTileN & 1u], 0);
                    if (!held) acc ^= kTileN;
                }
            }
        }
        for (uint32_t x = 0; x < kBufs; ++x) {                    // (given up: what was asked for still lands here)
            volatile int no_abort = 0;
            if (wanted >> x & 1u) mbar_wait_bounded(&tail.added[w][x], landed >> x & 1u, &no_abort);
        }
        bulk_wait_all();
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

template <bool kLoads, bool kHeld>
cudaError_t launch(int dev, dim3 grid, cudaStream_t stream, const CUtensorMap &tmY, const CUtensorMap &tmX,
                   const CUtensorMap &tmW, const CUtensorMap &tmAdd, const Params &p)
{
    constexpr size_t bytes = smem_bytes<kLoads>();
    static std::atomic<uint64_t> done{0};
    const uint64_t bit = 1ull << (dev & 63);
    if (!(done.load(std::memory_order_relaxed) & bit)) {
        const cudaError_t err = cudaFuncSetAttribute(expert_wgrad_kernel<kLoads, kHeld>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                     static_cast<int>(bytes));
        if (err != cudaSuccess) return err;
        done.fetch_or(bit, std::memory_order_relaxed);
    }
    expert_wgrad_kernel<kLoads, kHeld><<<grid, kThreads, bytes, stream>>>(tmY, tmX, tmW, tmAdd, p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_expert_wgrad(const ExpertWgradArgs &a, cudaStream_t stream)
{
    int dev = 0;
    cudaError_t err = expert_device(&dev);
    if (err != cudaSuccess) return err;
    CUtensorMap tmY, tmX, tmW, tmAdd;
    const uint64_t R = a.R > 0 ? a.R : 1;   // (no rows: the maps are not used)
    const uint64_t yd[2] = {static_cast<uint64_t>(a.rows), R};
    const uint32_t yb[2] = {64, kRows};
    const uint64_t xd[2] = {static_cast<uint64_t>(a.cols), R};
    const uint32_t xb[2] = {128, kRows};
    if (!encode_map(&tmY, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.R > 0 ? a.dY : a.dW, 2, yd, yb) ||
        !encode_map(&tmX, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.R > 0 ? a.X : a.dW, 2, xd, xb))
        return cudaErrorInvalidValue;
    // boxes of 16 columns x 32 rows
    const uint64_t wd[3] = {static_cast<uint64_t>(a.cols), static_cast<uint64_t>(a.rows), static_cast<uint64_t>(a.E)};
    const uint32_t wb[3] = {16, 32, 1};
    const bool out_ok = a.bf16_out ? encode_map(&tmW, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.dW, 3, wd, wb,
                                                CU_TENSOR_MAP_SWIZZLE_32B)
                                   : encode_map(&tmW, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, a.dW, 3, wd, wb,
                                                CU_TENSOR_MAP_SWIZZLE_64B);
    // (nothing to add: the map is not used)
    if (!out_ok || !encode_map(&tmAdd, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, a.add ? a.add : a.dW, 3, wd, wb,
                               CU_TENSOR_MAP_SWIZZLE_64B))
        return cudaErrorInvalidValue;
    Params p;
    p.X_scale = a.X_scale;
    p.offsets = a.offsets;
    p.R = a.R;
    p.E = a.E;
    p.has_add = a.add != nullptr;
    p.segment = a.bf16_out ? kSegmentBf16 : kSegment;
    p.rows = a.rows;
    p.cols = a.cols;
    p.x_ue8m0 = a.x_ue8m0;
    p.bf16_out = a.bf16_out;
    p.m_tiles = (a.rows + kTileM - 1) / kTileM;
    p.n_tiles = (a.cols + kTileN - 1) / kTileN;
    p.status = a.status;
    const int64_t tiles = static_cast<int64_t>(a.E) * p.m_tiles * p.n_tiles;
    const int pairs = device_sm_count(dev) / 2;
    const dim3 grid(2 * static_cast<unsigned>(tiles < pairs ? tiles : pairs));
    const bool several = a.R > p.segment;
    const auto run = a.bf16_out ? several ? a.add ? launch<true, true> : launch<false, true>
                                          : a.add ? launch<true, false> : launch<false, false>
                                : a.add || several ? launch<true, false> : launch<false, false>;
    return run(dev, grid, stream, tmY, tmX, tmW, tmAdd, p);
}

}  // namespace moe
