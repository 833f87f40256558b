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
//   warps 2, 3 and the last two  scale producers: gather the bytes of 16 128-blocks per row; warp 3
//               allocates TMEM
//   warps 4..7  epilogue: TMEM -> registers -> bf16, transposed through shared memory; with the gated
//               activation or its gradient (expert_gemm_epilogue.cuh) the warps from 4 on
//
// Measured (bursts, 1.94 GHz): 16384 tokens on 128 experts, top 8, 2048 x 2048: 354 to 372 us, 3.0 PFLOP/s, the
// tensor pipe 67% busy; the rest is the latency of a ring that 180 KiB in flight per SM do not quite cover (no unit
// is at its limit: the joined products, whose loop it is too, have L2 at 51 to 59% and read 12 to 13 TB/s from it; back
// to back the board's power limit makes it 417 us, and uniformly random codes draw so much that they take 391 in bursts).  The input gradient of 16381 unevenly routed
// tokens, 64 experts of 1024 x 4096: 122 us against 85 for its bytes.
#include <mutex>

#include "expert_gemm_epilogue.cuh"

namespace moe {
namespace {

template <Mode kMode>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(threads(kMode), 1)
    expert_gemm_kernel(const __grid_constant__ TokenMaps tmX, const __grid_constant__ CUtensorMap tmW,
                       const __grid_constant__ CUtensorMap tmY, const Params p)
{
    constexpr int kRing = stages(kMode);
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sf_ring = ring + kRing * kStageBytes;
    uint8_t *epi = sf_ring + kScaleSlots * kScaleSlotBytes;
    Tail &tail = *reinterpret_cast<Tail *>(epi + epi_bytes(kMode));
    volatile int *abort_flag = &tail.abort;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kRing; ++s) {
            mbar_init(&tail.full[s], rank == 0 ? 2 : 1);   // the leader's: its own stage and the other CTA's
            mbar_init(&tail.empty[s], 1);
        }
        for (int s = 0; s < kScaleSlots; ++s) {
            mbar_init(&tail.sf_full[s], 4);
            mbar_init(&tail.sf_empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tail.acc_full[b], 1);
            mbar_init(&tail.acc_empty[b], 8 * teams(kMode));
        }
        for (int i = 0; i < teams(kGated); ++i)
            for (int k = 0; k < 4; ++k) mbar_init(&tail.words[i][k], 1);
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
                    if constexpr (gated(kMode)) {
                        // 16 rows of the gate half, then the same 16 of the up half, four times
#pragma unroll
                        for (int g = 0; g < 4; ++g)
                            tma_load_5d(a + g * 32 * kBlk, &tmW, &tail.full[s], kb * kBlk, 0, (m0 >> 5) + g, 0, t.e, keep);
                    } else {
                        tma_load_3d(a, &tmW, &tail.full[s], p.transpose ? m0 : kb * kBlk, p.transpose ? kb * kBlk : m0, t.e, keep);
                    }
                    tma_load_2d(b, map, &tail.full[s], kb * kBlk, row0, keep);
                }
                __syncwarp();
                ++issued;
                if (++s == kRing) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
        if (!ok) {
            // let the copies already issued land before the CTA ends
            const uint32_t from = issued > kRing ? issued - kRing : 0u;
            for (uint32_t x = from; x < issued; ++x) {
                volatile int no_abort = 0;
                mbar_wait_bounded(&tail.full[x % kRing], (x / kRing) & 1u, &no_abort);
            }
        }
        if (rank != 0) {
            // the leader's commits arrive in this CTA's memory too: it stays until the last of them has
            volatile int no_abort = 0;
            mbar_wait_bounded(&tail.drain, 0, &no_abort, 32);
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
                if (++s == kRing) {
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
                    if (++s == kRing) {
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
    } else if (warp < 4 || warp >= 4 + 4 * teams(kMode)) {
        // Scale words: byte i of a row's word is the scale of 128-block 4 q + i.  Tokens: row r at
        // lane r % 32, word r / 32 of a 128-row atom; features: one word for the whole 128.  Two warps,
        // one for each atom, fill a slot with 16 blocks; two such teams take turns, so that a team has
        // two tiles' time (16 blocks each) for the loads' latency and the hand-over.  (With the activation's
        // epilogue the one team fills both slots.)
        constexpr bool kTurns = scale_teams(kMode) == 2;
        const int team = warp >= 4, half = warp & 1;
        const int m_blocks = (p.out + kBlk - 1) / kBlk;
        uint32_t turn = 0, ph = 0;
        bool bad = false, ok = true;
        for (Walk walk(pair, p.m_tiles); walk.tile < tiles && ok; walk.next(pairs, p.m_tiles)) {
            Tile t;
            t.e = -1;
            for (int k0 = 0; k0 < blocks && ok; k0 += 16, turn ^= 1u) {
                if (kTurns && turn != static_cast<uint32_t>(team)) continue;
                if (t.e < 0) t = walk.get(tail);
                // (blocks and rows that are not there read their neighbour's scale and are never used: the
                // loads carry no condition and are all in flight together)
                const int n = blocks - k0;
                uint32_t feat[4], tok[4][4];
                if (half == 0) {
                    // (gated: lane and row, modulo 32, are a row of the gate half below 16, of the up half from 16)
                    const int mb = gated(kMode) ? t.m0 / kTileM + (lane < 16 ? 0 : m_blocks >> 1)
                                   : t.m0 / kBlk + rank < m_blocks ? t.m0 / kBlk + rank : m_blocks - 1;
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
                ok = __all_sync(0xffffffffu, mbar_wait_bounded(&tail.sf_empty[turn], ph ^ 1u, abort_flag, 32));
                if (kTurns || turn) ph ^= 1u;
                uint4 *slot = reinterpret_cast<uint4 *>(sf_ring + turn * kScaleSlotBytes);
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
                if (lane == 0) mbar_arrive_at(&tail.sf_full[turn], 0);
            }
        }
        if (bad) tail.bad_scale = 1;
    } else {
        const EpilogueWarp wp{epi, tmem, static_cast<int>(rank), (warp >> 2) - 1, warp & 3, lane, pair, pairs, tiles};
        if constexpr (kMode == kPlain)
            plain_epilogue(p, tail, wp);
        else if constexpr (kMode == kGated)
            gated_epilogue(p, tail, wp);
        else if constexpr (kMode == kGatedOnly)
            gated_only_epilogue(p, tail, wp);
        else
            gated_grad_epilogue(p, tmY, tail, wp);
    }

    tc_fence_before_sync();
    cluster_sync();               // the leader's MMAs have read the other CTA's memory
    tc_fence_after_sync();
    if (warp == 3) tmem_dealloc_pair(tmem, kTmemCols);
    if (threadIdx.x == 0) {
        if (tail.abort) {
            report_status(p.status, MOE_ERR_TIMEOUT);
            if constexpr (gated(kMode)) {
                // This CTA may have given up a wait for scale words.  The other one sends none any more, being past its
                // last chunk too, and those on their way here land long before this time (1 ms by the clock) is over.
                // (A CTA that gave up no wait has had all of its words.)
                const uint64_t t0 = globaltimer_ns();
                for (int i = 0; i < (1 << 20) && globaltimer_ns() - t0 < 1000000; ++i) __nanosleep(1000);
            }
        }
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

namespace {

// What the three launches share: the tensor maps of the rows and of the weights, the scales' vector
// width, the grid.
template <Mode kMode>
cudaError_t launch(Params &p, const void *X, const void *W, int rows, int cols, cudaStream_t stream)
{
    int dev = 0;
    cudaError_t err = expert_device(&dev);
    if (err != cudaSuccess) return err;

    TokenMaps tmX;
    CUtensorMap tmW;
    const uint64_t xd[2] = {static_cast<uint64_t>(p.red), static_cast<uint64_t>(p.R)};
    for (int i = 0; i < kBoxes; ++i) {
        const uint32_t xb[2] = {kBlk, static_cast<uint32_t>(box_rows(i))};
        if (!encode_map(&tmX.map[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, X, 2, xd, xb)) return cudaErrorInvalidValue;
    }
    if (gated(kMode)) {
        // 16 rows of either half in one box
        const uint64_t wd[5] = {static_cast<uint64_t>(cols), 16, static_cast<uint64_t>(rows / 32), 2, static_cast<uint64_t>(p.E)};
        const uint32_t wb[5] = {kBlk, 16, 1, 2, 1};
        if (!encode_map(&tmW, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, W, 5, wd, wb)) return cudaErrorInvalidValue;
    } else {
        const uint64_t wd[3] = {static_cast<uint64_t>(cols), static_cast<uint64_t>(rows), static_cast<uint64_t>(p.E)};
        const uint32_t wb[3] = {128, 128, 1};
        if (!encode_map(&tmW, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, W, 3, wd, wb)) return cudaErrorInvalidValue;
    }

    CUtensorMap tmY = tmW;
    if (kMode == kGatedGrad && p.Y) {
        // a warp's 32 features of a chunk's tokens
        const uint64_t yd[2] = {2 * static_cast<uint64_t>(p.I), static_cast<uint64_t>(p.R)};
        const uint32_t yb[2] = {32, chunk_tokens(kGatedGrad)};
        if (!encode_map(&tmY, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, p.Y, 2, yd, yb, CU_TENSOR_MAP_SWIZZLE_64B))
            return cudaErrorInvalidValue;
    }

    static std::atomic<uint64_t> done{0};
    const uint64_t bit = 1ull << (dev & 63);
    if (!(done.load(std::memory_order_relaxed) & bit)) {
        err = cudaFuncSetAttribute(expert_gemm_kernel<kMode>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   static_cast<int>(smem_bytes(kMode)));
        if (err != cudaSuccess) return err;
        done.fetch_or(bit, std::memory_order_relaxed);
    }
    const uintptr_t xs = reinterpret_cast<uintptr_t>(p.X_scale);
    p.x_vec = (p.red / kBlk) % 4 == 0 && xs % (p.x_ue8m0 ? 4 : 16) == 0;
    if (p.x_ue8m0 && (p.red / kBlk) % 16 == 0 && xs % 16 == 0) p.x_vec = 2;
    p.m_tiles = (p.out + kTileM - 1) / kTileM;
    // the most tiles that R rows in E groups can make; no more pairs than that
    const int64_t most = (p.R / kTileN + (p.R < p.E ? p.R : p.E) + 1) * p.m_tiles;
    const int pairs = device_sm_count(dev) / 2;
    const int grid = 2 * static_cast<int>(most < pairs ? most : pairs);
    expert_gemm_kernel<kMode><<<grid, threads(kMode), smem_bytes(kMode), stream>>>(tmX, tmW, tmY, p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_expert_gemm(const ExpertGemmArgs &a, cudaStream_t stream)
{
    Params p{};
    p.X_scale = a.X_scale;
    p.W_scale = a.W_scale;
    p.offsets = a.offsets;
    p.R = a.R;
    p.E = a.E;
    p.out = a.transpose ? a.cols : a.rows;
    p.red = a.transpose ? a.rows : a.cols;
    p.transpose = a.transpose;
    p.x_ue8m0 = a.x_ue8m0;
    p.w_ue8m0 = a.w_ue8m0;
    p.Y = a.Y;
    p.status = a.status;
    return launch<kPlain>(p, a.X, a.W, a.rows, a.cols, stream);
}

cudaError_t launch_expert_swiglu(const ExpertSwigluArgs &a, cudaStream_t stream)
{
    Params p{};
    p.X_scale = a.X_scale;
    p.W_scale = a.W_scale;
    p.offsets = a.offsets;
    p.R = a.R;
    p.E = a.E;
    p.I = a.I;
    p.out = a.backward ? a.I : 2 * a.I;
    p.red = a.H;
    p.transpose = a.backward;
    p.x_ue8m0 = a.x_ue8m0;
    p.w_ue8m0 = a.w_ue8m0;
    p.k_ue8m0 = a.gu_ue8m0;
    p.out_ue8m0 = a.out_ue8m0;
    p.K = static_cast<uint8_t *>(a.GU);
    p.K_scale = a.GU_scale;
    p.A = static_cast<uint8_t *>(a.A);
    p.A_scale = a.A_scale;
    p.Y = a.dGU;
    p.Q = static_cast<uint8_t *>(a.dGU_fp8);
    p.Q_scale = a.dGU_scale;
    p.status = a.status;
    if (a.backward) return launch<kGatedGrad>(p, a.X, a.W, a.H, a.I, stream);
    return a.GU ? launch<kGated>(p, a.X, a.W, 2 * a.I, a.H, stream) : launch<kGatedOnly>(p, a.X, a.W, 2 * a.I, a.H, stream);
}

}  // namespace moe
