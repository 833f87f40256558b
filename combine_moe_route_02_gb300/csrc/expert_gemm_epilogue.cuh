// expert_gemm_epilogue.cuh -- what follows the product in its own launch: bf16 rows; the gated activation; the
// gated activation's gradient.
//
// A warp reads its quarter of the accumulator (32 lanes: features) in chunks of 32 tokens (columns), as fragments of
// 8x8: element 16 h + 4 c + 2 r + i of a lane is feature 16 h + 8 r + lane / 4 of token 8 c + 2 (lane % 4) + i.
// With s = 2 c + i a lane has eight tokens, the same ones as the lanes that agree with it modulo 4.
//
// E4M3 codes leave through shared memory.  stmatrix and ldmatrix move 8x8 matrices of two bytes; the two bytes here
// are the codes of features j and j + 8 (r = 0 and 1) of one token, so that 16 features are 16 bytes of a token's
// row in the order 0, 8, 1, 9, ...; four byte permutations put them right on the way to global memory.
#pragma once

#include "expert_gemm.cuh"

namespace moe {
namespace {

constexpr uint32_t kAll = 0xffffffffu;

struct EpilogueWarp {
    uint8_t *epi;                 // the epilogue's shared memory
    uint32_t tmem;
    int rank, team, w, lane;      // CTA of the pair, team of four warps, warp of the team
    int pair, pairs, tiles;
};

// The accumulator has been read: one arrival of each warp at the leader.
__device__ __forceinline__ void release_accumulator(Tail &tail, int b, int lane)
{
    tc_fence_before_sync();
    if (lane == 0) mbar_arrive_at(&tail.acc_empty[b], 0);
}

__device__ __forceinline__ void plain_epilogue(const Params &p, Tail &tail, const EpilogueWarp &e)
{
    const int w = e.w, lane = e.lane;
    uint8_t *buf = e.epi + w * 32 * 64;
    const uint32_t buf_addr = smem_u32(buf);
    const uint32_t lane_addr = e.tmem + (static_cast<uint32_t>(w * 32) << 16);
    int j = 0;
    for (Walk walk(e.pair, p.m_tiles); walk.tile < e.tiles; walk.next(e.pairs, p.m_tiles)) {
        const Tile t = walk.get(tail);
        const int b = j & 1;
        if (!__all_sync(kAll, mbar_wait_bounded(&tail.acc_full[b], (j >> 1) & 1, &tail.abort, 64))) break;
        tc_fence_after_sync();
        const int m = t.m0 + e.rank * kHalfM + w * 32;  // this warp's features
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
        release_accumulator(tail, b, lane);
        ++j;
    }
}

// ---------------------------------------------------------------------------
// Pieces of the activation's two epilogues
// ---------------------------------------------------------------------------
// Whether all of a team's 128 threads say so (they go on or stop together: a warp that left alone would leave the
// others at their next barrier).
__device__ __forceinline__ bool team_all(int team, bool ok)
{
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.and.aligned.pred q, %2, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(__all_sync(kAll, ok))), "r"(2 + team)
        : "memory");
    return r != 0;
}

// The teams take a tile's chunks in turn, and with every tile another team begins (kGated: a tile of 7 chunks is 3, 2
// and 2).
template <Mode kMode>
struct Chunks {
    static constexpr int kStep = teams(kMode) * chunk_tokens(kMode);
    int first;
    __device__ __forceinline__ explicit Chunks(int team) : first(team) {}
    __device__ __forceinline__ void next() { first = first == 0 ? teams(kMode) - 1 : first - 1; }
    __device__ __forceinline__ int begin() const { return first * chunk_tokens(kMode); }
};

// The largest of m[s] over the eight lanes that share tokens: lane l is left with that of s = l / 4, which is token
// lane_token(l).
__device__ __forceinline__ float max_of_lanes(const float (&m)[8], int lane)
{
    float a[4], b[2];
    const bool h16 = lane & 16, h8 = lane & 8, h4 = lane & 4;
#pragma unroll
    for (int k = 0; k < 4; ++k) a[k] = fmaxf(h16 ? m[k + 4] : m[k], __shfl_xor_sync(kAll, h16 ? m[k] : m[k + 4], 16));
#pragma unroll
    for (int k = 0; k < 2; ++k) b[k] = fmaxf(h8 ? a[k + 2] : a[k], __shfl_xor_sync(kAll, h8 ? a[k] : a[k + 2], 8));
    return fmaxf(h4 ? b[1] : b[0], __shfl_xor_sync(kAll, h4 ? b[0] : b[1], 4));
}
__device__ __forceinline__ int lane_token(int lane) { return (lane >> 3) * 8 + (lane & 3) * 2 + ((lane >> 2) & 1); }
// What the lane of token s of this lane's eight holds.
__device__ __forceinline__ uint32_t of_token(uint32_t word, int s, int lane) { return __shfl_sync(kAll, word, 4 * s + (lane & 3)); }

// Two tokens at a time (i = 0, 1): the values of feature r of chunk column c, and codes of features r = 0 and 1 of
// both tokens, the first token's in the low half.
__device__ __forceinline__ float2 both(const float *v, int at) { return make_float2(v[at], v[at + 1]); }
__device__ __forceinline__ float2 twice(float x) { return make_float2(x, x); }
__device__ __forceinline__ uint32_t codes_of(float2 r0, float2 r1)
{
    uint32_t q;
    asm("{\n\t.reg .b16 a, b;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 a, %3, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 b, %4, %2;\n\t"
        "mov.b32 %0, {a, b};\n\t}"
        : "=r"(q)
        : "f"(r0.x), "f"(r0.y), "f"(r1.x), "f"(r1.y));
    return q;
}
__device__ __forceinline__ float2 sigmoid2(float2 g)
{
    // (as sigmoid(), both at a time)
    const float2 t = __fmul2_rn(g, twice(-1.44269504088896340736f));
    float2 e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(t.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(t.y));
    e = __fadd2_rn(e, twice(1.f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(e.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(e.y));
    return r;
}

// 16 bytes of a row in the order 0, 8, 1, 9, ... put right, and back.
__device__ __forceinline__ uint4 in_order(const uint4 &x)
{
    return make_uint4(__byte_perm(x.x, x.y, 0x6420), __byte_perm(x.z, x.w, 0x6420), __byte_perm(x.x, x.y, 0x7531),
                      __byte_perm(x.z, x.w, 0x7531));
}
__device__ __forceinline__ uint4 in_pairs(const uint4 &x)
{
    return make_uint4(__byte_perm(x.x, x.z, 0x5140), __byte_perm(x.x, x.z, 0x7362), __byte_perm(x.y, x.w, 0x5140),
                      __byte_perm(x.y, x.w, 0x7362));
}

// Shared memory by its address (the ring's start is rounded up through an integer, so that accesses through pointers
// derived from it are generic ones).
__device__ __forceinline__ uint4 lds128(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void sts128(uint32_t a, const uint4 &v)
{
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t a)
{
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void sts32(uint32_t a, uint32_t v) { asm volatile("st.shared.b32 [%0], %1;" ::"r"(a), "r"(v) : "memory"); }

// Four 8x8 matrices of two bytes, transposed, to / from rows of 16 bytes: lane l gives the address of row l.
__device__ __forceinline__ void store_rows(uint32_t row_addr, const uint32_t (&m)[4])
{
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(row_addr), "r"(m[0]),
                 "r"(m[1]), "r"(m[2]), "r"(m[3])
                 : "memory");
}
__device__ __forceinline__ void load_rows(uint32_t row_addr, uint32_t (&m)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(m[0]), "=r"(m[1]), "=r"(m[2]), "=r"(m[3])
                 : "r"(row_addr)
                 : "memory");
}

// A word to CTA `rank`'s shared memory at this offset, counted there on the barrier at that one.
__device__ __forceinline__ void send_word(uint32_t addr, uint32_t word, uint32_t bar, uint32_t rank)
{
    asm volatile(
        "{\n\t.reg .b32 a, b;\n\t"
        "mapa.shared::cluster.u32 a, %0, %3;\n\t"
        "mapa.shared::cluster.u32 b, %2, %3;\n\t"
        "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b32 [a], %1, [b];\n\t}" ::"r"(addr),
        "r"(word), "r"(bar), "r"(rank)
        : "memory");
}

// ---------------------------------------------------------------------------
// Gated activation: a = g / (1 + exp(-g)) u of the product, in E4M3, and (checkpoint) g and u in E4M3.
//
// The rows of the weights lie in the tile so that a warp's 32 lanes of TMEM are 16 features of the gate half, then
// the same 16 of the up half (h = 0 and 1 of the fragments): a lane has both.  A block of 128 features is the pair's
// eight warps; each finds the scale bytes of its 16 features (the byte of the largest is the largest byte), sends a
// word of three for each token to both CTAs, and takes the largest of eight.
//
// Measured: 16384 tokens, 128 experts, top 8, H = 2048, I = 1024: 381 us in graphs of 20 after a pause, 2.9 PFLOP/s (in
// bursts of 5: 389), where the product alone with its bf16 rows and the same operands takes 367 (372); the launch without
// any epilogue 328; back to back 444, the product alone 420 (the board's power).  The tensor pipe is 63 to 66% busy, DRAM 59%.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void gated_epilogue(const Params &p, Tail &tail, const EpilogueWarp &e)
{
    const int team = e.team, w = e.w, lane = e.lane, tok = lane_token(lane);
    const uint32_t stage = smem_u32(e.epi) + team * 3 * 2048;         // codes of a, g, u: 32 tokens x 64 features each
    const uint32_t words = smem_u32(e.epi) + stage_bytes(kGated) + team * 2 * 1024;
    // 16-byte piece f of token t lies at place f ^ (t / 2 % 4)
    const uint32_t put = stage + lane * 64 + ((w ^ ((lane >> 1) & 3)) << 4);
    const int out_tok = w * 8 + (lane >> 2), piece = lane & 3;
    const uint32_t take = stage + out_tok * 64 + ((piece ^ ((out_tok >> 1) & 3)) << 4);
    const uint32_t lane_addr = e.tmem + (static_cast<uint32_t>(w * 32) << 16);
    const int nb = p.I / kBlk;
    int j = 0;
    uint32_t n = 0;                                    // this team's chunks
    bool ok = true;
    Chunks<kGated> chunks(team);
    constexpr int kChunkStep = Chunks<kGated>::kStep;
    for (Walk walk(e.pair, p.m_tiles); walk.tile < e.tiles; walk.next(e.pairs, p.m_tiles), chunks.next(), ++j) {
        const Tile t = walk.get(tail);
        const int b = j & 1, fb = t.m0 / kTileM;       // its block of 128 features
        ok = team_all(team, mbar_wait_bounded(&tail.acc_full[b], (j >> 1) & 1, &tail.abort, 64));
        if (!ok) break;
        tc_fence_after_sync();
        if (chunks.begin() >= t.rows) release_accumulator(tail, b, lane);
        for (int c0 = chunks.begin(); c0 < t.rows; c0 += kChunkStep, ++n) {
            float v[32];
            tmem_ld_fragments(lane_addr + b * kTileN + c0, v);
            tmem_ld_wait();
            if (c0 + kChunkStep >= t.rows) release_accumulator(tail, b, lane);
            float2 a[4][2];
            float ma[8], mg[8], mu[8];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float2 g = both(v, 4 * c + 2 * r);
                    a[c][r] = __fmul2_rn(__fmul2_rn(g, sigmoid2(g)), both(v, 16 + 4 * c + 2 * r));
                }
                ma[2 * c] = fmaxf(fabsf(a[c][0].x), fabsf(a[c][1].x));
                ma[2 * c + 1] = fmaxf(fabsf(a[c][0].y), fabsf(a[c][1].y));
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    mg[2 * c + i] = fmaxf(fabsf(v[4 * c + i]), fabsf(v[4 * c + 2 + i]));
                    mu[2 * c + i] = fmaxf(fabsf(v[16 + 4 * c + i]), fabsf(v[18 + 4 * c + i]));
                }
            }
            uint32_t word = block_scale_byte(max_of_lanes(ma, lane));
            word |= block_scale_byte(max_of_lanes(mu, lane)) << 16 | block_scale_byte(max_of_lanes(mg, lane)) << 24;
            // eight warps' words for each token; a buffer is written again two chunks later, when the words of the
            // chunk between have come from every warp, which each sent after it had read this one
            const uint32_t slot = words + (n & 1) * 1024;
            uint64_t *bar = &tail.words[team][n & 1];
            if (w == 0 && lane == 0) mbar_arrive_expect_tx(bar, 8 * 32 * 4);
            const uint32_t to = slot + ((e.rank * 4 + w) * 32 + tok) * 4;
            send_word(to, word, smem_u32(bar), 0);
            send_word(to, word, smem_u32(bar), 1);
            ok = mbar_wait_bounded(bar, (n >> 1) & 1, &tail.abort);
            // the top byte is the largest word's, the two others are compared as halves
            uint32_t top = 0, halves = 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint32_t x = lds32(slot + (k * 32 + tok) * 4);
                top = max(top, x);
                halves = __vmaxu2(halves, x & 0x00FF00FFu);
            }
            const uint32_t ba = halves & 0xFFu, bu = halves >> 16, bg = top >> 24;
            if (e.rank == 0 && c0 + tok < t.rows) {
                const int64_t row = t.row0 + c0 + tok;
                if (w == 0) store_scale(p.A_scale, p.out_ue8m0, row * nb + fb, ba);
                if (w == 1) store_scale(p.K_scale, p.out_ue8m0, row * 2 * nb + fb, bg);
                if (w == 2) store_scale(p.K_scale, p.out_ue8m0, (row * 2 + 1) * nb + fb, bu);
            }
            // the scales' reciprocals: a's, and as two bf16 numbers g's and u's
            const uint32_t ra = __float_as_uint(scale_reciprocal(ba)), rgu = (254u - bg) << 7 | (254u - bu) << 23;
            uint32_t q[3][4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float2 ia = make_float2(__uint_as_float(of_token(ra, 2 * c, lane)), __uint_as_float(of_token(ra, 2 * c + 1, lane)));
                q[0][c] = codes_of(__fmul2_rn(a[c][0], ia), __fmul2_rn(a[c][1], ia));
                const uint32_t t0 = of_token(rgu, 2 * c, lane), t1 = of_token(rgu, 2 * c + 1, lane);
                const float2 ig = make_float2(__uint_as_float(t0 << 16), __uint_as_float(t1 << 16));
                const float2 iu = make_float2(__uint_as_float(t0 & 0xFFFF0000u), __uint_as_float(t1 & 0xFFFF0000u));
                q[1][c] = codes_of(__fmul2_rn(both(v, 4 * c), ig), __fmul2_rn(both(v, 4 * c + 2), ig));
                q[2][c] = codes_of(__fmul2_rn(both(v, 16 + 4 * c), iu), __fmul2_rn(both(v, 18 + 4 * c), iu));
            }
            // (the codes of the chunk before have been read: its words came after that)
            store_rows(put, q[0]);
            store_rows(put + 2048, q[1]);
            store_rows(put + 4096, q[2]);
            ok = team_all(team, ok);
            if (!ok) break;
            if (c0 + out_tok < t.rows) {
                const int64_t row = t.row0 + c0 + out_tok;
                const int f = fb * kBlk + e.rank * 64 + piece * 16;
                *reinterpret_cast<uint4 *>(p.A + row * p.I + f) = in_order(lds128(take));
                uint8_t *k = p.K + row * 2 * p.I + f;
                *reinterpret_cast<uint4 *>(k) = in_order(lds128(take + 2048));
                *reinterpret_cast<uint4 *>(k + p.I) = in_order(lds128(take + 4096));
            }
        }
        if (!ok) break;
    }
}

// ---------------------------------------------------------------------------
// Without the checkpoint a lane keeps 16 values of a chunk, and there is room for two chunks: the words of one are on
// their way while the next is computed, across tiles too.
//
// A warp sends chunk n's words before it has read those of n - 1, and after those of n - 2 have come from every warp,
// which says that every warp has read those of n - 4: four buffers in turn.  The codes of chunk n are put where those of
// n - 2 lay, which the team has read before its barrier of n - 1: two.
//
// Measured: 16381 tokens of 64 experts, H = 1024, I = 2048 (8 blocks of reduction a tile: the epilogue sets the pace): 111 to
// 114 us in bursts, 127 back to back (waiting for each chunk's words at once 127 and 137); 99 and 110 without an epilogue.
// ---------------------------------------------------------------------------
struct PendingChunk {
    float2 a[4][2];
    int64_t row0;                 // its first row, how many it has, their block of features
    int rows, fb;
};

__device__ __forceinline__ bool finish_chunk(const Params &p, Tail &tail, const EpilogueWarp &e, const PendingChunk &c, uint32_t n)
{
    const int team = e.team, w = e.w, lane = e.lane, tok = lane_token(lane), nb = p.I / kBlk;
    const uint32_t stage = smem_u32(e.epi) + (team * 2 + (n & 1)) * 2048;
    const uint32_t slot = smem_u32(e.epi) + stage_bytes(kGatedOnly) + (team * 4 + (n & 3)) * 1024;
    const int out_tok = w * 8 + (lane >> 2), piece = lane & 3;
    bool ok = mbar_wait_bounded(&tail.words[team][n & 3], (n >> 2) & 1, &tail.abort);
    uint32_t word = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) word = max(word, lds32(slot + (k * 32 + tok) * 4));
    if (e.rank == 0 && w == 0 && tok < c.rows) store_scale(p.A_scale, p.out_ue8m0, (c.row0 + tok) * nb + c.fb, word);
    const uint32_t inv = __float_as_uint(scale_reciprocal(word));
    uint32_t q[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        const float2 i = make_float2(__uint_as_float(of_token(inv, 2 * x, lane)), __uint_as_float(of_token(inv, 2 * x + 1, lane)));
        q[x] = codes_of(__fmul2_rn(c.a[x][0], i), __fmul2_rn(c.a[x][1], i));
    }
    store_rows(stage + lane * 64 + ((w ^ ((lane >> 1) & 3)) << 4), q);
    ok = team_all(team, ok);
    if (ok && out_tok < c.rows)
        *reinterpret_cast<uint4 *>(p.A + (c.row0 + out_tok) * p.I + c.fb * kBlk + e.rank * 64 + piece * 16) =
            in_order(lds128(stage + out_tok * 64 + ((piece ^ ((out_tok >> 1) & 3)) << 4)));
    return ok;
}

__device__ __forceinline__ void gated_only_epilogue(const Params &p, Tail &tail, const EpilogueWarp &e)
{
    constexpr int kChunkStep = Chunks<kGatedOnly>::kStep;
    const int team = e.team, w = e.w, lane = e.lane, tok = lane_token(lane);
    const uint32_t words = smem_u32(e.epi) + stage_bytes(kGatedOnly) + team * 4 * 1024;
    const uint32_t lane_addr = e.tmem + (static_cast<uint32_t>(w * 32) << 16);
    int j = 0;
    uint32_t n = 0;                                    // this team's chunks
    bool ok = true;
    PendingChunk before;
    Chunks<kGatedOnly> chunks(team);
    for (Walk walk(e.pair, p.m_tiles); walk.tile < e.tiles; walk.next(e.pairs, p.m_tiles), chunks.next(), ++j) {
        const Tile t = walk.get(tail);
        const int b = j & 1;
        ok = team_all(team, mbar_wait_bounded(&tail.acc_full[b], (j >> 1) & 1, &tail.abort, 64));
        if (!ok) break;
        tc_fence_after_sync();
        if (chunks.begin() >= t.rows) release_accumulator(tail, b, lane);
        for (int c0 = chunks.begin(); c0 < t.rows; c0 += kChunkStep, ++n) {
            float v[32];
            tmem_ld_fragments(lane_addr + b * kTileN + c0, v);
            tmem_ld_wait();
            if (c0 + kChunkStep >= t.rows) release_accumulator(tail, b, lane);
            PendingChunk now;
            now.row0 = t.row0 + c0;
            now.rows = t.rows - c0;
            now.fb = t.m0 / kTileM;
            float m[8];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float2 g = both(v, 4 * c + 2 * r);
                    now.a[c][r] = __fmul2_rn(__fmul2_rn(g, sigmoid2(g)), both(v, 16 + 4 * c + 2 * r));
                }
                m[2 * c] = fmaxf(fabsf(now.a[c][0].x), fabsf(now.a[c][1].x));
                m[2 * c + 1] = fmaxf(fabsf(now.a[c][0].y), fabsf(now.a[c][1].y));
            }
            const uint32_t word = block_scale_byte(max_of_lanes(m, lane));
            uint64_t *bar = &tail.words[team][n & 3];
            if (w == 0 && lane == 0) mbar_arrive_expect_tx(bar, 8 * 32 * 4);
            const uint32_t to = words + (n & 3) * 1024 + ((e.rank * 4 + w) * 32 + tok) * 4;
            send_word(to, word, smem_u32(bar), 0);
            send_word(to, word, smem_u32(bar), 1);
            if (n > 0) {
                ok = finish_chunk(p, tail, e, before, n - 1);
                if (!ok) break;
            }
            before = now;
        }
        if (!ok) break;
    }
    if (ok && n > 0) finish_chunk(p, tail, e, before, n - 1);
}

// ---------------------------------------------------------------------------
// The activation's gradient: the product is da; g and u come from the checkpoint (codes and scales).
//   s = 1 / (1 + exp(-g));  dg = da u s (1 + g (1 - s));  du = da g s
// in bf16 and in E4M3.  A CTA's 128 features are a block, its scale bytes are joined over a team's four warps.
//
// Chunks of 16 tokens (c = 0, 1; element 8 h + 4 c + 2 r + i of a lane) keep a warp near 96 registers (two words are
// spilled), so that four teams fit: the work of a chunk is a chain of short steps, and what hides their latency is the
// number of warps.
//
// Measured: 16384 tokens, 128 experts, top 8, H = 2048, I = 1024: 314 to 321 us in short graphs, 348 back to back (power),
// 5.1 TB/s of its bytes; without any epilogue 200, the bytes alone 239.  Issue slots 50% busy, DRAM 70%.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void load_fragments16(uint32_t taddr, float (&v)[16])
{
    uint32_t r[16];
#pragma unroll
    for (int h = 0; h < 2; ++h)
        asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(r[8 * h]), "=r"(r[8 * h + 1]), "=r"(r[8 * h + 2]), "=r"(r[8 * h + 3]), "=r"(r[8 * h + 4]),
                       "=r"(r[8 * h + 5]), "=r"(r[8 * h + 6]), "=r"(r[8 * h + 7])
                     : "r"(taddr + (static_cast<uint32_t>(16 * h) << 16))
                     : "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// As store_transposed(), of 16 tokens.
__device__ __forceinline__ void store_transposed16(uint32_t buf, int lane, const float (&v)[16])
{
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        uint32_t m[4];
#pragma unroll
        for (int f = 0; f < 4; ++f) {
            const int at = 8 * (f >> 1) + 4 * c + 2 * (f & 1);
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[at], v[at + 1]);
            m[f] = *reinterpret_cast<const uint32_t *>(&h);
        }
        const int t = 8 * c + (lane & 7), f = lane >> 3;
        store_rows(buf + t * 64 + ((f ^ ((t >> 1) & 3)) << 4), m);
    }
}

// As max_of_lanes(), of four tokens: lane l is left with that of s = l / 8 (as lane l ^ 4 is).
__device__ __forceinline__ float max_of_lanes4(const float (&m)[4], int lane)
{
    const bool h16 = lane & 16, h8 = lane & 8;
    const float a = fmaxf(h16 ? m[2] : m[0], __shfl_xor_sync(kAll, h16 ? m[0] : m[2], 16));
    const float b = fmaxf(h16 ? m[3] : m[1], __shfl_xor_sync(kAll, h16 ? m[1] : m[3], 16));
    const float c = fmaxf(h8 ? b : a, __shfl_xor_sync(kAll, h8 ? a : b, 8));
    return fmaxf(c, __shfl_xor_sync(kAll, c, 4));
}

__device__ __forceinline__ void gated_grad_epilogue(const Params &p, const CUtensorMap &tmY, Tail &tail, const EpilogueWarp &e)
{
    constexpr int kTok = chunk_tokens(kGatedGrad), kChunkStep = Chunks<kGatedGrad>::kStep;
    const int team = e.team, w = e.w, lane = e.lane;
    const int tok = (lane >> 4) * 8 + (lane & 3) * 2 + ((lane >> 3) & 1);       // the token of s = lane / 8
    const uint32_t rows = smem_u32(e.epi) + (team * 4 + w) * 2048;       // bf16 rows of both halves, for the TMA
    const uint32_t buf = smem_u32(e.epi) + teams(kGatedGrad) * 4 * 2048 + (team * 4 + w) * 1024;    // codes
    const uint32_t words = smem_u32(e.epi) + stage_bytes(kGatedGrad) + team * 2 * 4 * kTok * 4;
    const uint32_t lane_addr = e.tmem + (static_cast<uint32_t>(w * 32) << 16);
    const int nb = p.I / kBlk;
    const int64_t pitch = 2 * static_cast<int64_t>(p.I);
    // E4M3 rows are read and written by two lanes for a token's 32 features; in shared memory the 16-byte pieces of
    // the gate's features 0..15, 16..31, the up half's: 16 tokens of each
    const int k_tok = lane >> 1, k_half = lane & 1;
    const uint32_t k_at = buf + k_half * 256 + k_tok * 16, m_at = buf + (lane >> 4) * 256 + (lane & 15) * 16;
    uint32_t n = 0;
    bool bad = false;
    uint4 kg = make_uint4(0, 0, 0, 0), ku = kg;
    uint32_t sg = 0, su = 0;
    // A chunk's part of the checkpoint is asked for while the chunk before is worked on, across tiles too.
    const auto fetch = [&](const Tile &t, int c0) {
        const int fb = t.m0 / kBlk + e.rank;
        if (fb >= nb || c0 >= t.rows) return;
        const int r = c0 + k_tok;
        const uint8_t *k = p.K + (t.row0 + (r < t.rows ? r : t.rows - 1)) * pitch + fb * kBlk + w * 32 + k_half * 16;
        kg = __ldcs(reinterpret_cast<const uint4 *>(k));
        ku = __ldcs(reinterpret_cast<const uint4 *>(k + p.I));
        const int q = c0 + (lane & 15);
        const int64_t at = (t.row0 + (q < t.rows ? q : t.rows - 1)) * 2 * nb + fb;
        sg = load_scale_bits(p.K_scale, p.k_ue8m0, at);
        su = load_scale_bits(p.K_scale, p.k_ue8m0, at + nb);
    };
    Chunks<kGatedGrad> chunks(team);
    Walk walk(e.pair, p.m_tiles);
    Tile next{};
    if (walk.tile < e.tiles) {
        next = walk.get(tail);
        fetch(next, chunks.begin());
    }
    for (int j = 0; walk.tile < e.tiles; ++j) {
        const Tile t = next;
        const int b = j & 1, fb = t.m0 / kBlk + e.rank, begin = chunks.begin();
        walk.next(e.pairs, p.m_tiles);
        chunks.next();
        next.rows = 0;
        if (walk.tile < e.tiles) next = walk.get(tail);
        if (!team_all(team, mbar_wait_bounded(&tail.acc_full[b], (j >> 1) & 1, &tail.abort, 64))) break;
        tc_fence_after_sync();
        // (the last tile of an odd number of blocks is half empty)
        if (fb >= nb || begin >= t.rows) {
            release_accumulator(tail, b, lane);
            fetch(next, chunks.begin());
            continue;
        }
        for (int c0 = begin; c0 < t.rows; c0 += kChunkStep, ++n) {
            const bool last = c0 + kChunkStep >= t.rows;
            float du[16], dg[16];
            load_fragments16(lane_addr + b * kTileN + c0, du);
            __syncwarp();
            sts128(k_at, in_pairs(kg));
            sts128(k_at + 512, in_pairs(ku));
            // both scales as bf16 numbers
            const uint32_t scales = __float_as_uint(scale_value(scale_bits_byte(sg, p.k_ue8m0, bad))) >> 16 |
                                    (__float_as_uint(scale_value(scale_bits_byte(su, p.k_ue8m0, bad))) & 0xFFFF0000u);
            __syncwarp();
            uint32_t k[2][4];                          // [gate, up][2 h + c]
            load_rows(m_at, k[0]);
            load_rows(m_at + 512, k[1]);
            fetch(last ? next : t, last ? chunks.begin() : c0 + kChunkStep);
            tmem_ld_wait();
            if (last) release_accumulator(tail, b, lane);
            float mg[4], mu[4];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const uint32_t t0 = __shfl_sync(kAll, scales, 8 * c + 2 * (lane & 3)), t1 = __shfl_sync(kAll, scales, 8 * c + 2 * (lane & 3) + 1);
                const float2 gs = make_float2(__uint_as_float(t0 << 16), __uint_as_float(t1 << 16));
                const float2 us = make_float2(__uint_as_float(t0 & 0xFFFF0000u), __uint_as_float(t1 & 0xFFFF0000u));
                mg[2 * c] = mg[2 * c + 1] = mu[2 * c] = mu[2 * c + 1] = 0.f;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    // the two tokens' codes of r = 0, then of r = 1
                    const uint32_t kg4 = __byte_perm(k[0][2 * h + c], 0, 0x3120), ku4 = __byte_perm(k[1][2 * h + c], 0, 0x3120);
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const int x = 8 * h + 4 * c + 2 * r;
                        const float2 g = __fmul2_rn(e4m3x2_to_f32x2(r ? kg4 >> 16 : kg4 & 0xFFFFu), gs);
                        const float2 u = __fmul2_rn(e4m3x2_to_f32x2(r ? ku4 >> 16 : ku4 & 0xFFFFu), us);
                        const float2 s = sigmoid2(g), as = __fmul2_rn(both(du, x), s);
                        const float2 slope = __ffma2_rn(g, __ffma2_rn(s, twice(-1.f), twice(1.f)), twice(1.f));
                        const float2 dg2 = __fmul2_rn(__fmul2_rn(as, u), slope), du2 = __fmul2_rn(as, g);
                        dg[x] = dg2.x, dg[x + 1] = dg2.y;
                        du[x] = du2.x, du[x + 1] = du2.y;
                        mg[2 * c] = fmaxf(mg[2 * c], fabsf(dg2.x)), mg[2 * c + 1] = fmaxf(mg[2 * c + 1], fabsf(dg2.y));
                        mu[2 * c] = fmaxf(mu[2 * c], fabsf(du2.x)), mu[2 * c + 1] = fmaxf(mu[2 * c + 1], fabsf(du2.y));
                    }
                }
            }
            const uint32_t slot = words + (n & 1) * 4 * kTok * 4;
            if (p.Q) sts32(slot + (w * kTok + tok) * 4, block_scale_byte(max_of_lanes4(mg, lane)) | block_scale_byte(max_of_lanes4(mu, lane)) << 16);
            if (p.Y) {
                if (lane == 0) bulk_wait_read<0>();    // the chunk before
                __syncwarp();
                store_transposed16(rows, lane, dg);
                store_transposed16(rows + 1024, lane, du);
                const int f = fb * kBlk + w * 32;
                if (c0 + kTok <= t.rows) {
                    // whole: two boxes (pieces of 16 bytes lie as the TMA's swizzle of 64 bytes has them)
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        const int32_t r = static_cast<int32_t>(t.row0) + c0;
                        tma_store_2d(&tmY, rows, f, r);
                        tma_store_2d(&tmY, rows + 1024, f + p.I, r);
                        bulk_commit();
                    }
                } else {
                    __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.Y) + (t.row0 + c0 + (lane >> 2)) * pitch + f + (lane & 3) * 8;
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int at = i * 8 + (lane >> 2);
                        const uint32_t y = rows + at * 64 + (((lane & 3) ^ ((at >> 1) & 3)) << 4);
                        if (c0 + at < t.rows) {
                            *reinterpret_cast<uint4 *>(dst + 8 * i * pitch) = lds128(y);
                            *reinterpret_cast<uint4 *>(dst + 8 * i * pitch + p.I) = lds128(y + 1024);
                        }
                    }
                }
            }
            if (p.Q) {
                // (a slot is written again two chunks later, behind the barrier of the one between)
                named_barrier_sync(2 + team, 128);
                uint32_t word = 0;
#pragma unroll
                for (int x = 0; x < 4; ++x) word = __vmaxu2(word, lds32(slot + (x * kTok + tok) * 4));
                if (c0 + tok < t.rows && w < 2 && !(lane & 4))
                    store_scale(p.Q_scale, p.out_ue8m0, (t.row0 + c0 + tok) * 2 * nb + w * nb + fb, w ? word >> 16 : word & 0xFFu);
                word = (0x00FE00FEu - word) << 7;      // the scales' reciprocals as bf16 numbers
                uint32_t q[2][4];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const uint32_t t0 = __shfl_sync(kAll, word, 16 * c + (lane & 3)), t1 = __shfl_sync(kAll, word, 16 * c + 8 + (lane & 3));
                    const float2 ig = make_float2(__uint_as_float(t0 << 16), __uint_as_float(t1 << 16));
                    const float2 iu = make_float2(__uint_as_float(t0 & 0xFFFF0000u), __uint_as_float(t1 & 0xFFFF0000u));
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int x = 8 * h + 4 * c;
                        q[0][2 * h + c] = codes_of(__fmul2_rn(both(dg, x), ig), __fmul2_rn(both(dg, x + 2), ig));
                        q[1][2 * h + c] = codes_of(__fmul2_rn(both(du, x), iu), __fmul2_rn(both(du, x + 2), iu));
                    }
                }
                __syncwarp();
                store_rows(m_at, q[0]);
                store_rows(m_at + 512, q[1]);
                __syncwarp();
                const uint4 yg = in_order(lds128(k_at)), yu = in_order(lds128(k_at + 512));
                if (c0 + k_tok < t.rows) {
                    uint8_t *dst = p.Q + (t.row0 + c0 + k_tok) * pitch + fb * kBlk + w * 32 + k_half * 16;
                    *reinterpret_cast<uint4 *>(dst) = yg;
                    *reinterpret_cast<uint4 *>(dst + p.I) = yu;
                }
            }
        }
    }
    if (bad) tail.bad_scale = 1;
    if (lane == 0) bulk_wait_all();
}

}  // namespace
}  // namespace moe
