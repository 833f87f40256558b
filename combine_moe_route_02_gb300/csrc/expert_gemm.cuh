// expert_gemm.cuh -- what the product kernel (expert_gemm.cu) and what follows it in the same launch
// (expert_gemm_epilogue.cuh) share: sizes, the shared-memory layout, the walk over the tiles, TMEM fragments.
#pragma once

#include "expert_internal.cuh"

namespace moe {
namespace {

constexpr int kTileM = 256;        // output features per tile, half of them in each CTA
constexpr int kHalfM = 128;
constexpr int kTileN = 224;        // most tokens per tile: two accumulators and the scales fit TMEM
constexpr int kBlk = 128;          // reduction block of a scale, and of a ring stage
constexpr int kScaleSlots = 2;
constexpr int kABytes = kHalfM * kBlk;
constexpr int kBBytes = kTileN / 2 * kBlk;      // half of the tokens
constexpr int kStageBytes = kABytes + kBBytes;
constexpr int kScaleQuadBytes = 512 + 1024;   // four blocks: 128 feature words, 256 token words
constexpr int kScaleSlotBytes = 4 * kScaleQuadBytes;

// What follows the product: nothing (bf16 rows out), the gated activation (the product is both halves of its
// input) with or without their checkpoint, or the activation's gradient (the product is the gradient of its output).
enum Mode { kPlain, kGated, kGatedOnly, kGatedGrad };
constexpr bool gated(Mode m) { return m == kGated || m == kGatedOnly; }
// The activation's modes have teams of four epilogue warps, which take chunks of tokens in turn, and one team of scale
// producers instead of two.  What a chunk costs is a chain of short steps, so the number of warps decides, and that goes by
// their registers.  kGated, kGatedOnly: three teams and chunks of 32 tokens, 16 warps, the most that have 128 registers a
// thread (16384 tokens, 128 experts, H = 2048, I = 1024 / 16381 tokens of H = 1024, I = 2048 without checkpoint, graphs of
// 20 passes, with kGated's epilogue for both: 433 / 134 us; chunks of 16 tokens and four teams 452 / 169, three 461 / 169,
// five 468 / 181: the exchange of words is paid for each chunk).  kGatedGrad, where no words cross the CTAs: four and 16, 20 warps of 96 (the first case: 321; three teams and
// 32 tokens 344, five teams and 80 registers 355).
constexpr int teams(Mode m) { return m == kPlain ? 1 : gated(m) ? 3 : 4; }
constexpr int chunk_tokens(Mode m) { return m == kGatedGrad ? 16 : 32; }
constexpr int scale_teams(Mode m) { return m == kPlain ? 2 : 1; }
constexpr int threads(Mode m) { return 32 * (2 + 2 * scale_teams(m) + 4 * teams(m)); }
constexpr int stages(Mode m) { return m == kGatedGrad ? 4 : 6; }
// Staging of the epilogue.  kPlain: 32 tokens x 64 bytes a warp; kGated: three arrays of that (codes of the activation
// and of both halves) a team; kGatedOnly: two in turn; kGatedGrad, 16 tokens: two of 64 bytes for the TMA (bf16 rows of both halves) and two of
// 32 (codes) a warp.  Then the words in which warps tell each other scales: two buffers in turn for each team (kGatedOnly: four), of a
// word for each token and warp (but for kGatedGrad of both CTAs).
constexpr int stage_bytes(Mode m) { return m == kPlain ? 4 * 2048 : m == kGated ? teams(m) * 3 * 2048 : m == kGatedOnly ? teams(m) * 2 * 2048 : teams(m) * 4 * 3072; }
constexpr int word_buffers(Mode m) { return m == kGatedOnly ? 4 : 2; }
constexpr int word_warps(Mode m) { return m == kPlain ? 0 : gated(m) ? 8 : 4; }
constexpr int epi_bytes(Mode m) { return stage_bytes(m) + teams(m) * word_buffers(m) * word_warps(m) * chunk_tokens(m) * 4; }
constexpr uint32_t kTmemCols = 512;
// Scales lie behind the two accumulators: 4 + 8 columns for four blocks.  Five places in turn: when one is
// written again its MMAs have completed, those of the tile before the last by the wait for its accumulator,
// nearer ones because at least as many blocks as the ring holds lie between.
constexpr uint32_t kSfCol = 2 * kTileN, kSfCols = 12, kSfPlaces = 5;
static_assert(kSfCol + kSfPlaces * kSfCols <= kTmemCols, "TMEM");
constexpr int kMaxE = 256;

struct Tail {
    uint64_t full[6], empty[6];
    uint64_t sf_full[kScaleSlots], sf_empty[kScaleSlots];
    uint64_t acc_full[2], acc_empty[2], drain;
    uint64_t words[teams(kGated)][4];    // kGated, kGatedOnly: the scale words of a team's chunk, two or four in turn
    uint32_t tmem_base;
    int abort, bad_index, bad_scale;
    int tiles;                    // token tiles of all groups
    int first[kMaxE + 1];         // first token tile of each group
    int begin[kMaxE], count[kMaxE], size[kMaxE];   // its rows, and the rows of its tiles but the last
};

constexpr size_t smem_bytes(Mode m)
{
    return 1024 + stages(m) * kStageBytes + kScaleSlots * kScaleSlotBytes + epi_bytes(m) + sizeof(Tail);
}
static_assert(smem_bytes(kPlain) <= 227 * 1024 && smem_bytes(kGated) <= 227 * 1024 &&
                  smem_bytes(kGatedOnly) <= 227 * 1024 && smem_bytes(kGatedGrad) <= 227 * 1024,
              "shared memory");

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
    void *Y;                      // bf16 rows: the product, or (kGatedGrad) the gradient of both halves, or nullptr
    // the activation's modes
    int I, out_ue8m0, k_ue8m0;
    uint8_t *A;                   // codes of the activation
    void *A_scale;
    uint8_t *K;                   // codes of both halves: the checkpoint, written by kGated, read by kGatedGrad
    void *K_scale;
    uint8_t *Q;                   // kGatedGrad: codes of the gradient of both halves, or nullptr
    void *Q_scale;
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

}  // namespace
}  // namespace moe
