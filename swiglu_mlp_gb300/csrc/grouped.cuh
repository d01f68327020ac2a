// grouped.cuh — products grouped by expert on tcgen05: 16-bit operands and
// microscaled 4-bit ones, with the plain, SwiGLU and SwiGLU-gradient epilogues.
//
//   C[i, n] = sum_k A[i, k] * W_g[n, k]      for the rows i of group g
//
// The product is computed transposed: the weight is the MMA's 256-row operand
// (128 rows per CTA of a pair) and the group's rows are its N, which every
// instruction may choose anew as any multiple of 16 up to TOKENS.  A group
// of r rows is cut into ceil(r / TOKENS) tiles of nearly equal width, so the
// padding is below 16 rows a tile, where 256-row tiles of A would pad every
// group to 256: with 16 experts of about 500 rows a third of the work.
//
// Warp 0 loads (TMA), warp 1 issues the MMAs, warps 2..9 empty the finished
// accumulator while the next tile's main loop runs (two accumulators in tensor
// memory).  Every CTA finds its tiles itself from the offsets on the device;
// the host never waits for them.
//
// 4-bit operands (kind::mxf4 / kind::mxf4nvf4, K = 64 per instruction): a
// stage holds 256 elements of K and their scales, which tcgen05.cp copies from
// the 512-byte scale tiles in shared memory to tensor memory ahead of the
// stage's MMAs (same issuing thread, so they execute in order).  Both CTAs
// need the scales of all of the tile's rows of A, and those of their own
// weight rows.
//
// What bounds it, and what it measured on one GB300:
//   many rows, 16 bits: the tensor pipe at the clock that the power limit
//     leaves.  SwiGLU, 16384 rows of 16 groups, K = 4096, N = 2 x 1792: 267 us,
//     1800 TFLOP/s, in a burst and 310 us, 1550, in a long run; gradient of half
//     as many rows, 8 groups: 146 us, 1650, and 167 us, 1440.
//   many rows, 4 bits: MMAs and the copies of their scales, one behind the other
//     in the tensor pipe, which is 70% busy.  8192 x 14336 x 4096, in a burst:
//     NVFP4 143 us, 6.7 PFLOP/s; MXFP4 135 us, 7.1.
//   few rows: the weights' way from memory and about 3.3 us that any call takes
//     (set-up, offsets, first load, last store).  8 groups of one row, 4096 x
//     9728 in 16 bits: 94 us, 6.8 TB/s; 16 rows, 229376 x 4096 in MXFP4: 78 us,
//     6.4 TB/s; 2 rows of 8 groups, 896 x 9728: 8.3 us, 4.2 TB/s.
//   between: not accounted for.  32 groups of 128 rows, 2048 x 2432 in MXFP4: 24
//     us, 3.5 TB/s, of which the latency of loads that miss L2 (1.3 to 2.3 us) is
//     a part at most: the weights of 6 stages on every SM are 15 MB in flight,
//     6.5 TB/s at 2.3 us.
#pragma once

#include "experts_launch.h"
#include "groups.cuh"
#include "tc_gemm.cuh"

namespace swg {

// ------------------------------------------------------------ PTX wrappers

__device__ __forceinline__ void tma_load_4d_pair(uint32_t dst, const void *tmap, uint32_t bar,
                                                 int32_t x, int32_t y, int32_t z, int32_t w)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
        : "memory");
}

// Scales of one tile (128 rows x 4 blocks, 512 bytes in shared memory) to four
// tensor-memory columns, repeated for the four lane quarters, in both CTAs.
__device__ __forceinline__ void tc_cp_scales_pair(uint32_t taddr, uint64_t desc)
{
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
                 : "memory");
}

template <bool NV>
__device__ __forceinline__ void tc_mma_f4_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                               uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                               uint32_t accumulate)
{
    if (NV)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X"
            " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X"
            " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
}

// wait_bounded by every lane of a converged warp.
__device__ __forceinline__ bool wait_bounded_warp(uint32_t bar, uint32_t parity,
                                                  volatile int *abort_flag, int *err)
{
    return __all_sync(0xffffffffu, wait_bounded(bar, parity, abort_flag, err));
}

// Descriptor of a scale tile: 8-row x 16-byte core matrices 128 bytes apart, no swizzle.
__device__ __forceinline__ uint64_t scale_desc(uint32_t addr)
{
    return (uint64_t)((addr >> 4) & 0x3FFF) | (8ull << 32) | (1ull << 46);
}

// ------------------------------------------------------------ configuration

enum GrpMath { MATH_16 = 0, MATH_MX = 1, MATH_NV = 2 };

// A's maps: boxes of 128, 96, 64, 32 and 16 rows.
constexpr int TOKEN_BOXES = 5;
constexpr int SMEM_MOST = 232448;        // bytes of shared memory that a CTA can have
__host__ __device__ constexpr int token_box(int i) { return i == 0 ? 128 : i == 1 ? 96 : 128 >> (i - 1); }

struct GrpMaps {
    CUtensorMap w;                       // weights
    CUtensorMap t[TOKEN_BOXES];          // rows of A
    CUtensorMap sw, st;                  // scale tiles of both (4-bit)
    CUtensorMap c, y;                    // 16-bit outputs, boxes of 64 columns x 32 rows (tma_out)
};

struct GrpParams {
    Groups groups;
    int N;
    int n_blocks, k_blocks;              // 256 columns; stages of 64 (16-bit) or 256 (4-bit) of K
    uint32_t idesc;                      // without N
    int w_mn;                            // weight MN-major (stored K x N)
    int w_4d;                            // ... as one 4-D box per stage
    int w_tiles;                         // rows of scale tiles per group of weights
    float alpha, beta;
    void *C;
    long long ldc;
    const void *dY;
    void *Y;
    int out_kind;
    int tma_out;                         // whole chunks of 32 rows leave through TMA stores
    // K cut into `splits` ranges of split_blocks stages: range s of a tile is a
    // unit of its own and goes to C + s * split_stride (FP32 partials).
    int splits, split_blocks;
    long long split_stride;
    int stages, stages_narrow;           // of the ring, see GrpCfg (4-bit)
    int ring_bytes;
    int *err;
};

// FEW: the form for at most 64 rows of A in all, which streams weights from
// memory.  Its stages hold 64 rows of A instead of 256 and are 8 to 10
// instead of 5 or 6, so that more of the weight is in flight.  (Two CTAs of
// half the depth per SM instead were slower: 8 groups of one row, 4096 x 1024
// each, 21.4 us against 18.2 with 6 stages.)
template <int MATH, bool FEW>
struct GrpCfg {
    static constexpr bool F4 = MATH != MATH_16;
    // Rows of A per tile: two accumulators fill tensor memory at 256.
    static constexpr int TOKENS = FEW ? 64 : 256;
    // A tile begins at a multiple of UNIT rows of its group (4-bit: 64 rows are
    // two columns of scales) and may be CANDIDATES widths, see choose_rows.
    static constexpr int UNIT = F4 ? 64 : 16;
    static constexpr int CANDIDATES = FEW ? 1 : F4 ? 3 : 8;
    static constexpr int NARROWEST = TOKENS - (CANDIDATES - 1) * UNIT;
    static constexpr int EPI_WARPS = FEW ? 4 : 8;
    static constexpr int THREADS = 64 + 32 * EPI_WARPS;
    static constexpr int TILES_PER_STAGE = MATH == MATH_NV ? 4 : 2;   // scale tiles along K
    static constexpr int SCALE_ROWS = FEW ? 1 : 2;                    // rows of tiles of A's scales
    static constexpr int SCALE_BYTES = F4 ? 512 * TILES_PER_STAGE : 0;
    static constexpr int STAGE_SCALES = (1 + SCALE_ROWS) * SCALE_BYTES;
    static constexpr int W_BYTES = 128 * 128;
    static constexpr int T_BYTES = TOKENS / 2 * 128;
    static constexpr int STAGE_BYTES = W_BYTES + T_BYTES + STAGE_SCALES;
    static constexpr int OUT_BYTES = F4 ? 2048 : 3072;   // per epilogue warp, see the epilogue
    static constexpr int BAR_BYTES = 512;
    static constexpr int FIXED = EPI_WARPS * OUT_BYTES + BAR_BYTES;
    __host__ __device__ static constexpr int table_bytes(int G) { return (F4 ? 3 : 2) * 4 * (G + 1) + G; }
    // The ring has as many stages as the table of G groups leaves room for, at
    // most 6 unless weights are streamed; a launch whose tiles have at most 192
    // rows lays out stages of that many.  (For 32 groups 6 instead of 5: MXFP4
    // 8192 x 14336 x 4096 133 us against 138, with 192 rows 4096 x 4096 x 14336
    // 70 against 74, in NVFP4 73 against 77.)
    static constexpr int T_NARROW = F4 && !FEW ? 192 / 2 * 128 : T_BYTES;
    static constexpr int NARROW_BYTES = W_BYTES + T_NARROW + STAGE_SCALES;
    static constexpr int RING = FEW ? 12 : 6;        // barriers for that many
    __host__ __device__ static constexpr int stages_of(int bytes, int G)
    {
        const int n = (SMEM_MOST - FIXED - table_bytes(G)) / bytes;
        return n < RING ? n : RING;
    }
    __host__ __device__ static constexpr int ring_bytes(int G)
    {
        const int wide = stages_of(STAGE_BYTES, G) * STAGE_BYTES;
        const int narrow = stages_of(NARROW_BYTES, G) * NARROW_BYTES;
        return wide > narrow ? wide : narrow;
    }
    static constexpr int smem_bytes(int G) { return ring_bytes(G) + FIXED + table_bytes(G); }
    static constexpr int TMEM_COLS = !FEW ? 512 : F4 ? 256 : 128;
    // Two buffers of a stage's scales at the end of tensor memory.  What they
    // take of it the two accumulators share: the second begins ACC_STRIDE
    // columns behind the first, and the columns that are in both are emptied
    // first (OVERLAP, see the epilogue).  With two apart, tiles have 192 rows
    // at most and the bound is what an SM gets from L2, 64 bytes a cycle: 34 KB
    // a stage in 290 ns for 200 ns of MMAs (8192 x 14336 x 4096 in NVFP4 156 us
    // against 143, MXFP4 144 against 139; 16 groups of 512 rows, 4096 x 4096,
    // 65 against 60 and 61 against 55).
    static constexpr int SCALE_COLS = F4 ? 12 * TILES_PER_STAGE : 0;
    static constexpr int SCALE_COL = TMEM_COLS - 2 * SCALE_COLS;
    static constexpr bool OVERLAP = 2 * TOKENS > SCALE_COL;
    static constexpr int ACC_STRIDE = OVERLAP ? (SCALE_COL - TOKENS) / 32 * 32 : TOKENS;
    static constexpr bool TWO_SHARED = OVERLAP && TOKENS - ACC_STRIDE > 64;
    static_assert(stages_of(STAGE_BYTES, MAX_GROUPS) >= 5, "pipeline too shallow");
    static_assert(STAGE_BYTES % 1024 == 0 && NARROW_BYTES % 1024 == 0, "swizzled tiles");
    static_assert(ACC_STRIDE + TOKENS <= SCALE_COL && 2 * ACC_STRIDE >= TOKENS, "tensor memory");
};

// a / b for a >= 0, b > 0.  Below 2^21 through the fast FP32 division: a + 1/2
// keeps the quotient 1/(2b) away from the next integer, more than its error of
// two units in the last place.  (Integer division is a chain of tens of
// dependent instructions; four of them per tile, before its first load, took
// 0.4 us.)
__device__ __forceinline__ int fast_div(int a, int b)
{
    if (a < (1 << 21)) return (int)__fdividef((float)a + 0.5f, (float)b);
    return a / b;
}

// Tiles of a group of `rows` rows, when they have at most `most`.
template <class C>
__device__ __forceinline__ int tiles_of(int rows, int most)
{
    return C::CANDIDATES == 1 ? ceil_div(rows, C::TOKENS) : fast_div(rows + most - 1, most);
}

// Rows of A covered by each tile of a group of `rows` (> 0) rows, but the
// last, when tiles have at most `most` rows.  (rows + t - 1 may pass 2^31.)
template <class C>
__device__ __forceinline__ int tile_step(int rows, int most)
{
    const int t = tiles_of<C>(rows, most);
    constexpr int UNIT = C::UNIT;
    return ceil_div(fast_div(rows - 1, t) + 1, UNIT) * UNIT;
}

// The most rows of A that a tile should have, chosen so that the last wave of
// tiles is not nearly empty: of TOKENS, TOKENS - unit, .. the one with the least
//   waves * (stages * max(rows of a tile, 176) + 700),
// a tile's measured time in units of 1.145 ns: a 16-bit stage takes 292 ns at
// 256 rows, 228 at 192, 212 at 160 and not less than 195 below (the loading
// and issuing), and a tile about 0.8 us besides.  994 tiles on 76 pairs are
// 13.1 waves at 256 rows; 1064 tiles of at most 240 make 14.0 and are 7% faster.
// In 4 bits, in cycles: a stage takes what its loads do (22 KB and 64 bytes a
// row, at 64 bytes a cycle) or its MMAs (2.8 a row in NVFP4, 2.55 in MXFP4), and
// a tile not less than its epilogue (21 a row).  1536 x 4096 x 8192: 22.3 us at
// the 192 rows that this gives, 26.7 at 256.
// A tile's rows are their mean over many waves; in few, the widest tiles hold
// the others up.  Among equals the narrowest.  (3000 rows in 16 groups, 2048 x
// 2048: 34.8 us; by the mean alone, and the widest of equals, 39.9.  5003 in 12,
// 2051 x 1003: 31.4 us against 33.7.)  The three 4-bit widths are told apart by
// the mean as well.
// cost_of_rows: that of tiles of at most `most` rows, given what the calling
// warp's lanes have of the groups' tiles and rows, and the widest tile.
template <class C>
__device__ __forceinline__ float cost_of_rows(int tiles, int rows, int widest, int n_blocks,
                                              int k_blocks, int pairs)
{
    tiles = __reduce_add_sync(0xffffffffu, tiles);
    rows = __reduce_add_sync(0xffffffffu, rows);
    const float waves = (float)fast_div(tiles * n_blocks + pairs - 1, pairs);
    const float mean = __fdividef((float)rows, fmaxf((float)tiles, 1.0f));
    float r = mean;
    if (!C::F4) {
        widest = __reduce_max_sync(0xffffffffu, widest);
        r += __fdividef((float)widest - mean, fmaxf(waves, 1.0f));
    }
    const float k = (float)k_blocks;
    const float tile = C::F4 ? fmaxf(k * fmaxf(330.0f + r, 2.7f * r), 21.0f * r) + 500.0f
                             : k * fmaxf(r, 176.0f) + 700.0f;
    return waves * tile;
}

// Warp w of the first eight has candidate w's cost; called by all threads, ends
// with a barrier.
template <class C>
__device__ __forceinline__ int choose_rows(float cost, float *costs)
{
    if ((threadIdx.x & 31) == 0 && (threadIdx.x >> 5) < C::CANDIDATES) costs[threadIdx.x >> 5] = cost;
    __syncthreads();
    int best = 0;
#pragma unroll
    for (int c = 1; c < C::CANDIDATES; ++c)
        if (C::F4 ? costs[c] < costs[best] : costs[c] <= costs[best]) best = c;
    return C::TOKENS - best * C::UNIT;
}

struct GrpTile {
    int g, nb;         // group, block of 256 weight rows
    int row0, rows;    // rows of A
    int local;         // row0 within the group
    int width;         // rows rounded up to 16: the MMA's N
};

// Tile u: groups in order; within a group bands of 8 tiles of A walk the
// weight blocks together, so that concurrently running pairs share both in L2.
__device__ __forceinline__ GrpTile grp_tile(const int *start, const int *first,
                                            const uint8_t *steps, int G, int n_blocks, int u)
{
    GrpTile t;
    t.g = group_of(first, G, n_blocks, u);
    const int tiles = first[t.g + 1] - first[t.g];
    const int local = u - first[t.g] * n_blocks;
    int mb;
    if (tiles == 1) {
        mb = 0;
        t.nb = local;
    } else {
        const int band = tiles <= 8 ? 0 : fast_div(local, 8 * n_blocks);
        const int in = local - band * 8 * n_blocks;
        const int bm = min(8, tiles - band * 8);
        t.nb = fast_div(in, bm);
        mb = band * 8 + in - t.nb * bm;
    }
    const int step = 16 * steps[t.g];
    t.local = mb * step;
    t.row0 = start[t.g] + t.local;
    t.rows = min(step, start[t.g + 1] - t.row0);
    t.width = (t.rows + 15) & ~15;
    return t;
}

// ------------------------------------------------------------ epilogue

__device__ __forceinline__ void st_shared_u16(uint32_t addr, uint32_t v)
{
    asm volatile("st.shared.u16 [%0], %1;" ::"r"(addr), "h"((unsigned short)v) : "memory");
}

__device__ __forceinline__ void st_shared_u32(uint32_t addr, uint32_t v)
{
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

__device__ __forceinline__ uint32_t to_16(float v, int out_kind)
{
    if (out_kind == OUT_F16) return __half_as_ushort(__float2half_rn(v));
    return __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// A warp's 32 lanes x 32 columns of the accumulator in fragments: for each 8
// columns i, r[4 i] and r[4 i + 1] are row lane / 4, columns 2 (lane % 4) and
// + 1; r[4 i + 2] and r[4 i + 3] the same of row lane / 4 + 8; r[16 + 4 i] ..
// those of rows + 16.
template <int FROM>
__device__ __forceinline__ void tmem_ld_16x32(uint32_t taddr, uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32"
        " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[FROM + 0]), "=r"(r[FROM + 1]), "=r"(r[FROM + 2]), "=r"(r[FROM + 3]),
          "=r"(r[FROM + 4]), "=r"(r[FROM + 5]), "=r"(r[FROM + 6]), "=r"(r[FROM + 7]),
          "=r"(r[FROM + 8]), "=r"(r[FROM + 9]), "=r"(r[FROM + 10]), "=r"(r[FROM + 11]),
          "=r"(r[FROM + 12]), "=r"(r[FROM + 13]), "=r"(r[FROM + 14]), "=r"(r[FROM + 15])
        : "r"(taddr));
}

__device__ __forceinline__ void tmem_ld_fragments(uint32_t taddr, uint32_t (&r)[32])
{
    tmem_ld_16x32<0>(taddr, r);
    tmem_ld_16x32<16>(taddr + (16u << 16), r);
}

// Four 8 x 8 matrices of 16-bit values, each stored transposed: matrix m's
// row j of 16 bytes goes to the address that lane 8 m + j gives.
__device__ __forceinline__ void stmatrix_x4_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                                  uint32_t d)
{
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr),
                 "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}

// A tile store from shared memory whose lines leave L2 first: results would
// push out the operands that other tiles still read (8192 x 14336 x 4096 in
// NVFP4: 161.8 -> 159.3 us).
__device__ __forceinline__ void tma_store_2d_first_out(const void *tmap, uint32_t src, int32_t x,
                                                       int32_t y)
{
    uint64_t policy;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
    asm volatile(
        "cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group.L2::cache_hint"
        " [%0, {%2, %3}], [%1], %4;" ::"l"(reinterpret_cast<uint64_t>(tmap)),
        "r"(src), "r"(x), "r"(y), "l"(policy)
        : "memory");
}

// Staging of 16-bit results: boxes of 32 rows x 64 columns (128 bytes a row) in
// the 128-byte swizzle, 16-byte piece j of row r at j ^ (r mod 8).
__device__ __forceinline__ uint32_t staged_at(uint32_t box, int r, int j)
{
    return box + (uint32_t)(r * 128 + ((j ^ (r & 7)) << 4));
}

// Pieces j0 .. j0 + PIECES - 1 of the first `rows` (of 32) rows of a staged box
// to rows of `out` ldo apart (out: the column of piece j0), 16 bytes per lane;
// columns from `limit` on are left out.
template <int PIECES>
__device__ __forceinline__ void copy_staged(uint32_t box, int j0, uint16_t *out, long long ldo,
                                            int rows, int limit, int lane)
{
    const int j = lane % PIECES, c = j * 8;
#pragma unroll
    for (int r = lane / PIECES; r < 32; r += 32 / PIECES) {
        if (r >= rows || c >= limit) continue;
        const uint4 v = ld_shared_v4(staged_at(box, r, j0 + j));
        uint16_t *dst = out + r * ldo + c;
        if (c + 8 <= limit) {
            *reinterpret_cast<uint4 *>(dst) = v;
        } else {
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (c + i < limit) dst[i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
        }
    }
}

// Columns `from` .. `limit` - 1 (counted from piece j0; at most 7, which a TMA
// store leaves out: it clips rows at 16-byte granules) of the same rows, a row
// per lane.
__device__ __forceinline__ void copy_last_columns(uint32_t box, int j0, uint16_t *out, long long ldo,
                                                  int rows, int from, int limit, int lane)
{
    if (lane >= rows) return;
    for (int c = from; c < limit; ++c) {
        uint16_t v;
        asm volatile("ld.shared.u16 %0, [%1];"
                     : "=h"(v)
                     : "r"(staged_at(box, lane, j0 + (c >> 3)) + (uint32_t)(c & 7) * 2)
                     : "memory");
        out[lane * ldo + c] = v;
    }
}

// One chunk of the epilogue: 32 rows of A (from `row`; `rows` of them exist) by
// the CTA's 128 accumulator rows, 32 per warp of a group of four, which stage
// their results together so that they leave as whole 128-byte lines: as
// 32-byte pieces of each warp's own, or 64-byte ones, the stores slowed the
// main loop's loads by a sixth.  (Staged at all because the results come out
// transposed, and because the operands take most of the L1 and shared-memory
// bandwidth: 2-byte shared and row-wise global stores cost 5% of 8192 x 4096 x
// 4096.)
struct Chunk {
    int row, rows;
    int cta_n0, n0;          // first accumulator column (of C) of the CTA, of this warp
    int q;                   // warp of the group
    uint32_t buf;            // the group's staging: boxes of 4 KB
    int bar;                 // its named barrier
    int lane;
};
constexpr int GROUP_THREADS = 128;

// The group's staging may be written again: what its first warp's TMA stores
// were to read, they have, and every warp has copied what it copies itself.
__device__ __forceinline__ void staging_free(const Chunk &c)
{
    if (c.q == 0 && c.lane == 0) bulk_wait_read_all();
    named_bar_sync(c.bar, GROUP_THREADS);
}

// What the group has staged is visible to the TMA; true in the thread that
// issues its stores.
__device__ __forceinline__ bool staging_done(const Chunk &c)
{
    fence_proxy_async_smem();
    named_bar_sync(c.bar, GROUP_THREADS);
    return c.q == 0 && c.lane == 0;
}

// 16-bit results of the plain product.
template <int KIND>
__device__ __forceinline__ void emit_store_16(const GrpParams &p, const CUtensorMap *tm,
                                              const uint32_t (&r)[32], const Chunk &c)
{
    staging_free(c);
    const uint32_t box = c.buf + (uint32_t)(c.q >> 1) * 4096;
    const int j0 = (c.q & 1) * 4;                   // this warp's pieces of its rows
    const int m = c.lane >> 3, j8 = c.lane & 7;     // the 16 bytes that this lane addresses
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        auto pk = [&](int k) {
            return pack2(p.alpha * __uint_as_float(r[4 * i + k]),
                         p.alpha * __uint_as_float(r[4 * i + k + 1]), KIND);
        };
        stmatrix_x4_trans(staged_at(box, 8 * i + j8, j0 + m), pk(0), pk(2), pk(16), pk(18));
    }
    uint16_t *out = reinterpret_cast<uint16_t *>(p.C) + c.row * p.ldc + c.n0;
    if (p.tma_out && c.rows == 32) {
        const int whole = p.N & ~7;
        if (staging_done(c)) {
            if (c.cta_n0 < whole) tma_store_2d_first_out(tm, c.buf, c.cta_n0, c.row);
            if (c.cta_n0 + 64 < whole) tma_store_2d_first_out(tm, c.buf + 4096, c.cta_n0 + 64, c.row);
            bulk_commit_group();
        }
        if (p.N != whole && c.n0 < p.N && c.n0 + 32 > whole)
            copy_last_columns(box, j0, out, p.ldc, 32, whole - c.n0, p.N - c.n0, c.lane);
    } else {
        __syncwarp();
        copy_staged<4>(box, j0, out, p.ldc, c.rows, p.N - c.n0, c.lane);
    }
}

template <int KIND>
struct Kind {
    static constexpr int value = KIND;
};

// FP32 results (and partials of K ranges), beta, and K = 0 (no accumulator):
// each lane is a column, its stores (and loads of C) of one row are 64 or 128
// bytes a warp.
template <int KIND>
__device__ __forceinline__ void emit_store_direct(const GrpParams &p, uint32_t taddr,
                                                  long long offset, int row, int rows, int n0,
                                                  int lane)
{
    const int n = n0 + lane;
#pragma unroll 1
    for (int j0 = 0; j0 < rows; j0 += 16) {
        uint32_t acc[16] = {};
        if (p.k_blocks > 0) {
            tmem_ld_16cols(taddr + j0, acc);
            tmem_ld_wait(acc);
        }
        if (n >= p.N) continue;
        const long long o = offset + (row + j0) * p.ldc + n;
        float v[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = p.alpha * __uint_as_float(acc[j]);
        if (p.beta != 0.0f) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
                if (j0 + j < rows) v[j] += p.beta * load_out(p.C, o + j * p.ldc, KIND);
        }
#pragma unroll
        for (int j = 0; j < 16; ++j)
            if (j0 + j < rows) store_out(p.C, o + j * p.ldc, v[j], KIND);
    }
}

// SwiGLU and its gradient.  Lanes 2i and 2i + 1 hold Gate and Up of one output
// column.  They swap halves, so that the even lane has both for the even rows
// and the odd lane for the odd ones.  dY comes as 16 columns of row `lane` of the
// chunk and goes through the warp's own part of the staging to the lanes that
// need it, fetched a chunk ahead (fetched by each lane, element by element, and
// only when the chunk before was done, 16 groups of 512 rows, 1024 x 1024,
// took 61 us instead of 39).
template <int EPI>
__device__ __forceinline__ void emit_swiglu(const GrpParams &p, const GrpMaps &maps,
                                            const uint32_t (&acc)[32], const uint4 (&dY)[2],
                                            const Chunk &c)
{
    staging_free(c);
    const int odd = c.lane & 1;
    // where this lane's results go: of the 64 output columns, and of the 128 of dH
    const uint32_t y_box = c.buf + (EPI == GRP_SWIGLU ? 0 : 8192);
    const int y_j0 = c.q * 2;
    const uint32_t h_box = c.buf + (uint32_t)(c.q >> 1) * 4096;
    const int h_j0 = (c.q & 1) * 4;
    uint32_t dy[16];                                // of this lane's 16 rows
    if (EPI == GRP_DSWIGLU) {
        st_shared_v4(staged_at(h_box, c.lane, h_j0), dY[0]);
        st_shared_v4(staged_at(h_box, c.lane, h_j0 + 1), dY[1]);
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            uint16_t v;
            asm volatile("ld.shared.u16 %0, [%1];"
                         : "=h"(v)
                         : "r"(staged_at(h_box, 2 * j + odd, h_j0 + (c.lane >> 4)) +
                               (uint32_t)((c.lane >> 1) & 7) * 2)
                         : "memory");
            dy[j] = (uint32_t)v << 16;
        }
        __syncwarp();
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        const uint32_t send = odd ? acc[2 * j] : acc[2 * j + 1];
        const float got = __uint_as_float(__shfl_xor_sync(0xffffffffu, send, 1));
        const float g = p.alpha * (odd ? got : __uint_as_float(acc[2 * j]));
        const float u = p.alpha * (odd ? __uint_as_float(acc[2 * j + 1]) : got);
        const int r = 2 * j + odd;
        const uint32_t y_at = staged_at(y_box, r, y_j0 + (c.lane >> 4)) + (uint32_t)((c.lane >> 1) & 7) * 2;
        if (EPI == GRP_SWIGLU) {
            st_shared_u16(y_at, to_16(silu_f32(g) * u, OUT_BF16));
        } else {
            const float s = __fdividef(1.0f, 1.0f + __expf(-g));
            const float d = __uint_as_float(dy[j]);
            const float gs = g * s;
            st_shared_u32(staged_at(h_box, r, h_j0 + (c.lane >> 3)) + (uint32_t)((c.lane >> 1) & 3) * 4,
                          pack2(d * u * (s + gs * (1.0f - s)), d * gs, OUT_BF16));
            if (p.Y) st_shared_u16(y_at, to_16(gs * u, OUT_BF16));
        }
    }
    if (p.tma_out && c.rows == 32) {
        if (staging_done(c)) {
            if (EPI == GRP_SWIGLU) {
                tma_store_2d_first_out(&maps.c, y_box, c.cta_n0 / 2, c.row);
            } else {
                tma_store_2d_first_out(&maps.c, c.buf, c.cta_n0, c.row);
                if (c.cta_n0 + 64 < p.N)
                    tma_store_2d_first_out(&maps.c, c.buf + 4096, c.cta_n0 + 64, c.row);
                if (p.Y) tma_store_2d_first_out(&maps.y, y_box, c.cta_n0 / 2, c.row);
            }
            bulk_commit_group();
        }
        return;
    }
    __syncwarp();
    if (EPI == GRP_SWIGLU) {
        copy_staged<2>(y_box, y_j0, reinterpret_cast<uint16_t *>(p.C) + c.row * p.ldc + c.n0 / 2, p.ldc,
                       c.rows, (p.N - c.n0) / 2, c.lane);
    } else {
        copy_staged<4>(h_box, h_j0, reinterpret_cast<uint16_t *>(p.C) + c.row * p.ldc + c.n0, p.ldc,
                       c.rows, p.N - c.n0, c.lane);
        if (p.Y)
            copy_staged<2>(y_box, y_j0,
                           reinterpret_cast<uint16_t *>(p.Y) + c.row * (long long)(p.N / 2) + c.n0 / 2,
                           p.N / 2, c.rows, (p.N - c.n0) / 2, c.lane);
    }
}

// One stage of 4-bit operands: the scales to tensor memory (from column sf on:
// 4 columns per tile of this CTA's weight rows, then 8 per tile of A -- its
// rows 0..127 and 128..255), then four K steps.  Consecutive stages alternate
// between two sets of columns.
template <int MATH, class C>
__device__ __forceinline__ void issue_f4(uint32_t d_tmem, uint64_t w, uint64_t t, uint64_t s,
                                         uint32_t idesc, uint32_t sf, uint32_t t_shift,
                                         uint32_t accum)
{
    const uint32_t st = sf + 4 * C::TILES_PER_STAGE;
#pragma unroll
    for (int i = 0; i < C::TILES_PER_STAGE; ++i) {
        tc_cp_scales_pair(sf + 4 * i, s + i * 32);
        tc_cp_scales_pair(st + 8 * i, s + (C::SCALE_BYTES >> 4) + i * 32);
        if (C::SCALE_ROWS == 2)
            tc_cp_scales_pair(st + 8 * i + 4, s + 2 * (C::SCALE_BYTES >> 4) + i * 32);
    }
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
        if (MATH == MATH_NV) {
            tc_mma_f4_pair<true>(d_tmem, w + kk * 2, t + kk * 2, idesc, sf + 4 * kk,
                                 st + t_shift + 8 * kk, accum | kk);
        } else {
            // two blocks of 32 per instruction: bytes 0, 1 or 2, 3 of a tile's four
            const uint32_t id = (kk & 1) * 2;
            tc_mma_f4_pair<false>(d_tmem, w + kk * 2, t + kk * 2, idesc | (id << 29) | (id << 4),
                                  sf + 4 * (kk >> 1), st + t_shift + 8 * (kk >> 1), accum | kk);
        }
    }
}

// ------------------------------------------------------------ kernel

template <int MATH, int EPI, bool FEW>
__global__ void __launch_bounds__(GrpCfg<MATH, FEW>::THREADS, 1)
    grouped_kernel(const __grid_constant__ GrpMaps maps, const GrpParams p)
{
    using C = GrpCfg<MATH, FEW>;
    constexpr bool F4 = C::F4;
    constexpr int RING = C::RING;
    constexpr int RING_16 = C::ring_bytes(MAX_GROUPS);   // of 16-bit operands, for any G
    constexpr int STAGES_16 = C::stages_of(C::STAGE_BYTES, MAX_GROUPS);
    static_assert(F4 || C::ring_bytes(1) == RING_16);
    extern __shared__ __align__(1024) uint8_t grouped_smem[];
    // stages (W, rows of A, scales), output staging, barriers, group table
    uint8_t *sW = grouped_smem;
    uint8_t *sOut = grouped_smem + (F4 ? p.ring_bytes : RING_16);
    uint64_t *bars = reinterpret_cast<uint64_t *>(sOut + C::EPI_WARPS * C::OUT_BYTES);
    uint64_t *full = bars;
    uint64_t *empty = bars + RING;
    uint64_t *acc_full = bars + 2 * RING;
    uint64_t *acc_empty = bars + 2 * RING + 2;
    uint64_t *mma_done = bars + 2 * RING + 4;
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(bars + 2 * RING + 5);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
    int *scratch = reinterpret_cast<int *>(tmem_holder + 4);      // 16 ints, 8 floats
    int *start = reinterpret_cast<int *>(sOut + C::EPI_WARPS * C::OUT_BYTES + C::BAR_BYTES);
    int *first = start + p.groups.G + 1;
    int *stile = first + p.groups.G + 1;          // rows of scale tiles before each group
    // 16 rows of A: a tile of each group covers this many of them
    uint8_t *steps = reinterpret_cast<uint8_t *>(F4 ? stile + p.groups.G + 1 : stile);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (threadIdx.x == 0) {
        if (p.k_blocks > 0) {                        // fetched from memory on first use
            tma_prefetch_desc(&maps.w);
            tma_prefetch_desc(&maps.t[TOKEN_BOXES - 1]);
            if (F4) {
                tma_prefetch_desc(&maps.sw);
                tma_prefetch_desc(&maps.st);
            }
        }
        for (int s = 0; s < RING; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&acc_full[b]), 1);
            mbar_init(smem_u32(&acc_empty[b]), 2 * C::EPI_WARPS);   // (one with OVERLAP)
        }
        mbar_init(smem_u32(mma_done), 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(tmem_holder), C::TMEM_COLS);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem_base = __shfl_sync(0xffffffffu, *tmem_holder, 0);
    // Up to here only this pair's own resources; now the offsets may be read.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int G = p.groups.G;
    // So few rows that a group has at most one tile, and one of the narrowest width?
    const bool narrow = FEW || p.groups.M <= C::NARROWEST;
    static_assert(!F4 || C::NARROWEST <= 128, "one scale tile");
    int most = C::TOKENS;
    const int n_blocks = p.n_blocks * p.splits, pairs = (int)(gridDim.x >> 1);
    const int candidate = C::TOKENS - min(warp, C::CANDIDATES - 1) * C::UNIT;
    float *costs = reinterpret_cast<float *>(scratch + 16);
    if (narrow && G < 32 * WARP_ROUNDS) {
        if (warp == 0) {
            const WarpGroups w = warp_groups(p.groups, p.err, true);
            int before = 0;                          // groups with rows: they have a tile
#pragma unroll
            for (int r = 0; r < WARP_ROUNDS; ++r) {
                const int i = 32 * r + lane, rows = w.rows(r);
                const unsigned has = __ballot_sync(0xffffffffu, rows > 0);
                const int tile = before + __popc(has & ((1u << lane) - 1));
                if (i <= G) {
                    start[i] = w.start[r];
                    first[i] = tile;
                    if (F4) stile[i] = tile;
                    if (i < G) steps[i] = (uint8_t)(ceil_div(max(1, rows), C::UNIT) * (C::UNIT / 16));
                }
                before += __popc(has);
            }
        }
        __syncthreads();
    } else if (!FEW && G < (F4 ? 128 : 64)) {
        // Every warp reads the groups; the first eight find the widths' costs, the
        // first two write the tables.  (16 bits, 100 groups of 20 rows: 12.7 us so,
        // 12.3 through shared memory; 8 of 512: 8.5 and 9.1.)
        const WarpGroups w = warp_groups(p.groups, p.err, warp == 0);
        int tiles = 0, rows = 0, widest = 0;
#pragma unroll
        for (int r = 0; r < WARP_ROUNDS; ++r) {
            if (32 * r >= G) break;
            const int n = w.rows(r);
            tiles += tiles_of<C>(n, candidate);
            rows += n;
            if (!C::F4 && n > 0) widest = max(widest, tile_step<C>(n, candidate));
        }
        most = choose_rows<C>(
            cost_of_rows<C>(tiles, rows, widest, n_blocks, p.split_blocks, pairs), costs);
        if (warp == 0) {
#pragma unroll
            for (int r = 0; r < WARP_ROUNDS; ++r) {
                const int i = 32 * r + lane;
                if (i <= G) start[i] = w.start[r];
                if (i < G) steps[i] = (uint8_t)(tile_step<C>(max(1, w.rows(r)), most) / 16);
            }
            warp_tile_sums(w, first, [most](int n) { return tiles_of<C>(n, most); });
        } else if (F4 && warp == 1) {
            warp_tile_sums(w, stile, [](int n) { return ceil_div(n, 128); });
        }
        __syncthreads();
    } else {
        group_starts<C::THREADS>(p.groups, start, p.err);
        if (!narrow) {
            int tiles = 0, rows = 0, widest = 0;
            for (int g = lane; g < G; g += 32) {
                const int n = start[g + 1] - start[g];
                tiles += tiles_of<C>(n, candidate);
                rows += n;
                if (!C::F4 && n > 0) widest = max(widest, tile_step<C>(n, candidate));
            }
            most = choose_rows<C>(
                cost_of_rows<C>(tiles, rows, widest, n_blocks, p.split_blocks, pairs), costs);
        }
        for (int g = threadIdx.x; g < G; g += C::THREADS)
            steps[g] = (uint8_t)(tile_step<C>(max(1, start[g + 1] - start[g]), most) / 16);
        tile_sums<C::THREADS>(G, start, first, scratch,
                              [most](int n) { return tiles_of<C>(n, most); });
        if (F4)
            tile_sums<C::THREADS>(G, start, stile, scratch, [](int n) { return ceil_div(n, 128); });
    }
    // the ring
    const bool small = C::T_NARROW < C::T_BYTES && (narrow || most <= 192);
    const int S = !F4 ? STAGES_16 : small ? p.stages_narrow : p.stages;
    const uint32_t t_size = small ? C::T_NARROW : C::T_BYTES;
    uint8_t *sT = sW + S * C::W_BYTES;
    uint8_t *sS = sT + S * t_size;
    const int units = first[G] * p.n_blocks * p.splits;
    const int u0 = (int)(blockIdx.x >> 1), du = (int)(gridDim.x >> 1);

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        if (p.k_blocks > 0) {
            const uint32_t empty0 = smem_u32(empty), full0 = smem_u32(full);
            const uint32_t full_leader0 = mapa_shared(full0, 0);
            const uint32_t w_dst0 = smem_u32(sW), t_dst0 = smem_u32(sT), s_dst0 = smem_u32(sS);
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true, wrapped = false;
            for (int u = u0; u < units && ok; u += du) {
                const int split = p.splits == 1 ? 0 : u % p.splits;
                const GrpTile t = grp_tile(start, first, steps, G, p.n_blocks,
                                           p.splits == 1 ? u : u / p.splits);
                const int kb0 = split * p.split_blocks;
                const int kb1 = min(kb0 + p.split_blocks, p.k_blocks);
                const int half = __shfl_sync(0xffffffffu, t.width, 0) / 2;
                const int g = __shfl_sync(0xffffffffu, t.g, 0);
                // the lowest box that holds this CTA's rows of A
                int box = 0;
                while (box + 1 < TOKEN_BOXES && half <= token_box(box + 1)) ++box;
                const CUtensorMap *t_map = &maps.t[box];
                const int t_row = __shfl_sync(0xffffffffu, t.row0, 0) + (int)rank * half;
                const int n0 = __shfl_sync(0xffffffffu, t.nb, 0) * 256 + (int)rank * 128;
                const int w_tile = g * p.w_tiles + n0 / 128;
                const int t_tile = F4 ? __shfl_sync(0xffffffffu, stile[t.g] + t.local / 128, 0) : 0;
                const uint32_t t_bytes = (uint32_t)token_box(box) * 128u;
                const uint32_t bytes = C::W_BYTES + t_bytes + C::STAGE_SCALES;
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!wait_bounded_warp(empty0 + 8 * stage, phase ^ 1, abort_flag, p.err)) {
                        ok = false;
                        break;
                    }
                    const uint32_t fb = full_leader0 + 8 * stage;
                    const uint32_t w_dst = w_dst0 + stage * C::W_BYTES;
                    const uint32_t t_dst = t_dst0 + stage * t_size;
                    const uint32_t s_dst = s_dst0 + stage * C::STAGE_SCALES;
                    const int k0 = kb * (F4 ? 128 : 64);     // inner coordinate of the boxes
                    const int x = kb * (C::SCALE_BYTES / 8);
                    if (elect_one()) {
                        // both CTAs' bytes complete on the leader's barrier
                        if (leader) mbar_arrive_expect_tx(full0 + 8 * stage, 2 * bytes);
                        if (!p.w_mn) {
                            tma_load_3d_pair(w_dst, &maps.w, fb, k0, n0, g);
                        } else if (p.w_4d) {
                            tma_load_4d_pair(w_dst, &maps.w, fb, 0, k0, n0 / 64, g);
                        } else {
                            tma_load_3d_pair(w_dst, &maps.w, fb, n0, k0, g);
                            tma_load_3d_pair(w_dst + 8192, &maps.w, fb, n0 + 64, k0, g);
                        }
                        tma_load_2d_pair(t_dst, t_map, fb, k0, t_row);
                        if (F4) {
                            tma_load_2d_pair(s_dst, &maps.sw, fb, x, w_tile);
                            tma_load_2d_pair(s_dst + C::SCALE_BYTES, &maps.st, fb, x, t_tile);
                        }
                    }
                    if (++stage == S) {
                        stage = 0;
                        phase ^= 1;
                        wrapped = true;
                    }
                }
            }
            // Never leave with loads in flight into this CTA's shared memory.
            if (leader) {
                // (stages before `stage` were last used in this lap of the ring, the others
                // in the one before)
                for (int s = 0; s < S; ++s)
                    if (s < stage || wrapped)
                        wait_bounded(full0 + 8 * s, s < stage ? phase : phase ^ 1, abort_flag,
                                     p.err, false, DRAIN_LIMIT_NS);
            } else if (!ok) {
                const uint64_t t0 = global_timer_ns();
                while (global_timer_ns() - t0 < 200000ull) {
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        if (leader && p.k_blocks > 0) {
            // Descriptors of the first stage; stages and K steps are added in
            // units of 16 bytes (shared memory stays below the field's 2^14).
            const uint64_t w_desc = smem_desc(smem_u32(sW), p.w_mn ? 8192u : 16u, 1024);
            const uint64_t t_desc = smem_desc(smem_u32(sT), 16, 1024);
            const uint64_t s_desc = scale_desc(smem_u32(sS));
            const uint32_t w_kstep = p.w_mn ? 128u : 2u;
            const uint32_t empty0 = smem_u32(empty), full0 = smem_u32(full);
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            int n = 0;
            for (int u = u0; u < units && ok; u += du, ++n) {
                const int split = p.splits == 1 ? 0 : u % p.splits;
                const GrpTile t = grp_tile(start, first, steps, G, p.n_blocks,
                                           p.splits == 1 ? u : u / p.splits);
                const int kb0 = split * p.split_blocks;
                const int kb1 = min(kb0 + p.split_blocks, p.k_blocks);
                const uint32_t idesc =
                    __shfl_sync(0xffffffffu, p.idesc | ((uint32_t)(t.width >> 3) << 17), 0);
                // a tile of A that begins at the second half of its scale tile
                const uint32_t t_shift = __shfl_sync(0xffffffffu, (t.local & 64) ? 2u : 0u, 0);
                const int acc = n & 1;
                // the accumulator, or what it shares with the last tile's, is empty
                if (!wait_bounded_warp(smem_u32(&acc_empty[C::OVERLAP ? 0 : acc]),
                                       ((C::OVERLAP ? n : n >> 1) & 1) ^ 1, abort_flag, p.err)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + acc * C::ACC_STRIDE;
                uint32_t accum = 0;
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!wait_bounded_warp(full0 + 8 * stage, phase, abort_flag, p.err)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t w_stage = w_desc + (uint64_t)(stage * (C::W_BYTES >> 4));
                    const uint64_t t_stage = t_desc + (uint64_t)(stage * (t_size >> 4));
                    // (Always four K steps: behind K the loads give zeros.  Testing
                    // for the last steps made the issuing, not the tensor pipe,
                    // the bound: 8192 x 4096 x 4096 in 176 us instead of 159.)
                    if (elect_one()) {
                        if (MATH == MATH_16) {
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                tc_mma_f16_pair(d_tmem, w_stage + kk * w_kstep, t_stage + kk * 2,
                                                idesc, accum | kk);
                        } else {
                            const uint64_t sd = s_desc + (uint64_t)(stage * (C::STAGE_SCALES >> 4));
                            issue_f4<MATH, C>(d_tmem, w_stage, t_stage, sd, idesc,
                                           tmem_base + C::SCALE_COL + (kb & 1) * C::SCALE_COLS, t_shift,
                                              accum);
                        }
                        tc_commit_pair(empty0 + 8 * stage);
                    }
                    accum = 1;
                    if (++stage == S) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
                if (!ok) break;
                if (elect_one()) tc_commit_pair(smem_u32(&acc_full[acc]));
                __syncwarp();
            }
            // Never free tensor memory under a running MMA.
            if (elect_one()) tc_commit_pair_local(smem_u32(mma_done));
            __syncwarp();
            wait_bounded(smem_u32(mma_done), 0, abort_flag, p.err, false, DRAIN_LIMIT_NS);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ epilogue
        const int q = warp & 3;                 // tensor-memory lane quarter of this warp
        const int h = (warp - EPI_WARP0) / 4;   // of HALVES warps a quarter: every HALVES-th
        constexpr int HALVES = C::EPI_WARPS / 4;    // chunk of 32 rows of A
        Chunk ch;
        ch.q = q;
        ch.buf = smem_u32(sOut + h * 4 * C::OUT_BYTES);
        ch.bar = 1 + h;
        ch.lane = lane;
        int n = 0;
        for (int u = u0; u < units; u += du, ++n) {
            const int split = p.splits == 1 ? 0 : u % p.splits;
            const GrpTile t = grp_tile(start, first, steps, G, p.n_blocks,
                                       p.splits == 1 ? u : u / p.splits);
            const int acc = n & 1;
            ch.cta_n0 = t.nb * 256 + (int)rank * 128;
            ch.n0 = ch.cta_n0 + q * 32;
            const int n0 = ch.n0;
            const bool work = ch.cta_n0 < p.N;      // (the same for the whole group)
            const int chunks = ceil_div(t.rows, 32);
            // This group's chunks, of HALVES groups': h, h + HALVES, ..  With OVERLAP
            // the first accumulator's from the last on, so that the columns that
            // it shares with the second come first, and `keep` is the number of
            // the group's chunks that have none: at that many left, the next tile
            // may be accumulated.
            const int mine = work ? (chunks - h + HALVES - 1) / HALVES : 0;
            const bool down = C::OVERLAP && acc == 0;
            auto chunk_at = [&](int i) { return h + HALVES * (down ? mine - 1 - i : i); };
            int keep = 0;
            if (C::OVERLAP) {
                constexpr int SHARED = (C::TOKENS - C::ACC_STRIDE) / 32, OWN = C::ACC_STRIDE / 32;
                keep = down ? min(mine, (OWN - h + HALVES - 1) / HALVES)
                            : max(0, mine - (SHARED - h + HALVES - 1) / HALVES);
            }
            auto release = [&] {
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive_remote_tmem(mapa_shared(smem_u32(&acc_empty[C::OVERLAP ? 0 : acc]), 0));
            };
            // dY of a chunk is fetched while the one before is worked on
            uint4 dy_next[2];
            auto load_dy = [&](int i) {
                if (EPI != GRP_DSWIGLU) return;
                const int col = n0 / 2, r = chunk_at(i) * 32 + lane;
                const uint4 *src = reinterpret_cast<const uint4 *>(
                    reinterpret_cast<const uint16_t *>(p.dY) + (t.row0 + r) * (long long)(p.N / 2) + col);
#pragma unroll
                for (int j = 0; j < 2; ++j)          // (N / 2 is a multiple of 8)
                    dy_next[j] = r < t.rows && col + 8 * j < p.N / 2 ? src[j] : make_uint4(0, 0, 0, 0);
            };
            if (mine > 0) load_dy(0);
            if (p.k_blocks > 0) {
                const bool ok = wait_bounded(smem_u32(&acc_full[acc]), (n >> 1) & 1, abort_flag, p.err);
                // the whole group leaves, or none of it
                if (!named_bar_and(ch.bar, GROUP_THREADS, ok)) break;
                tc_fence_after();
                if (keep == mine) release();
            }
            const uint32_t t_row = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + acc * C::ACC_STRIDE;
            const bool direct = EPI == GRP_STORE &&
                                (p.out_kind == OUT_F32 || p.beta != 0.0f || p.k_blocks == 0);
            auto load = [&](int i, uint32_t(&r)[32]) {
                if (EPI == GRP_STORE) {
                    tmem_ld_fragments(t_row + chunk_at(i) * 32, r);
                } else if (p.k_blocks > 0) {
                    tmem_ld_32cols(t_row + chunk_at(i) * 32, r);
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) r[j] = 0;
                }
            };
            auto emit = [&](int i, const uint32_t(&r)[32]) {
                const int c = chunk_at(i);
                ch.row = t.row0 + c * 32;
                ch.rows = min(32, t.rows - c * 32);
                if (EPI == GRP_STORE) {
                    if (p.out_kind == OUT_F16)
                        emit_store_16<OUT_F16>(p, &maps.c, r, ch);
                    else
                        emit_store_16<OUT_BF16>(p, &maps.c, r, ch);
                } else {
                    const uint4 dy[2] = {dy_next[0], dy_next[1]};
                    if (i + 1 < mine) load_dy(i + 1);
                    emit_swiglu<EPI>(p, maps, r, dy, ch);
                }
            };
            int i = 0;
            if (C::TWO_SHARED && !direct && mine - keep == 2) {
                // both are read before the first is written out: the next
                // tile's MMAs wait for them (8192 x 14336 x 4096 151 -> 143 us)
                uint32_t r[32], second[32];
                load(0, r);
                load(1, second);
                tmem_ld_wait(r);
                tmem_ld_wait(second);
                release();
                emit(0, r);
                emit(1, second);
                i = 2;
            }
#pragma unroll 1
            for (; i < mine; ++i) {
                const bool last = p.k_blocks > 0 && mine - i == keep + 1;
                if (direct) {
                    const int c = chunk_at(i);
                    auto store = [&](auto kind) {
                        emit_store_direct<decltype(kind)::value>(
                            p, t_row + c * 32, split * p.split_stride, t.row0 + c * 32,
                            min(32, t.rows - c * 32), n0, lane);
                    };
                    if (p.out_kind == OUT_F32)
                        store(Kind<OUT_F32>());
                    else if (p.out_kind == OUT_F16)
                        store(Kind<OUT_F16>());
                    else
                        store(Kind<OUT_BF16>());
                    if (last) release();
                    continue;
                }
                uint32_t r[32];
                load(i, r);
                tmem_ld_wait(r);
                if (last) release();
                emit(i, r);
            }
        }
        if (q == 0 && lane == 0) bulk_wait_read_all();      // before this CTA's shared memory goes
    }

    // Neither CTA frees its tensor memory or exits while the leader's MMAs or
    // the peer's arrivals can still reach it.
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    if (warp == 1) tmem_dealloc_pair(tmem_base, C::TMEM_COLS);
}

}  // namespace swg
