// k_w4.cu — products of few rows with weights of 4 bits and group scales:
// C = alpha A W^T + beta C, and SwiGLU over alternating rows of W, dense or by
// expert.
//
// For few rows the weights' bytes are what the operator cannot do without; the
// kernel streams them once.  Decoding is most of its instructions: seven shifts and masks
// for eight codes, on a pipe that takes one every two cycles (a row through 14336 rows of
// 4096: 3.7 us of it, 4.5 of memory, 8.9 in all; 28672 x 4096: 16.0, 3.9 TB/s; 64 rows of 64
// experts, 2432 x 896: 15.8, of which 6.7 memory).  No pipe is full: a warp waits for its
// step, reads it, decodes and multiplies in turn, and the 12 to 16 warps that the shared
// memory of an SM has room for fill 47 and 56% of its issue slots and 42 and 45% of that pipe
// (the first and the last of these).  The rows of
// W are the 16 rows of an mma.sync m16n8k16 (FP32 accumulators), up to eight rows
// of A its columns: at one row of A 7/8 of the instruction's work is for nothing,
// but it is free, and the rows of W arrive in fragments as they lie in memory:
// codes become 16-bit numbers in registers, by one mask per two codes and one
// subtraction of the zero point, exactly.  (The tcgen05 instructions take their
// operands from shared or tensor memory, 128 rows of them: the decoded weights would
// pass through it once more, four times their size.  Decoding into tensor memory, which
// takes registers directly, has not been tried.)  Sums of a group of columns
// are scaled in FP32 as a whole, so that no product with a scale is ever rounded to
// 16 bits.
//
// w4_kernel: a CTA has one chunk of at most eight rows of A; its four warps are teams of
// `team` along K, and each team has 32 rows of W (64: a third fewer warps fit, 20.3 us
// instead of 17.4 for the experts above).  A team's warps take steps of 256
// columns in turn.  Each warp has a ring of its own that TMA fills: an elected lane asks
// for a step's codes (32 rows of 128 bytes), scales, zero points and columns of A, all from
// values that the warp shares (addresses of its lanes' own took a loop over the lanes, a
// seventh of all instructions), which leaves the issue slots to the decoding;
// cp.async by all lanes, with its addresses and edges, took as many instructions
// again.  A team's sums are added at the end, in order.  w4_many_kernel, for more
// rows or where there are too few rows of W, stands below it.
#include <algorithm>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "groups.cuh"
#include "host.h"
#include "launch.h"
#include "w4.h"

namespace swg {
namespace {

constexpr int WARPS = 4;
constexpr int MT = 2;                    // tiles of 16 rows of W per warp
constexpr int ROWS = 16 * MT;
constexpr int TOKENS = 8;                // rows of A per chunk
constexpr int STEP = 256;                // columns per warp and step
constexpr int CODES = ROWS * STEP / 2;   // bytes of a step
constexpr int SUMS = ROWS + 2;           // floats of a row of A's sums, padded
constexpr int STAGES = 2;
constexpr int SM_SHARED = 233472, CTA_SHARED = 232448;   // bytes of an SM (1024 of each CTA are the system's), most of a CTA

// d = a b (FIRST) or d += a b, a 16 x 16 (row fragments), b 16 x 8.
template <bool BF16, bool FIRST>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1)
{
    const float c[4] = {FIRST ? 0.0f : d[0], FIRST ? 0.0f : d[1], FIRST ? 0.0f : d[2], FIRST ? 0.0f : d[3]};
    if (BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

// A number whose units' place takes a code: 128 in bfloat16 (7 fraction bits),
// 1024 in binary16 (10), twice in a register.
template <bool BF16> constexpr uint32_t UNITS = BF16 ? 0x43004300u : 0x64006400u;

// Codes 2 i and 2 i + 1 of a word, less the zero point (given as UNITS + z).
// `units` is UNITS kept in a register: an instruction takes only one of mask and
// units as a constant, and would become two.
template <bool BF16>
__device__ __forceinline__ uint32_t decode(uint32_t word, int i, uint32_t units, uint32_t zero)
{
    uint32_t q;
    asm("lop3.b32 %0, %1, 0x000f000f, %2, 0xea;" : "=r"(q) : "r"(word >> (4 * i)), "r"(units));   // (a & b) | c
    if (BF16) {
        const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&q),
                                         *reinterpret_cast<const __nv_bfloat162 *>(&zero));
        return *reinterpret_cast<const uint32_t *>(&d);
    }
    const __half2 d = __hsub2(*reinterpret_cast<const __half2 *>(&q), *reinterpret_cast<const __half2 *>(&zero));
    return *reinterpret_cast<const uint32_t *>(&d);
}

template <bool BF16>
__device__ __forceinline__ float2 scale_pair(uint32_t s)
{
    return BF16 ? __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&s))
                : __half22float2(*reinterpret_cast<const __half2 *>(&s));
}

__device__ __forceinline__ void tma_load_3d_cta(uint32_t dst, const void *map, uint32_t bar, int x, int y, int z)
{
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar),
                 "r"(x), "r"(y), "r"(z)
                 : "memory");
}

struct W4Maps {
    CUtensorMap q, s, z, a;
};

// Shared memory: rings of codes, of A, of scales and zero points, barriers; then the
// teams' sums in its place.
// (of a box of `rows` rows of W)
__host__ __device__ constexpr int scales_bytes(int per, int rows) { return STEP / (32 * per) * rows * 2; }
__host__ __device__ constexpr int params_bytes(int per, bool zero, int rows) { return scales_bytes(per, rows) * (zero ? 3 : 2) / 2; }
__host__ __device__ constexpr int params_pitch(int per, bool zero, int rows) { return (params_bytes(per, zero, rows) + 127) / 128 * 128; }  // (TMA's rule)
__host__ __device__ constexpr int a_bytes(int tokens) { return STEP * 2 * tokens; }
__host__ __device__ constexpr int a_pitch(int tokens) { return tokens == 1 ? 1024 : a_bytes(tokens); }   // (whole times 1024)
__host__ __device__ constexpr int shared_bytes(int per, bool zero, int tokens)
{
    return WARPS * STAGES * (CODES + a_pitch(tokens) + params_pitch(per, zero, ROWS)) + 256;
}
static_assert(WARPS * STAGES * 8 + 8 <= 256, "barriers and the abort flag");

// Of a row's 128 bytes TMA puts 16-byte piece c to place c ^ (row % 8), the row being that
// of shared memory.  Lane (quad, t) computes with two neighbouring rows of each 16, a
// Gate and its Up, as rows quad and quad + 8 of the instruction; which, is chosen so
// that reads of 4, 8 or 16 bytes a lane meet no bank twice: rows 2 pi and 2 pi + 1, pi
// the quad with its lower bits swapped, the odd one first in quads 4 to 7.  Word j of
// the eight that lane t has of a row is columns 32 PER (j / PER) + 8 PER t + 8 (j % PER)
// .. + 7 (PER: a scale's columns in units of 32): the words of a place in all four
// lanes of a row share a scale.
struct Lane {
    int pi, odd, t;
    int w0, w1;                                      // where the first and second row's first word is in a box
    int x[8];                                        // ... and the columns of A of the eight words in a step of them
    uint32_t units, order;                           // (order: of the rows' scales)
};

// `row` of A, whose lines are `lines` apart from one 64 columns to the next.  (Steps
// of A begin at multiples of eight lines: all of this is the same for each.)
template <bool BF16, int PER>
__device__ __forceinline__ Lane lane_of(int row, int lines)
{
    Lane l;
    const int lane = threadIdx.x & 31, quad = lane >> 2;
    l.t = lane & 3;
    l.pi = (quad & 4) | (quad & 1) << 1 | (quad >> 1 & 1);
    l.odd = quad >> 2;
    const int row0 = 2 * l.pi + l.odd, row1 = 2 * l.pi + 1 - l.odd;
    const int piece = PER == 4 ? l.t : PER == 2 ? l.t >> 1 : 0, within = PER == 4 ? 0 : PER == 2 ? (l.t & 1) * 8 : l.t * 4;
    l.w0 = row0 * (STEP / 2) + ((piece ^ row0) & 7) * 16 + within;
    l.w1 = row1 * (STEP / 2) + ((piece ^ row1) & 7) * 16 + within;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int c = i / PER * (4 * PER) + PER * l.t + i % PER;     // columns in units of 8: block of 64, piece of it
        const int line = (c >> 3) * lines + row;
        l.x[i] = line * 128 + ((c ^ line) & 7) * 16;
    }
    asm volatile("mov.b32 %0, %1;" : "=r"(l.units) : "n"(UNITS<BF16>));
    l.order = l.odd ? 0x1032u : 0x3210u;
    return l;
}

// acc += the products of a step: codes and params as TMA left them, and rows of A in
// lines of 128 bytes, at these offsets of shared memory (codes 128, A 1024 bytes
// aligned); NT tiles of eight rows of A; MT pieces of 16 rows of W, from `piece` of the
// slot's box of BOX rows on.  whole: the second half has columns too.
template <bool BF16, int PER, bool ZERO, int BOX, int NT>
__device__ __forceinline__ void multiply(const Lane &l, const unsigned char *shared, int codes, int params, int a, bool whole,
                                         int piece, float (&acc)[MT][NT][4])
{
    const uint32_t *scale = reinterpret_cast<const uint32_t *>(shared + params) + piece * 8 + l.pi;
    const uint16_t *zero = reinterpret_cast<const uint16_t *>(shared + params + scales_bytes(PER, BOX)) + piece * 8 + l.pi;
    const uint32_t scale0 = l.odd ? 0x3244u : 0x1044u, scale1 = l.odd ? 0x1044u : 0x3244u;
    const int w0 = codes + piece * 16 * (STEP / 2) + l.w0, w1 = codes + piece * 16 * (STEP / 2) + l.w1;
    float part[MT][NT][4];
    uint32_t z0[MT], z1[MT];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        if (half == 1 && !whole) break;
        uint32_t w[2 * MT][4];                       // both rows of each 16
#pragma unroll
        for (int r = 0; r < 2 * MT; ++r) {
            // (a 16-byte piece further is one bit of the address turned over)
            const unsigned char *const at = shared + r / 2 * 16 * (STEP / 2);
            const int w_at = r % 2 ? w1 : w0;
            if (PER == 4) {
                const uint4 v = *reinterpret_cast<const uint4 *>(at + (w_at ^ (half * 64)));
                w[r][0] = v.x, w[r][1] = v.y, w[r][2] = v.z, w[r][3] = v.w;
            } else if (PER == 2) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint2 v = *reinterpret_cast<const uint2 *>(at + (w_at ^ (half * 64 + h * 32)));
                    w[r][2 * h] = v.x, w[r][2 * h + 1] = v.y;
                }
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) w[r][j] = *reinterpret_cast<const uint32_t *>(at + (w_at ^ (half * 64 + j * 16)));
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint4 x[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) x[n] = *reinterpret_cast<const uint4 *>(shared + n * 1024 + (a + l.x[4 * half + j]));
            const int b = (4 * half + j) / PER;      // the scale's place among the step's
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                if (j % PER == 0) {
                    z0[m] = z1[m] = UNITS<BF16> + 0x00080008u;
                    if (ZERO) {
                        const uint32_t z = __byte_perm(zero[(b * (BOX / 16) + m) * 8], 0, l.odd ? 0x4401 : 0x4410);
                        z0[m] = UNITS<BF16> + (z & 15u) * 0x00010001u;
                        z1[m] = UNITS<BF16> + (z >> 8 & 15u) * 0x00010001u;
                    }
                }
                const uint32_t w0 = w[2 * m][j], w1 = w[2 * m + 1][j];
                uint32_t f[8];                       // the fragments of two instructions
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    f[2 * i] = decode<BF16>(w0, i, l.units, z0[m]);
                    f[2 * i + 1] = decode<BF16>(w1, i, l.units, z1[m]);
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    if (j % PER == 0)
                        mma16816<BF16, true>(part[m][n], f[0], f[1], f[2], f[3], x[n].x, x[n].y);
                    else
                        mma16816<BF16, false>(part[m][n], f[0], f[1], f[2], f[3], x[n].x, x[n].y);
                    mma16816<BF16, false>(part[m][n], f[4], f[5], f[6], f[7], x[n].z, x[n].w);
                }
                if (j % PER == PER - 1) {
                    float2 s;
                    if (BF16)                        // (a bfloat16 is the upper half of its FP32)
                        s = make_float2(__uint_as_float(__byte_perm(scale[(b * (BOX / 16) + m) * 8], 0, scale0)),
                                        __uint_as_float(__byte_perm(scale[(b * (BOX / 16) + m) * 8], 0, scale1)));
                    else
                        s = scale_pair<BF16>(__byte_perm(scale[(b * (BOX / 16) + m) * 8], 0, l.order));
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        acc[m][n][0] = fmaf(s.x, part[m][n][0], acc[m][n][0]);
                        acc[m][n][1] = fmaf(s.x, part[m][n][1], acc[m][n][1]);
                        acc[m][n][2] = fmaf(s.y, part[m][n][2], acc[m][n][2]);
                        acc[m][n][3] = fmaf(s.y, part[m][n][3], acc[m][n][3]);
                    }
                }
            }
        }
    }
}

// Columns n, n + 1 of a row of A.
__device__ __forceinline__ void store_pair(const W4Args &p, int row, int n, float x, float y)
{
    if (n >= p.w.N) return;
    const long long o = row * p.ldc;
    x *= p.alpha;
    y *= p.alpha;
    if (p.swiglu) {
        store_out(p.C, o + n / 2, silu_f32(x) * y, p.out_kind);
        return;
    }
    if (p.beta != 0.0f) x += p.beta * load_out(p.C, o + n, p.out_kind);
    store_out(p.C, o + n, x, p.out_kind);
    if (n + 1 < p.w.N) {
        if (p.beta != 0.0f) y += p.beta * load_out(p.C, o + n + 1, p.out_kind);
        store_out(p.C, o + n + 1, y, p.out_kind);
    }
}

// Rows 2 pi and 2 pi + 1 of what a lane has of 16 rows of W, for row h of A.
__device__ __forceinline__ float2 rows_of(const Lane &l, const float (&c)[4], int h)
{
    return l.odd ? make_float2(c[2 + h], c[h]) : make_float2(c[h], c[2 + h]);
}

// `tokens`: rows of A of a chunk, 1, 2, 4 or 8.  `team`: a power of two.
template <bool BF16, int PER, bool ZERO>
__global__ void __launch_bounds__(32 * WARPS, 4)
    w4_kernel(const __grid_constant__ W4Maps maps, const W4Args p, int tiles, int tokens, int team, int *err)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    extern __shared__ __align__(1024) unsigned char shared[];
    constexpr int BLOCKS = STEP / (32 * PER), PARAMS = params_pitch(PER, ZERO, ROWS);
    const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);     // (known to be the same in all lanes)
    const int wk = warp & (team - 1), quad = lane >> 2;
    const int of_a = a_pitch(tokens);
    const int codes = warp * STAGES * CODES, a = WARPS * STAGES * CODES + warp * STAGES * of_a;
    const int params = WARPS * STAGES * (CODES + of_a) + warp * STAGES * PARAMS;
    unsigned char *const at_bars = shared + WARPS * STAGES * (CODES + of_a + PARAMS);
    const uint32_t bars = smem_u32(at_bars) + warp * STAGES * 8;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(at_bars + WARPS * STAGES * 8);
    if (lane == 0) {
#pragma unroll
        for (int i = 0; i < STAGES; ++i) mbar_init(bars + 8 * i, 1);
        fence_barrier_init();
        if (warp == 0) *abort_flag = 0;
    }
    const int chunk = blockIdx.x / tiles, tile = blockIdx.x - chunk * tiles;
    const int n0 = (tile * (WARPS / team) + warp / team) * ROWS;
    __syncthreads();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int g, row0, rows;
    if (!find_chunk(p.groups, tokens, chunk, err, g, row0, rows)) return;

    const int steps = n0 < p.w.N ? (p.w.K + STEP - 1) / STEP : 0;
    auto load = [&](int step, int slot) {            // by one lane
        if (elect_one()) {
            const uint32_t bar = bars + 8 * slot, to = smem_u32(shared) + params + slot * PARAMS;
            mbar_arrive_expect_tx(bar, CODES + params_bytes(PER, ZERO, ROWS) + a_bytes(tokens));
            tma_load_3d_cta(smem_u32(shared) + codes + slot * CODES, &maps.q, bar, step * (STEP / 2), n0, g);
            tma_load_3d_cta(to, &maps.s, bar, n0, step * BLOCKS, g);
            if (ZERO) tma_load_3d_cta(to + scales_bytes(PER, ROWS), &maps.z, bar, n0, step * BLOCKS, g);
#pragma unroll
            for (int c = 0; c < 4; ++c)
                tma_load_2d(smem_u32(shared) + a + slot * of_a + c * tokens * 128, &maps.a, bar, step * STEP + c * 64, row0);
        }
    };
#pragma unroll 1
    for (int i = 0; i < STAGES; ++i)
        if (wk + i * team < steps) load(wk + i * team, i);

    // (lanes of rows of A that do not exist compute with another, for nothing)
    const Lane l = lane_of<BF16, PER>(min(quad, tokens - 1), tokens);
    float acc[MT][1][4] = {};
    bool stopped = false;
    int step = wk, slot = 0;
    uint32_t parity = 0;
    for (; step < steps; step += team) {
        if (!__all_sync(0xffffffffu, wait_bounded(bars + 8 * slot, parity, abort_flag, err))) {
            stopped = true;
            break;
        }
        multiply<BF16, PER, ZERO, ROWS, 1>(l, shared, codes + slot * CODES, params + slot * PARAMS, a + slot * of_a,
                                           step * STEP + STEP / 2 < p.w.K, 0, acc);
        __syncwarp();
        if (step + STAGES * team < steps) load(step + STAGES * team, slot);
        slot = slot + 1 == STAGES ? 0 : slot + 1;
        parity ^= slot == 0;
    }
    if (stopped)                                     // what is still on its way lands before the CTA ends
        for (int i = 0; i < STAGES; ++i, step += team) {
            if (step < steps) wait_bounded(bars + 8 * slot, parity, abort_flag, err, false, DRAIN_LIMIT_NS);
            slot = slot + 1 == STAGES ? 0 : slot + 1;
            parity ^= slot == 0;
        }
    if (team == 1) {
        if (stopped) return;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float2 v = rows_of(l, acc[m][0], h);
                if (2 * l.t + h < rows) store_pair(p, row0 + 2 * l.t + h, n0 + m * 16 + 2 * l.pi, v.x, v.y);
            }
        return;
    }
    // [warp][row of A][row of W]
    float *sums = reinterpret_cast<float *>(shared);
    __syncthreads();
    if (*abort_flag) return;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (2 * l.t + h < rows)
                *reinterpret_cast<float2 *>(sums + (warp * tokens + 2 * l.t + h) * SUMS + m * 16 + 2 * l.pi) = rows_of(l, acc[m][0], h);
    __syncthreads();
    const float *of_team = sums + (warp & ~(team - 1)) * tokens * SUMS;
    for (int o = wk * 32 + lane; o < rows * (ROWS / 2); o += team * 32) {
        const int row = o / (ROWS / 2), pair = o % (ROWS / 2);
        float x = 0.0f, y = 0.0f;
        for (int w = 0; w < team; ++w) {
            const float2 v = *reinterpret_cast<const float2 *>(of_team + (w * tokens + row) * SUMS + 2 * pair);
            x += v.x;
            y += v.y;
        }
        store_pair(p, row0 + row, n0 + 2 * pair, x, y);
    }
}

// ------------------------------------------------------------ more rows of A

// Chunks of 8, 16 or 32 rows of A, NT = 1, 2 or 4 tiles of 8.  A code decoded is used NT
// times, and from NT = 2 on the mma.sync instructions bound it: one takes 17 cycles of
// its quarter of an SM, as measured (32 rows, 4096 x 14336: 13.4 us on all SMs).  Rows
// of A are as much to read as codes then, so four warps of 32 rows of W share them: a
// CTA has 128 rows of W and a range of the steps, a fifth warp feeds its ring, two CTAs
// fill an SM, and the CTAs of a cluster that have a tile's ranges add their sums
// through shared memory, in order.  (One CTA of 256 rows for each SM: 41 us, since only
// 15 clusters of eight of that size are resident, and 35.9 with clusters of four; this
// 19.0; chunks of eight rows of the other kernel 29.3.)
constexpr int MANY_ROWS = WARPS * ROWS, MANY_BOX = 64, MANY_BOXES = MANY_ROWS / MANY_BOX;
constexpr int MANY_CODES = MANY_BOX * STEP / 2;
constexpr int MANY_THREADS = 32 * (WARPS + 1);
constexpr int MANY_STAGES = 3;
constexpr int MANY_SUMS = MANY_ROWS + 2;             // floats of a row of A's sums, padded
constexpr int MOST_RANGES = 8;

__host__ __device__ constexpr int many_stage(int per, bool zero, int nt)
{
    return MANY_BOXES * (MANY_CODES + params_pitch(per, zero, MANY_BOX)) + a_bytes(8 * nt);
}
__host__ __device__ constexpr int many_shared(int per, bool zero, int nt) { return MANY_STAGES * many_stage(per, zero, nt) + 256; }
static_assert(2 * (many_shared(1, true, 4) + 1024) <= SM_SHARED, "two CTAs on an SM");
static_assert(MANY_SUMS * 32 * 4 <= MANY_STAGES * MANY_BOXES * MANY_CODES, "the sums take the ring's place");

__device__ __forceinline__ float2 load_cluster(uint32_t at)
{
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at) : "memory");
    return v;
}

template <bool BF16, int PER, bool ZERO, int NT>
__global__ void __launch_bounds__(MANY_THREADS, 2)
    w4_many_kernel(const __grid_constant__ W4Maps maps, const W4Args p, int tiles, int ranges, int *err)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    extern __shared__ __align__(1024) unsigned char shared[];
    constexpr int BLOCKS = STEP / (32 * PER), PARAMS = params_pitch(PER, ZERO, MANY_BOX), TOKENS_MANY = 8 * NT;
    constexpr int A = MANY_STAGES * MANY_BOXES * MANY_CODES, P = A + MANY_STAGES * a_bytes(TOKENS_MANY), B = P + MANY_STAGES * MANY_BOXES * PARAMS;
    const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    const uint32_t full = smem_u32(shared) + B, empty = full + 8 * MANY_STAGES;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(shared + B + 16 * MANY_STAGES);
    // (a cluster's CTAs, the ranges of a tile, follow one another)
    const int range = blockIdx.x % ranges, unit = blockIdx.x / ranges, chunk = unit / tiles, tile = unit - chunk * tiles;
    const int n0 = tile * MANY_ROWS, boxes = min(MANY_BOXES, (p.w.N - n0 + MANY_BOX - 1) / MANY_BOX), used = boxes * (WARPS / MANY_BOXES);
    if (threadIdx.x == 0) {
#pragma unroll
        for (int i = 0; i < MANY_STAGES; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, used);
        }
        fence_barrier_init();
        *abort_flag = 0;
    }
    __syncthreads();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int g, row0, rows;
    if (!find_chunk(p.groups, TOKENS_MANY, chunk, err, g, row0, rows)) return;   // (the whole cluster)

    const int steps = (p.w.K + STEP - 1) / STEP, first = (int)((long long)steps * range / ranges);
    const int count = (int)((long long)steps * (range + 1) / ranges) - first;
    float acc[MT][NT][4] = {};
    const Lane l = lane_of<BF16, PER>(lane >> 2, TOKENS_MANY);
    if (warp == WARPS) {
        int i = 0;
        for (; i < count; ++i) {
            const int slot = i % MANY_STAGES, step = first + i;
            const uint32_t bar = full + 8 * slot;
            if (i >= MANY_STAGES &&
                !__all_sync(0xffffffffu, wait_bounded(empty + 8 * slot, (uint32_t)((i / MANY_STAGES) - 1) & 1u, abort_flag, err)))
                break;
            if (elect_one()) {
                mbar_arrive_expect_tx(bar, boxes * (MANY_CODES + params_bytes(PER, ZERO, MANY_BOX)) + a_bytes(TOKENS_MANY));
                for (int w = 0; w < boxes; ++w) {
                    const uint32_t to = smem_u32(shared) + P + (slot * MANY_BOXES + w) * PARAMS;
                    tma_load_3d_cta(smem_u32(shared) + (slot * MANY_BOXES + w) * MANY_CODES, &maps.q, bar, step * (STEP / 2), n0 + w * MANY_BOX, g);
                    tma_load_3d_cta(to, &maps.s, bar, n0 + w * MANY_BOX, step * BLOCKS, g);
                    if (ZERO) tma_load_3d_cta(to + scales_bytes(PER, MANY_BOX), &maps.z, bar, n0 + w * MANY_BOX, step * BLOCKS, g);
                }
                for (int c = 0; c < 4; ++c)
                    tma_load_2d(smem_u32(shared) + A + slot * a_bytes(TOKENS_MANY) + c * TOKENS_MANY * 128, &maps.a, bar, step * STEP + c * 64, row0);
            }
            __syncwarp();
        }
        // (all that is on its way lands before the sums take its place, after a wait that ran out too)
        for (int j = max(i - MANY_STAGES, 0); j < i; ++j)
            wait_bounded(full + 8 * (j % MANY_STAGES), (uint32_t)(j / MANY_STAGES) & 1u, abort_flag, err, false, DRAIN_LIMIT_NS);
        __syncwarp();
    } else if (warp < used) {
        const int box = warp / (WARPS / MANY_BOXES);
        for (int i = 0; i < count; ++i) {
            const int slot = i % MANY_STAGES;
            if (!__all_sync(0xffffffffu, wait_bounded(full + 8 * slot, (uint32_t)(i / MANY_STAGES) & 1u, abort_flag, err))) break;
            multiply<BF16, PER, ZERO, MANY_BOX, NT>(l, shared, (slot * MANY_BOXES + box) * MANY_CODES, P + (slot * MANY_BOXES + box) * PARAMS,
                                                    A + slot * a_bytes(TOKENS_MANY), (first + i) * STEP + STEP / 2 < p.w.K,
                                                    warp * MT % (MANY_BOX / 16), acc);
            __syncwarp();
            if (lane == 0) mbar_arrive(empty + 8 * slot);
        }
    }
    // Sums: [row of A][row of W], in the ring's place.
    __syncthreads();
    float *sums = reinterpret_cast<float *>(shared);
    if (warp < used) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    *reinterpret_cast<float2 *>(sums + (8 * n + 2 * l.t + h) * MANY_SUMS + (warp * MT + m) * 16 + 2 * l.pi) =
                        rows_of(l, acc[m][n], h);
    }
    if (ranges > 1) cluster_sync_all();
    else __syncthreads();
    // A share of the pairs of rows of W for each CTA of the cluster.
    const int pairs = MANY_ROWS / 2 / ranges, from = range * pairs;
    if (!*abort_flag)
        for (int o = threadIdx.x; o < rows * pairs; o += MANY_THREADS) {
            const int row = o / pairs, pair = from + o - row * pairs;
            if (n0 + 2 * pair >= p.w.N) continue;
            const uint32_t at = smem_u32(sums + row * MANY_SUMS + 2 * pair);
            float x = 0.0f, y = 0.0f;
            for (int r = 0; r < ranges; ++r) {
                const float2 v = ranges > 1 ? load_cluster(mapa_shared(at, r)) : *reinterpret_cast<const float2 *>(sums + row * MANY_SUMS + 2 * pair);
                x += v.x;
                y += v.y;
            }
            store_pair(p, row0 + row, n0 + 2 * pair, x, y);
        }
    if (ranges > 1) cluster_sync_all();              // no CTA leaves while its sums are read
}

// An upper bound of the chunks over all groups, and with offsets one more, whose
// CTAs find nothing: on the way they look at every offset and report what they
// have to clamp.
long long chunks_of(const Groups &g, int tokens)
{
    return g.offsets == nullptr ? (g.M + tokens - 1) / tokens : g.M / tokens + std::min(g.G, g.M) + 1;
}

struct Shape {
    int tokens;                                      // rows of A of a chunk
    bool many;                                       // of w4_many_kernel
};

// (Times in us, bfloat16, groups of 128 with zero points, each of the same build on both
// sides.)
Shape shape_of(const W4Args &p, int sms)
{
    const Groups &g = p.groups;
    const int steps = (p.w.K + STEP - 1) / STEP;
    const long long items = (p.w.N + ROWS - 1ll) / ROWS;
    // Groups: chunks of four times their mean and four rows at least, since another chunk
    // reads and decodes the weights again (64 rows of 64 experts of 2432 x 896, scales of 32
    // columns: 21.9 with chunks of 1, 18.5 with 2, 18.3 with 4, 18.9 with 8; 4 rows, 8 experts of
    // 8192 x 2048: 9.1 with 2, 6.8 with 4, 8.6 with 8; 8 rows, 16 experts of 4096 x 1024: 6.7 with
    // 2, 7.5 with 4, 8.2 with 8).  More than eight rows from a mean of 16 on, where the fuller
    // instructions outweigh the emptier chunks (16 experts of 4096 x 1024: means of 8 23.7 and
    // 17.4, 12 24.8 and 22.3, 16 26.3 and 27.0, 32 37.8 and 44.8).
    if (g.offsets != nullptr && g.M >= 16ll * g.G) return {32, true};
    const int want = g.offsets == nullptr ? g.M : (int)std::min<long long>(g.M, std::max(4ll, (4ll * g.M + g.G - 1) / g.G));
    // More than eight rows (4096 x 14336, 32 rows: 19.0 and 29.3; 14336 x 4096, 9 rows: 15.0
    // and 15.9), unless there is too little to do for a cluster's barriers (2048 x 8192, 16
    // rows: 9.0 and 7.4; 8192 x 1024, 16 rows: 6.3 and 5.1).
    if (g.offsets == nullptr && want > TOKENS && (want + TOKENS - 1) / TOKENS * items * steps > 28ll * sms)
        return {want <= 16 ? 16 : 32, true};
    // Up to eight, where rows are long and few: a cluster has up to 32 warps for a tile, a
    // team four (one row, 1024 x 8192: 5.7 and 7.5; 2048 x 8192: 7.4 and 7.5; but 4096 x 14336
    // 14.1 and 12.3).
    if (steps > 24 && (g.offsets == nullptr ? 1 : std::min(g.G, g.M)) * items * 2 < sms) return {TOKENS, true};
    return {want <= 1 ? 1 : want <= 2 ? 2 : want <= 4 ? 4 : TOKENS, false};
}

template <bool BF16, int PER, bool ZERO>
cudaError_t launch(const W4Args &p, const W4Maps &maps, int tokens, int sms, int *err, cudaStream_t s)
{
    // As small teams as leave 16 warps for each SM, as many as are resident (8 experts of
    // 4096 x 4096, 8 rows: 13.9, and 17.7 with 12 warps).
    const int steps = (p.w.K + STEP - 1) / STEP;
    const long long items = (p.groups.offsets ? std::min(p.groups.G, p.groups.M) : chunks_of(p.groups, tokens)) * ((p.w.N + ROWS - 1ll) / ROWS);
    int team = 1;
    while (team < WARPS && team < steps && items * team < 16ll * sms) team *= 2;
    const size_t sums = (size_t)WARPS * tokens * SUMS * 4;
    auto kernel = w4_kernel<BF16, PER, ZERO>;
    static DeviceOnce once;
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev)) return e;
    if (once.needed(dev)) {
        if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, CTA_SHARED)) return e;
        once.mark(dev);
    }
    const int per_cta = ROWS * (WARPS / team), tiles = (p.w.N + per_cta - 1) / per_cta;
    const long long ctas = chunks_of(p.groups, tokens) * tiles;
    size_t room = std::max((size_t)shared_bytes(PER, ZERO, tokens), sums);
    // CTAs that are resident at once are spread evenly: no more of them fit an SM than its
    // share (one row, 14336 x 4096: 448 CTAs, 9.5 and 11.8 when some SMs have four and some
    // two; 4096 x 4096: 4.8 and 5.4).  Of groups it is not known how many have work.
    const long long share = (ctas + sms - 1) / sms;
    if (p.groups.offsets == nullptr && share < 8) room = std::max(room, std::min<size_t>(SM_SHARED / (share + 1) - 1024 + 128, CTA_SHARED));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(32 * WARPS);
    cfg.dynamicSmemBytes = room;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, maps, p, tiles, tokens, team, err);
}

template <bool BF16, int PER, bool ZERO, int NT>
cudaError_t launch_many(const W4Args &p, const W4Maps &maps, int sms, int *err, cudaStream_t s)
{
    // As many ranges of the steps as the SMs have places for CTAs, two each (in us, with 1, 2,
    // 4 and 8: 32 rows, 14336 x 4096 32.3, 22.6, 26.2, 32.6; 4096 x 14336 61.8, 34.7, 27.6, 19.0).
    const int steps = (p.w.K + STEP - 1) / STEP, tiles = (p.w.N + MANY_ROWS - 1) / MANY_ROWS;
    const long long chunks = chunks_of(p.groups, 8 * NT);
    // (of groups half a chunk more for each than their rows fill: 64 rows of 4 experts of 4096 x
    // 4096 21.5 in two ranges, 30.5 in one, 25.2 in four)
    const long long units = (p.groups.offsets ? p.groups.M / (8 * NT) + (std::min(p.groups.G, p.groups.M) + 1) / 2 : chunks) * tiles;
    int ranges = 1;
    while (ranges < MOST_RANGES && 2 * ranges <= steps && ranges * units <= sms) ranges *= 2;
    auto kernel = w4_many_kernel<BF16, PER, ZERO, NT>;
    static DeviceOnce once;
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev)) return e;
    if (once.needed(dev)) {
        if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, many_shared(PER, ZERO, NT))) return e;
        once.mark(dev);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(chunks * tiles * ranges));
    cfg.blockDim = dim3(MANY_THREADS);
    cfg.dynamicSmemBytes = many_shared(PER, ZERO, NT);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ranges;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, maps, p, tiles, ranges, err);
}

template <bool BF16, int PER, bool ZERO>
cudaError_t launch_any(const W4Args &p, const W4Maps &maps, Shape shape, int sms, int *err, cudaStream_t s)
{
    return !shape.many               ? launch<BF16, PER, ZERO>(p, maps, shape.tokens, sms, err, s)
           : shape.tokens == TOKENS ? launch_many<BF16, PER, ZERO, 1>(p, maps, sms, err, s)
           : shape.tokens == 16     ? launch_many<BF16, PER, ZERO, 2>(p, maps, sms, err, s)
                                    : launch_many<BF16, PER, ZERO, 4>(p, maps, sms, err, s);
}

template <bool BF16, int PER>
cudaError_t launch_zero(const W4Args &p, const W4Maps &maps, Shape shape, int sms, int *err, cudaStream_t s)
{
    return p.w.Z != nullptr ? launch_any<BF16, PER, true>(p, maps, shape, sms, err, s) : launch_any<BF16, PER, false>(p, maps, shape, sms, err, s);
}

template <bool BF16>
cudaError_t launch_group(const W4Args &p, const W4Maps &maps, Shape shape, int sms, int *err, cudaStream_t s)
{
    return p.w.group == 32   ? launch_zero<BF16, 1>(p, maps, shape, sms, err, s)
           : p.w.group == 64 ? launch_zero<BF16, 2>(p, maps, shape, sms, err, s)
                             : launch_zero<BF16, 4>(p, maps, shape, sms, err, s);
}

}  // namespace

bool w4_fits(const W4Args &p) { return chunks_of(p.groups, 1) * ((p.w.N + 31ll) / 32) <= 0x7fffffff; }

cudaError_t launch_w4(const W4Args &p, int sms, int *err, cudaStream_t s, bool &mapped)
{
    W4Maps maps{};
    const Shape shape = shape_of(p, sms);
    mapped = true;
    if (p.w.K > 0) {
        const uint64_t N = p.w.N, G = p.groups.G, blocks = p.w.blocks(), row = p.w.row_bytes(), lds = p.w.lds;
        const uint32_t per_step = STEP / p.w.group;
        const uint64_t qd[] = {row, N, G}, qs[] = {row, G > 1 ? row * N : row};
        const uint32_t box = shape.many ? MANY_BOX : ROWS, qb[] = {STEP / 2, box, 1}, sb[] = {box, per_step, 1};
        const uint64_t sd[] = {lds, blocks, G}, ss[] = {lds * 2, G > 1 ? lds * 2 * blocks : lds * 2}, zs[] = {lds, G > 1 ? lds * blocks : lds};
        const uint64_t ad[] = {(uint64_t)p.w.K, (uint64_t)p.groups.M}, as[] = {(uint64_t)p.lda * 2};
        const uint32_t ab[] = {64, (uint32_t)shape.tokens};
        mapped = encode_tiled(&maps.q, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, p.w.Q, qd, qs, qb, 128) &&
                 encode_tiled(&maps.s, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, p.w.S, sd, ss, sb, 0) &&
                 (p.w.Z == nullptr || encode_tiled(&maps.z, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, p.w.Z, sd, zs, sb, 0)) &&
                 encode_tiled(&maps.a, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, p.A, ad, as, ab, 128);
        if (!mapped) return cudaErrorInvalidValue;
    }
    return p.bf16 ? launch_group<true>(p, maps, shape, sms, err, s) : launch_group<false>(p, maps, shape, sms, err, s);
}

}  // namespace swg
