// k_w4.cu — products of few rows with weights of 4 bits and group scales:
// C = alpha A W^T + beta C, and SwiGLU over alternating rows of W, dense or by
// expert.
//
// For few rows the weights' bytes are what the operator cannot do without, so the
// kernel streams them once and keeps the arithmetic behind that.  The rows of
// W are the 16 rows of an mma.sync m16n8k16 (FP32 accumulators), up to eight rows
// of A its columns: at one row of A 7/8 of the instruction's work is for nothing,
// but it is free, and the rows of W arrive in fragments as they lie in memory:
// codes become 16-bit numbers in registers, by one mask per two codes and one
// subtraction of the zero point, exactly.  (The tcgen05 instructions take their
// operands from shared or tensor memory, 128 rows of them: the decoded weights would
// pass through it once more, four times their size.)  Sums of a group of columns
// are scaled in FP32 as a whole, so that no product with a scale is ever rounded to
// 16 bits.
//
// A CTA has 16 MT rows of W and one chunk of rows of A; its eight warps take steps
// of 128 columns in turn, so that a row's 512 bytes are asked for together.
// Each warp has a ring of its own in shared memory, filled by cp.async a few
// steps ahead (codes, scales, zero points and A: no barrier but the warp's), and
// the warps' sums are added at the end, in order.
#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "groups.cuh"
#include "launch.h"
#include "w4.h"

namespace swg {
namespace {

constexpr int WARPS = 8;
constexpr int TOKENS = 8;                // rows of A per chunk
constexpr int STEP = 128;                // columns per warp and step
constexpr int ROW_PITCH = 80;            // bytes of a row's 128 codes in the ring: eight rows' 16-byte
                                         // pieces, read four bytes a lane, fall on all banks

// Copies 16 bytes, of which those from `bytes` on are zero and not read.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, int bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint32_t ld_shared(uint32_t a)
{
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t ld_shared_u16(uint32_t a)
{
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}

// d += a b, a 16 x 16 (row fragments), b 16 x 8.
template <bool BF16>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1)
{
    if (BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A number whose units' place takes a code: 128 in bfloat16 (7 fraction bits),
// 1024 in binary16 (10), twice in a register.
template <bool BF16> constexpr uint32_t UNITS = BF16 ? 0x43004300u : 0x64006400u;

// Codes 2 i and 2 i + 1 of a word, less the zero point (given as UNITS + z).
template <bool BF16>
__device__ __forceinline__ uint32_t decode(uint32_t word, int i, uint32_t zero)
{
    const uint32_t q = ((word >> (4 * i)) & 0x000f000fu) | UNITS<BF16>;
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

// Bytes of a stage of a warp's ring.
__host__ __device__ constexpr int codes_bytes(int mt) { return mt * 16 * ROW_PITCH; }
__host__ __device__ constexpr int scales_bytes(int mt, int per) { return STEP / (32 * per) * mt * 16 * 2; }
__host__ __device__ constexpr int stage_bytes(int mt, int per, int tokens)
{
    return codes_bytes(mt) + scales_bytes(mt, per) * 3 / 2 + tokens * STEP * 2;
}

// PER: a scale's columns in units of 32.  `tokens`: rows of A that a chunk can
// have, at most TOKENS.
template <bool BF16, int MT, int PER, int STAGES>
__global__ void __launch_bounds__(32 * WARPS) w4_kernel(const W4Args p, int tiles, int tokens, int *err)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    extern __shared__ __align__(16) unsigned char shared[];
    constexpr int ROWS = 16 * MT, BLOCKS = STEP / (32 * PER);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int unit = blockIdx.x / tiles, n0 = (blockIdx.x - unit * tiles) * ROWS;
    int g, row0, rows;
    if (!find_chunk<TOKENS>(p.groups, unit, err, g, row0, rows)) return;

    const int stage = stage_bytes(MT, PER, tokens);
    const uint32_t ring = smem_u32(shared) + warp * STAGES * stage;
    const int steps = (p.w.K + STEP - 1) / STEP, row_bytes = p.w.row_bytes(), blocks = p.w.blocks();
    const uint8_t *codes = p.w.Q + (long long)g * p.w.N * row_bytes;
    const long long first_block = (long long)g * blocks;

    auto load = [&](int step, int slot) {
        const uint32_t at = ring + slot * stage;
        // codes: row r of a 16 in place r / 2 + 8 (r % 2), so that a lane's two rows
        // are neighbours in W (a Gate and its Up)
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i) {
            const int r = i * 8 + (lane >> 2), n = n0 + r, c = step * 64 + (lane & 3) * 16;
            const int place = (r & ~15) + ((r & 15) >> 1) + 8 * (r & 1);
            const bool in = n < p.w.N && c < row_bytes;
            copy16(at + place * ROW_PITCH + (lane & 3) * 16, codes + (in ? (long long)n * row_bytes + c : 0),
                   in ? 16 : 0);
        }
        const uint32_t scales = at + codes_bytes(MT);
        if (lane < BLOCKS * MT * 2) {
            const int b = lane / (MT * 2), part = lane % (MT * 2), block = step * BLOCKS + b;
            const bool in = block < blocks && n0 + part * 8 < p.w.lds;
            copy16(scales + lane * 16,
                   static_cast<const uint16_t *>(p.w.S) + (in ? (first_block + block) * p.w.lds + n0 + part * 8 : 0),
                   in ? 16 : 0);
        }
        if (p.w.Z != nullptr && lane < BLOCKS * MT) {
            const int b = lane / MT, part = lane % MT, block = step * BLOCKS + b;
            const bool in = block < blocks && n0 + part * 16 < p.w.lds;
            copy16(scales + scales_bytes(MT, PER) + lane * 16,
                   p.w.Z + (in ? (first_block + block) * p.w.lds + n0 + part * 16 : 0), in ? 16 : 0);
        }
        // A: lane (row, t) has columns 32 j + 8 t .. + 7 of the step, as it will read them
        const uint32_t a = scales + scales_bytes(MT, PER) * 3 / 2;
        if ((lane >> 2) < rows) {
            const char *row = static_cast<const char *>(p.A) + (long long)(row0 + (lane >> 2)) * p.lda * 2;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int k = step * STEP + j * 32 + (lane & 3) * 8;
                const int left = min(max(p.w.K - k, 0), 8) * 2;
                copy16(a + (j * tokens * 4 + lane) * 16, row + (left > 0 ? (long long)k * 2 : 0), left);
            }
        }
    };

    float acc[MT][4] = {};
    const int mine = steps > warp ? (steps - warp + WARPS - 1) / WARPS : 0;
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) {
        if (i < mine) load(warp + i * WARPS, i);
        copies_commit();
    }
    int slot = 0;
    for (int i = 0; i < mine; ++i) {
        copies_wait<STAGES - 2>();
        __syncwarp();
        const uint32_t at = ring + slot * stage, scales = at + codes_bytes(MT);
        const uint32_t a = scales + scales_bytes(MT, PER) * 3 / 2;
        float part[MT][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint4 x = make_uint4(0, 0, 0, 0);
            if ((lane >> 2) < rows) x = ld_shared_v4(a + (j * tokens * 4 + lane) * 16);
            const int b = j / PER;                   // the scale's place among the step's
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                if (j % PER == 0) part[m][0] = part[m][1] = part[m][2] = part[m][3] = 0.0f;
                const uint32_t row = at + (m * 16 + (lane >> 2)) * ROW_PITCH + j * 16 + (lane & 3) * 4;
                const uint32_t w0 = ld_shared(row), w1 = ld_shared(row + 8 * ROW_PITCH);
                const int pair = b * MT * 8 + m * 8 + (lane >> 2);
                uint32_t z0 = UNITS<BF16> + 0x00080008u, z1 = z0;
                if (p.w.Z != nullptr) {
                    const uint32_t z = ld_shared_u16(scales + scales_bytes(MT, PER) + pair * 2);
                    z0 = UNITS<BF16> + (z & 15u) * 0x00010001u;
                    z1 = UNITS<BF16> + (z >> 8 & 15u) * 0x00010001u;
                }
                mma16816<BF16>(part[m], decode<BF16>(w0, 0, z0), decode<BF16>(w1, 0, z1), decode<BF16>(w0, 1, z0),
                               decode<BF16>(w1, 1, z1), x.x, x.y);
                mma16816<BF16>(part[m], decode<BF16>(w0, 2, z0), decode<BF16>(w1, 2, z1), decode<BF16>(w0, 3, z0),
                               decode<BF16>(w1, 3, z1), x.z, x.w);
                if (j % PER == PER - 1) {
                    const float2 s = scale_pair<BF16>(ld_shared(scales + pair * 4));
                    acc[m][0] = fmaf(s.x, part[m][0], acc[m][0]);
                    acc[m][1] = fmaf(s.x, part[m][1], acc[m][1]);
                    acc[m][2] = fmaf(s.y, part[m][2], acc[m][2]);
                    acc[m][3] = fmaf(s.y, part[m][3], acc[m][3]);
                }
            }
        }
        __syncwarp();
        const int next = i + STAGES - 1;
        if (next < mine) load(warp + next * WARPS, slot == 0 ? STAGES - 1 : slot - 1);
        copies_commit();
        slot = slot + 1 == STAGES ? 0 : slot + 1;
    }
    copies_wait<0>();
    __syncthreads();

    // The warps' sums, in order: [warp][token][row], rows padded by 2.
    constexpr int PITCH = ROWS + 2;
    float *sums = reinterpret_cast<float *>(shared);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int token = 2 * (lane & 3) + h, row = m * 16 + 2 * (lane >> 2);
            if (token < rows)
                *reinterpret_cast<float2 *>(sums + (warp * tokens + token) * PITCH + row) =
                    make_float2(acc[m][h], acc[m][2 + h]);
        }
    __syncthreads();
    constexpr int PAIRS = ROWS / 2;
    for (int i = threadIdx.x; i < rows * PAIRS; i += 32 * WARPS) {
        const int token = i / PAIRS, n = n0 + 2 * (i - token * PAIRS);
        if (n >= p.w.N) continue;
        float x = 0.0f, y = 0.0f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            const float2 v = *reinterpret_cast<const float2 *>(sums + (w * tokens + token) * PITCH + n - n0);
            x += v.x;
            y += v.y;
        }
        const long long o = (row0 + token) * p.ldc;
        if (p.swiglu) {
            store_out(p.C, o + n / 2, silu_f32(p.alpha * x) * (p.alpha * y), p.out_kind);
            continue;
        }
        x *= p.alpha;
        y *= p.alpha;
        if (p.beta != 0.0f) x += p.beta * load_out(p.C, o + n, p.out_kind);
        store_out(p.C, o + n, x, p.out_kind);
        if (n + 1 < p.w.N) {
            if (p.beta != 0.0f) y += p.beta * load_out(p.C, o + n + 1, p.out_kind);
            store_out(p.C, o + n + 1, y, p.out_kind);
        }
    }
}

// An upper bound of the chunks over all groups, and with offsets one more, whose
// CTAs find nothing: on the way they look at every offset and report what they
// have to clamp.
long long chunks_of(const Groups &g)
{
    return g.offsets == nullptr ? (g.M + TOKENS - 1) / TOKENS : g.M / TOKENS + std::min(g.G, g.M) + 1;
}

template <bool BF16, int MT, int PER>
cudaError_t launch(const W4Args &p, int *err, cudaStream_t s)
{
    constexpr int STAGES = 4;
    const int tokens = std::min(p.groups.M, TOKENS), tiles = (p.w.N + 16 * MT - 1) / (16 * MT);
    const size_t ring = (size_t)WARPS * STAGES * stage_bytes(MT, PER, tokens);
    const size_t sums = (size_t)WARPS * tokens * (16 * MT + 2) * 4;
    const size_t bytes = std::max(ring, sums);
    auto kernel = w4_kernel<BF16, MT, PER, STAGES>;
    static DeviceOnce once;
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev)) return e;
    if (once.needed(dev)) {
        if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 WARPS * STAGES * stage_bytes(MT, PER, TOKENS)))
            return e;
        once.mark(dev);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(chunks_of(p.groups) * tiles));
    cfg.blockDim = dim3(32 * WARPS);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p, tiles, tokens, err);
}

template <bool BF16, int MT>
cudaError_t launch_group(const W4Args &p, int *err, cudaStream_t s)
{
    return p.w.group == 32   ? launch<BF16, MT, 1>(p, err, s)
           : p.w.group == 64 ? launch<BF16, MT, 2>(p, err, s)
                             : launch<BF16, MT, 4>(p, err, s);
}

}  // namespace

bool w4_fits(const W4Args &p) { return chunks_of(p.groups) * ((p.w.N + 15ll) / 16) <= 0x7fffffff; }

cudaError_t launch_w4(const W4Args &p, int sms, int *err, cudaStream_t s)
{
    const bool wide = (long long)std::min(p.groups.G, p.groups.M) * p.w.N >= 64ll * sms;
    if (p.bf16) return wide ? launch_group<true, 2>(p, err, s) : launch_group<true, 1>(p, err, s);
    return wide ? launch_group<false, 2>(p, err, s) : launch_group<false, 1>(p, err, s);
}

}  // namespace swg
