// api_experts.cu — the C ABI of the expert-MLP operators: products grouped by
// expert with ragged sizes, and microscaled 4-bit floating point.  As in
// api.cu, every argument is validated before any CUDA call.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "swiglu_mlp.h"
#include "experts_launch.h"
#include "grouped.cuh"
#include "host.h"

namespace {

constexpr int64_t kMaxStride = 0x7fffffff;
// The kernels number rows and columns in 32 bits and round them up to whole
// tiles, up to 511 beyond the last.
constexpr int64_t kMaxDim = 0x80000000ll - 1024;

int64_t ceil_to(int64_t a, int64_t b) { return (a + b - 1) / b * b; }
bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The 16-bit dtypes of gemm.
bool io_types(int dtype, swg::GrpKind &in, int &out, int &out_bytes)
{
    switch (dtype) {
    case SWG_F16_F32OUT: in = swg::GRP_F16; out = swg::OUT_F32; out_bytes = 4; return true;
    case SWG_BF16: in = swg::GRP_BF16; out = swg::OUT_BF16; out_bytes = 2; return true;
    case SWG_F16: in = swg::GRP_F16; out = swg::OUT_F16; out_bytes = 2; return true;
    case SWG_BF16_F32OUT: in = swg::GRP_BF16; out = swg::OUT_F32; out_bytes = 4; return true;
    default: return false;
    }
}

bool type_bytes(int type, int &bytes)
{
    switch (type) {
    case SWG_TYPE_F16: case SWG_TYPE_BF16: bytes = 2; return true;
    case SWG_TYPE_F32: bytes = 4; return true;
    default: return false;
    }
}

// Rules on groups shared by every entry point; *empty: nothing to do.
int check_groups(const int32_t *offsets, int64_t G)
{
    if (G < 0) return SWG_ERR_INVALID_ARG;
    if (G > SWG_MAX_GROUPS) return SWG_ERR_UNSUPPORTED;
    if (offsets == nullptr && G > 1) return SWG_ERR_INVALID_ARG;
    if (offsets != nullptr && (reinterpret_cast<uintptr_t>(offsets) & 3u)) return SWG_ERR_MISALIGNED;
    return SWG_OK;
}

bool too_big(std::initializer_list<int64_t> dims, std::initializer_list<int64_t> strides = {})
{
    for (int64_t x : dims)
        if (x > kMaxDim) return true;
    for (int64_t x : strides)
        if (x > kMaxStride) return true;
    return false;
}

int block_of(int format) { return format == SWG_NVFP4 ? 16 : 32; }
bool known_format(int format) { return format == SWG_MXFP4 || format == SWG_NVFP4; }

// The most tiles of at most `rows` rows that M > 0 rows of G groups can have: a
// row in every group, and the others in whole tiles of one.
int64_t most_tiles(int64_t M, int64_t G, int64_t rows)
{
    const int64_t g = std::min(G, M);
    return (M - g) / rows + g;
}

// How many K ranges a product of `results` results in `tiles` tiles (an upper
// bound) on `pairs` pairs of CTAs is cut into: as many as there are pairs for, of
// at least 8 stages each, when that saves a tile more than the second kernel
// and the FP32 partials, written and read, cost: a stage takes 0.2 us, the kernel
// and what goes with it 2.8, 8 bytes of partials a result and range the rest.
// (One row, 4096 x 4096: 17.1 us in one range and 11.6 in four; 64 rows, 8192 x
// 8192 in 4 bits: 11.0 in one and 12.3 in two.)  More than 8, up to 16, only of at
// least 16 stages (64 rows, 16384 x 256: 12.1 us in 16, 13.3 in 8; 16 rows, 8192
// x 1024: 10.3 and 9.8; in 32 both are slower).
int pick_splits(int64_t tiles, int k_blocks, int64_t results, int pairs)
{
    const int64_t most = std::max(8, std::min(16, k_blocks / 16));
    const int64_t s = std::min<int64_t>({most, pairs / std::max<int64_t>(tiles, 1), k_blocks / 8});
    if (s < 2) return 1;
    const double cost = 14 + 6e-6 * (double)s * (double)results;
    return k_blocks - k_blocks / s >= cost ? (int)s : 1;
}

// Tensor maps and parameters of a grouped product, and its launch.
int run_grouped(const swg::GrpArgs &a, swg::GrpKind kind, swg::GrpEpi epi, void *stream)
{
    using swg::encode_tiled;
    swg::DeviceInfo d;
    if (int rc = swg::device_info(d)) return rc;
    const bool f4 = kind >= swg::GRP_MXFP4, nv = kind == swg::GRP_NVFP4;
    const int64_t M = a.groups.M, G = a.groups.G, N = a.N, K = a.K;
    const bool few = M <= swg::GrpCfg<swg::MATH_16, true>::TOKENS;
    const int tokens = few ? swg::GrpCfg<swg::MATH_16, true>::TOKENS
                           : swg::GrpCfg<swg::MATH_16, false>::TOKENS;
    const int narrowest = few  ? tokens
                          : f4 ? swg::GrpCfg<swg::MATH_MX, false>::NARROWEST
                               : swg::GrpCfg<swg::MATH_16, false>::NARROWEST;
    // Boxes of A's rows: of box i (see GrpMaps) those that tiles of at most
    // `half` rows per CTA can ask for.
    const int64_t half = std::min<int64_t>(tokens, ceil_to(M, 16)) / 2;
    auto box_rows = [&](int i) { return (uint32_t)swg::token_box(i); };
    auto box_used = [&](int i) { return i + 1 == swg::TOKEN_BOXES || half > swg::token_box(i + 1); };

    swg::GrpParams p{};
    p.groups = a.groups;
    p.N = a.N;
    p.n_blocks = (int)((N + 255) / 256);
    const int bk = f4 ? 256 : 64;
    p.k_blocks = (int)((K + bk - 1) / bk);
    p.w_mn = a.b_kn;
    p.w_tiles = (int)((N + 127) / 128);
    p.alpha = a.alpha;
    p.beta = a.beta;
    p.C = a.C;
    p.ldc = a.ldc;
    p.dY = a.dY;
    p.Y = a.Y;
    p.out_kind = a.out_kind;
    p.err = d.err;

    swg::GrpMaps m{};
    bool ok = true;
    if (K > 0 && !f4) {
        // instruction descriptor, kind::f16: FP32 accumulators (bits 4-5 = 1), types (7-9,
        // 10-12: 1 = bf16), weight MN-major (15), M >> 4 (24-28); N is set per tile (17-22)
        const uint32_t t = kind == swg::GRP_BF16 ? 1u : 0u;
        p.idesc = (1u << 4) | (t << 7) | (t << 10) | ((uint32_t)p.w_mn << 15) | (16u << 24);
        const CUtensorMapDataType type = kind == swg::GRP_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                               : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
        const uint64_t ldb = (uint64_t)a.ldb * 2;
        const uint64_t sb = G > 1 ? (uint64_t)a.strideB * 2 : ldb * (p.w_mn ? K : N);
        if (!p.w_mn) {
            const uint64_t dims[] = {(uint64_t)K, (uint64_t)N, (uint64_t)G}, st[] = {ldb, sb};
            const uint32_t box[] = {64, 128, 1};
            ok = encode_tiled(&m.w, type, 3, a.B, dims, st, box, 128);
        } else if (N % 64 == 0) {
            // 64 columns at a time as their own dimension: one box of 64 x 64 x 2
            const uint64_t dims[] = {64, (uint64_t)K, (uint64_t)N / 64, (uint64_t)G};
            const uint64_t st[] = {ldb, 128, sb};
            const uint32_t box[] = {64, 64, 2, 1};
            ok = encode_tiled(&m.w, type, 4, a.B, dims, st, box, 128);
            p.w_4d = 1;
        } else {
            const uint64_t dims[] = {(uint64_t)N, (uint64_t)K, (uint64_t)G}, st[] = {ldb, sb};
            const uint32_t box[] = {64, 64, 1};
            ok = encode_tiled(&m.w, type, 3, a.B, dims, st, box, 128);
        }
        for (int i = 0; i < swg::TOKEN_BOXES && ok; ++i) {
            if (!box_used(i)) continue;
            const uint64_t dims[] = {(uint64_t)K, (uint64_t)M}, st[] = {(uint64_t)a.lda * 2};
            const uint32_t box[] = {64, box_rows(i)};
            ok = encode_tiled(&m.t[i], type, 2, a.A, dims, st, box, 128);
        }
    } else if (K > 0) {
        // kind::mxf4 and mxf4nvf4: E2M1 operands (7-9, 10-12: 1), scale type (23: 1 = E8M0,
        // 0 = E4M3), M >> 4 (24-28); the scales' byte in their column (4-5, 29-30) per instruction
        p.idesc = (1u << 7) | (1u << 10) | (nv ? 0u : 1u << 23) | (16u << 24);
        const uint64_t row = (uint64_t)ceil_to(K, 32) / 2;
        const uint64_t sb = G > 1 ? (uint64_t)a.strideB : (uint64_t)a.ldb * N;
        const uint64_t wd[] = {row, (uint64_t)N, (uint64_t)G}, wst[] = {(uint64_t)a.ldb, sb};
        const uint32_t wbox[] = {128, 128, 1};
        ok = encode_tiled(&m.w, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, a.B, wd, wst, wbox, 128);
        for (int i = 0; i < swg::TOKEN_BOXES && ok; ++i) {
            if (!box_used(i)) continue;
            const uint64_t dims[] = {row, (uint64_t)M}, st[] = {(uint64_t)a.lda};
            const uint32_t box[] = {128, box_rows(i)};
            ok = encode_tiled(&m.t[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, a.A, dims, st, box, 128);
        }
        // Scale tiles as rows of 64-bit elements, one row per 128 rows of the
        // matrix: a box is one stage's tiles (1 KB or 2 KB) of one row, for A of as many as a tile spans
        const int tile_k = nv ? 64 : 128;
        const uint64_t tiles = (uint64_t)(K + tile_k - 1) / tile_k * 64;
        const uint64_t sst[] = {tiles * 8};
        const uint64_t swd[] = {tiles, (uint64_t)(p.w_tiles * G)};
        const uint64_t std_[] = {tiles, (uint64_t)(M / 128 + G)};
        const uint32_t per = nv ? 256u : 128u;
        const uint32_t swbox[] = {per, 1}, stbox[] = {per, few ? 1u : 2u};
        ok = ok && encode_tiled(&m.sw, CU_TENSOR_MAP_DATA_TYPE_UINT64, 2, a.SB, swd, sst, swbox, 0);
        ok = ok && encode_tiled(&m.st, CU_TENSOR_MAP_DATA_TYPE_UINT64, 2, a.SA, std_, sst, stbox, 0);
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // (Where tiles may be narrower, that comes before ranges of K: 256 rows, 8192 x
    // 8192: 37 us in two tiles, 45 in two ranges.)
    const int64_t tiles = most_tiles(M, G, narrowest) * (int64_t)p.n_blocks;
    const int splits = pick_splits(tiles, p.k_blocks, M * N, d.sms / 2);
    p.splits = 1;
    p.split_blocks = p.k_blocks;
    if (splits > 1) {
        // Partials of the K ranges to the workspace, then their sum and the epilogue.
        p.split_blocks = (p.k_blocks + splits - 1) / splits;
        p.splits = (p.k_blocks + p.split_blocks - 1) / p.split_blocks;
        swg::ReduceArgs r{};
        r.ld = ceil_to(N, 8);
        r.stride = r.ld * M;
        float *ws = nullptr;
        std::unique_lock<std::mutex> held;           // until the sum of the partials is queued
        if (int rc = swg::stream_workspace(s, sizeof(float) * (size_t)p.splits * (size_t)r.stride, ws, held))
            return rc;
        r.ws = ws;
        r.splits = p.splits;
        r.rows = (int)M;
        r.N = a.N;
        r.groups = a.groups;
        r.C = a.C;
        r.ldc = a.ldc;
        r.dY = a.dY;
        r.Y = a.Y;
        r.alpha = a.alpha;
        r.beta = a.beta;
        r.out_kind = a.out_kind;
        p.C = ws;
        p.ldc = r.ld;
        p.split_stride = r.stride;
        p.alpha = 1.0f;
        p.beta = 0.0f;
        p.out_kind = swg::OUT_F32;
        if (!ok) return swg::record_cuda_error();
        const long long units = tiles * p.splits;
        if (int rc = swg::count_launch(
                f4 ? swg::launch_grouped_f4(nv, swg::GRP_STORE, few, m, p, units, d.sms, s)
                   : swg::launch_grouped_16(swg::GRP_STORE, few, m, p, units, d.sms, s)))
            return rc;
        return swg::count_launch(swg::launch_reduce(r, epi, d.sms, s));
    }
    // 16-bit outputs in boxes of 64 columns x 32 rows.  TMA clips a row at 16-byte
    // granules: the last N % 8 columns are not the map's.
    auto out_map = [&](CUtensorMap *map, void *ptr, int64_t cols, int64_t ld) {
        const uint64_t dims[] = {(uint64_t)cols, (uint64_t)M}, st[] = {(uint64_t)ld * 2};
        const uint32_t box[] = {64, 32};
        return encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, ptr, dims, st, box, 128);
    };
    p.tma_out = M >= 32;
    if (epi == swg::GRP_STORE)
        p.tma_out = p.tma_out && a.out_kind != swg::OUT_F32 && a.beta == 0.0f && N >= 8;
    if (p.tma_out) {
        ok = ok && out_map(&m.c, a.C, epi == swg::GRP_SWIGLU ? N / 2 : N & ~7, a.ldc);
        if (a.Y) ok = ok && out_map(&m.y, a.Y, N / 2, N / 2);
    }
    if (!ok) return swg::record_cuda_error();
    return swg::count_launch(f4 ? swg::launch_grouped_f4(nv, epi, few, m, p, tiles, d.sms, s)
                                : swg::launch_grouped_16(epi, few, m, p, tiles, d.sms, s));
}

}  // namespace

extern "C" {

int gemm_grouped(int transB, int64_t G, int64_t M, int64_t N, int64_t K, float alpha,
                 const void *A, int64_t lda, const void *B, int64_t ldb, int64_t strideB,
                 const int32_t *offsets, float beta, void *C, int64_t ldc, int dtype, void *stream)
{
    swg::GrpKind in;
    int out, out_bytes;
    if (!io_types(dtype, in, out, out_bytes)) return SWG_ERR_UNSUPPORTED;
    if (transB != SWG_OP_N && transB != SWG_OP_T) return SWG_ERR_INVALID_ARG;
    if (M < 0 || N < 0 || K < 0) return SWG_ERR_INVALID_ARG;
    if (int rc = check_groups(offsets, G)) return rc;
    if (M == 0 || N == 0 || G == 0) return SWG_OK;
    const int64_t b_rows = transB ? N : K, b_cols = transB ? K : N;
    if (C == nullptr || ldc < N) return SWG_ERR_INVALID_ARG;
    if (K > 0 && (A == nullptr || B == nullptr || lda < K || ldb < b_cols))
        return SWG_ERR_INVALID_ARG;
    if (too_big({M, N, K}, {lda, ldb, ldc})) return SWG_ERR_UNSUPPORTED;
    if (K > 0 && G > 1 && strideB < (b_rows - 1) * ldb + b_cols) return SWG_ERR_INVALID_ARG;
    if (!aligned16(C) || (ldc * out_bytes) % 16 != 0) return SWG_ERR_MISALIGNED;
    if (K > 0 && (!aligned16(A) || !aligned16(B) || lda % 8 != 0 || ldb % 8 != 0 ||
                  (G > 1 && strideB % 8 != 0)))
        return SWG_ERR_MISALIGNED;
    swg::GrpArgs p{};
    p.groups = {offsets, (int)G, (int)M};
    p.N = (int)N;
    p.K = (int)K;
    p.A = A;
    p.lda = lda;
    p.B = B;
    p.ldb = ldb;
    p.strideB = G > 1 ? strideB : 0;
    p.b_kn = transB == SWG_OP_N;
    p.C = C;
    p.ldc = ldc;
    p.alpha = alpha;
    p.beta = beta;
    p.out_kind = out;
    return run_grouped(p, in, swg::GRP_STORE, stream);
}

int gemm_grouped_wgrad(int64_t G, int64_t M, int64_t N, int64_t K, float alpha, const void *A,
                       int64_t lda, const void *D, int64_t ldd, const int32_t *offsets, float beta,
                       void *C, int64_t ldc, int64_t strideC, int dtype, void *stream)
{
    swg::GrpKind in;
    int out, out_bytes;
    if (!io_types(dtype, in, out, out_bytes)) return SWG_ERR_UNSUPPORTED;
    if (M < 0 || N < 0 || K < 0) return SWG_ERR_INVALID_ARG;
    if (int rc = check_groups(offsets, G)) return rc;
    if (N == 0 || K == 0 || G == 0) return SWG_OK;
    if (C == nullptr || ldc < N) return SWG_ERR_INVALID_ARG;
    if (M > 0 && (A == nullptr || D == nullptr || lda < K || ldd < N)) return SWG_ERR_INVALID_ARG;
    if (too_big({M, N, K}, {lda, ldd, ldc})) return SWG_ERR_UNSUPPORTED;
    if (G > 1 && strideC < (K - 1) * ldc + N) return SWG_ERR_INVALID_ARG;
    if (!aligned16(C) || (ldc * out_bytes) % 16 != 0 || (G > 1 && (strideC * out_bytes) % 16 != 0))
        return SWG_ERR_MISALIGNED;
    if (M > 0 && (!aligned16(A) || !aligned16(D) || lda % 8 != 0 || ldd % 8 != 0))
        return SWG_ERR_MISALIGNED;
    swg::WgradArgs p{};
    p.groups = {offsets, (int)G, (int)M};
    p.N = (int)N;
    p.K = (int)K;
    p.A = A;
    p.lda = lda;
    p.D = D;
    p.ldd = ldd;
    p.C = C;
    p.ldc = ldc;
    p.strideC = G > 1 ? strideC : 0;
    p.alpha = alpha;
    p.beta = beta;
    p.in_bf16 = in == swg::GRP_BF16;
    p.out_kind = out;
    swg::DeviceInfo d;
    if (int rc = swg::device_info(d)) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // The rows of a group cut into ranges, as pick_splits cuts K; how many rows
    // a group has is not known here, so their mean decides.
    const int64_t tiles = G * ((K + 255) / 256) * ((N + 255) / 256);
    p.splits = pick_splits(tiles, (int)(M / 64 / G), G * K * N, d.sms / 2);
    swg::ReduceArgs r{};
    std::unique_lock<std::mutex> held;               // until the sum of the partials is queued
    if (p.splits > 1) {
        r.ld = ceil_to(N, 8);
        r.stride = r.ld * K * G;
        float *ws = nullptr;
        if (int rc = swg::stream_workspace(s, sizeof(float) * (size_t)p.splits * (size_t)r.stride, ws, held))
            return rc;
        r.ws = ws;
        r.splits = p.splits;
        r.rows = (int)(K * G);
        r.N = (int)N;
        r.per_group = (int)K;
        r.C = C;
        r.ldc = ldc;
        r.strideC = p.strideC;
        r.alpha = alpha;
        r.beta = beta;
        r.out_kind = out;
        p.C = ws;
        p.ldc = r.ld;
        p.strideC = r.ld * K;
        p.split_stride = r.stride;
        p.alpha = 1.0f;
        p.beta = 0.0f;
        p.out_kind = swg::OUT_F32;
    }
    bool mapped = true;
    const cudaError_t e = swg::launch_wgrad(p, d.sms, d.err, s, mapped);
    if (!mapped) return swg::record_cuda_error();
    if (int rc = swg::count_launch(e)) return rc;
    return p.splits > 1 ? swg::count_launch(swg::launch_reduce(r, swg::GRP_STORE, d.sms, s)) : SWG_OK;
}

static int swiglu_grouped_impl(const void *A, const void *W, const void *dY, void *Y, void *dH,
                               const int32_t *offsets, int64_t G, int64_t M, int64_t N, int64_t K,
                               bool grad, void *stream)
{
    if (M < 0 || N < 0 || K < 0) return SWG_ERR_INVALID_ARG;
    if (int rc = check_groups(offsets, G)) return rc;
    if (M == 0 || N == 0 || G == 0) return SWG_OK;
    if (grad ? dY == nullptr || dH == nullptr : Y == nullptr) return SWG_ERR_INVALID_ARG;
    if (K > 0 && (A == nullptr || W == nullptr)) return SWG_ERR_INVALID_ARG;
    if (too_big({M, N, K}) || too_big({2 * N})) return SWG_ERR_UNSUPPORTED;
    if (!aligned16(Y) || !aligned16(dY) || !aligned16(dH) || N % 8 != 0) return SWG_ERR_MISALIGNED;
    if (K > 0 && (!aligned16(A) || !aligned16(W) || K % 8 != 0)) return SWG_ERR_MISALIGNED;
    swg::GrpArgs p{};
    p.groups = {offsets, (int)G, (int)M};
    p.N = (int)(2 * N);
    p.K = (int)K;
    p.A = A;
    p.lda = K;
    p.B = W;
    p.ldb = 2 * N;
    p.strideB = G > 1 ? 2 * N * K : 0;
    p.b_kn = 1;
    p.C = grad ? dH : Y;
    p.ldc = grad ? 2 * N : N;
    p.dY = dY;
    p.Y = grad ? Y : nullptr;
    p.alpha = 1.0f;
    p.out_kind = swg::OUT_BF16;
    return run_grouped(p, swg::GRP_BF16, grad ? swg::GRP_DSWIGLU : swg::GRP_SWIGLU, stream);
}

int swiglu_grouped(const void *A, const void *W_fused, void *Y, const int32_t *offsets, int64_t G,
                   int64_t M, int64_t N, int64_t K, void *stream)
{
    return swiglu_grouped_impl(A, W_fused, nullptr, Y, nullptr, offsets, G, M, N, K, false, stream);
}

int swiglu_grouped_grad(const void *A, const void *W_fused, const void *dY, void *Y, void *dH,
                        const int32_t *offsets, int64_t G, int64_t M, int64_t N, int64_t K,
                        void *stream)
{
    return swiglu_grouped_impl(A, W_fused, dY, Y, dH, offsets, G, M, N, K, true, stream);
}

int64_t mx4_scale_bytes(int format, int64_t G, int64_t M, int64_t K)
{
    if (!known_format(format) || G < 0 || M < 0 || K < 0 || too_big({G, M, K})) return -1;
    const int64_t tiles_k = ceil_to(K, 4 * block_of(format)) / (4 * block_of(format));
    return 512 * tiles_k * (M / 128 + G);
}

static int mx4_convert(int format, int64_t G, int64_t M, int64_t K, const void *X, int64_t ldx,
                       int xtype, float scale, const int32_t *offsets, const void *Q, int64_t ldq,
                       const void *S, bool back, void *stream)
{
    int bytes;
    if (!known_format(format) || !type_bytes(xtype, bytes)) return SWG_ERR_UNSUPPORTED;
    if (M < 0 || K < 0) return SWG_ERR_INVALID_ARG;
    if (int rc = check_groups(offsets, G)) return rc;
    if (M == 0 || K == 0 || G == 0) return SWG_OK;
    if (X == nullptr || Q == nullptr || S == nullptr || ldx < K) return SWG_ERR_INVALID_ARG;
    if (!(scale > 0.0f) || !std::isfinite(scale)) return SWG_ERR_INVALID_ARG;
    if (too_big({M, K}, {ldx, ldq})) return SWG_ERR_UNSUPPORTED;
    if (ldq < ceil_to(K, 32) / 2) return SWG_ERR_INVALID_ARG;
    if (!aligned16(X) || !aligned16(Q) || !aligned16(S) || (ldx * bytes) % 16 != 0 || ldq % 16 != 0)
        return SWG_ERR_MISALIGNED;
    swg::Mx4Args p{};
    p.groups = {offsets, (int)G, (int)M};
    p.K = (int)K;
    p.format = format;
    p.X = const_cast<void *>(X);
    p.ldx = ldx;
    p.type = xtype;
    p.scale = scale;
    p.Q = static_cast<uint8_t *>(const_cast<void *>(Q));
    p.ldq = ldq;
    p.S = static_cast<uint8_t *>(const_cast<void *>(S));
    swg::DeviceInfo d;
    if (int rc = swg::device_info(d)) return rc;
    return swg::count_launch(swg::launch_mx4(p, back, d.err, static_cast<cudaStream_t>(stream)));
}

int mx4_quantize(int format, int64_t G, int64_t M, int64_t K, const void *X, int64_t ldx,
                 int xtype, float scale, const int32_t *offsets, void *Q, int64_t ldq, void *S,
                 void *stream)
{
    return mx4_convert(format, G, M, K, X, ldx, xtype, scale, offsets, Q, ldq, S, false, stream);
}

int mx4_dequantize(int format, int64_t G, int64_t M, int64_t K, const void *Q, int64_t ldq,
                   const void *S, float scale, const int32_t *offsets, void *X, int64_t ldx,
                   int xtype, void *stream)
{
    return mx4_convert(format, G, M, K, X, ldx, xtype, scale, offsets, Q, ldq, S, true, stream);
}

int gemm_mx4(int format, int64_t G, int64_t M, int64_t N, int64_t K, float alpha, const void *A,
             int64_t lda, const void *SA, const void *B, int64_t ldb, int64_t strideB,
             const void *SB, const int32_t *offsets, float beta, void *C, int64_t ldc, int ctype,
             void *stream)
{
    int bytes;
    if (!known_format(format) || !type_bytes(ctype, bytes)) return SWG_ERR_UNSUPPORTED;
    if (M < 0 || N < 0 || K < 0) return SWG_ERR_INVALID_ARG;
    if (int rc = check_groups(offsets, G)) return rc;
    if (M == 0 || N == 0 || G == 0) return SWG_OK;
    if (C == nullptr || ldc < N) return SWG_ERR_INVALID_ARG;
    if (K > 0 && (!A || !SA || !B || !SB)) return SWG_ERR_INVALID_ARG;
    if (too_big({M, N, K}, {lda, ldb, ldc})) return SWG_ERR_UNSUPPORTED;
    const int64_t row = ceil_to(K, 32) / 2;
    if (K > 0 && (lda < row || ldb < row)) return SWG_ERR_INVALID_ARG;
    if (K > 0 && G > 1 && strideB < (N - 1) * ldb + row) return SWG_ERR_INVALID_ARG;
    if (!aligned16(C) || (ldc * bytes) % 16 != 0) return SWG_ERR_MISALIGNED;
    if (K > 0 && (!aligned16(A) || !aligned16(SA) || !aligned16(B) || !aligned16(SB) ||
                  lda % 16 != 0 || ldb % 16 != 0 || (G > 1 && strideB % 16 != 0)))
        return SWG_ERR_MISALIGNED;
    swg::GrpArgs p{};
    p.groups = {offsets, (int)G, (int)M};
    p.N = (int)N;
    p.K = (int)K;
    p.A = A;
    p.lda = lda;
    p.SA = static_cast<const uint8_t *>(SA);
    p.B = B;
    p.ldb = ldb;
    p.strideB = G > 1 ? strideB : 0;
    p.SB = static_cast<const uint8_t *>(SB);
    p.C = C;
    p.ldc = ldc;
    p.alpha = alpha;
    p.beta = beta;
    p.out_kind = ctype == SWG_TYPE_F32 ? swg::OUT_F32 : ctype == SWG_TYPE_F16 ? swg::OUT_F16
                                                                              : swg::OUT_BF16;
    return run_grouped(p, format == SWG_NVFP4 ? swg::GRP_NVFP4 : swg::GRP_MXFP4, swg::GRP_STORE,
                       stream);
}

int swiglu_mx4(int format, const void *A, const void *SA, const void *W, const void *SW, void *Y,
               const int32_t *offsets, int64_t G, int64_t M, int64_t N, int64_t K, float alpha,
               void *stream)
{
    if (!known_format(format)) return SWG_ERR_UNSUPPORTED;
    if (M < 0 || N < 0 || K < 0) return SWG_ERR_INVALID_ARG;
    if (int rc = check_groups(offsets, G)) return rc;
    if (M == 0 || N == 0 || G == 0) return SWG_OK;
    if (Y == nullptr || (K > 0 && (!A || !SA || !W || !SW))) return SWG_ERR_INVALID_ARG;
    if (too_big({M, N, K}) || too_big({2 * N})) return SWG_ERR_UNSUPPORTED;
    if (!aligned16(Y) || N % 8 != 0) return SWG_ERR_MISALIGNED;
    if (K > 0 && (!aligned16(A) || !aligned16(SA) || !aligned16(W) || !aligned16(SW)))
        return SWG_ERR_MISALIGNED;
    const int64_t row = ceil_to(K, 32) / 2;
    swg::GrpArgs p{};
    p.groups = {offsets, (int)G, (int)M};
    p.N = (int)(2 * N);
    p.K = (int)K;
    p.A = A;
    p.lda = row;
    p.SA = static_cast<const uint8_t *>(SA);
    p.B = W;
    p.ldb = row;
    p.strideB = G > 1 ? 2 * N * row : 0;
    p.SB = static_cast<const uint8_t *>(SW);
    p.C = Y;
    p.ldc = N;
    p.alpha = alpha;
    p.out_kind = swg::OUT_BF16;
    return run_grouped(p, format == SWG_NVFP4 ? swg::GRP_NVFP4 : swg::GRP_MXFP4, swg::GRP_SWIGLU,
                       stream);
}

}  // extern "C"
