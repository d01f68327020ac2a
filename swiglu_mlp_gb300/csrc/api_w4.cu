// api_w4.cu — the C ABI of 4-bit weights with group scales.  As in api.cu,
// every argument is validated before any CUDA call.
#include <cuda_runtime.h>

#include <cstdint>

#include "swiglu_mlp.h"
#include "host.h"
#include "tc_gemm.cuh"
#include "w4.h"

namespace {

constexpr int64_t kMaxDim = 0x80000000ll - 1024;
constexpr int64_t kMaxStride = 0x7fffffff;

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool half_type(int type) { return type == SWG_TYPE_F16 || type == SWG_TYPE_BF16; }

bool type_bytes(int type, int &bytes)
{
    if (half_type(type)) bytes = 2;
    else if (type == SWG_TYPE_F32) bytes = 4;
    else return false;
    return true;
}

// Weights of N rows in each group.
int check_weight(int64_t N, const void *Q, const void *S, const void *Z, int64_t lds, int64_t group)
{
    if (Q == nullptr || S == nullptr || lds < N) return SWG_ERR_INVALID_ARG;
    if (group != 32 && group != 64 && group != 128) return SWG_ERR_UNSUPPORTED;
    if (lds > kMaxStride) return SWG_ERR_UNSUPPORTED;
    if (!aligned16(Q) || !aligned16(S) || !aligned16(Z) || lds % 16 != 0) return SWG_ERR_MISALIGNED;
    return SWG_OK;
}

swg::W4Weight weight(int64_t N, int64_t K, const void *Q, const void *S, const void *Z, int64_t lds, int64_t group)
{
    swg::W4Weight w{};
    w.Q = static_cast<const uint8_t *>(Q);
    w.S = S;
    w.Z = static_cast<const uint8_t *>(Z);
    w.lds = lds;
    w.N = (int)N;
    w.K = (int)K;
    w.group = (int)group;
    return w;
}

int convert(int64_t G, int64_t N, int64_t K, const void *X, int64_t ldx, int xtype, int64_t group, const void *Q,
            const void *S, const void *Z, int64_t lds, int stype, bool back, void *stream)
{
    int bytes;
    if (!type_bytes(xtype, bytes) || !half_type(stype)) return SWG_ERR_UNSUPPORTED;
    if (G < 0 || N < 0 || K < 0) return SWG_ERR_INVALID_ARG;
    if (G == 0 || N == 0 || K == 0) return SWG_OK;
    if (X == nullptr || ldx < K) return SWG_ERR_INVALID_ARG;
    // (CTAs of 32 rows and 256 columns in a grid of 2^31 - 1 by 65535)
    if (N > kMaxDim || G > kMaxDim || ldx > kMaxStride || G * ((N + 31) / 32) > kMaxStride || K > 256 * 65535)
        return SWG_ERR_UNSUPPORTED;
    if (int rc = check_weight(N, Q, S, Z, lds, group)) return rc;
    if (!aligned16(X) || ldx * bytes % 16 != 0) return SWG_ERR_MISALIGNED;
    swg::W4Convert p{};
    p.G = (int)G;
    p.w = weight(N, K, Q, S, Z, lds, group);
    p.stype = stype;
    p.X = const_cast<void *>(X);
    p.ldx = ldx;
    p.type = xtype;
    swg::DeviceInfo d;
    if (int rc = swg::device_info(d)) return rc;
    return swg::count_launch(swg::launch_w4_convert(p, back, static_cast<cudaStream_t>(stream)));
}

int product(int64_t G, int64_t M, int64_t N, int64_t K, float alpha, const void *A, int64_t lda, const void *Q,
            const void *S, const void *Z, int64_t lds, int64_t group, const int32_t *offsets, float beta, void *C,
            int64_t ldc, int type, int ctype, bool swiglu, void *stream)
{
    int bytes;
    if (!half_type(type) || !type_bytes(ctype, bytes)) return SWG_ERR_UNSUPPORTED;
    if (G < 0 || M < 0 || N < 0 || K < 0) return SWG_ERR_INVALID_ARG;
    if (G > SWG_MAX_GROUPS) return SWG_ERR_UNSUPPORTED;
    if (offsets == nullptr && G > 1) return SWG_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(offsets) & 3u) return SWG_ERR_MISALIGNED;
    if (M == 0 || N == 0 || G == 0) return SWG_OK;
    if (C == nullptr || ldc < N) return SWG_ERR_INVALID_ARG;
    if (K > 0 && (A == nullptr || lda < K)) return SWG_ERR_INVALID_ARG;
    if (M > kMaxDim || N > kMaxDim || K > kMaxDim || lda > kMaxStride || ldc > kMaxStride)
        return SWG_ERR_UNSUPPORTED;
    const int64_t rows = swiglu ? 2 * N : N;
    if (rows > kMaxDim) return SWG_ERR_UNSUPPORTED;
    if (K > 0) {
        if (int rc = check_weight(rows, Q, S, Z, lds, group)) return rc;
    } else {
        group = 128;
    }
    if (!aligned16(C) || ldc * bytes % 16 != 0) return SWG_ERR_MISALIGNED;
    if (K > 0 && (!aligned16(A) || lda % 8 != 0)) return SWG_ERR_MISALIGNED;
    swg::W4Args p{};
    p.groups = {offsets, (int)G, (int)M};
    p.w = weight(rows, K, Q, S, Z, lds, group);
    p.A = A;
    p.lda = lda;
    p.bf16 = type == SWG_TYPE_BF16;
    p.C = C;
    p.ldc = ldc;
    p.alpha = alpha;
    p.beta = beta;
    p.out_kind = ctype == SWG_TYPE_F32 ? swg::OUT_F32 : ctype == SWG_TYPE_F16 ? swg::OUT_F16 : swg::OUT_BF16;
    p.swiglu = swiglu;
    if (!swg::w4_fits(p)) return SWG_ERR_UNSUPPORTED;
    swg::DeviceInfo d;
    if (int rc = swg::device_info(d)) return rc;
    bool mapped = true;
    const cudaError_t e = swg::launch_w4(p, d.sms, d.err, static_cast<cudaStream_t>(stream), mapped);
    return mapped ? swg::count_launch(e) : swg::record_cuda_error();
}

}  // namespace

extern "C" {

int w4_quantize(int64_t G, int64_t N, int64_t K, const void *X, int64_t ldx, int xtype, int64_t group, void *Q,
                void *S, void *Z, int64_t lds, int stype, void *stream)
{
    return convert(G, N, K, X, ldx, xtype, group, Q, S, Z, lds, stype, false, stream);
}

int w4_dequantize(int64_t G, int64_t N, int64_t K, const void *Q, const void *S, const void *Z, int64_t lds,
                  int stype, int64_t group, void *X, int64_t ldx, int xtype, void *stream)
{
    return convert(G, N, K, X, ldx, xtype, group, Q, S, Z, lds, stype, true, stream);
}

int gemm_w4(int64_t G, int64_t M, int64_t N, int64_t K, float alpha, const void *A, int64_t lda, const void *Q,
            const void *S, const void *Z, int64_t lds, int64_t group, const int32_t *offsets, float beta, void *C,
            int64_t ldc, int type, int ctype, void *stream)
{
    return product(G, M, N, K, alpha, A, lda, Q, S, Z, lds, group, offsets, beta, C, ldc, type, ctype, false,
                   stream);
}

int swiglu_w4(int64_t G, int64_t M, int64_t N, int64_t K, float alpha, const void *A, int64_t lda, const void *Q,
              const void *S, const void *Z, int64_t lds, int64_t group, const int32_t *offsets, void *Y,
              int64_t ldy, int type, void *stream)
{
    return product(G, M, N, K, alpha, A, lda, Q, S, Z, lds, group, offsets, 0.0f, Y, ldy, type, type, true,
                   stream);
}

}  // extern "C"
