// experts.h — internal interface between the C ABI of the expert-MLP
// operators (api_experts.cu) and their kernels: products grouped by expert
// with ragged sizes, and microscaled 4-bit floating point.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace swg {

constexpr int MAX_GROUPS = 1024;

// Operand kinds of a grouped product.
enum GrpKind { GRP_F16 = 0, GRP_BF16 = 1, GRP_MXFP4 = 2, GRP_NVFP4 = 3 };
// What becomes of the accumulators.
enum GrpEpi {
    GRP_STORE = 0,     // C = alpha * acc + beta * C
    GRP_SWIGLU = 1,    // Y = SiLU(alpha g) * (alpha u) of column pairs
    GRP_DSWIGLU = 2    // the gradient of that in g and u, and optionally Y
};

// Rows of A sorted by group; offsets == nullptr: one group of all M rows.
struct Groups {
    const int32_t *offsets;
    int G;
    int M;
};

struct GrpArgs {
    Groups groups;
    int N, K;                  // columns of the accumulator (2N-space of SwiGLU), contraction
    const void *A;             // 16-bit: M x K, row stride lda elements; 4-bit: bytes, lda in bytes
    long long lda;
    const void *B;             // group g at B + g * strideB (elements; bytes for 4-bit)
    long long ldb, strideB;
    int b_kn;                  // B stored K x N (op N); 0: N x K (op T, and every 4-bit B)
    const uint8_t *SA, *SB;    // scale tiles (4-bit)
    void *C;                   // output; Y or dH for the SwiGLU forms
    long long ldc;
    const void *dY;            // GRP_DSWIGLU: M x N/2 bf16
    void *Y;                   // GRP_DSWIGLU: M x N/2 bf16 or nullptr
    float alpha, beta;
    int out_kind;              // OutKind
};

}  // namespace swg
