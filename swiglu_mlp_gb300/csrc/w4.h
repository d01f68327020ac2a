// w4.h — internal interface between the C ABI of 4-bit weights with group
// scales (api_w4.cu) and their kernels (k_w4.cu, k_w4_convert.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "experts.h"

namespace swg {

// w[n][k] = S[k / group][n] * (q[n][k] - Z[k / group][n]), Z = 8 where it is nullptr.
struct W4Weight {
    const uint8_t *Q;                  // G x N rows of row_bytes
    const void *S;                     // G x blocks x lds, 16-bit
    const uint8_t *Z;                  // the same of bytes, or nullptr
    long long lds;                     // a multiple of 16
    int N, K;                          // of each group
    int group;                         // 32, 64 or 128 columns per scale
    __host__ __device__ int blocks() const { return (K + group - 1) / group; }
    __host__ __device__ int row_bytes() const { return (K + 31) / 32 * 16; }
};

struct W4Args {
    Groups groups;                     // rows of A by group
    W4Weight w;                        // N: its rows (2N of the SwiGLU)
    const void *A;                     // M x K, binary16 or bfloat16 (as S)
    long long lda;
    int bf16;
    void *C;                           // M x N (SwiGLU: M x N / 2)
    long long ldc;
    float alpha, beta;
    int out_kind;                      // OutKind
    int swiglu;
};
// The number of CTAs has to fit 32 bits.
bool w4_fits(const W4Args &p);
// mapped: whether the tensor maps could be encoded (if not, nothing was launched).
cudaError_t launch_w4(const W4Args &p, int sms, int *err, cudaStream_t s, bool &mapped);

struct W4Convert {
    int G;
    W4Weight w;                        // (written by quantize)
    int stype;                         // swg_type of S: 0 binary16, 1 bfloat16
    void *X;                           // G * N x K of swg_type `type`
    long long ldx;
    int type;
};
cudaError_t launch_w4_convert(const W4Convert &p, bool back, cudaStream_t s);

}  // namespace swg
