// experts_launch.h — launches of the expert-MLP kernels.
#pragma once

#include "experts.h"

namespace swg {

struct Mx4Args {
    Groups groups;
    int K;
    int format;                // 0 MXFP4, 1 NVFP4
    void *X;                   // read by quantize, written by dequantize
    long long ldx;             // elements
    int type;                  // swg_type
    float scale;
    uint8_t *Q;
    long long ldq;             // bytes
    uint8_t *S;
};
cudaError_t launch_mx4(const Mx4Args &p, bool back, int *err, cudaStream_t s);

struct GrpMaps;
struct GrpParams;
// `units`: an upper bound of the tiles over all groups; `few`: the form for few
// rows of A (GrpCfg).
cudaError_t launch_grouped_16(GrpEpi epi, bool few, const GrpMaps &m, const GrpParams &p, long long units,
                              int sms, cudaStream_t s);
cudaError_t launch_grouped_f4(bool nv, GrpEpi epi, bool few, const GrpMaps &m, const GrpParams &p,
                              long long units, int sms, cudaStream_t s);

// The sum of FP32 partials of K ranges, in their order, and the epilogue:
// rows x N accumulators, range s at ws + s * stride, rows ld floats apart.
struct ReduceArgs {
    const float *ws;
    long long ld, stride;
    int splits;
    int rows, N;               // N: columns of the accumulator
    Groups groups;             // rows outside the groups are left alone (offsets may be null)
    int per_group;             // > 0: row r is row r % per_group of matrix r / per_group of C
    void *C;
    long long ldc, strideC;
    const void *dY;
    void *Y;
    float alpha, beta;
    int out_kind;
};
cudaError_t launch_reduce(const ReduceArgs &p, GrpEpi epi, int sms, cudaStream_t s);

struct WgradArgs {
    Groups groups;
    int N, K;
    const void *A;
    long long lda;
    const void *D;
    long long ldd;
    void *C;
    long long ldc, strideC;
    float alpha, beta;
    int in_bf16;
    int out_kind;
    int splits;                // ranges of a group's rows: range s to C + s * split_stride (FP32)
    long long split_stride;
};
// mapped: whether the tensor maps could be encoded (if not, nothing was launched).
cudaError_t launch_wgrad(const WgradArgs &a, int sms, int *err, cudaStream_t s, bool &mapped);

}  // namespace swg
