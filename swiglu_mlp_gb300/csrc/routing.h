// routing.h — internal interface between the C ABI of routing (api_routing.cu)
// and its kernels: choosing experts and sorting rows by them (k_route.cu),
// moving rows to the experts and back (k_rows.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace swg {

constexpr int MAX_EXPERTS = 1024;
constexpr int MAX_TOP = 32;            // experts per token
constexpr int MAX_EXPERT_GROUPS = 32;

enum RouteScore { SCORE_SOFTMAX = 0, SCORE_SIGMOID = 1 };

// Rows sorted by expert (see expert_sort).
struct Plan {
    int32_t *offsets, *source, *position;
};

struct RouteArgs {
    const void *logits;                // T x E of swg_type `type`, row stride ld elements
    long long ld;
    int type;
    const float *bias;                 // E or nullptr
    int T, E, top;
    int score;                         // RouteScore
    int groups, top_groups, group_sum; // groups == 1: no choice of groups
    int normalise;
    float scale;
    int32_t *experts;                  // T x top
    float *weights;
    Plan plan;                         // offsets == nullptr: none
};

// How many chunks of tokens a call with a plan is cut into; more than one need
// a workspace of chunks x E ints.
int plan_chunks(int T, int top, bool route, int sms);
cudaError_t launch_route(const RouteArgs &p, int chunks, int32_t *counts, cudaStream_t s);
// The plan of T x top experts.  More than one chunk: `counts` holds how many slots of each
// chunk go to each expert, from launch_route or launch_count with as many chunks.  One chunk:
// counted here, `counts` is not used.  err: where wrong experts are reported, or nullptr.
cudaError_t launch_sort(int T, int E, int top, const int32_t *experts, const Plan &plan, int chunks,
                        int32_t *counts, int *err, cudaStream_t s);
cudaError_t launch_count(int T, int E, int top, const int32_t *experts, int chunks, int32_t *counts,
                         cudaStream_t s);

struct RouteGradArgs {
    const void *logits;
    long long ld;
    int type;
    int T, E, top;
    int score, normalise;
    float scale;
    const int32_t *experts;
    const float *d_weights;
    void *d_logits;                    // T x E of `type`
    long long ldd;
};
cudaError_t launch_route_grad(const RouteGradArgs &p, int *err, cudaStream_t s);

struct RowsArgs {
    int T, D, top;
    int R;                             // rows that `rows` and `d_rows` have
    int type;                          // swg_type of X, rows, d_out, d_rows
    int out_type;                      // combine: of out, `type` or any for FP32 rows
    const int32_t *position;           // T x top
    const float *weights;              // T x top or nullptr: ones
    const void *X;                     // dispatch: T x D; combine_grad: d_out
    long long ldx;
    void *rows;                        // R x D
    long long ldr;
    void *out;                         // combine: T x D; combine_grad: d_rows (R x D)
    long long ldo;
    float beta;                        // combine: out = sum + beta * out
    float *d_weights;                  // combine_grad: T x top or nullptr
};
cudaError_t launch_dispatch(const RowsArgs &p, int sms, int *err, cudaStream_t s);
cudaError_t launch_combine(const RowsArgs &p, int sms, int *err, cudaStream_t s);
cudaError_t launch_combine_grad(const RowsArgs &p, int *err, cudaStream_t s);

}  // namespace swg
