/*
 * swiglu_mlp.h — C ABI of the GB300 (sm_103a) GEMM and fused-SwiGLU library.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - Matrices are ROW-MAJOR: element (i, j) of a matrix with row stride ld
 *   sits at offset i*ld + j ("GEMM o Coração Matemático", §2, row-major
 *   linearisation).  ld counts elements, not bytes.
 * - op(X) is X (SWG_OP_N) or its transpose (SWG_OP_T) of the STORED row-major
 *   matrix ("GEMM o Coração Matemático", §1: reading a matrix as transposed
 *   needs no copy).
 * - All pointers except alpha/beta scalars are DEVICE pointers on the current
 *   CUDA device.  The caller owns every tensor; the library never frees them.
 * - `stream` is a cudaStream_t passed as void* (NULL = legacy default stream).
 *   Calls are asynchronous: SWG_OK means the work was validated and enqueued.
 * - Every argument is validated BEFORE any CUDA call; a rejected call writes
 *   nothing and launches nothing.
 * - Accumulation is always FP32, in tensor memory; outputs are rounded once,
 *   round-to-nearest-even, at the store.
 * - There is no CPU fallback: an unsupported case returns an error.
 * - Device-side waits are bounded: a kernel that cannot make progress within
 *   about two seconds stops, records SWG_ERR_DEVICE_TIMEOUT in a device error
 *   word, and exits; read it with swg_get_device_error().
 */
#ifndef SWIGLU_MLP_H
#define SWIGLU_MLP_H

#include <stdint.h>

/* Exported with default visibility even when the library is built with
 * -fvisibility=hidden. */
#if defined(__GNUC__)
#define SWG_API __attribute__((visibility("default")))
#else
#define SWG_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    SWG_OK = 0,
    SWG_ERR_INVALID_ARG = 1,    /* negative size, null pointer, ld too small, bad enum */
    SWG_ERR_MISALIGNED = 2,     /* a pointer or row stride breaks the 16-byte rule */
    SWG_ERR_UNSUPPORTED = 3,    /* valid request this library does not implement */
    SWG_ERR_CUDA = 4,           /* a CUDA runtime/driver call failed */
    SWG_ERR_NO_MEMORY = 5,      /* library workspace allocation failed */
    SWG_ERR_DEVICE_TIMEOUT = 6  /* a kernel gave up on a bounded wait */
} swg_status;

typedef enum { SWG_OP_N = 0, SWG_OP_T = 1 } swg_op;

/* Storage types.  A and B share one input type; C and D share one output type.
 * The e4m3 types quantise A and B to 8 bits, with per-tensor dequantisation
 * scales ("GEMM o Coração Matemático", §12.4: quantised operands with a
 * scale); the scales are applied by folding them into alpha
 * (alpha * scale_A * scale_B).  The 8-bit layout is E4M3 of the OCP 8-bit
 * floating-point format (as torch's float8_e4m3fn): 1 sign, 4 exponent bits
 * with bias 7, 3 fraction bits, no infinities, largest finite value 448.  They require
 * op(A) = A and op(B) = B^T, i.e. A stored M x K and B stored N x K (both
 * K-contiguous), and lda and ldb multiples of 16.  Split-K exists for them
 * only with M <= 64 (few rows, e.g. decode): such calls run the transposed
 * product with the K loop split, automatically or with split_k > 1, and
 * reduce the partials in split order (one or two rows with split_k = 0 run
 * the one-launch FP32-pipe kernel described under gemm); split_k > 1 with
 * M > 64 and other op combinations return SWG_ERR_UNSUPPORTED. */
typedef enum {
    SWG_F16_F32OUT = 0,   /* A, B binary16;  C, D binary32 */
    SWG_BF16 = 1,         /* A, B, C, D bfloat16            */
    SWG_F16 = 2,          /* A, B, C, D binary16            */
    SWG_BF16_F32OUT = 3,  /* A, B bfloat16;  C, D binary32  */
    SWG_E4M3_BF16OUT = 4, /* A, B e4m3;      C, D bfloat16  */
    SWG_E4M3_F32OUT = 5   /* A, B e4m3;      C, D binary32  */
} swg_dtype;

/*
 * gemm — D = alpha * op(A) * op(B) + beta * C, written in place over C.
 *
 * Defined by "GEMM o Coração Matemático", §1 (the BLAS GEMM statement, element
 * by element: D_ij = alpha * sum_p op(A)_ip op(B)_pj + beta * C_ij) and by
 * "为什么 GEMM 是 CUDA 的必修课" (the opening definition C = A B with 2K flops
 * per element).
 *
 *   transA, transB  SWG_OP_N or SWG_OP_T.
 *   M, N, K         op(A) is M x K, op(B) is K x N, C/D is M x N.  All >= 0.
 *                   M == 0 or N == 0: nothing to do, returns SWG_OK.
 *                   K == 0: D = beta * C (D = 0 when beta == 0).
 *   alpha, beta     host scalars.  When beta == 0, C is NOT read (so NaN or
 *                   garbage in C does not reach D).
 *   A, lda          stored M x K (op N) or K x M (op T); lda >= stored columns.
 *   B, ldb          stored K x N (op N) or N x K (op T); ldb >= stored columns.
 *   C, ldc          M x N, ldc >= N; read (when beta != 0) and overwritten.
 *   dtype           a swg_dtype.
 *   Alignment       A, B, C must be 16-byte aligned and lda, ldb, ldc times
 *                   the element size must be multiples of 16 bytes (tensor
 *                   memory accelerator rule); otherwise SWG_ERR_MISALIGNED.
 *   Sizes           M, N, K, lda, ldb, ldc <= 2^31 - 1, else SWG_ERR_UNSUPPORTED.
 *   Aliasing        A or B overlapping C is undefined.
 *   Split-K         chosen automatically when the output has too few tiles to
 *                   fill the GPU ("为什么 GEMM 是 CUDA 的必修课", 关键技术 item 5);
 *                   the partial sums are reduced in a fixed order, so repeated
 *                   calls give bit-identical results.
 *                   Few rows (M <= 64) with an automatic split: the K ranges
 *                   of each output tile run as one thread-block cluster of up
 *                   to 4 CTAs that sum their FP32 partials through shared
 *                   memory, in range order -- one kernel, no workspace --
 *                   when that occupies at least half of the SMs or splits K
 *                   as often as the workspace path would.  More rows with an
 *                   automatic split: the same over 128 x 256 tiles (2 or 4
 *                   ranks per tile) when all their clusters are resident at
 *                   once and fill at least half of the SMs.
 *                   SWG_CLUSTER_SPLITK=0 turns both off.
 *                   Otherwise the FP32 partials live
 *                   in a library-owned workspace, allocated (cudaMalloc) on
 *                   first use per (device, stream) and replaced by a larger
 *                   one when a larger split needs it; replaced workspaces stay
 *                   allocated (queued work may still use them) until
 *                   swg_shutdown() frees them all.  Two kernels are
 *                   launched: the GEMM and a dependent reduction.
 *                   Threads that share a stream queue the two together, each
 *                   call's before the next's; cudaStreamPerThread is a stream
 *                   of its own in every thread.
 *   One or two rows M <= 2 with 16-bit or e4m3 A and B (decode of one or two
 *                   tokens), K <= 8 * 8192 / M and N <= 2^30: one kernel on the FP32 pipes
 *                   instead ("GEMM o Coração Matemático", §14: the product
 *                   streams op(B) once and is bound by memory).  Its K split
 *                   is summed inside the kernel, again in a fixed order; it
 *                   uses no workspace.  Setting the environment variable
 *                   SWG_GEMV=0 sends these calls to the tensor-core path.
 *   Graph capture   every call can be captured into a CUDA graph on a stream
 *                   once the same call (or one needing at least as much
 *                   workspace) has run on that stream; a call that would have
 *                   to allocate while its stream is capturing returns
 *                   SWG_ERR_UNSUPPORTED and launches nothing.  Calls of the
 *                   one-or-two-rows kernel and of the cluster-reduced split
 *                   need no earlier run.  A graph keeps its partials in a
 *                   workspace of its own, allocated (cudaMalloc, no part of
 *                   the graph) during the capture and reused by later
 *                   captures once the graph and what was instantiated from
 *                   it are destroyed.  So it may run on any stream, beside
 *                   other graphs and calls; only two executable graphs
 *                   instantiated from one capture must not run at once.
 */
SWG_API int gemm(int transA, int transB, int64_t M, int64_t N, int64_t K, float alpha,
         const void *A, int64_t lda, const void *B, int64_t ldb, float beta,
         void *C, int64_t ldc, int dtype, void *stream);

/*
 * gemm_ex — gemm with an explicit split-K factor.
 *   split_k == 0  automatic choice (what gemm does, including the kernel for
 *                 one or two rows);
 *   split_k == 1  no split;
 *   split_k >= 2  split the K loop into at most min(split_k, 16) contiguous
 *                 ranges (fewer when K has fewer 64-wide blocks).
 * Every other argument and rule is that of gemm.
 */
SWG_API int gemm_ex(int transA, int transB, int64_t M, int64_t N, int64_t K,
            float alpha, const void *A, int64_t lda, const void *B,
            int64_t ldb, float beta, void *C, int64_t ldc, int dtype,
            int split_k, void *stream);

/*
 * swiglu_mlp — Y = SiLU(A * W1) (.) (A * W2) as ONE GEMM over the interleaved
 * weight W_fused, with SiLU(x) = x / (1 + e^-x).
 *
 * Defined by "Sobreposição de Ativação em Nível de Tile para Inferência
 * Eficiente de LLM": Definição do Problema (the SwiGLU MLP) and Metodologia,
 * Kernel-2 (one GEMM over W_fused in R^{K x 2N} whose even columns are Gate
 * and odd columns Up; the epilogue reads each column pair of the accumulator
 * and stores SiLU(gate) * up).  Gate and Up stay in tensor memory and
 * registers; neither is written to global memory.
 *
 *   A        bfloat16, M x K, row stride K.
 *   W_fused  bfloat16, K x 2N, row stride 2N: W_fused[k][2n] = W1[k][n],
 *            W_fused[k][2n+1] = W2[k][n] (see swiglu_interleave).
 *   Y        bfloat16, M x N, row stride N (written).
 *   Alignment  all three pointers 16-byte aligned, K % 8 == 0 and
 *            N % 8 == 0; otherwise SWG_ERR_MISALIGNED.
 *   M == 0 or N == 0: nothing to do.  K == 0: Y = SiLU(0) * 0 = 0.
 *   One or two rows (M <= 2, decode; K <= 8 * 8192 / M): one kernel on the
 *            FP32 pipes streams W_fused once and forms SiLU(gate) * up per
 *            column pair in its final, fixed-order reduction (the gemm
 *            kernel for one or two rows); SWG_GEMV=0 keeps the tensor-core
 *            tiles.
 *   At most 64 rows (decode of a few sequences): one 128 x 128 tile per
 *            128 columns of the 2N-space, its K range split over a
 *            thread-block cluster of up to 4 CTAs whose Gate and Up partials
 *            (first M rows) are summed through shared memory, in range
 *            order, before the pair-multiply (one kernel, no workspace), when
 *            the tiles leave at least half of the SMs free
 *            ("为什么 GEMM 是 CUDA 的必修课", 关键技术 item 5); otherwise, and
 *            with SWG_CLUSTER_SPLITK=0, the persistent tiles.
 */
SWG_API int swiglu_mlp(const void *A, const void *W_fused, void *Y, int64_t M,
               int64_t N, int64_t K, void *stream);

/*
 * swiglu_mlp_fp8 — Y = SiLU(s * A W1) (.) (s * A W2) with e4m3 A and weights,
 * s = scale_A * scale_W (per-tensor dequantisation scales), FP32
 * accumulation, bfloat16 Y.  Same operation and sources as swiglu_mlp; the
 * 8-bit form follows "GEMM o Coração Matemático", §12.4 (quantised operands
 * with a scale); the 8-bit layout is the OCP E4M3 format described at
 * swg_dtype.
 *
 *   A          e4m3, M x K, row stride K.
 *   W_fused_t  e4m3, 2N x K, row stride K: the TRANSPOSED interleaved weight,
 *              row 2n = W1 column n (Gate), row 2n+1 = W2 column n (Up)
 *              (8-bit operands are read K-contiguous).
 *   Y          bfloat16, M x N, row stride N (written).
 *   scale      s above; applied to Gate and Up before the SiLU.
 *   Alignment  pointers 16-byte aligned, K % 16 == 0, N % 8 == 0.
 *   One or two rows (M <= 2): the same one-kernel path as swiglu_mlp, reading
 *              W_fused_t in 256 x 64 byte boxes.
 */
SWG_API int swiglu_mlp_fp8(const void *A, const void *W_fused_t, void *Y,
                           int64_t M, int64_t N, int64_t K, float scale,
                           void *stream);

/*
 * swiglu_mlp_dual — the same Y = SiLU(A * W1) (.) (A * W2), computed directly
 * from SEPARATE W1 and W2 with no interleaved copy of the weights.
 *
 * Defined by "Sobreposição de Ativação em Nível de Tile para Inferência
 * Eficiente de LLM", Metodologia, Kernel-1 (Gate and Up from their own weight
 * matrices, SiLU on the Gate accumulator, the product formed in the
 * epilogue).  One kernel: each output tile's accumulator holds the Gate
 * columns in its first half and the matching Up columns in its second half,
 * and the epilogue stores SiLU(gate) * up; neither reaches memory.
 *
 *   A       bfloat16, M x K, row stride K.
 *   W1, W2  bfloat16, each K x N, row stride N.
 *   Y       bfloat16, M x N, row stride N (written).
 *   Alignment, sizes and the K == 0 case as for swiglu_mlp.
 *   One or two rows (M <= 2): the one-kernel path of swiglu_mlp, reading 64
 *           columns of W1 beside the same 64 columns of W2 per stage.
 */
SWG_API int swiglu_mlp_dual(const void *A, const void *W1, const void *W2,
                            void *Y, int64_t M, int64_t N, int64_t K,
                            void *stream);

/*
 * swiglu_mlp_forward — the whole gated MLP of a transformer block:
 *     Out = (SiLU(A * W1) (.) (A * W2)) * W_down + beta * Out
 * "GEMM o Coração Matemático", §13.3 (the feed-forward block as two GEMMs
 * around an activation) with the gated activation of "Sobreposição de
 * Ativação em Nível de Tile para Inferência Eficiente de LLM", Definição do
 * Problema.  beta = 1 adds a residual already held in Out.
 *
 *   A        bfloat16, M x K, row stride K (K = model width).
 *   W_fused  bfloat16, K x 2N, row stride 2N (interleaved Gate/Up, as for
 *            swiglu_mlp).
 *   W_down   bfloat16, N x K, row stride K.
 *   Y        bfloat16, M x N, row stride N: receives the gated activation
 *            (caller-owned; Gate and Up themselves never reach memory).
 *   Out      bfloat16, M x K, row stride K: read when beta != 0, written.
 *   Two kernels run on `stream`: swiglu_mlp's fused kernel, then gemm.
 *   Alignment: pointers 16-byte aligned, K % 8 == 0, N % 8 == 0, else
 *   SWG_ERR_MISALIGNED.  M == 0 or K == 0: nothing to do.  All arguments are
 *   checked before the first launch.
 */
SWG_API int swiglu_mlp_forward(const void *A, const void *W_fused,
                               const void *W_down, void *Y, void *Out,
                               int64_t M, int64_t N, int64_t K, float beta,
                               void *stream);

/*
 * swiglu_interleave — builds W_fused (K x 2N, row stride 2N) from W1 and W2
 * (each K x N, row stride N), bfloat16: column 2n <- W1 column n (Gate),
 * column 2n+1 <- W2 column n (Up).  Same page and section as swiglu_mlp.
 * A one-off weight-layout step, not part of the per-token hot path.
 * Pointers 16-byte aligned and N % 4 == 0, else SWG_ERR_MISALIGNED.
 */
SWG_API int swiglu_interleave(const void *W1, const void *W2, void *W_fused,
                      int64_t K, int64_t N, void *stream);

/*
 * gemm_splitk_noalloc — gemm_ex without any device allocation.  The pages
 * have no counterpart to this call.  It is for callers that cannot call
 * cudaMalloc once they are running: a host framework that has already
 * reserved nearly all device memory in its own pool (where a cudaMalloc
 * would fail, or fragment that pool), or a serving loop that forbids
 * cudaMalloc/cudaFree because either can synchronise the whole device.
 *
 * Same arguments, rules and results as gemm_ex: for every input it launches
 * the kernels gemm_ex would launch, with the same tiles, split count and
 * fixed-order reduction, so the two give bit-identical D.  The one
 * difference: a split-K call that keeps FP32 partial sums in global memory
 * keeps them in a fixed array of SWG_NOALLOC_SCRATCH_BYTES (plus two 64 KiB
 * guard bands) that is part of the library's device image, instead of a
 * workspace from cudaMalloc (few-row calls whose K ranges are reduced inside
 * a thread-block cluster keep none there).  The caller still passes A, B
 * and C.
 *
 *   Limit        a split needs splits * M * round_up(N, 4) * 4 bytes of
 *                partials; a call that would need more than
 *                SWG_NOALLOC_SCRATCH_BYTES returns SWG_ERR_UNSUPPORTED and
 *                launches nothing (pass a smaller split_k, or use gemm_ex).
 *   Allocation   none: no cudaMalloc, cudaFree or allocating library call.
 *   Residency    the array is device memory of the library's module.  With
 *                CUDA's default lazy module loading it is committed on a
 *                device the first time this library runs there (the first
 *                call of any of its entry points), and with
 *                CUDA_MODULE_LOADING=EAGER when the library is loaded; it
 *                stays until the process exits.  A caller about to reserve
 *                nearly all device memory should make one call on each
 *                device first.
 *   First call   on each device looks up the array's device address
 *                (cudaGetSymbolAddress) with that device current; make that
 *                first call before any stream capture.
 *   Sharing      all calls, on every stream, use the one array, and it keeps
 *                the last call's contents (each call writes every partial it
 *                reads, so nothing needs clearing).  Calls that overlap on the
 *                GPU race with each other: order them, e.g. on one stream.
 *                (Threads may share that stream: a call's kernels are queued
 *                together.)
 *   Reset        call swg_shutdown() before cudaDeviceReset(): it makes the
 *                next call look the address up again.
 */
#define SWG_NOALLOC_SCRATCH_BYTES (16u * 1024u * 1024u)
SWG_API int gemm_splitk_noalloc(int transA, int transB, int64_t M, int64_t N,
                                int64_t K, float alpha, const void *A,
                                int64_t lda, const void *B, int64_t ldb,
                                float beta, void *C, int64_t ldc, int dtype,
                                int split_k, void *stream);

/* ------------------------------------------------------------------------
 * Products grouped by expert, with ragged sizes.  (The pages have no
 * counterpart; the mathematics is the GEMM statement applied to each group.)
 *
 * The M rows of A (and C) are sorted by group: group g owns rows
 * offsets[g] .. offsets[g+1] - 1.  `offsets` is a DEVICE array of G + 1
 * int32 values, non-decreasing within [0, M]; it is read on the stream, so a
 * kernel queued earlier may write it, and the host never waits for it.
 * offsets == NULL with G == 1: one group of all M rows.  Groups may be empty.
 * Rows outside [offsets[0], offsets[G]) are neither read into a result nor
 * written.  Offsets that break the rule are clamped to it by the kernels
 * (nothing is accessed out of bounds), and the device error word becomes
 * SWG_ERR_INVALID_ARG.  G <= SWG_MAX_GROUPS, else SWG_ERR_UNSUPPORTED.
 * 16-bit dtypes only (SWG_F16_F32OUT, SWG_BF16, SWG_F16, SWG_BF16_F32OUT);
 * alignment, size and graph-capture rules are gemm's, for every pointer,
 * row stride and group stride, but M, N, K (and 2N of the SwiGLU calls) are at
 * most 2^31 - 1024, here and in the 4-bit calls below.
 */
#define SWG_MAX_GROUPS 1024

/*
 * gemm_grouped — C[i,:] = alpha * A[i,:] * op(B_g) + beta * C[i,:] for the
 * rows i of every group g.  With op = N this is the forward product, with
 * op = T (the same stored B) the gradient of its input.
 *   A, lda            M x K.
 *   B, ldb, strideB   group g at B + g * strideB elements, stored K x N
 *                     (transB = SWG_OP_N) or N x K (SWG_OP_T).
 *   C, ldc            M x N; not read when beta == 0.
 *   K == 0: C = beta * C.
 */
SWG_API int gemm_grouped(int transB, int64_t G, int64_t M, int64_t N, int64_t K, float alpha,
                         const void *A, int64_t lda, const void *B, int64_t ldb,
                         int64_t strideB, const int32_t *offsets, float beta, void *C,
                         int64_t ldc, int dtype, void *stream);

/*
 * gemm_grouped_wgrad — the gradient of each group's weight:
 * C_g = alpha * A_g^T * D_g + beta * C_g, where A_g and D_g are the group's
 * rows of A (M x K) and D (M x N).  C_g is K x N at C + g * strideC elements,
 * row stride ldc.  An empty group gives beta * C_g (0 when beta == 0).
 */
SWG_API int gemm_grouped_wgrad(int64_t G, int64_t M, int64_t N, int64_t K, float alpha,
                               const void *A, int64_t lda, const void *D, int64_t ldd,
                               const int32_t *offsets, float beta, void *C, int64_t ldc,
                               int64_t strideC, int dtype, void *stream);

/*
 * swiglu_grouped — swiglu_mlp with each group's own weight:
 * Y[i,:] = SiLU(A[i,:] W1_g) (.) (A[i,:] W2_g).
 *   A        bfloat16, M x K.   W_fused  bfloat16, G x K x 2N (each group's
 *   weight interleaved as for swiglu_mlp).   Y  bfloat16, M x N.
 *   All contiguous; K % 8 == 0 and N % 8 == 0, pointers 16-byte aligned.
 */
SWG_API int swiglu_grouped(const void *A, const void *W_fused, void *Y, const int32_t *offsets,
                           int64_t G, int64_t M, int64_t N, int64_t K, void *stream);

/*
 * swiglu_grouped_grad — the gradient of swiglu_grouped in its pre-activations.
 * With g = A W1_g, u = A W2_g (computed again; they are never stored) and
 * s = 1 / (1 + e^-g):
 *   dH[i][2n]   = dY[i][n] * u * s * (1 + g * (1 - s))      (Gate)
 *   dH[i][2n+1] = dY[i][n] * g * s                          (Up)
 * and, when Y is not NULL, Y[i][n] = g * s * u as swiglu_grouped gives it.
 *   dY, Y    bfloat16, M x N.   dH  bfloat16, M x 2N (interleaved like
 *   W_fused).  The gradients of A and W_fused follow as
 *   gemm_grouped(SWG_OP_T) of dH and W_fused, and gemm_grouped_wgrad of A
 *   and dH.  Other rules as for swiglu_grouped.
 */
SWG_API int swiglu_grouped_grad(const void *A, const void *W_fused, const void *dY, void *Y,
                                void *dH, const int32_t *offsets, int64_t G, int64_t M,
                                int64_t N, int64_t K, void *stream);

/* ------------------------------------------------------------------------
 * Microscaled 4-bit floating point (no counterpart on the pages).  Values are
 * E2M1 (1 sign, 2 exponent, 1 fraction bit: 0, .5, 1, 1.5, 2, 3, 4, 6) in
 * blocks along K that share a scale:
 *   SWG_MXFP4  blocks of 32; scale 2^e in E8M0 (a byte e + 127), with
 *              e = floor(log2(max |x|)) - 2, as the OCP microscaling formats
 *              specification (v1.0) gives its conversion;
 *   SWG_NVFP4  blocks of 16; scale an unsigned E4M3 value: max |x| / 6
 *              rounded to nearest even, at least 2^-9, at most 448.
 * A value x becomes x / scale rounded to the nearest E2M1 value, ties to even
 * code, magnitudes beyond 6 to 6.  A block that holds a NaN or an infinity
 * gets the NaN scale (0xFF, 0x7F): it reads back as NaN, and so do the sums
 * that use it.  A block of zeros gets the smallest scale.
 *
 * Storage of an M x K matrix: two codes per byte, column 2j in the low half of
 * byte j of its row, rows ld BYTES apart (a multiple of 16, at least
 * 16 * ceil(K / 32)); the codes from column K up to a multiple of 32 are zero.
 * Scales are kept in tiles of 128 rows x 4 blocks (512 bytes): row r, block b
 * of a tile at byte 16 * (r % 32) + 4 * (r / 32) + b.  The tiles of 128 rows
 * across K follow one another, then those of the next 128 rows; each GROUP of
 * rows begins a new row of tiles, and rows and blocks that do not exist hold 0.
 * mx4_scale_bytes gives the size that is enough for any offsets.
 * offsets, G: as above; offsets == NULL: one group (G is then 1).
 */
typedef enum { SWG_MXFP4 = 0, SWG_NVFP4 = 1 } swg_mx4;
typedef enum { SWG_TYPE_F16 = 0, SWG_TYPE_BF16 = 1, SWG_TYPE_F32 = 2 } swg_type;

/* 512 * ceil(K / (4 blocks)) * (floor(M / 128) + G); -1 for bad arguments. */
SWG_API int64_t mx4_scale_bytes(int format, int64_t G, int64_t M, int64_t K);

/*
 * mx4_quantize — X (M x K, row stride ldx, of type xtype) times `scale`
 * (finite, > 0; the product is formed in FP32) to 4 bits: codes to Q, scale
 * tiles to S.  X, Q, S 16-byte aligned, row strides multiples of 16 bytes.
 * Its gradient is taken straight through: that of the identity times `scale`.
 */
SWG_API int mx4_quantize(int format, int64_t G, int64_t M, int64_t K, const void *X, int64_t ldx,
                         int xtype, float scale, const int32_t *offsets, void *Q, int64_t ldq,
                         void *S, void *stream);

/* mx4_dequantize — X = scale * the values of (Q, S), the product formed in FP32
 * and rounded to xtype. */
SWG_API int mx4_dequantize(int format, int64_t G, int64_t M, int64_t K, const void *Q,
                           int64_t ldq, const void *S, float scale, const int32_t *offsets,
                           void *X, int64_t ldx, int xtype, void *stream);

/*
 * gemm_mx4 — C[i,:] = alpha * A[i,:] * B_g^T + beta * C[i,:] with A (M x K)
 * and B_g (N x K each) in 4 bits of the same format, FP32 accumulation, C of
 * type ctype.  Dense: G = 1, offsets = NULL.
 *   A, lda, SA       as mx4_quantize writes them with the same offsets.
 *   B, ldb, strideB  group g's codes at B + g * strideB bytes (a multiple of
 *                    16), rows ldb bytes apart.
 *   SB               scale tiles, each group's N rows beginning a new row of
 *                    tiles (ceil(N / 128) of them per group).
 *   alpha            also takes the dequantisation scales of both operands.
 */
SWG_API int gemm_mx4(int format, int64_t G, int64_t M, int64_t N, int64_t K, float alpha,
                     const void *A, int64_t lda, const void *SA, const void *B, int64_t ldb,
                     int64_t strideB, const void *SB, const int32_t *offsets, float beta,
                     void *C, int64_t ldc, int ctype, void *stream);

/*
 * swiglu_mx4 — Y[i,:] = SiLU(alpha A[i,:] W1_g) (.) (alpha A[i,:] W2_g) with
 * 4-bit A and weights: W holds, for each group, 2N rows of K codes, row 2n =
 * W1 column n (Gate) and row 2n + 1 = W2 column n (Up), as swiglu_mlp_fp8's
 * W_fused_t.  A's and W's rows are 16 * ceil(K / 32) bytes apart, groups of W
 * 2N rows apart; Y bfloat16, M x N contiguous, N % 8 == 0.
 */
SWG_API int swiglu_mx4(int format, const void *A, const void *SA, const void *W, const void *SW,
                       void *Y, const int32_t *offsets, int64_t G, int64_t M, int64_t N,
                       int64_t K, float alpha, void *stream);

/* ------------------------------------------------------------------------
 * Routing: which experts a token goes to, and its rows there and back (no
 * counterpart on the pages).  A slot is one of the `top` places of a token:
 * slot t * top + j is token t's j'th.  Arrays of slots are contiguous
 * (T x top).  T * top, R and D are at most 2^31 - 1024, the experts at most
 * SWG_MAX_EXPERTS, top at most SWG_MAX_TOP, else SWG_ERR_UNSUPPORTED.
 * X, rows, out and their gradients share one swg_type (but for FP32 rows, see
 * expert_combine); they are 16-byte aligned, row strides multiples of 16 bytes.  Logits
 * need only their type's alignment (four logits at a multiple of their size are read
 * faster: rows of a multiple of four, up to 256 experts and 8 of them a token).
 * None of the outputs may overlap an input, but out of expert_combine, which is
 * read for beta != 0.
 */
typedef enum { SWG_SOFTMAX = 0, SWG_SIGMOID = 1 } swg_score;
#define SWG_MAX_EXPERTS 1024
#define SWG_MAX_TOP 32
#define SWG_MAX_EXPERT_GROUPS 32

/*
 * expert_route — the experts of each token and their weights, and, unless
 * offsets is NULL, the plan of rows that expert_sort gives.
 *   logits, ldl   T x E of swg_type `type`.
 *   score         s = softmax(logits) over the token's E experts, or the sigmoid of
 *                 each.
 *   bias          E floats or NULL.  Experts are chosen by c = s + bias, compared
 *                 as FP64 has them (without a bias in the order of the
 *                 logits); equal ones by the lowest index.  The weights are those of s.
 *   groups        >= 1, dividing E: experts e with equal e / (E / groups) are a
 *                 group, of which the top_groups best are chosen first.  A group is
 *                 worth its largest c (group_sum = 1) or the sum of its two
 *                 largest (2).  groups <= SWG_MAX_EXPERT_GROUPS.
 *   top           experts per token, at most E / groups * top_groups.
 *   normalise     non-zero: weights are scale * s_j / (the sum of the chosen s);
 *                 zero: scale * s_j.  (scale finite.)
 *   experts, weights   T x top: largest c first.
 * An expert whose logit or bias is -inf is not chosen; a slot that none is left for
 * gets expert -1 and weight 0.  A token with a NaN logit, or a NaN among the c of
 * experts that are not masked (for softmax also by a logit of +inf), goes to experts
 * 0 .. top - 1 with weights of NaN.
 * Calls with a plan of more than 64 tokens keep counts in the stream's workspace:
 * what gemm says of split calls and graph capture holds for them.
 */
SWG_API int expert_route(int score, int64_t T, int64_t E, int64_t top, const void *logits, int64_t ldl,
                         int type, const float *bias, int64_t groups, int64_t top_groups,
                         int group_sum, int normalise, float scale, int32_t *experts, float *weights,
                         int32_t *offsets, int32_t *source, int32_t *position, void *stream);

/*
 * expert_sort — the plan of rows sorted by expert, for experts [T x top] as
 * expert_route gives them (or any numbers from -1 to E - 1).
 *   offsets    E + 1: where each expert's rows begin; offsets[E] rows in all.
 *              The offsets of the grouped products.
 *   source     T * top: the slot that row r is of; an expert's rows are in the order
 *              of their slots.  -1 behind the last row.
 *   position   T x top: the row of each slot, -1 where it has no expert.
 * Experts beyond the rule count as -1, and the device error word becomes
 * SWG_ERR_INVALID_ARG.  T == 0: offsets of 0.  More than 4096 slots: workspace as
 * for expert_route.
 */
SWG_API int expert_sort(int64_t T, int64_t E, int64_t top, const int32_t *experts, int32_t *offsets,
                        int32_t *source, int32_t *position, void *stream);

/*
 * expert_route_grad — d_logits (T x E of `type`, all written) from d_weights
 * (T x top floats), the experts taken as given:
 *   normalised, p_j = s_j / sum s:  softmax dl_j = scale p_j (d_j - sum p d),
 *                                   sigmoid that times (1 - s_j);
 *   not normalised:                 softmax dl_e = s_e (g_e - sum g s), g_e the sum of
 *                                   scale * d over the slots with expert e,
 *                                   sigmoid dl_j = scale s_j (1 - s_j) d_j.
 * Slots of expert -1 count for nothing; other numbers beyond [0, E) neither, and
 * they are reported.  The bias has no gradient.
 */
SWG_API int expert_route_grad(int score, int64_t T, int64_t E, int64_t top, const void *logits,
                              int64_t ldl, int type, const int32_t *experts, int normalise, float scale,
                              const float *d_weights, void *d_logits, int64_t ldd, void *stream);

/*
 * expert_dispatch — rows[position[t][j],:] = X[t,:] for every slot with a row: X
 * T x D, rows R x D.  Other rows keep their values.  Positions beyond [0, R) have no
 * row; those other than -1 are reported (device error word), also where there are no
 * rows or no columns to move.  The positions have to
 * differ (as expert_sort's do): a row of several slots gets pieces of any of theirs.
 * Its gradient is expert_combine without weights.
 */
SWG_API int expert_dispatch(int64_t T, int64_t R, int64_t D, int64_t top, const void *X, int64_t ldx,
                            int type, const int32_t *position, void *rows, int64_t ldr, void *stream);

/*
 * expert_combine — out[t,:] = sum_j weights[t][j] * rows[position[t][j],:] + beta *
 * out[t,:] over the slots with a row, in FP32 and in the order of the slots, rounded
 * once to otype: the rows' type, or any of the three where they are FP32.  weights
 * NULL: ones.  out is not read when beta == 0.
 */
SWG_API int expert_combine(int64_t T, int64_t R, int64_t D, int64_t top, const void *rows, int64_t ldr,
                           int type, const int32_t *position, const float *weights, float beta,
                           void *out, int64_t ldo, int otype, void *stream);

/*
 * expert_combine_grad — the gradients of that:
 *   d_rows[position[t][j],:] = weights[t][j] * d_out[t,:]      (other rows keep theirs)
 *   d_weights[t][j] = <rows[position[t][j],:], d_out[t,:]>     (0 without a row)
 * d_out and d_rows are of the rows' type: FP32 for FP32 rows, whatever type their sum had.
 * weights NULL: ones.  d_weights NULL: not computed, and rows is not read.  The
 * positions have to differ (as expert_sort's do): a row of several slots gets pieces of
 * any of their gradients.
 */
SWG_API int expert_combine_grad(int64_t T, int64_t R, int64_t D, int64_t top, const void *d_out,
                                int64_t ldd, const void *rows, int64_t ldr, int type,
                                const int32_t *position, const float *weights, void *d_rows,
                                int64_t lddr, float *d_weights, void *stream);

/* ------------------------------------------------------------------------
 * Weights of 4 bits with group scales, rows of A in 16 bits (no counterpart on
 * the pages): for decoding, where the weights' bytes are the time.
 *   w[n][k] = S[k / group][n] * (q[n][k] - Z[k / group][n]),  q and Z from 0 to 15;
 *   Z NULL: 8 everywhere.  group: 32, 64 or 128 columns (else SWG_ERR_UNSUPPORTED).
 * Storage of an expert's N x K weight; the G experts' follow one another:
 *   Q   N rows of 16 * ceil(K / 32) bytes.  Eight columns of a row are a 32-bit
 *       word (little-endian): columns 0, 2, 4, 6 in bits 0, 4, 8, 12 and columns 1,
 *       3, 5, 7 in bits 16, 20, 24, 28.
 *   S   ceil(K / group) rows of lds elements, binary16 or bfloat16; lds >= N, a
 *       multiple of 16.
 *   Z   the same of bytes (the lower 4 bits count).
 * Pointers 16-byte aligned, row strides of X, A, C, Y multiples of 16 bytes.  Sizes
 * as for the grouped products; K of the conversions at most 256 * 65535.
 */

/*
 * w4_quantize — X (G * N rows of K, swg_type xtype) to 4 bits.  With m the largest
 * magnitude of a group of columns in a row, and lo <= 0 <= hi its range:
 *   Z NULL:  S = m / 7,           q = round(x / S) + 8;
 *   else:    S = (hi - lo) / 15,  Z = round(-lo / S),  q = round(x / S) + Z;
 * quotients in FP32, S rounded to stype (the largest finite value at most) before
 * it is used, ties to even, q and Z clamped to 0 .. 15, x / S = 0 where S is 0.  A
 * group of columns with a NaN or an infinity gets a NaN S and reads back as NaN.
 * Codes from column K up to a multiple of 32 are 0.
 */
SWG_API int w4_quantize(int64_t G, int64_t N, int64_t K, const void *X, int64_t ldx, int xtype,
                        int64_t group, void *Q, void *S, void *Z, int64_t lds, int stype, void *stream);

/* w4_dequantize — X = the values, formed in FP32 and rounded to xtype. */
SWG_API int w4_dequantize(int64_t G, int64_t N, int64_t K, const void *Q, const void *S, const void *Z,
                          int64_t lds, int stype, int64_t group, void *X, int64_t ldx, int xtype,
                          void *stream);

/*
 * gemm_w4 — C[i,:] = alpha * A[i,:] * W_g^T + beta * C[i,:] for the rows i of every
 * group g (offsets, G: as for gemm_grouped; NULL and 1: dense), FP32 accumulation.
 *   A, S   of swg_type `type` (16 bits).   C   of ctype.
 * Meant for few rows of each expert: up to about 32 it is faster than the product with
 * 16-bit weights, beyond them w4_dequantize and gemm or gemm_grouped are.
 */
SWG_API int gemm_w4(int64_t G, int64_t M, int64_t N, int64_t K, float alpha, const void *A, int64_t lda,
                    const void *Q, const void *S, const void *Z, int64_t lds, int64_t group,
                    const int32_t *offsets, float beta, void *C, int64_t ldc, int type, int ctype,
                    void *stream);

/*
 * swiglu_w4 — Y[i,:] = SiLU(alpha A[i,:] W1_g^T) (.) (alpha A[i,:] W2_g^T), M x N of
 * `type`.  W has 2N rows for each group: row 2n = W1's n'th (Gate), row 2n + 1 = W2's
 * (Up); lds >= 2N.  Y is rounded to 16 bits, as gemm_w4 takes its A: a layer of both rounds
 * its hidden values once, each by up to 2^-8 (bfloat16) or 2^-11 (binary16).
 */
SWG_API int swiglu_w4(int64_t G, int64_t M, int64_t N, int64_t K, float alpha, const void *A, int64_t lda,
                      const void *Q, const void *S, const void *Z, int64_t lds, int64_t group,
                      const int32_t *offsets, void *Y, int64_t ldy, int type, void *stream);

/*
 * swg_debug_workspace_guards — diagnostic for tests (no counterpart on the
 * pages).  With the environment variable SWG_TEST_WS_GUARD=1 set before a
 * workspace is created, every split-K workspace and the fixed array of
 * gemm_splitk_noalloc sit between 64 KiB guard bands of the byte 0xA5.  This
 * call synchronises `stream` and the current device, then stores in
 * *bad_bytes how many guard bytes of the current device's workspaces have
 * changed (0 when no kernel wrote outside its partials; workspaces made
 * without the variable are skipped).  SWG_ERR_INVALID_ARG for a null
 * bad_bytes, SWG_ERR_CUDA if a copy fails.
 */
SWG_API int swg_debug_workspace_guards(void *stream, int64_t *bad_bytes);

/* Human-readable name of a swg_status value (static string, never NULL). */
SWG_API const char *swg_status_string(int status);

/*
 * Synchronises `stream`, then reads and clears the current device's error
 * word.  Returns SWG_OK when no kernel reported a problem since the last call,
 * SWG_ERR_DEVICE_TIMEOUT when a bounded wait ran out, SWG_ERR_CUDA when the
 * synchronisation itself failed.
 */
SWG_API int swg_get_device_error(void *stream);

/*
 * swg_selftest_wait_timeout — diagnostic: exercises the bounded-wait path the
 * pipeline kernels use, on purpose.  Launches one small kernel that waits, with
 * the kernels' own wait routine, on a barrier nothing ever completes; after
 * limit_ns (1 ns .. 1 s) it gives up, records SWG_ERR_DEVICE_TIMEOUT in the
 * device error word and exits, leaving the context usable.  The next
 * swg_get_device_error() on that stream returns SWG_ERR_DEVICE_TIMEOUT (and
 * clears it).  No counterpart on the pages: it tests this library's failure
 * reporting without faulting or hanging the GPU.
 */
SWG_API int swg_selftest_wait_timeout(int64_t limit_ns, void *stream);

/* Why the calling thread's most recent call returned SWG_ERR_CUDA: the CUDA
 * runtime error code (cudaError_t), or 10000 + the driver's CUresult when
 * encoding a tensor map failed; 0 if no call of this thread has failed that
 * way.  Thread-local; a later successful call does not clear it. */
SWG_API int swg_last_cuda_error(void);

/* Name of a code returned by swg_last_cuda_error (static storage). */
SWG_API const char *swg_cuda_error_name(int code);

/* Number of kernels this library has launched in this process (all devices). */
SWG_API uint64_t swg_launch_count(void);

/* Frees every library-owned workspace on every device, including replaced
 * ones, and forgets every cached per-device lookup (device addresses,
 * occupancy, kernel attributes), so it is also the call to make before
 * cudaDeviceReset().  Safe to call twice; later calls allocate and look up
 * afresh.  Call only when no library work is in flight and no captured graph
 * with a split call in it will be replayed. */
SWG_API void swg_shutdown(void);

#ifdef __cplusplus
}
#endif

#endif /* SWIGLU_MLP_H */
