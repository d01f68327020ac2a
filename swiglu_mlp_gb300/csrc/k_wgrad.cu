// k_wgrad.cu — weight gradients grouped by expert on tcgen05:
//
//   C_g[k, n] = alpha * sum_i A[i, k] * D[i, n] + beta * C_g[k, n]
//
// over the rows i of group g.  The rows are the contraction, so both operands
// are MN-major and a group's last block of 64 rows also holds rows of the
// next group.  MMA steps of 16 rows that lie behind the group are skipped; in
// the step where it ends the loading warp overwrites the foreign rows with
// zeros in shared memory (at most 15 rows, once per tile), in both operands,
// because a NaN or an infinity there times zero would not vanish.
//
// Tiles are 256 (k) x 256 (n) per CTA pair with two accumulators, as in
// grouped.cuh.  A group without rows runs no main loop: its tiles store
// beta * C_g, or zeros.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "grouped_launch.cuh"

namespace swg {
namespace {

struct WgradMaps {
    CUtensorMap a, d;
};

struct WgradParams {
    Groups groups;
    int N, K;
    int k_tiles, n_tiles;
    int a_3d, d_3d;                      // 64-column atoms of an operand as one 3-D box
    uint32_t idesc;
    float alpha, beta;
    void *C;
    long long ldc, strideC;
    int out_kind;
    int *err;
};

constexpr int WG_STAGES = 5;             // a sixth would not leave room for the output staging
constexpr int OP_BYTES = 128 * 128;      // 64 rows x 128 columns of one operand per CTA
constexpr int OUT_BYTES = 32 * 32 * 4;   // per epilogue warp
constexpr int SMEM_BYTES = 1024 + WG_STAGES * 2 * OP_BYTES + NUM_EPI_WARPS * OUT_BYTES + 256 +
                           2 * 4 * (MAX_GROUPS + 1);
static_assert(SMEM_BYTES <= 232448, "beyond the per-CTA shared memory");

__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_addr)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
                 : "memory");
}

__device__ __forceinline__ void fence_acquire_cluster()
{
    asm volatile("fence.acq_rel.cluster;" ::: "memory");
}

struct WgradTile {
    int g, kb, nb, row0, rows;
};

__device__ __forceinline__ WgradTile wgrad_tile(const WgradParams &p, const int *start, int u)
{
    const int per = p.k_tiles * p.n_tiles;
    WgradTile t;
    t.g = u / per;
    const int local = u - t.g * per;
    const int band = local / (8 * p.n_tiles);
    const int in = local - band * 8 * p.n_tiles;
    const int bm = min(8, p.k_tiles - band * 8);
    t.nb = in / bm;
    t.kb = band * 8 + in - t.nb * bm;
    t.row0 = start[t.g];
    t.rows = start[t.g + 1] - t.row0;
    return t;
}

// 32 x 32 accumulators of this warp (row `k`: its lane's, columns n ..): to
// C through `buf`, in which 16-byte chunk j of row r sits at j ^ (r mod 8).
__device__ __forceinline__ void wgrad_emit(const WgradParams &p, const uint32_t (&acc)[32], int g,
                                           int k0, int n, uint32_t buf, int lane)
{
#pragma unroll
    for (int j = 0; j < 8; ++j)
        st_shared_v4(buf + (uint32_t)(lane * 128 + ((j ^ (lane & 7)) << 4)),
                     make_uint4(acc[4 * j], acc[4 * j + 1], acc[4 * j + 2], acc[4 * j + 3]));
    __syncwarp();
    const long long base = (long long)g * p.strideC + n;
    if (p.out_kind == OUT_F32) {
        const int j = lane & 7;
#pragma unroll 4
        for (int r = lane >> 3; r < 32; r += 4) {
            const uint4 w = ld_shared_v4(buf + (uint32_t)(r * 128 + ((j ^ (r & 7)) << 4)));
            if (k0 + r >= p.K || n + 4 * j >= p.N) continue;
            float *dst = reinterpret_cast<float *>(p.C) + base + (k0 + r) * p.ldc + 4 * j;
            float v[4] = {p.alpha * __uint_as_float(w.x), p.alpha * __uint_as_float(w.y),
                          p.alpha * __uint_as_float(w.z), p.alpha * __uint_as_float(w.w)};
            if (n + 4 * j + 4 <= p.N) {
                if (p.beta != 0.0f) {
                    const float4 c = *reinterpret_cast<const float4 *>(dst);
                    v[0] += p.beta * c.x;
                    v[1] += p.beta * c.y;
                    v[2] += p.beta * c.z;
                    v[3] += p.beta * c.w;
                }
                *reinterpret_cast<float4 *>(dst) = make_float4(v[0], v[1], v[2], v[3]);
            } else {
                for (int i = 0; i < 4 && n + 4 * j + i < p.N; ++i)
                    dst[i] = p.beta != 0.0f ? v[i] + p.beta * dst[i] : v[i];
            }
        }
    } else {
        const int j = (lane & 3) * 2;
#pragma unroll 4
        for (int r = lane >> 2; r < 32; r += 8) {
            const uint4 a = ld_shared_v4(buf + (uint32_t)(r * 128 + ((j ^ (r & 7)) << 4)));
            const uint4 b = ld_shared_v4(buf + (uint32_t)(r * 128 + (((j + 1) ^ (r & 7)) << 4)));
            if (k0 + r >= p.K || n + 4 * j >= p.N) continue;
            const long long o = base + (k0 + r) * p.ldc + 4 * j;
            uint16_t *dst = reinterpret_cast<uint16_t *>(p.C) + o;
            const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = p.alpha * __uint_as_float(w[i]);
            if (p.beta != 0.0f) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (n + 4 * j + i < p.N) v[i] += p.beta * load_out(p.C, o + i, p.out_kind);
            }
            if (n + 4 * j + 8 <= p.N) {
                *reinterpret_cast<uint4 *>(dst) =
                    make_uint4(pack2(v[0], v[1], p.out_kind), pack2(v[2], v[3], p.out_kind),
                               pack2(v[4], v[5], p.out_kind), pack2(v[6], v[7], p.out_kind));
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (n + 4 * j + i < p.N) dst[i] = (uint16_t)to_16(v[i], p.out_kind);
            }
        }
    }
    __syncwarp();
}

__global__ void __launch_bounds__(NUM_THREADS, 1)
    wgrad_kernel(const __grid_constant__ WgradMaps maps, const WgradParams p)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t *sA = smem;
    uint8_t *sD = sA + WG_STAGES * OP_BYTES;
    uint8_t *sOut = sD + WG_STAGES * OP_BYTES;
    uint64_t *bars = reinterpret_cast<uint64_t *>(sOut + NUM_EPI_WARPS * OUT_BYTES);
    uint64_t *full = bars;
    uint64_t *empty = bars + WG_STAGES;
    uint64_t *acc_full = bars + 2 * WG_STAGES;
    uint64_t *acc_empty = bars + 2 * WG_STAGES + 2;
    uint64_t *mma_done = bars + 2 * WG_STAGES + 4;
    uint64_t *landed = bars + 2 * WG_STAGES + 5;     // a group's last block, in this CTA
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(bars + 2 * WG_STAGES + 6);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
    int *start = reinterpret_cast<int *>(reinterpret_cast<uint8_t *>(bars) + 256);
    int *first = start + MAX_GROUPS + 1;

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (threadIdx.x == 0) {
        for (int s = 0; s < WG_STAGES; ++s) {
            mbar_init(smem_u32(&full[s]), 2);        // the loading warps of both CTAs
            mbar_init(smem_u32(&empty[s]), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&acc_full[b]), 1);
            mbar_init(smem_u32(&acc_empty[b]), 2 * NUM_EPI_WARPS);
        }
        mbar_init(smem_u32(mma_done), 1);
        mbar_init(smem_u32(landed), 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(tmem_holder), 512);
        tmem_relinquish_pair();
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (warp == 2) group_table(p.groups, start, first, p.err, [](int) { return 1; });
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_holder;
    const int units = p.groups.G * p.k_tiles * p.n_tiles;
    const int u0 = (int)(blockIdx.x >> 1), du = (int)(gridDim.x >> 1);

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        int stage = 0;
        uint32_t phase = 0;
        uint32_t armed = 0, armed_parity = 0;
        uint32_t landed_phase = 0;
        bool ok = true;
        for (int u = u0; u < units && ok; u += du) {
            const WgradTile t = wgrad_tile(p, start, u);
            const int ka = t.kb * 256 + (int)rank * 128;
            const int nd = t.nb * 256 + (int)rank * 128;
            const int blocks = ceil_div(t.rows, 64);
            for (int b = 0; b < blocks; ++b) {
                const int left = t.rows - b * 64;            // rows of the group from here on
                const bool ends = left < 64 && (left & 15) != 0;
                bool got = true;
                const uint32_t full_leader = mapa_shared(smem_u32(&full[stage]), 0);
                const uint32_t a_dst = smem_u32(sA + stage * OP_BYTES);
                const uint32_t d_dst = smem_u32(sD + stage * OP_BYTES);
                if (lane == 0) {
                    got = wait_bounded(smem_u32(&empty[stage]), phase ^ 1, abort_flag, p.err);
                    if (got) {
                        uint32_t bar = full_leader;
                        if (ends) {
                            bar = smem_u32(landed);
                            mbar_arrive_expect_tx(bar, 2 * OP_BYTES);
                        } else if (leader) {
                            mbar_arrive_expect_tx(smem_u32(&full[stage]), 4 * OP_BYTES);
                        } else {
                            mbar_arrive_cluster(full_leader);
                        }
                        armed |= 1u << stage;
                        armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
                        const int row = t.row0 + b * 64;
                        if (p.a_3d) {
                            tma_load_3d_pair(a_dst, &maps.a, bar, 0, row, ka / 64);
                        } else {
                            tma_load_2d_pair(a_dst, &maps.a, bar, ka, row);
                            tma_load_2d_pair(a_dst + 8192, &maps.a, bar, ka + 64, row);
                        }
                        if (p.d_3d) {
                            tma_load_3d_pair(d_dst, &maps.d, bar, 0, row, nd / 64);
                        } else {
                            tma_load_2d_pair(d_dst, &maps.d, bar, nd, row);
                            tma_load_2d_pair(d_dst + 8192, &maps.d, bar, nd + 64, row);
                        }
                        if (ends) got = wait_bounded(bar, landed_phase, abort_flag, p.err);
                    }
                }
                got = __all_sync(0xffffffffu, got);
                if (!got) {
                    ok = false;
                    break;
                }
                if (ends) {
                    landed_phase ^= 1;
                    // rows [left, left rounded up to 16) of the four 64-column atoms
                    const uint32_t zero0 = (uint32_t)left * 128, zero1 = (uint32_t)((left + 15) & ~15) * 128;
                    for (uint32_t o = zero0 + lane * 16; o < zero1; o += 512) {
                        st_shared_v4(a_dst + o, make_uint4(0, 0, 0, 0));
                        st_shared_v4(a_dst + 8192 + o, make_uint4(0, 0, 0, 0));
                        st_shared_v4(d_dst + o, make_uint4(0, 0, 0, 0));
                        st_shared_v4(d_dst + 8192 + o, make_uint4(0, 0, 0, 0));
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(full_leader);
                }
                if (++stage == WG_STAGES) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
        // Never leave with loads in flight into this CTA's shared memory.
        if (lane == 0) {
            if (leader) {
                for (int s = 0; s < WG_STAGES; ++s)
                    if (armed & (1u << s))
                        wait_bounded(smem_u32(&full[s]), (armed_parity >> s) & 1, abort_flag,
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
        if (lane == 0 && leader) {
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            int n = 0;                                   // tiles with rows so far
            for (int u = u0; u < units && ok; u += du) {
                const WgradTile t = wgrad_tile(p, start, u);
                if (t.rows == 0) continue;
                const int acc = n & 1;
                if (!wait_bounded(smem_u32(&acc_empty[acc]), ((n >> 1) & 1) ^ 1, abort_flag, p.err)) {
                    ok = false;
                    break;
                }
                ++n;
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + acc * 256;
                const int blocks = ceil_div(t.rows, 64);
                for (int b = 0; b < blocks; ++b) {
                    if (!wait_bounded(smem_u32(&full[stage]), phase, abort_flag, p.err)) {
                        ok = false;
                        break;
                    }
                    fence_acquire_cluster();             // the peer's zeros, if any
                    tc_fence_after();
                    const int steps = min(4, ceil_div(t.rows - b * 64, 16));
                    const uint32_t a_base = smem_u32(sA + stage * OP_BYTES);
                    const uint32_t d_base = smem_u32(sD + stage * OP_BYTES);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        if (kk >= steps) break;
                        tc_mma_f16_pair(d_tmem, smem_desc(a_base + kk * 2048, 8192, 1024),
                                        smem_desc(d_base + kk * 2048, 8192, 1024), p.idesc,
                                        (b > 0 || kk > 0) ? 1u : 0u);
                    }
                    tc_commit_pair(smem_u32(&empty[stage]));
                    if (++stage == WG_STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
                if (!ok) break;
                tc_commit_pair(smem_u32(&acc_full[acc]));
            }
            tc_commit_pair_local(smem_u32(mma_done));
            wait_bounded(smem_u32(mma_done), 0, abort_flag, p.err, false, DRAIN_LIMIT_NS);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ epilogue
        const int q = warp & 3;
        const int h = (warp - EPI_WARP0) / 4;
        const uint32_t buf = smem_u32(sOut + (warp - EPI_WARP0) * OUT_BYTES);
        int n = 0;
        for (int u = u0; u < units; u += du) {
            const WgradTile t = wgrad_tile(p, start, u);
            const int acc = n & 1;
            if (t.rows > 0) {
                bool ok = wait_bounded(smem_u32(&acc_full[acc]), (n >> 1) & 1, abort_flag, p.err);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
            }
            const uint32_t t_row = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + acc * 256;
            const int k0 = t.kb * 256 + (int)rank * 128 + q * 32;
#pragma unroll 1
            for (int c = h; c < 8; c += 2) {
                const int col = t.nb * 256 + c * 32;
                if (k0 >= p.K || col >= p.N) break;
                uint32_t r[32];
                if (t.rows > 0) {
                    tmem_ld_32cols(t_row + c * 32, r);
                    tmem_ld_wait(r);
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) r[j] = 0;
                }
                wgrad_emit(p, r, t.g, k0, col, buf, lane);
            }
            if (t.rows > 0) {
                ++n;
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote_tmem(mapa_shared(smem_u32(&acc_empty[acc]), 0));
            }
        }
    }

    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    if (warp == 1) tmem_dealloc_pair(tmem_base, 512);
}

}  // namespace

cudaError_t launch_wgrad(const WgradArgs &a, int sms, int *err, cudaStream_t s, bool &mapped)
{
    const int64_t M = a.groups.M, N = a.N, K = a.K;
    WgradMaps m{};
    WgradParams p{};
    p.groups = a.groups;
    p.N = a.N;
    p.K = a.K;
    p.k_tiles = (int)((K + 255) / 256);
    p.n_tiles = (int)((N + 255) / 256);
    const uint32_t t = a.in_bf16 ? 1u : 0u;
    // kind::f16, FP32 accumulators, both operands MN-major, 256 x 256
    p.idesc = (1u << 4) | (t << 7) | (t << 10) | (1u << 15) | (1u << 16) | (32u << 17) | (16u << 24);
    p.alpha = a.alpha;
    p.beta = a.beta;
    p.C = a.C;
    p.ldc = a.ldc;
    p.strideC = a.strideC;
    p.out_kind = a.out_kind;
    p.err = err;
    auto encode = [&](CUtensorMap *map, const void *ptr, int64_t cols, int64_t ld, int &in_3d) {
        const CUtensorMapDataType type =
            a.in_bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
        if (cols % 64 == 0) {
            const uint64_t dims[] = {64, (uint64_t)M, (uint64_t)cols / 64}, st[] = {(uint64_t)ld * 2, 128};
            const uint32_t box[] = {64, 64, 2};
            in_3d = 1;
            return encode_tiled(map, type, 3, ptr, dims, st, box, true);
        }
        const uint64_t dims[] = {(uint64_t)cols, (uint64_t)M}, st[] = {(uint64_t)ld * 2};
        const uint32_t box[] = {64, 64};
        in_3d = 0;
        return encode_tiled(map, type, 2, ptr, dims, st, box, true);
    };
    mapped = M == 0 || (encode(&m.a, a.A, K, a.lda, p.a_3d) && encode(&m.d, a.D, N, a.ldd, p.d_3d));
    if (!mapped) return cudaErrorInvalidValue;
    const long long units = (long long)a.groups.G * p.k_tiles * p.n_tiles;
    return launch_pairs<wgrad_kernel>(SMEM_BYTES, units, sms, s, m, p);
}

}  // namespace swg
