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
//
// What bounds it: for long groups the tensor pipe at the clock that the power
// limit leaves (16 groups of about 1024 rows, 1792 x 4096, bf16: 147 us, 1640
// TFLOP/s, in a burst and 168 us, 1430, in a long run; 75% of the pipe's cycles);
// for short ones writing C (64 groups of 16
// rows, 2048 x 1024: 63 us for 268 MB, 4.3 TB/s; 64 of 3, 1024 x 1024: 36 us, 3.8;
// a plain fill reaches 4.1), and 4 us that any call takes (48 groups of about 4
// rows, 896 x 521 with rows 1072 bytes apart: 19 to 24 us for 45 MB).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "grouped_launch.cuh"

namespace swg {
namespace {

struct WgradMaps {
    CUtensorMap a, d;                    // boxes of 64 rows
    CUtensorMap a16, d16;                // boxes of 16 rows
    CUtensorMap c;                       // 16-bit output, boxes of 64 columns x 32 rows (tma_out)
};

struct WgradParams {
    Groups groups;
    int N, K;
    int k_tiles, n_tiles;
    int n_step;                          // columns per tile, a multiple of 64
    int a_3d, d_3d;                      // 64-column atoms of an operand as one 3-D box
    uint32_t idesc;
    float alpha, beta;
    void *C;
    long long ldc, strideC;
    int out_kind;
    int staged;                          // 16-bit output, beta = 0: through shared memory
    int tma_out;                         // ... and from there with TMA stores
    int splits;                          // ranges of a group's rows, each a unit
    long long split_stride;
    int *err;
};

constexpr int WG_STAGES = 6;             // the ring
constexpr int LAST = WG_STAGES;          // a slot for a group's last rows, see Blocks
constexpr int LAST_FROM = 256;           // rows from which on it is used
constexpr int LAST_BYTES = 16 * 256;     // 16 rows x 128 columns of one operand
constexpr int FIX_WARP = EPI_WARP0 + NUM_EPI_WARPS;
constexpr int WG_THREADS = NUM_THREADS + 32;
constexpr int OP_BYTES = 128 * 128;      // 64 rows x 128 columns of one operand per CTA
constexpr int BAR_BYTES = 512;
constexpr int OUT_BYTES = 2048;          // 32 x 32 16-bit results per epilogue warp
constexpr int SMEM_BYTES = 1024 + WG_STAGES * 2 * OP_BYTES + 2 * LAST_BYTES + NUM_EPI_WARPS * OUT_BYTES + BAR_BYTES +
                           4 * (MAX_GROUPS + 1);
static_assert(SMEM_BYTES <= 232448, "beyond the per-CTA shared memory");

__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_addr)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
                 : "memory");
}

// Whether the phase has completed, acquiring at cluster scope: what the
// peer's threads wrote before their arrivals is visible.
__device__ __forceinline__ bool mbar_try_wait_cluster(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// Whether a block with `left` rows of the group from its first on (64 rows and
// more: all of them) also holds foreign rows in an MMA step that is run.
__device__ __forceinline__ bool ends_inside(int left) { return left < 64 && (left & 15) != 0; }

// A group's last block, where it ends inside an MMA step, is ready later than
// others: it lands, the fixing warp overwrites the foreign rows, and only then
// may the MMAs read it.  In the ring that held every tile up by 0.8 us.  So
// longer groups load the 16 rows of that step apart from the ring, after the
// first WG_STAGES blocks (by when the tile before has been done with the slot),
// and multiply them last (16 groups of 1000 rows, 1792 x 4096: 156 -> 144 us).
struct Blocks {
    int ring;        // blocks of 64 rows that go through the ring
    int rows;        // rows of the group in them
    bool apart;      // and the rest, fewer than 16, apart
};

__device__ __forceinline__ Blocks blocks_of(int rows)
{
    const bool apart = (rows & 15) != 0 && rows >= LAST_FROM;
    const int in_ring = apart ? rows & ~15 : rows;
    return {ceil_div(in_ring, 64), in_ring, apart};
}

struct WgradTile {
    int g, kb, nb, split, row0, rows;
};

__device__ __forceinline__ WgradTile wgrad_tile(const WgradParams &p, const int *start, int u)
{
    WgradTile t;
    t.split = 0;
    if (p.splits > 1) {
        const int tile = fast_div(u, p.splits);
        t.split = u - tile * p.splits;
        u = tile;
    }
    const int per = p.k_tiles * p.n_tiles;
    t.g = fast_div(u, per);
    const int local = u - t.g * per;
    const int band = p.k_tiles <= 8 ? 0 : fast_div(local, 8 * p.n_tiles);
    const int in = local - band * 8 * p.n_tiles;
    const int bm = min(8, p.k_tiles - band * 8);
    t.nb = fast_div(in, bm);
    t.kb = band * 8 + in - t.nb * bm;
    t.row0 = start[t.g];
    t.rows = start[t.g + 1] - t.row0;
    if (p.splits > 1) {                  // whole blocks of 64 rows
        const int range = ceil_div(ceil_div(t.rows, 64), p.splits) * 64;
        const int from = min(t.rows, t.split * range);
        t.row0 += from;
        t.rows = min(range, t.rows - from);
    }
    return t;
}

__global__ void __launch_bounds__(WG_THREADS, 1)
    wgrad_kernel(const __grid_constant__ WgradMaps maps, const WgradParams p)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t *sA = smem;
    uint8_t *sD = sA + WG_STAGES * OP_BYTES;
    uint8_t *sLast = sD + WG_STAGES * OP_BYTES;       // A's last rows, then D's
    uint8_t *sOut = sLast + 2 * LAST_BYTES;
    uint64_t *bars = reinterpret_cast<uint64_t *>(sOut + NUM_EPI_WARPS * OUT_BYTES);
    constexpr int SLOTS = WG_STAGES + 1;
    uint64_t *full = bars;
    uint64_t *empty = bars + SLOTS;
    uint64_t *landed = bars + 2 * SLOTS;             // a group's last block, in this CTA
    uint64_t *acc_full = bars + 3 * SLOTS;
    uint64_t *acc_empty = bars + 3 * SLOTS + 2;
    uint64_t *mma_done = bars + 3 * SLOTS + 4;
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(bars + 3 * SLOTS + 5);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
    int *start = reinterpret_cast<int *>(reinterpret_cast<uint8_t *>(bars) + BAR_BYTES);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (threadIdx.x == 0) {
        for (int s = 0; s < SLOTS; ++s) {
            mbar_init(smem_u32(&full[s]), 2);        // a thread of each CTA
            mbar_init(smem_u32(&empty[s]), 1);
            mbar_init(smem_u32(&landed[s]), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&acc_full[b]), 1);
            mbar_init(smem_u32(&acc_empty[b]), 2 * NUM_EPI_WARPS);
        }
        mbar_init(smem_u32(mma_done), 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(tmem_holder), 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    // Up to here only this pair's own resources; now the offsets may be read.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    group_starts<WG_THREADS>(p.groups, start, p.err);
    const uint32_t tmem_base = __shfl_sync(0xffffffffu, *tmem_holder, 0);
    const int units = p.groups.G * p.k_tiles * p.n_tiles * p.splits;
    const int u0 = (int)(blockIdx.x >> 1), du = (int)(gridDim.x >> 1);

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        int stage = 0;
        uint32_t phase = 0, last_phase = 0;
        uint32_t armed = 0, armed_parity = 0;
        const uint32_t empty0 = smem_u32(empty), full0 = smem_u32(full), landed0 = smem_u32(landed);
        const uint32_t full_leader0 = mapa_shared(full0, 0);
        const uint32_t a0 = smem_u32(sA), d0 = smem_u32(sD), last0 = smem_u32(sLast);
        bool ok = true;
        for (int u = u0; u < units && ok; u += du) {
            const WgradTile t = wgrad_tile(p, start, u);
            const int rows = __shfl_sync(0xffffffffu, t.rows, 0);
            const int row0 = __shfl_sync(0xffffffffu, t.row0, 0);
            const int ka = t.kb * 256 + (int)rank * 128;
            const int nd = t.nb * p.n_step + (int)rank * (p.n_step / 2);
            const Blocks blocks = blocks_of(rows);
            // Loads 64 rows (`last`: the 16 of a last step) from `row` on into slot
            // s, whose barriers are in phase ph.  Both CTAs' bytes and one arrival
            // of each complete the leader's barrier.  Where foreign rows must go,
            // the rows land on a barrier of this CTA instead, and the fixing warp
            // arrives for it.
            auto load = [&](auto last, int s, uint32_t ph, int row, bool ends) {
                constexpr bool rows16 = decltype(last)::value;
                if (!wait_bounded_warp(empty0 + 8 * s, ph ^ 1, abort_flag, p.err)) return false;
                armed |= 1u << s;
                armed_parity = (armed_parity & ~(1u << s)) | (ph << s);
                constexpr uint32_t bytes = rows16 ? LAST_BYTES : OP_BYTES;
                const uint32_t a_dst = rows16 ? last0 : a0 + s * OP_BYTES;
                const uint32_t d_dst = rows16 ? last0 + LAST_BYTES : d0 + s * OP_BYTES;
                const CUtensorMap *ma = rows16 ? &maps.a16 : &maps.a;
                const CUtensorMap *md = rows16 ? &maps.d16 : &maps.d;
                const uint32_t fb = full0 + 8 * s;
                const uint32_t bar = ends ? landed0 + 8 * s : full_leader0 + 8 * s;
                if (elect_one()) {
                    if (ends)
                        mbar_arrive_expect_tx(bar, 2 * bytes);
                    else if (leader)
                        mbar_arrive_expect_tx(fb, 4 * bytes);
                    else
                        mbar_arrive_remote_tmem(bar);            // nothing to release
                    if (p.a_3d) {
                        tma_load_3d_pair(a_dst, ma, bar, 0, row, ka / 64);
                    } else {
                        tma_load_2d_pair(a_dst, ma, bar, ka, row);
                        tma_load_2d_pair(a_dst + bytes / 2, ma, bar, ka + 64, row);
                    }
                    if (p.d_3d) {
                        tma_load_3d_pair(d_dst, md, bar, 0, row, nd / 64);
                    } else {
                        tma_load_2d_pair(d_dst, md, bar, nd, row);
                        tma_load_2d_pair(d_dst + bytes / 2, md, bar, nd + 64, row);
                    }
                }
                __syncwarp();
                return true;
            };
            const int ahead = blocks.apart ? min(blocks.ring, WG_STAGES) : -1;
            for (int b = 0; b <= blocks.ring && ok; ++b) {
                if (b == ahead) {
                    ok = load(std::true_type{}, LAST, last_phase, row0 + blocks.rows, true);
                    last_phase ^= 1;
                }
                if (b == blocks.ring || !ok) break;
                ok = load(std::false_type{}, stage, phase, row0 + b * 64,
                          ends_inside(blocks.rows - b * 64));
                if (++stage == WG_STAGES) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
        // Never leave with loads in flight into this CTA's shared memory.
        if (leader) {
            for (int s = 0; s < SLOTS; ++s)
                if (armed & (1u << s))
                    wait_bounded(smem_u32(&full[s]), (armed_parity >> s) & 1, abort_flag, p.err,
                                 false, DRAIN_LIMIT_NS);
        } else if (!ok) {
            const uint64_t t0 = global_timer_ns();
            while (global_timer_ns() - t0 < 200000ull) {
            }
        }
        __syncwarp();
    } else if (warp == FIX_WARP) {
        // ------------------------------------------------------------ foreign rows
        int stage = 0;
        uint32_t phases = 0;                             // next parity of each landed[]
        bool ok = true;
        for (int u = u0; u < units && ok; u += du) {
            const WgradTile t = wgrad_tile(p, start, u);
            const Blocks blocks = blocks_of(t.rows);
            if (t.rows & 15) {
                const int s = blocks.apart ? LAST : (stage + blocks.ring - 1) % WG_STAGES;
                ok = wait_bounded(smem_u32(&landed[s]), (phases >> s) & 1, abort_flag, p.err);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                phases ^= 1u << s;
                // from the group's end to a multiple of 16 rows, in the four 64-column atoms
                const int left = blocks.apart ? t.rows & 15 : t.rows & 63;
                const uint32_t atom = blocks.apart ? LAST_BYTES / 2 : OP_BYTES / 2;
                const uint32_t a_dst = smem_u32(blocks.apart ? sLast : sA + s * OP_BYTES);
                const uint32_t d_dst = smem_u32(blocks.apart ? sLast + LAST_BYTES : sD + s * OP_BYTES);
                const uint32_t end = (uint32_t)((left + 15) & ~15) * 128;
                for (uint32_t o = (uint32_t)left * 128 + lane * 16; o < end; o += 512) {
                    st_shared_v4(a_dst + o, make_uint4(0, 0, 0, 0));
                    st_shared_v4(a_dst + atom + o, make_uint4(0, 0, 0, 0));
                    st_shared_v4(d_dst + o, make_uint4(0, 0, 0, 0));
                    st_shared_v4(d_dst + atom + o, make_uint4(0, 0, 0, 0));
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&full[s]), 0));
            }
            stage = (stage + blocks.ring) % WG_STAGES;
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        if (leader) {
            int stage = 0;
            uint32_t phase = 0, last_phase = 0;
            bool ok = true;
            int n = 0;                                   // tiles with rows so far
            // K-step kk of a stage is 16 rows (2048 bytes) further in each atom
            const uint64_t a_desc = smem_desc(smem_u32(sA), 8192, 1024);
            const uint64_t d_desc = smem_desc(smem_u32(sD), 8192, 1024);
            const uint64_t last_desc = smem_desc(smem_u32(sLast), LAST_BYTES / 2, 1024);
            for (int u = u0; u < units && ok; u += du) {
                const int rows = __shfl_sync(0xffffffffu, wgrad_tile(p, start, u).rows, 0);
                if (rows == 0) continue;
                const int acc = n & 1;
                if (!wait_bounded_warp(smem_u32(&acc_empty[acc]), ((n >> 1) & 1) ^ 1, abort_flag, p.err)) {
                    ok = false;
                    break;
                }
                ++n;
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + acc * 256;
                const Blocks blocks = blocks_of(rows);
                // Block b of the tile, with `left` rows of it from its first on.
                auto multiply = [&](int b, int left, int s, uint32_t ph) {
                    if (!wait_bounded_warp(smem_u32(&full[s]), ph, abort_flag, p.err)) return false;
                    if (ends_inside(left)) mbar_try_wait_cluster(smem_u32(&full[s]), ph);
                    tc_fence_after();
                    const uint64_t ad = a_desc + (uint64_t)(s * (OP_BYTES >> 4));
                    const uint64_t dd = d_desc + (uint64_t)(s * (OP_BYTES >> 4));
                    if (elect_one()) {
                        if (left > 48) {                 // every block but a group's last
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                tc_mma_f16_pair(d_tmem, ad + kk * 128, dd + kk * 128, p.idesc, b | kk);
                        } else {
                            for (int kk = 0; kk < ceil_div(left, 16); ++kk)
                                tc_mma_f16_pair(d_tmem, ad + kk * 128, dd + kk * 128, p.idesc, b | kk);
                        }
                        tc_commit_pair(smem_u32(&empty[s]));
                    }
                    __syncwarp();
                    return true;
                };
                for (int b = 0; b < blocks.ring && ok; ++b) {
                    ok = multiply(b, blocks.rows - b * 64, stage, phase);
                    if (++stage == WG_STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
                if (ok && blocks.apart) {
                    const uint32_t bar = smem_u32(&full[LAST]);
                    ok = wait_bounded_warp(bar, last_phase, abort_flag, p.err);
                    if (!ok) break;
                    mbar_try_wait_cluster(bar, last_phase);
                    tc_fence_after();
                    if (elect_one()) {
                        tc_mma_f16_pair(d_tmem, last_desc, last_desc + (LAST_BYTES >> 4), p.idesc, 1u);
                        tc_commit_pair(smem_u32(&empty[LAST]));
                    }
                    __syncwarp();
                    last_phase ^= 1;
                }
                if (!ok) break;
                if (elect_one()) tc_commit_pair(smem_u32(&acc_full[acc]));
                __syncwarp();
            }
            if (elect_one()) tc_commit_pair_local(smem_u32(mma_done));
            __syncwarp();
            wait_bounded(smem_u32(mma_done), 0, abort_flag, p.err, false, DRAIN_LIMIT_NS);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ epilogue
        // Each lane holds 32 consecutive columns of its row of C.  16-bit results
        // pass through shared memory: the two warps of a lane quarter stage 32
        // rows x 64 columns, whole 128-byte lines, which leave with a TMA store
        // (but the last columns of rows that do not end on 16 bytes).  Stored by
        // the lanes themselves they touch 32 lines per instruction, and the main
        // loop, whose operands use the same memory, took a fifth longer.
        const int q = warp & 3;
        const int h = (warp - EPI_WARP0) / 4;
        const int row = q * 32 + lane;
        const uint32_t box = smem_u32(sOut + q * 2 * OUT_BYTES);
        const int bar = 1 + q;
        constexpr int PAIR_THREADS = 64;
        const bool issuer = h == 0 && lane == 0;
        TileParams tp{};
        tp.alpha = p.alpha;
        tp.beta = p.beta;
        tp.D = p.C;
        tp.out_kind = p.out_kind;
        int n = 0;
        for (int u = u0; u < units; u += du) {
            const WgradTile t = wgrad_tile(p, start, u);
            const int acc = n & 1;
            if (t.rows > 0) {
                const bool ok = wait_bounded(smem_u32(&acc_full[acc]), (n >> 1) & 1, abort_flag, p.err);
                if (!named_bar_and(bar, PAIR_THREADS, ok)) break;    // both warps leave, or none
                tc_fence_after();
            }
            const uint32_t t_row = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + acc * 256;
            const int k = t.kb * 256 + (int)rank * 128 + row;
            const long long out = (long long)t.g * p.strideC + (long long)k * p.ldc +
                                  t.split * p.split_stride;
            uint32_t r[32];
#pragma unroll 1
            for (int c = 0; c < p.n_step / 64; ++c) {
                const int col0 = t.nb * p.n_step + c * 64;
                if (k - lane >= p.K || col0 >= p.N) break;       // (the same for both warps)
                const int col = col0 + h * 32;
                if (t.rows > 0) {
                    tmem_ld_32cols(t_row + c * 64 + h * 32, r);
                    tmem_ld_wait(r);
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) r[j] = 0;
                }
                if (p.staged) {
                    if (issuer) bulk_wait_read_all();
                    named_bar_sync(bar, PAIR_THREADS);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t w[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            w[i] = pack2(p.alpha * __uint_as_float(r[8 * j + 2 * i]),
                                         p.alpha * __uint_as_float(r[8 * j + 2 * i + 1]), p.out_kind);
                        st_shared_v4(staged_at(box, lane, h * 4 + j), make_uint4(w[0], w[1], w[2], w[3]));
                    }
                    uint16_t *dst = reinterpret_cast<uint16_t *>(p.C) + out - lane * p.ldc + col;
                    const int rows = p.K - (k - lane);
                    if (p.tma_out) {
                        const int whole = p.N & ~7;
                        fence_proxy_async_smem();
                        named_bar_sync(bar, PAIR_THREADS);
                        if (issuer && col0 < whole) {
                            tma_store_3d(&maps.c, box, col0, k, t.g);
                            bulk_commit_group();
                        }
                        if (p.N != whole && col < p.N && col + 32 > whole)
                            copy_last_columns(box, h * 4, dst, p.ldc, rows, whole - col, p.N - col, lane);
                    } else {
                        __syncwarp();
                        copy_staged<4>(box, h * 4, dst, p.ldc, rows, p.N - col, lane);
                    }
                } else if (k < p.K && col < p.N) {
                    float v[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
                    store_row_chunk(tp, out + col, v, min(32, p.N - col));
                }
            }
            if (t.rows > 0) {
                ++n;
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote_tmem(mapa_shared(smem_u32(&acc_empty[acc]), 0));
            }
        }
        if (issuer) bulk_wait_read_all();           // before this CTA's shared memory goes
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
    // Tiles of nearly equal width: 521 columns are 3 x 192, not 256, 256 and 9
    p.n_tiles = (int)((N + 255) / 256);
    p.n_step = (int)((N + 64 * p.n_tiles - 1) / (64 * p.n_tiles) * 64);
    const uint32_t t = a.in_bf16 ? 1u : 0u;
    // kind::f16, FP32 accumulators, both operands MN-major, 256 x n_step
    p.idesc = (1u << 4) | (t << 7) | (t << 10) | (1u << 15) | (1u << 16) |
              ((uint32_t)(p.n_step >> 3) << 17) | (16u << 24);
    p.alpha = a.alpha;
    p.beta = a.beta;
    p.C = a.C;
    p.ldc = a.ldc;
    p.strideC = a.strideC;
    p.out_kind = a.out_kind;
    p.err = err;
    // (3-D: 64 columns at a time as their own dimension, where a CTA's columns
    // begin at multiples of 64)
    auto encode = [&](CUtensorMap *map, const void *ptr, int64_t cols, int64_t ld, uint32_t rows,
                      bool whole, int &in_3d) {
        const CUtensorMapDataType type =
            a.in_bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
        if (whole && cols % 64 == 0) {
            const uint64_t dims[] = {64, (uint64_t)M, (uint64_t)cols / 64}, st[] = {(uint64_t)ld * 2, 128};
            const uint32_t box[] = {64, rows, 2};
            in_3d = 1;
            return encode_tiled(map, type, 3, ptr, dims, st, box, 128);
        }
        const uint64_t dims[] = {(uint64_t)cols, (uint64_t)M}, st[] = {(uint64_t)ld * 2};
        const uint32_t box[] = {64, rows};
        in_3d = 0;
        return encode_tiled(map, type, 2, ptr, dims, st, box, 128);
    };
    mapped = M == 0 || (encode(&m.a, a.A, K, a.lda, 64, true, p.a_3d) &&
                        encode(&m.d, a.D, N, a.ldd, 64, p.n_step % 128 == 0, p.d_3d));
    if (M >= LAST_FROM)
        mapped = mapped && encode(&m.a16, a.A, K, a.lda, 16, true, p.a_3d) &&
                 encode(&m.d16, a.D, N, a.ldd, 16, p.n_step % 128 == 0, p.d_3d);
    p.splits = a.splits;
    p.split_stride = a.split_stride;
    p.staged = a.out_kind != OUT_F32 && a.beta == 0.0f;
    p.tma_out = p.staged && N >= 8;
    if (p.tma_out) {
        const uint64_t ld = (uint64_t)a.ldc * 2;
        const uint64_t dims[] = {(uint64_t)(N & ~7), (uint64_t)K, (uint64_t)a.groups.G};
        const uint64_t st[] = {ld, a.groups.G > 1 ? (uint64_t)a.strideC * 2 : ld * K};
        const uint32_t box[] = {64, 32, 1};
        mapped = mapped && encode_tiled(&m.c, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, a.C, dims, st, box, 128);
    }
    if (!mapped) return cudaErrorInvalidValue;
    const long long units = (long long)a.groups.G * p.k_tiles * p.n_tiles * p.splits;
    return launch_pairs<wgrad_kernel, WG_THREADS>(SMEM_BYTES, SMEM_BYTES, units, sms, s, m, p);
}

}  // namespace swg
