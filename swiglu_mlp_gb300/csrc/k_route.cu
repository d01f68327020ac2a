// k_route.cu — the router: the experts of each token with their weights, rows
// sorted by expert, and the gradient of the logits.
//
// route_kernel: a warp has a token, lane l the experts l, l + 32, ...  As many lanes'
// largest as experts are wanted give a bound that few others pass; those are ranked by
// comparing all with all, the lowest index of equals first.  (One after the other by
// a maximum over the warp, eight of 256 took four times the instructions.)  Without a
// bias the order of the scores is that of the logits, which
// compare exactly.  With one, or where groups are valued by a sum, the choices
// (score + bias) are formed in FP32 and compared with a bound of their error;
// where two are nearer than that, and not the same logit and bias, the candidates are
// decided once more in FP64.  So the choice is that of the definition, whatever
// the rounding of the exponential.
//
// route_team_kernel, up to 256 experts and eight of them: the same by eight lanes for
// each token, 480 instructions a token against 1412 (16384 tokens, eight of
// 256 experts by four of eight groups, with the plan: 29.6 us, 10 of them sorting, against
// 44; 8192 tokens, two of 16 experts, with the gradient: 11.8 against 14.9; 4 tokens, six of
// 64 experts, one CTA: 4.8 against 5.3).  The logits themselves take 2.5 us.  Instructions
// and their latencies bound it: the 16 warps that their registers leave room for fill 42% of
// the issue slots, and a CTA's 108 tokens are one full round of 64 and one of 44.
//
// Sorting is counting: every chunk of tokens counts its experts in shared memory,
// and the second kernel adds up the chunks before its own and ranks its slots
// in order: 10 us for 131072 slots of 256 experts, latencies one after the other (counts
// of 152 chunks, running sums, the scattered rows).  One chunk: the same CTA goes on,
// without a second kernel.
#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "chunks.h"
#include "groups.cuh"
#include "launch.h"
#include "routing.h"

namespace swg {
namespace {

constexpr unsigned ALL = 0xffffffffu;
constexpr int SORT_THREADS = 1024;

__device__ __forceinline__ float load_any(const void *x, long long i, int type)
{
    if (type == 2) return static_cast<const float *>(x)[i];
    if (type == 1) return __bfloat162float(static_cast<const __nv_bfloat16 *>(x)[i]);
    return __half2float(static_cast<const __half *>(x)[i]);
}

__device__ __forceinline__ void store_any(void *x, long long i, float v, int type)
{
    if (type == 2)
        static_cast<float *>(x)[i] = v;
    else if (type == 1)
        static_cast<__nv_bfloat16 *>(x)[i] = __float2bfloat16_rn(v);
    else
        static_cast<__half *>(x)[i] = __float2half_rn(v);
}

__device__ __forceinline__ float minus_inf() { return __int_as_float(0xff800000); }

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(ALL, v, d);
    return v;
}
__device__ __forceinline__ double warp_sum(double v)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(ALL, v, d);
    return v;
}

// Unsigned numbers in the order of the values (not NaN), equal zeros equal; more than 0.
__device__ __forceinline__ uint32_t ordered(float x)
{
    const uint32_t b = __float_as_uint(x + 0.0f);      // (-0 becomes 0)
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ uint64_t ordered(double x)
{
    const uint64_t b = (uint64_t)__double_as_longlong(x + 0.0);
    return b ^ ((uint64_t)((int64_t)b >> 63) | 0x8000000000000000ull);
}
__device__ __forceinline__ float value_of(uint32_t k)
{
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

__device__ __forceinline__ uint32_t warp_max(uint32_t k) { return __reduce_max_sync(ALL, k); }
__device__ __forceinline__ uint64_t warp_max(uint64_t k)
{
    const uint32_t hi = __reduce_max_sync(ALL, (uint32_t)(k >> 32));
    const uint32_t lo = __reduce_max_sync(ALL, (uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
    return (uint64_t)hi << 32 | lo;
}

// The sigmoid of x times e^-shift, shift 0 or from x up to 0: by the exponential of -|x|, so that
// no divisor passes 2 and scores keep their digits as far down as FP32 goes, and with a
// shift beyond that.  1 - sigmoid(x) is sigmoid(-x).  (FAST: the division that is off by 2 units.)
template <bool FAST>
__device__ __forceinline__ float sigmoid(float x, float shift = 0.0f)
{
    const float a = x < 0.0f ? expf(x - shift) : 1.0f, b = 1.0f + expf(-fabsf(x));
    return FAST ? __fdividef(a, b) : a / b;
}

// The largest over the warp (of no NaN).
__device__ __forceinline__ float warp_max(float m)
{
    float r;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(m));
    return r;
}

// Takes the largest key (lane l, place i: expert l + 32 i) out, the lowest expert of
// equals; -1 when only -inf is left.
template <int V>
__device__ __forceinline__ int take_best(float (&key)[V], float &best)
{
    const int lane = threadIdx.x & 31;
    float k = key[0];
    int at = 0;
#pragma unroll
    for (int i = 1; i < V; ++i)
        if (key[i] > k) {
            k = key[i];
            at = i;
        }
    best = warp_max(k);
    if (best == minus_inf()) return -1;
    const int e = (int)__reduce_min_sync(ALL, k == best ? (unsigned)(lane + 32 * at) : 0xffffffffu);
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (lane + 32 * i == e) key[i] = minus_inf();
    return e;
}

// Place of expert e's choice in a warp's scratch: one value further for every
// 32, so that groups of 32 do not share banks.
__device__ __forceinline__ int at_scratch(int e) { return e + (e >> 5); }

// Lanes that look at a group in the scratch together: as many as there are for each,
// a power of two.  (A group's home is the first of them.)
__device__ __forceinline__ int log_group_lanes(int groups) { return 31 - __clz(32 / groups); }

// The group's two largest choices, at its home, from those in the warp's scratch (-inf
// where masked).
template <class F>
__device__ __forceinline__ void largest_two(int groups, int size, int log_lanes, const F *scratch, F &a, F &b)
{
    const int lane = threadIdx.x & 31, lanes = 1 << log_lanes, g = lane >> log_lanes;
    a = b = (F)minus_inf();
    if (g < groups)
        for (int i = lane & (lanes - 1); i < size; i += lanes) {
            const F v = scratch[at_scratch(g * size + i)];
            const F less = v < a ? v : a;
            a = v > a ? v : a;
            b = less > b ? less : b;
        }
    for (int d = 1; d < lanes; d <<= 1) {
        const F a2 = __shfl_xor_sync(ALL, a, d), b2 = __shfl_xor_sync(ALL, b, d);
        const F less = a2 < a ? a2 : a, more = b2 > b ? b2 : b;
        a = a2 > a ? a2 : a;
        b = less > more ? less : more;
    }
}

// The best groups as a bit mask over their homes, from the two largest choices there
// (a > -inf only there).  Where the worst of them is not further than `tol` > 0 above the best of the
// others, `near` are those that may change places, and `last` is, at a group's home,
// the smallest choice in its value.
template <class F>
__device__ __forceinline__ unsigned best_groups(const RouteArgs &p, F a, F b, F tol, unsigned &near, F &last)
{
    const int lane = threadIdx.x & 31;
    const F low = (F)minus_inf();
    const bool both = p.group_sum == 2 && b > low;
    const F value = both ? a + b : a;
    last = both ? b : a;
    auto key = ordered(value);
    if (!(a > low)) key = 0;
    const auto own = key;
    unsigned keep = 0;
    auto best = key;
    for (int j = 0; j < p.top_groups; ++j) {
        best = warp_max(key);
        if (best == 0) break;
        const int home = __ffs(__ballot_sync(ALL, key == best)) - 1;
        keep |= 1u << home;
        if (lane == home) key = 0;
    }
    near = 0;
    if constexpr (sizeof(F) == 4)
        if (tol > (F)0 && best != 0) {
            const uint32_t rest = warp_max(key);
            const float w = value_of(best), r = value_of(rest);
            if (rest != 0 && !(w - r > tol))
                near = __ballot_sync(ALL, own != 0 && (keep >> lane & 1 ? value - r <= tol : w - value <= tol));
        }
    return keep;
}

// The token's experts in FP64: lane j's is the j'th.  For what the candidates alone do
// not decide (many equal choices, biases of +inf).
template <int V>
__device__ __noinline__ int choose_exactly(const RouteArgs &p, long long row, double *scratch)
{
    constexpr int TOGETHER = V < 8 ? V : 8;
    const int lane = threadIdx.x & 31;
    const double low = (double)minus_inf();
    double c[V];
    uint64_t key[V];
    double m = low, z = 0.0;
    uint32_t masked = 0;
#pragma unroll TOGETHER
    for (int i = 0; i < V; ++i) {
        const int e = lane + 32 * i;
        c[i] = e < p.E ? (double)load_any(p.logits, row + e, p.type) : low;
        if (c[i] == low) masked |= 1u << i;
        m = c[i] > m ? c[i] : m;
    }
    for (int d = 16; d > 0; d >>= 1) {
        const double o = __shfl_xor_sync(ALL, m, d);
        m = o > m ? o : m;
    }
    const bool softmax = p.score == SCORE_SOFTMAX;
#pragma unroll TOGETHER
    for (int i = 0; i < V; ++i) {
        const double e = exp(softmax ? c[i] - m : -c[i]);
        z += e;
        c[i] = softmax ? e : 1.0 / (1.0 + e);
    }
    const double sum = softmax ? warp_sum(z) : 1.0;
#pragma unroll TOGETHER
    for (int i = 0; i < V; ++i) {
        const int e = lane + 32 * i;
        if (softmax) c[i] /= sum;                    // (as in exact_choice: both round alike)
        if (p.bias != nullptr && e < p.E) c[i] += (double)p.bias[e];
        if (c[i] == low) masked |= 1u << i;
        // (without a bias the order is that of the logits, groups apart)
        const double by = p.bias != nullptr || e >= p.E ? c[i] : (double)load_any(p.logits, row + e, p.type);
        key[i] = masked >> i & 1 ? 0 : ordered(by);
    }
    if (p.groups > 1) {
        const int size = p.E / p.groups, log_lanes = log_group_lanes(p.groups);
        __syncwarp();
#pragma unroll TOGETHER
        for (int i = 0; i < V; ++i) {
            const int e = lane + 32 * i;
            if (e < p.E) scratch[at_scratch(e)] = masked >> i & 1 ? low : c[i];
        }
        __syncwarp();
        unsigned near;
        double last, a, b;
        largest_two<double>(p.groups, size, log_lanes, scratch, a, b);
        if ((lane & ((1 << log_lanes) - 1)) != 0) a = low;
        const unsigned keep = best_groups<double>(p, a, b, 0.0, near, last);
#pragma unroll TOGETHER
        for (int i = 0; i < V; ++i) {
            const int e = lane + 32 * i;
            if (e >= p.E || !(keep >> (e / size << log_lanes) & 1)) key[i] = 0;
        }
    }
    int mine = -1;
    for (int j = 0; j < p.top; ++j) {
        uint64_t k = 0;
        int at = 0;
#pragma unroll TOGETHER
        for (int i = 0; i < V; ++i)
            if (key[i] > k) {
                k = key[i];
                at = i;
            }
        const uint64_t best = warp_max(k);
        if (best == 0) break;
        const int e = (int)__reduce_min_sync(ALL, k == best ? (unsigned)(lane + 32 * at) : 0xffffffffu);
#pragma unroll TOGETHER
        for (int i = 0; i < V; ++i)
            if (lane + 32 * i == e) key[i] = 0;
        if (lane == j) mine = e;
    }
    return mine;
}

// A candidate for a token's experts.
struct Candidate {
    float key;
    int expert;
};
constexpr int SCRATCH = 32 * sizeof(Candidate);      // bytes of a warp's, before its choices

// What follows decides in FP64 where FP32 cannot.  It is seldom run, and then with
// nothing of it in the instruction caches, of which every 128 bytes come from afar: so
// it looks at the candidates alone, one per lane, in few instructions.  (All choices
// of a token in FP64: 16 us.)

// Expert e's choice; of the softmax with the sum of exact_sum.
__device__ __noinline__ double exact_choice(const RouteArgs &p, long long row, int e, float m, double sum)
{
    const double x = (double)load_any(p.logits, row + e, p.type);
    const bool softmax = p.score == SCORE_SOFTMAX;
    const double y = exp(softmax ? x - (double)m : -x);
    const double s = softmax ? y / sum : 1.0 / (1.0 + y);
    return p.bias != nullptr ? s + (double)p.bias[e] : s;
}

__device__ __noinline__ double exact_sum(const RouteArgs &p, long long row, float m)
{
    double z = 0.0;
#pragma unroll 1
    for (int e = threadIdx.x & 31; e < p.E; e += 32) z += exp((double)load_any(p.logits, row + e, p.type) - (double)m);
    return warp_sum(z);
}

// The groups once more: candidates (n <= 32, their group's first lane in `home`) of the
// groups that are `near`; `keep` gets the best of these by their exact values.
__device__ __noinline__ unsigned exact_groups(const RouteArgs &p, unsigned keep, unsigned near, bool on, int home, double choice)
{
    const int lane = threadIdx.x & 31;
    uint64_t value = 0;                              // at a group's first lane
    for (unsigned left = near; left != 0; left &= left - 1) {
        const int g = __ffs(left) - 1;
        uint64_t key = on && home == g ? ordered(choice) : 0;
        const uint64_t a = warp_max(key);
        const unsigned with = __ballot_sync(ALL, key == a);
        if (lane == __ffs(with) - 1) key = 0;
        const uint64_t b = p.group_sum == 2 ? warp_max(key) : 0;
        auto of = [](uint64_t k) { return __longlong_as_double((long long)(k >> 63 ? k ^ 0x8000000000000000ull : ~k)); };
        if (lane == g) value = ordered(b != 0 ? of(a) + of(b) : of(a));
    }
    int rank = 0;
    for (unsigned left = near; left != 0; left &= left - 1) {
        const int g = __ffs(left) - 1;
        const uint64_t other = __shfl_sync(ALL, value, g);
        rank += other > value || (other == value && g < lane);
    }
    const int places = __popc(keep & near);
    return (keep & ~near) | __ballot_sync(ALL, (near >> lane & 1) && rank < places);
}

// What a warp keeps from token to token.
template <int V>
struct Experts {
    float bias[V];                                   // of this lane's, 0 without
    float most;                                      // the largest magnitude among all biases
    int size, rows;                                  // of a group: experts, and how many places of every lane (0: not whole ones)
    int log_lanes;                                   // (0 with whole places: group g's home is lane g)
    uint8_t home[V];                                 // of their groups
};

template <int V>
__device__ __forceinline__ Experts<V> experts_of(const RouteArgs &p)
{
    const int lane = threadIdx.x & 31;
    Experts<V> of;
    of.most = 0.0f;
    of.size = p.E / p.groups;
    of.rows = of.size % 32 == 0 ? of.size / 32 : 0;
    of.log_lanes = of.rows > 0 ? 0 : log_group_lanes(p.groups);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = lane + 32 * i;
        of.bias[i] = p.bias != nullptr && e < p.E ? p.bias[e] : 0.0f;
        // (a bias of -inf masks its expert; behind the last, the logits do)
        if (of.bias[i] != minus_inf()) of.most = of.bias[i] == of.bias[i] ? fmaxf(of.most, fabsf(of.bias[i])) : -minus_inf();
        of.home[i] = (uint8_t)(min(e, p.E - 1) / of.size << of.log_lanes);
    }
    of.most = warp_max(of.most);
    return of;
}

// The experts of a token, lane j's the j'th (-1: none), and lane j's weight, from
// logits l (lane l's those of experts l, l + 32, ..; -inf behind the last).
template <int V>
__device__ __forceinline__ int choose(const RouteArgs &p, long long row, const float (&l)[V], const Experts<V> &of,
                                      unsigned char *scratch, float &weight)
{
    const int lane = threadIdx.x & 31;
    const bool grouped = p.groups > 1, biased = p.bias != nullptr;
    const bool by_score = biased || (grouped && p.group_sum == 2);
    const bool softmax = p.score == SCORE_SOFTMAX;
    float *choices = reinterpret_cast<float *>(scratch + SCRATCH);
    float m = l[0];
#pragma unroll
    for (int i = 1; i < V; ++i) m = fmaxf(m, l[i]);
    bool nan = false;
    float key[V], by_group[V];                       // what experts and groups go by; -inf where masked
    bool sure = true;
    float tol = 0.0f;
    if (by_score) {
        // Scores by the fast exponential, which is off by at most 2 + 1.2 |x| units (2^-23 of
        // its value), and division (2 units).  tol bounds by how much the difference of two
        // choices is off.
        // Softmax: x = l - m, whose rounding is half a unit of e^x for each of |x|.  What the
        // sum and its inverse are off by is common to all scores and takes that part of a
        // difference, which is at most the largest score.  The terms' errors, 2 + 1.7 |x|
        // weighted by e^x, are at most 9.3 units of the sum of 1024 (one term 0, the others
        // all near -5.2), its 15 additions in a tree 7.5, the inverse 2.  Each score's own
        // e^x, (2 + 1.7 |x|) e^x <= 2 units of the largest, and its product, a half: of two
        // choices 5.  In all 24 units of the largest score; twice that is taken.
        // Sigmoid: s (1 - s) (2 + 1.2 |x|) + 2.5 s is at most 3.6 units of the largest score
        // where that is a half or more, and 4.5 + 1.2 |m| where all logits are negative: twice
        // that, of two choices, is at most the 12 + 2.4 |m| that are taken.
        m = warp_max(m == m ? m : minus_inf());
        float s[V];
        float largest;
        if (softmax) {
            float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < V; ++i) {
                s[i] = __expf(l[i] - m);
                sum[i % 4] += s[i];
            }
            largest = __fdividef(1.0f, warp_sum((sum[0] + sum[1]) + (sum[2] + sum[3])));
#pragma unroll
            for (int i = 0; i < V; ++i) s[i] *= largest;
            tol = largest * 0x1.8p-18f;
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) s[i] = __fdividef(1.0f, 1.0f + __expf(-l[i]));
            largest = m < -80.0f ? 0.0f : __fdividef(1.0f, 1.0f + __expf(-m));
            tol = largest * (12.0f + 2.4f * fmaxf(-m, 0.0f)) * 0x1p-23f;
        }
        // Choices are rounded to FP32 (2^-23 of both; of the values of two groups, which are
        // compared with 2 tol, 2^-21), and 2^-120 stands for scores that FP32 has no digits for.
        tol += 0x1p-22f * (largest + of.most) + 0x1p-120f;
        sure = tol < 1.0f;                           // (not with a bias of +inf, or of NaN)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            s[i] += of.bias[i];
            if (l[i] == minus_inf()) s[i] = minus_inf();
            nan = nan || s[i] != s[i];
            key[i] = biased || s[i] == minus_inf() ? s[i] : l[i];
            by_group[i] = s[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            key[i] = l[i];
            nan = nan || l[i] != l[i];
            by_group[i] = l[i];
        }
        if (softmax && !p.normalise) m = warp_max(m == m ? m : minus_inf());
    }
    // A padding token: no logit is left.  (A NaN anywhere, or for softmax +inf, is
    // found before that.)
    const bool some = m > minus_inf();
    nan = nan || (softmax && m == -minus_inf());
    if (__any_sync(ALL, nan)) {
        weight = __int_as_float(0x7fffffff);
        return lane < p.top ? lane : -1;
    }
    if (!__any_sync(ALL, some)) {
        weight = 0.0f;
        return -1;
    }
    Candidate *buffer = reinterpret_cast<Candidate *>(scratch);
    if (grouped) {
        if (of.rows == 0) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (lane + 32 * i < p.E) choices[at_scratch(lane + 32 * i)] = by_group[i];
            __syncwarp();
        }
        unsigned near;
        float last, a = minus_inf(), b = minus_inf();
        if (of.rows > 0) {
            // Groups of whole places of every lane: from the registers, group after group.
            float a1 = minus_inf(), b1 = minus_inf();
            int g = 0, left = of.rows;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float v = by_group[i], less = fminf(v, a1);
                a1 = fmaxf(v, a1);
                b1 = fmaxf(less, b1);
                if (--left > 0) continue;
                const float top = warp_max(a1);
                const bool is = lane == __ffs(__ballot_sync(ALL, a1 == top)) - 1;
                const float next = p.group_sum == 2 ? warp_max(is ? b1 : a1) : minus_inf();
                if (lane == g) {
                    a = top;
                    b = next;
                }
                ++g;
                left = of.rows;
                a1 = b1 = minus_inf();
            }
        } else {
            largest_two<float>(p.groups, of.size, of.log_lanes, choices, a, b);
            if ((lane & ((1 << of.log_lanes) - 1)) != 0) a = minus_inf();
        }
        unsigned keep = best_groups<float>(p, a, b, 2.0f * tol, near, last);
        if (near != 0) {
            // what of the groups' largest may be in their values
            int n = 0;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float least = __shfl_sync(ALL, last, of.home[i]) - tol;
                const int e = lane + 32 * i;
                const bool in = e < p.E && (near >> of.home[i] & 1) && by_group[i] >= least && by_group[i] > minus_inf();
                const unsigned all = __ballot_sync(ALL, in);
                const int at = n + __popc(all & ((1u << lane) - 1));
                if (in && at < 32) buffer[at] = {__int_as_float(of.home[i]), e};
                n += __popc(all);
            }
            if (n <= 32) {
                __syncwarp();
                const Candidate c = buffer[max(min(lane, n - 1), 0)];
                const double sum = softmax ? exact_sum(p, row, m) : 1.0;
                keep = exact_groups(p, keep, near, lane < n, __float_as_int(c.key), exact_choice(p, row, c.expert, m, sum));
                __syncwarp();
            } else {
                sure = false;
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (!(keep >> of.home[i] & 1)) key[i] = minus_inf();
    }

    // The bound: the wanted number of lanes have a key that is not below it.
    float k = key[0], bound = minus_inf();
#pragma unroll
    for (int i = 1; i < V; ++i) k = fmaxf(k, key[i]);
    for (int left = p.top + biased; left > 0;) {     // (with a bias the next best has to be looked at too)
        bound = warp_max(k);
        if (bound == minus_inf()) break;
        const bool is = k == bound;
        left -= __popc(__ballot_sync(ALL, is));
        if (is) k = minus_inf();
    }
    if (biased) bound -= 1.01f * tol;
    bound = fmaxf(bound, -0x1.fffffep127f);          // (not what is masked)
    int n = 0;
    const unsigned below = (1u << lane) - 1;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const unsigned all = __ballot_sync(ALL, key[i] >= bound);
        // (where they are more than 32 the buffer is not read)
        if (key[i] >= bound) buffer[(n + __popc(all & below)) & 31] = {key[i], lane + 32 * i};
        n += __popc(all);
    }
    int mine = -1;
    if (n <= 32) {
        // ranked: candidates lie in the order of their experts
        __syncwarp();
        Candidate c = {minus_inf(), -1};
        if (lane < n) c = buffer[lane];
        int rank = 0;
        for (int j = 0; j < n; ++j) {
            const float other = __shfl_sync(ALL, c.key, j);
            rank += other > c.key || (other == c.key && j < lane);
        }
        __syncwarp();
        if (lane < n) buffer[rank] = c;
        __syncwarp();
        if (lane < n) c = buffer[lane];
        if (lane < min(n, p.top)) mine = c.expert;
        if (biased) {
            // Neighbours that are nearer than the error, and not the same logit and bias,
            // make the order unsure: down to the first behind the last chosen, or
            // behind those that are equal to it.
            const float last = __shfl_sync(ALL, c.key, p.top - 1), before = __shfl_up_sync(ALL, c.key, 1);
            const int expert = __shfl_up_sync(ALL, c.expert, 1);
            bool wrong = false;
            if (lane > 0 && lane < n && (lane <= p.top || before == last) && !(before - c.key > tol))
                wrong = load_any(p.logits, row + expert, p.type) != load_any(p.logits, row + c.expert, p.type) ||
                        p.bias[expert] != p.bias[c.expert];
            if (__any_sync(ALL, wrong) && sure) {
                const double sum = softmax ? exact_sum(p, row, m) : 1.0;
                const double exact = exact_choice(p, row, max(c.expert, 0), m, sum);
                rank = 0;
                for (int j = 0; j < n; ++j) {
                    const double other = __shfl_sync(ALL, exact, j);
                    const int of_other = __shfl_sync(ALL, c.expert, j);
                    rank += other > exact || (other == exact && of_other < c.expert);
                }
                __syncwarp();
                if (lane < n) buffer[rank] = c;
                __syncwarp();
                if (lane < min(n, p.top)) mine = buffer[lane].expert;
            }
        }
    } else {
        // One after the other.
        int last = -1;
        float before = 0.0f;
        for (int j = 0; sure && j < p.top; ++j) {
            float now;
            const int e = take_best<V>(key, now);
            if (e < 0) break;
            if (biased && j > 0 && !(before - now > tol))
                sure = load_any(p.logits, row + e, p.type) == load_any(p.logits, row + last, p.type) && p.bias[e] == p.bias[last];
            if (lane == j) mine = e;
            before = now;
            last = e;
        }
        if (biased && sure && last >= 0) {           // what is left and not apart from the last has to be the same too
            const float x = load_any(p.logits, row + last, p.type), y = p.bias[last];
            bool wrong = false;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = lane + 32 * i;         // (read again: this is seldom run)
                if (key[i] > minus_inf() && !(before - key[i] > tol))
                    wrong = wrong || load_any(p.logits, row + e, p.type) != x || p.bias[e] != y;
            }
            sure = !__any_sync(ALL, wrong);
        }
    }
    if (!sure) mine = choose_exactly<V>(p, row, reinterpret_cast<double *>(scratch + SCRATCH));

    // Weights: scores of the chosen, from their logits.  (The fast division is off by 2
    // units; its divisors are far from 2^126, where it ends.)
    const bool on = mine >= 0;
    const float x = on ? load_any(p.logits, row + mine, p.type) : minus_inf();
    float s;
    if (!p.normalise) {
        if (softmax) {
            float z = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) z += expf(l[i] - m);
            s = __fdividef(expf(x - m), warp_sum(z));
        } else {
            s = sigmoid<true>(x);
        }
        weight = on ? p.scale * s : 0.0f;
    } else {
        // What the scores have in common cancels: the chosen experts' own
        // softmax; of sigmoids the exponential of the largest logit where that is below 0, or
        // their sum might be 0 in FP32.
        const float top = warp_max(x);
        s = !on ? 0.0f : softmax ? expf(x - top) : sigmoid<true>(x, fminf(top, 0.0f));
        const float sum = warp_sum(s);
        weight = on ? p.scale * __fdividef(s, sum) : 0.0f;
    }
    return mine;
}

// ------------------------------------------------------------------- plan

// Warps that rank a chunk's slots, each with counts of its own: as many as 32 KB hold.
__host__ __device__ constexpr int rank_warps(int E, int most)
{
    return E * most <= 8192 ? most : E * 16 <= 8192 && most >= 16 ? 16 : 8;
}
__host__ __device__ constexpr int sort_ints(int E, int most) { return 2 * E + 64 + rank_warps(E, most) * E; }

// The slots lo .. hi - 1 into the plan.  total[e], before[e] (shared): how many
// slots have expert e in all, and before lo.  NT threads, all of them; `room`: the
// rest of sort_ints.
template <int NT>
__device__ void rank_slots(const int32_t *experts, int lo, int hi, int slots, int E, const Plan &plan,
                           int *total, const int *before, int *room)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, ranking = rank_warps(E, NT / 32);
    int *sums = room, *start = room + 64;            // start[w][e]: the next place of warp w's slots of e
    int from, to;
    slots_of_warp(lo, hi, ranking, warp, from, to);
    // (the first slots of each lane, which are all there are of most chunks, are asked for once)
    const int early = from + lane < to ? experts[from + lane] : -1;
    for (int i = tid; i < ranking * E; i += NT) start[i] = 0;
    __syncthreads();
    for (int i = from + lane; i < to; i += 32) {
        const int e = i == from + lane ? early : experts[i];
        if ((unsigned)e < (unsigned)E) atomicAdd(&start[warp * E + e], 1);
    }
    // total becomes its running sum: where each expert begins
    int carried = 0;
    for (int base = 0; base < E; base += NT) {
        const int e = base + tid, n = e < E ? total[e] : 0;
        int v = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(ALL, v, d);
            if (lane >= d) v += o;
        }
        if (lane == 31) sums[warp] = v;
        __syncthreads();
        int s = lane < NT / 32 ? sums[lane] : 0;
        const int all = __reduce_add_sync(ALL, s), lower = __reduce_add_sync(ALL, lane < warp ? s : 0);
        if (e < E) total[e] = carried + lower + v - n;
        carried += all;
        __syncthreads();
    }
    for (int e = tid; e < E; e += NT) {
        int next = total[e] + before[e];
        if (blockIdx.x == 0) plan.offsets[e] = total[e];
#pragma unroll 8
        for (int w = 0; w < ranking; ++w) {
            const int n = start[w * E + e];
            start[w * E + e] = next;
            next += n;
        }
    }
    if (blockIdx.x == 0 && tid == 0) plan.offsets[E] = carried;
    __syncthreads();
    for (int i = from; i < to; i += 32) {
        const int slot = i + lane;
        const int e = i == from ? early : slot < to ? experts[slot] : -1;
        const bool on = (unsigned)e < (unsigned)E;
        const unsigned peers = __match_any_sync(ALL, on ? e : -1);
        int place = -1;
        if (on) place = start[warp * E + e] + __popc(peers & ((1u << lane) - 1));
        __syncwarp();
        if (on && (peers >> lane) == 1u) start[warp * E + e] = place + 1;       // the last of its peers
        __syncwarp();
        if (slot < to) plan.position[slot] = place;
        if (on) plan.source[place] = slot;
    }
    uint32_t first, step;
    behind_rows(carried, blockIdx.x, gridDim.x, NT, tid, first, step);
    for (uint32_t r = first; r < (uint32_t)slots; r += step) plan.source[r] = -1;
}

template <int V, int NT>
__global__ void __launch_bounds__(NT) route_kernel(const __grid_constant__ RouteArgs p, int scratch_bytes, int32_t *counts)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    extern __shared__ __align__(16) unsigned char shared[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    unsigned char *scratch = shared + warp * scratch_bytes;
    int *count = reinterpret_cast<int *>(shared + (NT / 32) * scratch_bytes);
    const bool planned = p.plan.offsets != nullptr;
    if (planned) {
        for (int e = tid; e < 2 * p.E; e += NT) count[e] = 0;       // and, of one chunk, those before it: none
        __syncthreads();
    }
    int from, to;
    chunk_of(p.T, gridDim.x, blockIdx.x, from, to);
    const Experts<V> of = experts_of<V>(p);
    float l[V], next[V];
    auto load = [&](int t) {
        const long long row = t * p.ld + lane;
        if (p.type == 2) {
#pragma unroll
            for (int i = 0; i < V; ++i) next[i] = lane + 32 * i < p.E ? load_any(p.logits, row + 32 * i, 2) : minus_inf();
        } else if (p.type == 1) {
#pragma unroll
            for (int i = 0; i < V; ++i) next[i] = lane + 32 * i < p.E ? load_any(p.logits, row + 32 * i, 1) : minus_inf();
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) next[i] = lane + 32 * i < p.E ? load_any(p.logits, row + 32 * i, 0) : minus_inf();
        }
    };
    if (from + warp < to) load(from + warp);
    for (int t = from + warp; t < to; t += NT / 32) {
#pragma unroll
        for (int i = 0; i < V; ++i) l[i] = next[i];
        if (t + NT / 32 < to) load(t + NT / 32);
        float weight;
        const int e = choose<V>(p, t * p.ld, l, of, scratch, weight);
        if (lane < p.top) {
            p.experts[(long long)t * p.top + lane] = e;
            p.weights[(long long)t * p.top + lane] = weight;
            if (planned && e >= 0) atomicAdd(&count[e], 1);
        }
        __syncwarp();
    }
    if (!planned) return;
    __syncthreads();
    if (gridDim.x > 1) {
        for (int e = tid; e < p.E; e += NT) counts[(long long)blockIdx.x * p.E + e] = count[e];
        return;
    }
    rank_slots<NT>(p.experts, 0, p.T * p.top, p.T * p.top, p.E, p.plan, count, count + p.E, count + 2 * p.E);
}

// ----------------------------------------------------- four tokens of a warp

// For up to 256 experts, eight of them a token: eight lanes, a team, have a token.  A
// token's instructions are then mostly those of its logits, 4 W a lane, four
// neighbouring ones of every 32 (W pieces); what goes over lanes, and each
// instruction of it, serves four tokens.  Steps as in choose: groups from
// registers by halving (lane q has piece q's two largest at the end), a bound from the
// largest of sixteenths of the experts, and a ranking of what passes.  What
// FP32 cannot decide, the warp does together, one token after the other.
// (16 warps of 128 registers: four values of every piece stay in them from the scores to the
// ranking.  One CTA an SM is said to the compiler, or it may spill to 64 for a second: two of 16
// experts of 8192 tokens, with the gradient, 11.8 and 12.9 us.)
constexpr int TEAM_THREADS = 512, TEAM_TOP = 8;
constexpr int TEAM_BUFFER = 33;                      // 32 candidates, padded

__host__ __device__ constexpr int keys_pitch(int w) { return 4 * w + 4; }           // floats of a lane
__host__ __device__ constexpr int team_bytes(int w) { return 32 * keys_pitch(w) * 4 + 2 * 4 * TEAM_BUFFER * 8; }   // of a warp
static_assert(SCRATCH + 8 * (256 + 8) <= 32 * keys_pitch(8) * 4 && SCRATCH + 8 * (32 + 1) <= 32 * keys_pitch(1) * 4, "a token's choices");

template <class F>
__device__ __forceinline__ float over_team(float v, F f)
{
#pragma unroll
    for (int d = 4; d > 0; d >>= 1) v = f(v, __shfl_xor_sync(ALL, v, d));
    return v;
}
__device__ __forceinline__ float team_max(float v) { return over_team(v, [](float a, float b) { return fmaxf(a, b); }); }
__device__ __forceinline__ float team_sum(float v) { return over_team(v, [](float a, float b) { return a + b; }); }

__device__ __forceinline__ void merge_two(float &a, float &b, float a2, float b2)
{
    b = fmaxf(fminf(a, a2), fmaxf(b, b2));
    a = fmaxf(a, a2);
}

// Four neighbouring logits.
__device__ __forceinline__ void load_four(const void *x, long long i, int type, float *v)
{
    if (type == 2) {
        const float4 a = *reinterpret_cast<const float4 *>(static_cast<const float *>(x) + i);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        return;
    }
    const uint2 a = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(x) + i);
    float2 lo, hi;
    if (type == 1) {
        lo = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&a.x));
        hi = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&a.y));
    } else {
        lo = __half22float2(*reinterpret_cast<const __half2 *>(&a.x));
        hi = __half22float2(*reinterpret_cast<const __half2 *>(&a.y));
    }
    v[0] = lo.x, v[1] = lo.y, v[2] = hi.x, v[3] = hi.y;
}

// A whole warp's way, for what is left: many equal choices, biases of +inf.
template <int V>
__device__ __noinline__ int choose_alone(const RouteArgs &p, long long row, unsigned char *scratch, float *weight)
{
    const int lane = threadIdx.x & 31;
    const Experts<V> of = experts_of<V>(p);
    float l[V];
#pragma unroll
    for (int i = 0; i < V; ++i) l[i] = lane + 32 * i < p.E ? load_any(p.logits, row + lane + 32 * i, p.type) : minus_inf();
    return choose<V>(p, row, l, of, scratch, *weight);
}

// Groups whose values are nearer than FP32 tells (bits of `near`, and of `keep` the
// best so far, at their first pieces): the best, or nothing when more than 32 experts
// matter for that.  `last`: at lane g the smallest choice in group g's value.  The choices as
// route_team_kernel forms them.
__device__ __noinline__ bool settle_groups(const RouteArgs &p, long long row, unsigned &keep, unsigned near, float last, float m,
                                           float largest, float tol, int rows, uint64_t *buffer)
{
    const int lane = threadIdx.x & 31;
    const bool softmax = p.score == SCORE_SOFTMAX;
    int n = 0;
#pragma unroll 1
    for (int i = 0; 32 * i < p.E; ++i) {
        const int home = i & ~(rows - 1), e = lane + 32 * i;
        const float least = __shfl_sync(ALL, last, home) - tol;
        if (!(near >> home & 1)) continue;
        const float x = load_any(p.logits, row + e, p.type);
        float s = softmax ? __expf(x - m) * largest : __fdividef(1.0f, 1.0f + __expf(-x));
        if (p.bias != nullptr) s += p.bias[e];
        const bool in = x > minus_inf() && s >= least && s > minus_inf();
        const unsigned all = __ballot_sync(ALL, in);
        const int at = n + __popc(all & ((1u << lane) - 1));
        if (in && at < 32) buffer[at] = (uint64_t)home << 32 | (uint32_t)e;
        n += __popc(all);
    }
    if (n == 0 || n > 32) return false;
    __syncwarp();
    const uint64_t c = buffer[min(lane, n - 1)];
    const double sum = softmax ? exact_sum(p, row, m) : 1.0;
    keep = exact_groups(p, keep, near, lane < n, (int)(c >> 32), exact_choice(p, row, (int)(uint32_t)c, m, sum));
    __syncwarp();
    return true;
}

// The order of n <= 32 ranked candidates once more, by their exact choices.
__device__ __noinline__ void settle_order(const RouteArgs &p, long long row, int n, float m, uint64_t *sorted)
{
    const int lane = threadIdx.x & 31;
    const double sum = p.score == SCORE_SOFTMAX ? exact_sum(p, row, m) : 1.0;
    const uint64_t c = sorted[min(lane, n - 1)];
    const int expert = (int)~(uint32_t)c;
    const double exact = exact_choice(p, row, expert, m, sum);
    int rank = 0;
#pragma unroll 1
    for (int j = 0; j < n; ++j) {
        const double other = __shfl_sync(ALL, exact, j);
        const int of_other = __shfl_sync(ALL, expert, j);
        rank += other > exact || (other == exact && of_other < expert);
    }
    __syncwarp();
    if (lane < n) sorted[rank] = c;
    __syncwarp();
}

template <int W>
__global__ void __launch_bounds__(TEAM_THREADS, 1) route_team_kernel(const __grid_constant__ RouteArgs p, int32_t *counts)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    extern __shared__ __align__(16) unsigned char shared[];
    constexpr int WARPS = TEAM_THREADS / 32, N = 4 * W;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, team = lane >> 3, q = lane & 7;
    unsigned char *const scratch = shared + warp * team_bytes(W);
    float *const keys = reinterpret_cast<float *>(scratch) + lane * keys_pitch(W);
    uint64_t *const buffers = reinterpret_cast<uint64_t *>(scratch + 32 * keys_pitch(W) * 4);
    uint64_t *const buffer = buffers + team * TEAM_BUFFER, *const sorted = buffer + 4 * TEAM_BUFFER;
    float *const biases = reinterpret_cast<float *>(shared + WARPS * team_bytes(W));
    int *const count = reinterpret_cast<int *>(biases + 32 * W);
    const bool planned = p.plan.offsets != nullptr, biased = p.bias != nullptr, grouped = p.groups > 1;
    const bool by_score = biased || (grouped && p.group_sum == 2), softmax = p.score == SCORE_SOFTMAX;
    if (planned)
        for (int e = tid; e < 2 * p.E; e += TEAM_THREADS) count[e] = 0;
    for (int e = tid; e < 32 * W; e += TEAM_THREADS) biases[e] = biased && e < p.E ? p.bias[e] : 0.0f;
    __syncthreads();
    float most = 0.0f;                               // as in experts_of
    for (int i = 0; i < W; ++i) {
        const float b = biases[lane + 32 * i];
        if (b != minus_inf()) most = b == b ? fmaxf(most, fabsf(b)) : -minus_inf();
    }
    most = warp_max(most);
    int from, to;
    chunk_of(p.T, gridDim.x, blockIdx.x, from, to);
    const unsigned mates = 0xffu << (8 * team);
    const int rows = grouped ? p.E / p.groups / 32 : 1;              // pieces of a group, a power of two
#pragma unroll 1
    for (int first = from + 4 * warp; first < to; first += 4 * WARPS) {
        const int t = min(first + team, to - 1);
        const bool real = first + team < to;
        const long long row = t * p.ld;
        float l[N], v[N];                            // logits; what groups, then experts go by
#pragma unroll
        for (int i = 0; i < W; ++i) {
            if (32 * i + 4 * q < p.E) {
                load_four(p.logits, row + 32 * i + 4 * q, p.type, l + 4 * i);
            } else {
                l[4 * i] = l[4 * i + 1] = l[4 * i + 2] = l[4 * i + 3] = minus_inf();
            }
        }
        float m = l[0], tol = 0.0f, largest = 1.0f, z = 1.0f;
        bool nan = false, sure = true;
#pragma unroll
        for (int j = 1; j < N; ++j) m = fmaxf(m, l[j]);
        m = team_max(m == m ? m : minus_inf());
        if (by_score) {
            // (scores and the bound of their error as in choose; the sum has as many additions)
            if (softmax) {
                float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    v[j] = __expf(l[j] - m);
                    sum[j % 4] += v[j];
                }
                largest = __fdividef(1.0f, team_sum((sum[0] + sum[1]) + (sum[2] + sum[3])));
#pragma unroll
                for (int j = 0; j < N; ++j) v[j] *= largest;
                tol = largest * 0x1.8p-18f;
            } else {
#pragma unroll
                for (int j = 0; j < N; ++j) v[j] = __fdividef(1.0f, 1.0f + __expf(-l[j]));
                largest = m < -80.0f ? 0.0f : __fdividef(1.0f, 1.0f + __expf(-m));
                tol = largest * (12.0f + 2.4f * fmaxf(-m, 0.0f)) * 0x1p-23f;
            }
            tol += 0x1p-22f * (largest + most) + 0x1p-120f;
            sure = tol < 1.0f;
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const float4 b = *reinterpret_cast<const float4 *>(biases + 32 * i + 4 * q);
                v[4 * i] += b.x;
                v[4 * i + 1] += b.y;
                v[4 * i + 2] += b.z;
                v[4 * i + 3] += b.w;
            }
#pragma unroll
            for (int j = 0; j < N; ++j) {
                if (l[j] == minus_inf()) v[j] = minus_inf();
                nan = nan || v[j] != v[j];
            }
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j) {
                v[j] = l[j];
                nan = nan || l[j] != l[j];
            }
        }
        if (softmax && !p.normalise) {
            float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int j = 0; j < N; ++j) sum[j % 4] += expf(l[j] - m);
            z = team_sum((sum[0] + sum[1]) + (sum[2] + sum[3]));
        }
        // (a NaN, for softmax +inf as well; a padding token, without a logit)
        nan = (__ballot_sync(ALL, nan || (softmax && m == -minus_inf())) & mates) != 0;
        const bool usual = real && !nan && m > minus_inf();

        if (grouped) {
            float a[W], b[W];
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const float h0 = fmaxf(v[4 * i], v[4 * i + 1]), h1 = fmaxf(v[4 * i + 2], v[4 * i + 3]);
                const float l0 = fminf(v[4 * i], v[4 * i + 1]), l1 = fminf(v[4 * i + 2], v[4 * i + 3]);
                a[i] = fmaxf(h0, h1);
                b[i] = fmaxf(fminf(h0, h1), fmaxf(l0, l1));
            }
#pragma unroll
            for (int d = W / 2; d > 0; d >>= 1)      // a half of the pieces for each half of the lanes
#pragma unroll
                for (int i = 0; i < d; ++i) {
                    const bool up = q & d;
                    const float a2 = __shfl_xor_sync(ALL, up ? a[i] : a[i + d], d), b2 = __shfl_xor_sync(ALL, up ? b[i] : b[i + d], d);
                    a[i] = up ? a[i + d] : a[i];
                    b[i] = up ? b[i + d] : b[i];
                    merge_two(a[i], b[i], a2, b2);
                }
#pragma unroll
            for (int d = W; d < 8; d <<= 1) merge_two(a[0], b[0], __shfl_xor_sync(ALL, a[0], d), __shfl_xor_sync(ALL, b[0], d));
            for (int d = 1; d < rows; d <<= 1) merge_two(a[0], b[0], __shfl_xor_sync(ALL, a[0], d), __shfl_xor_sync(ALL, b[0], d));
            // lane q: piece q % W's group, whose home is the lane of its first piece
            const bool both = p.group_sum == 2 && b[0] > minus_inf();
            const float value = both ? a[0] + b[0] : a[0], last = both ? b[0] : a[0];
            const bool is = q < W && (q & (rows - 1)) == 0 && a[0] > minus_inf();
            const uint32_t own = is ? ordered(value) : 0;
            int rank = 0;
#pragma unroll
            for (int d = 1; d < 8; ++d) {
                const uint32_t other = __shfl_sync(ALL, own, q + d, 8);
                rank += other > own || (other == own && q + d >= 8);
            }
            const unsigned kept = __ballot_sync(ALL, is && rank < p.top_groups);
            const unsigned worst = __ballot_sync(ALL, is && rank == p.top_groups - 1) & mates;
            const unsigned next = __ballot_sync(ALL, is && rank == p.top_groups) & mates;
            const float w = __shfl_sync(ALL, value, __ffs(worst | 1u << 31) - 1), r = __shfl_sync(ALL, value, __ffs(next | 1u << 31) - 1);
            const float tol2 = 2.0f * tol;
            const bool close = by_score && usual && sure && next != 0 && !(w - r > tol2);
            const unsigned near = __ballot_sync(ALL, close && is && (rank < p.top_groups ? value - r <= tol2 : w - value <= tol2));
            unsigned keep = kept >> (8 * team) & 0xffu;
            if (near != 0) {
#pragma unroll 1
                for (int f = 0; f < 4; ++f) {
                    const unsigned of = near >> (8 * f) & 0xffu;
                    if (of == 0) continue;
                    unsigned found = kept >> (8 * f) & 0xffu;
                    const bool done = settle_groups(p, __shfl_sync(ALL, row, 8 * f), found, of, __shfl_sync(ALL, last, 8 * f + q),
                                                    __shfl_sync(ALL, m, 8 * f), __shfl_sync(ALL, largest, 8 * f),
                                                    __shfl_sync(ALL, tol, 8 * f), rows, buffers);
                    if (team == f) {
                        keep = found;
                        sure = sure && done;
                    }
                }
            }
            for (int d = 1; d < rows; d <<= 1) keep |= keep << d;    // all pieces of a group
#pragma unroll
            for (int j = 0; j < N; ++j) {
                if (!biased) v[j] = l[j];
                if (!(keep >> (j / 4) & 1)) v[j] = minus_inf();
            }
        }

        // The bound: of the team's 16 parts, two of each lane, as many have a value
        // that is not below it as are wanted.
        float h0 = fmaxf(v[0], v[1]), h1 = fmaxf(v[2], v[3]);
#pragma unroll
        for (int i = 1; i < W; ++i) {
            h0 = fmaxf(h0, fmaxf(v[4 * i], v[4 * i + 1]));
            h1 = fmaxf(h1, fmaxf(v[4 * i + 2], v[4 * i + 3]));
        }
        int above0 = h1 > h0, above1 = h0 > h1;
#pragma unroll
        for (int d = 1; d < 8; ++d) {
            const float o0 = __shfl_sync(ALL, h0, q + d, 8), o1 = __shfl_sync(ALL, h1, q + d, 8);
            above0 += (o0 > h0) + (o1 > h0);
            above1 += (o0 > h1) + (o1 > h1);
        }
        const int want = p.top + biased;             // (with a bias the next best has to be looked at too)
        float bound = over_team(fminf(above0 < want ? h0 : -minus_inf(), above1 < want ? h1 : -minus_inf()),
                                [](float x, float y) { return fminf(x, y); });
        if (biased) bound -= 1.01f * tol;
        bound = fmaxf(bound, -0x1.fffffep127f);      // (not what is masked)
        unsigned pass = 0;
#pragma unroll
        for (int j = 0; j < N; ++j) pass |= v[j] >= bound ? 1u << j : 0u;
#pragma unroll
        for (int i = 0; i < W; ++i) *reinterpret_cast<float4 *>(keys + 4 * i) = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        if (!usual) pass = 0;
        const int mine_pass = __popc(pass);
        int at = mine_pass;
#pragma unroll
        for (int d = 1; d < 8; d <<= 1) {
            const int o = __shfl_up_sync(ALL, at, d, 8);
            if (q >= d) at += o;
        }
        int n = __shfl_sync(ALL, at, 7, 8);
        at -= mine_pass;
        if (n > 32) {
            sure = false;
            pass = 0;
            n = 0;
        }
        // candidates: their keys' order above, the complement of the expert below
        for (; pass != 0; pass &= pass - 1, ++at) {
            const int j = __ffs(pass) - 1;
            buffer[at] = (uint64_t)ordered(keys[j]) << 32 | (uint32_t)~(32 * (j >> 2) + 4 * q + (j & 3));
        }
        __syncwarp();
        const int longest = (int)__reduce_max_sync(ALL, (unsigned)n);
        for (int base = 0; base < longest; base += 16) {
            const uint64_t c0 = base + q < n ? buffer[base + q] : ~0ull, c1 = base + q + 8 < n ? buffer[base + q + 8] : ~0ull;
            int rank0 = 0, rank1 = 0;
            for (int j = 0; j < longest; ++j) {
                const uint64_t other = j < n ? buffer[j] : 0;
                rank0 += other > c0;
                rank1 += other > c1;
            }
            if (base + q < n) sorted[rank0] = c0;
            if (base + q + 8 < n) sorted[rank1] = c1;
        }
        __syncwarp();
        if (biased) {
            // Neighbours nearer than the error, and not the same logit and bias: as in choose.
            bool wrong = false;
            const uint32_t edge = p.top - 1 < n ? (uint32_t)(sorted[p.top - 1] >> 32) : 0;
            for (int r = q + 1; r < n; r += 8) {
                const uint64_t one = sorted[r - 1], two = sorted[r];
                const uint32_t k1 = (uint32_t)(one >> 32), k2 = (uint32_t)(two >> 32);
                if ((r <= p.top || k1 == edge) && !(value_of(k1) - value_of(k2) > tol)) {
                    const int e1 = (int)~(uint32_t)one, e2 = (int)~(uint32_t)two;
                    wrong = wrong || load_any(p.logits, row + e1, p.type) != load_any(p.logits, row + e2, p.type) || biases[e1] != biases[e2];
                }
            }
            const unsigned any = __ballot_sync(ALL, wrong && sure);
            if (any != 0) {
#pragma unroll 1
                for (int f = 0; f < 4; ++f)
                    if (any >> (8 * f) & 0xffu)
                        settle_order(p, __shfl_sync(ALL, row, 8 * f), __shfl_sync(ALL, n, 8 * f), __shfl_sync(ALL, m, 8 * f),
                                     buffers + (4 + f) * TEAM_BUFFER);
            }
        }
        int mine = q < min(n, p.top) ? (int)~(uint32_t)sorted[q] : -1;

        // Weights, as in choose.
        const bool on = mine >= 0;
        const float x = on ? load_any(p.logits, row + mine, p.type) : minus_inf();
        float weight;
        if (!p.normalise) {
            const float s = softmax ? __fdividef(expf(x - m), z) : sigmoid<true>(x);
            weight = on ? p.scale * s : 0.0f;
        } else {
            const float top = team_max(x);
            float s = 0.0f;
            if (on) s = softmax ? expf(x - top) : sigmoid<true>(x, fminf(top, 0.0f));
            const float sum = team_sum(s);
            weight = on ? p.scale * __fdividef(s, sum) : 0.0f;
        }
        if (nan) {
            mine = q < p.top ? q : -1;
            weight = __int_as_float(0x7fffffff);
        }
        const unsigned left = __ballot_sync(ALL, usual && !sure);
        if (left != 0) {
#pragma unroll 1
            for (int f = 0; f < 4; ++f) {
                if (!(left >> (8 * f) & 0xffu)) continue;
                float w;
                __syncwarp();
                const int e = choose_alone<W>(p, __shfl_sync(ALL, row, 8 * f), scratch, &w);
                __syncwarp();
                const int e8 = __shfl_sync(ALL, e, q);
                const float w8 = __shfl_sync(ALL, w, q);
                if (team == f) {
                    mine = e8;
                    weight = w8;
                }
            }
        }
        if (real && q < p.top) {
            p.experts[(long long)t * p.top + q] = mine;
            p.weights[(long long)t * p.top + q] = weight;
            if (planned && mine >= 0) atomicAdd(&count[mine], 1);
        }
        __syncwarp();
    }
    if (!planned) return;
    __syncthreads();
    if (gridDim.x > 1) {
        for (int e = tid; e < p.E; e += TEAM_THREADS) counts[(long long)blockIdx.x * p.E + e] = count[e];
        return;
    }
    rank_slots<TEAM_THREADS>(p.experts, 0, p.T * p.top, p.T * p.top, p.E, p.plan, count, count + p.E, count + 2 * p.E);
}

__global__ void __launch_bounds__(SORT_THREADS)
    count_kernel(int T, int E, int top, const int32_t *experts, int32_t *counts)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    extern __shared__ __align__(16) unsigned char shared[];
    int *count = reinterpret_cast<int *>(shared);
    for (int e = threadIdx.x; e < E; e += SORT_THREADS) count[e] = 0;
    __syncthreads();
    int from, to;
    chunk_of(T, gridDim.x, blockIdx.x, from, to);
    for (int i = from * top + threadIdx.x; i < to * top; i += SORT_THREADS) {
        const int e = experts[i];
        if ((unsigned)e < (unsigned)E) atomicAdd(&count[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += SORT_THREADS) counts[(long long)blockIdx.x * E + e] = count[e];
}

// counts == nullptr: one chunk, counted here.
__global__ void __launch_bounds__(SORT_THREADS)
    sort_kernel(int T, int E, int top, const int32_t *experts, Plan plan, const int32_t *counts, int *err)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    extern __shared__ __align__(16) unsigned char shared[];
    int *total = reinterpret_cast<int *>(shared), *before = total + E;
    const int tid = threadIdx.x;
    for (int e = tid; e < 2 * E; e += SORT_THREADS) total[e] = 0;
    __syncthreads();
    int from, to;
    chunk_of(T, gridDim.x, blockIdx.x, from, to);
    from *= top;
    to *= top;
    bool bad = false;
    if (counts == nullptr) {
        for (int i = from + tid; i < to; i += SORT_THREADS) {
            const int e = experts[i];
            if ((unsigned)e < (unsigned)E) atomicAdd(&total[e], 1);
        }
    } else {
        // a row of counts per chunk: several threads per column, a part of the rows each
        const int parts = max(SORT_THREADS / E, 1), part = tid / E;
        if (part < parts)
            for (int e = tid - part * E; e < E; e += SORT_THREADS) {
                int all = 0, lower = 0;
#pragma unroll 32
                for (int c = part; c < (int)gridDim.x; c += parts) {
                    const int n = counts[(long long)c * E + e];
                    all += n;
                    lower += c < (int)blockIdx.x ? n : 0;
                }
                atomicAdd(&total[e], all);
                atomicAdd(&before[e], lower);
            }
    }
    if (err != nullptr)
        for (int i = from + tid; i < to; i += SORT_THREADS) bad = bad || experts[i] < -1 || experts[i] >= E;
    if (__syncthreads_or(bad) && tid == 0) atomicCAS(err, 0, ERR_INVALID);
    rank_slots<SORT_THREADS>(experts, from, to, T * top, E, plan, total, before, before + E);
}

// --------------------------------------------------------------- gradient

// Of the weights scale * p_j (p the scores of the chosen, normalised or not) in
// the logits.  Normalised: softmax p_j (d_j - sum p d), sigmoid that times 1 - s_j,
// zero for experts that were not chosen.  Not: softmax s_e (g_e - sum g s) with
// g_e the d of e's slots, sigmoid s_j (1 - s_j) d_j.  One pass over the logits, a
// warp per token.
template <int V>
__global__ void __launch_bounds__(256) route_grad_kernel(const RouteGradArgs p, int *err)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * 8 + (threadIdx.x >> 5);
    if (t >= p.T) return;
    const bool softmax = p.score == SCORE_SOFTMAX;
    const long long row = t * p.ld, out = t * p.ldd, slot = (long long)t * p.top + lane;
    int mine = lane < p.top ? p.experts[slot] : -1;
    const bool wrong = mine < -1 || mine >= p.E;
    if (__any_sync(ALL, wrong) && lane == 0) atomicCAS(err, 0, ERR_INVALID);
    if (wrong) mine = -1;
    const bool on = mine >= 0;
    const float d = on ? p.scale * p.d_weights[slot] : 0.0f;
    const float x = on ? load_any(p.logits, row + mine, p.type) : minus_inf();
    float l[V];
    float g = d;                                     // what the slot gives its expert's logit
    float sum = 0.0f, z = 1.0f, m = 0.0f;
    bool full = softmax && !p.normalise;             // every logit has a gradient
    if (p.normalise) {
        const float top = warp_max(x);
        float s = 0.0f;
        if (on) s = softmax ? expf(x - top) : sigmoid<false>(x, fminf(top, 0.0f));
        const float all = warp_sum(s);
        const float share = on ? s / all : 0.0f;
        const float mean = warp_sum(share * d);
        g = on ? share * (d - mean) : 0.0f;
        if (!softmax && on) g *= sigmoid<false>(-x);
    } else if (!softmax) {
        g = on ? d * sigmoid<false>(x) * sigmoid<false>(-x) : 0.0f;
    }
    if (full) {
        m = minus_inf();
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = lane + 32 * i;
            l[i] = e < p.E ? load_any(p.logits, row + e, p.type) : minus_inf();
            m = fmaxf(m, l[i]);
        }
        m = warp_max(m);
        z = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            l[i] = l[i] == minus_inf() ? 0.0f : expf(l[i] - m);
            z += l[i];
        }
        z = warp_sum(z);
        sum = warp_sum(on ? d * (expf(x - m) / z) : 0.0f);
    }
    float a[V];
#pragma unroll
    for (int i = 0; i < V; ++i) a[i] = 0.0f;
    for (int j = 0; j < p.top; ++j) {                // in order: an expert may be in several slots
        const int e = __shfl_sync(ALL, mine, j);
        const float v = __shfl_sync(ALL, g, j);
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (lane + 32 * i == e) a[i] += v;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = lane + 32 * i;
        if (e >= p.E) continue;
        float v = a[i];
        if (full) v = l[i] == 0.0f ? 0.0f : l[i] / z * (v - sum);
        store_any(p.d_logits, out + e, v, p.type);
    }
}

// ---------------------------------------------------------------- launches

template <class K, class... A>
cudaError_t go(K kernel, DeviceOnce &once, int ctas, int threads, size_t shared, cudaStream_t s, A... args)
{
    if (shared > 48 * 1024) {
        int dev = 0;
        if (cudaError_t e = cudaGetDevice(&dev)) return e;
        if (once.needed(dev)) {
            if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024))
                return e;
            once.mark(dev);
        }
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = shared;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int V, int NT>
cudaError_t route_form(const RouteArgs &p, int ctas, int32_t *counts, cudaStream_t s)
{
    // choices in FP32, or in FP64 where sums or a bias make that needed
    const int wide = p.bias != nullptr || p.group_sum == 2 ? 8 : 4;
    const int scratch = SCRATCH + (p.groups > 1 ? ((p.E + p.E / 32 + 1) * wide + 15) & ~15 : 0);
    const size_t shared = (size_t)scratch * (NT / 32) + (p.plan.offsets ? 4 * sort_ints(p.E, NT / 32) : 0);
    static DeviceOnce once;
    return go(route_kernel<V, NT>, once, ctas, NT, shared, s, p, scratch, counts);
}

template <int W>
cudaError_t team_form(const RouteArgs &p, int ctas, int32_t *counts, cudaStream_t s)
{
    const size_t shared = TEAM_THREADS / 32 * (size_t)team_bytes(W) + 128 * W + (p.plan.offsets ? 4 * sort_ints(p.E, TEAM_THREADS / 32) : 0);
    static DeviceOnce once;
    return go(route_team_kernel<W>, once, ctas, TEAM_THREADS, shared, s, p, counts);
}

// Whether route_team_kernel takes them: its logits come four at a time.
bool for_teams(const RouteArgs &p)
{
    const int rows = p.E / p.groups / 32;            // pieces of a group
    return p.E <= 256 && p.top <= TEAM_TOP && p.E % 4 == 0 && p.ld % 4 == 0 &&
           reinterpret_cast<uintptr_t>(p.logits) % (p.type == 2 ? 16 : 8) == 0 &&
           (p.groups == 1 || (p.E / p.groups % 32 == 0 && (rows & (rows - 1)) == 0));
}

int values_per_lane(int E) { return (E + 31) / 32; }

}  // namespace

// One chunk (and one kernel) for few tokens; else a CTA per SM at most, with a
// warp for each of its tokens as far as that goes.
int plan_chunks(int T, int top, bool route, int sms)
{
    if (route) return T <= 64 ? 1 : std::min((T + 31) / 32, sms);
    return (long long)T * top <= 4096 ? 1 : (int)std::min<long long>(((long long)T * top + 1023) / 1024, sms);
}

cudaError_t launch_route(const RouteArgs &p, int chunks, int32_t *counts, cudaStream_t s)
{
    const int v = values_per_lane(p.E);
    const int ctas = p.plan.offsets ? chunks : 0;
    if (for_teams(p)) {
        const int n = ctas ? ctas : (p.T + TEAM_THREADS / 8 - 1) / (TEAM_THREADS / 8);
        return v <= 1 ? team_form<1>(p, n, counts, s) : v <= 2 ? team_form<2>(p, n, counts, s) : v <= 4 ? team_form<4>(p, n, counts, s) : team_form<8>(p, n, counts, s);
    }
#define FORM(V, NT) return route_form<V, NT>(p, ctas ? ctas : (p.T + NT / 32 - 1) / (NT / 32), counts, s)
    if (ctas) {
        if (v <= 1) FORM(1, 1024);
        if (v <= 2) FORM(2, 1024);
        if (v <= 4) FORM(4, 1024);
        if (v <= 8) FORM(8, 1024);
        if (v <= 16) FORM(16, 512);
        FORM(32, 512);
    }
    if (v <= 1) FORM(1, 256);
    if (v <= 2) FORM(2, 256);
    if (v <= 4) FORM(4, 256);
    if (v <= 8) FORM(8, 256);
    if (v <= 16) FORM(16, 256);
    FORM(32, 256);
#undef FORM
}

cudaError_t launch_count(int T, int E, int top, const int32_t *experts, int chunks, int32_t *counts,
                         cudaStream_t s)
{
    static DeviceOnce once;
    return go(count_kernel, once, chunks, SORT_THREADS, 4 * (size_t)E, s, T, E, top, experts, counts);
}

cudaError_t launch_sort(int T, int E, int top, const int32_t *experts, const Plan &plan, int chunks,
                        int32_t *counts, int *err, cudaStream_t s)
{
    static DeviceOnce once;
    return go(sort_kernel, once, chunks, SORT_THREADS, 4 * (size_t)sort_ints(E, SORT_THREADS / 32), s, T, E, top, experts, plan,
              (const int32_t *)(chunks > 1 ? counts : nullptr), err);
}

cudaError_t launch_route_grad(const RouteGradArgs &p, int *err, cudaStream_t s)
{
    const int v = values_per_lane(p.E), ctas = (p.T + 7) / 8;
    static DeviceOnce once;
    auto with = [&](auto kernel) { return go(kernel, once, ctas, 256, 0, s, p, err); };
    if (v <= 1) return with(route_grad_kernel<1>);
    if (v <= 2) return with(route_grad_kernel<2>);
    if (v <= 4) return with(route_grad_kernel<4>);
    if (v <= 8) return with(route_grad_kernel<8>);
    if (v <= 16) return with(route_grad_kernel<16>);
    return with(route_grad_kernel<32>);
}

}  // namespace swg
