// k_route.cu — the router: the experts of each token with their weights, rows
// sorted by expert, and the gradient of the logits.
//
// A warp has a token, lane l the experts l, l + 32, ...  As many lanes' largest as
// experts are wanted give a bound that few others pass; those are ranked by
// comparing all with all, the lowest index of equals first.  (One after the other by
// a maximum over the warp, eight of 256 took four times the instructions.)  Without a
// bias the order of the scores is that of the logits, which
// compare exactly.  With one, or where groups are valued by a sum, the choices
// (score + bias) are formed in FP32 and compared with a bound of their error;
// where two are nearer than that, and not the same logit and bias, the token is
// decided once more in FP64.  So the choice is that of the definition, whatever
// the rounding of the exponential.
//
// Sorting is counting: every chunk of tokens counts its experts in shared memory,
// and the second kernel adds up the chunks before its own and ranks its slots
// in order.  (One chunk: the same CTA goes on, without a second kernel.)
#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

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
    const double inverse = softmax ? 1.0 / warp_sum(z) : 1.0;
#pragma unroll TOGETHER
    for (int i = 0; i < V; ++i) {
        const int e = lane + 32 * i;
        c[i] *= inverse;
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
        // Scores by the fast exponential, which is off by at most 2 + 1.2 |x| units,
        // and division (2 units).  Softmax: x = l - m, and |x| e^x is at most 0.4: 3 units
        // of the largest score for the exponential, as much for the sum's terms, 8 for
        // its 15 additions in a tree, 1 more: two choices, 2^-18 of it and a half.
        // Sigmoid: s (1 - s) (2 + 1.2 |x|) + 2 s, of the largest score 6 units, where all
        // logits are negative 1.2 |m| more.
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
        // (2^-120: scores that FP32 has no digits left for)
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
        int last = -1;
        float before = 0.0f;
        for (int j = 0; sure; ++j) {                 // one after the other, as far as that
            float now;
            const int e = take_best<V>(key, now);
            if (e < 0) break;
            const bool apart = !biased || j == 0 || before - now > tol;
            if (!apart) {
                const float x = load_any(p.logits, row + e, p.type), y = load_any(p.logits, row + last, p.type);
                sure = x == y && p.bias[e] == p.bias[last];
            }
            if (j >= p.top && apart) break;
            if (j < p.top && lane == j) mine = e;
            before = now;
            last = e;
        }
    }
    if (!sure) mine = choose_exactly<V>(p, row, reinterpret_cast<double *>(scratch + SCRATCH));

    // Weights: scores of the chosen, from their logits.  (The fast division is off by 2
    // units; its divisors are far from where it ends.)
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
            s = __fdividef(1.0f, 1.0f + expf(-x));
        }
        weight = on ? p.scale * s : 0.0f;
    } else {
        // What the scores have in common cancels: the chosen experts' own
        // softmax; of sigmoids too where all are so small that 1 + e^x is 1,
        // and their sum may be 0 in FP32.
        const float top = warp_max(x);
        if (softmax || top < -40.0f)
            s = on ? expf(x - top) : 0.0f;
        else
            s = on ? __fdividef(1.0f, 1.0f + expf(-x)) : 0.0f;
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
    const int per = ((hi - lo + ranking - 1) / ranking + 31) & ~31;
    const int from = min(lo + warp * per, hi), to = warp < ranking ? min(from + per, hi) : from;
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
    for (int r = carried + blockIdx.x * NT + tid; r < slots; r += gridDim.x * NT) plan.source[r] = -1;
}

// The tokens of chunk c of n.
__device__ __forceinline__ void chunk_of(int T, int n, int c, int &from, int &to)
{
    const int per = (T + n - 1) / n;
    from = min((long long)c * per, (long long)T);
    to = min(from + per, T);
}

template <int V, int NT>
__global__ void __launch_bounds__(NT) route_kernel(const RouteArgs p, int scratch_bytes, int32_t *counts)
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
        if (on) s = softmax || top < -40.0f ? expf(x - top) : 1.0f / (1.0f + expf(-x));
        const float all = warp_sum(s);
        const float share = on ? s / all : 0.0f;
        const float mean = warp_sum(share * d);
        g = on ? share * (d - mean) : 0.0f;
        if (!softmax && on) g *= 1.0f / (1.0f + expf(x));
    } else if (!softmax) {
        const float s = 1.0f / (1.0f + expf(-x));
        g = on ? d * s * (1.0f / (1.0f + expf(x))) : 0.0f;
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
