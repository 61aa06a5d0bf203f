// Balanced routing: scores, a bias for the choice, sets of experts.
//
//   score    s = sigmoid(x), or softmax(x) over the token's experts.
//   key      c = s + bias: what is chosen by.  An expert at x = -inf or NaN has
//            none (-inf) and is never chosen.
//   sets     groups / sets neighbouring experts each.  A set's value is the sum
//            of its two largest keys (the one it has; -inf for none); the
//            `kept` largest values stay, equal ones by the lower set.
//   choose   the `choices` largest keys of those sets, equal ones by the lower
//            expert.  weight_j = scale s_j / sum of the chosen s (normalize) or
//            scale s_j.
//   grad     sigmoid  d_j = w_j (1 - s_j) (g_j - dot)   (not normalize: no dot)
//            softmax  d_j = w_j (g_j - dot)             (not normalize: below)
//            dot = sum_j w_j g_j / scale, at the chosen experts, zero elsewhere;
//            softmax as it is: d_e = (w g at the chosen) - s_e sum_j w_j g_j.
//
// The slots are then sorted as in route.hpp, by the same kernels.
//
// Which expert is chosen goes by differences of keys: in 32 bits the last bits
// of an exponential decided one choice in about twenty thousand tokens (256
// experts).  A choice is first made in 32 bits with bounds on their errors; where
// two keys, or two sets, whose order matters are nearer than those the wavefront
// chooses again in 64 bits.  With biases that differ from expert to expert those are
// few: 1 token in 1000.  Equal keys are nearer than any bound, and logits of 16 bits
// with equal biases, or none, have many: of random ones (256 experts, 8 choices) 3 tokens
// in 10, 3 of 4 wavefronts.
//
// A token is held by LANES lanes.  A set takes a power of two of them
// (`lanes`), each `each` neighbouring experts, so that a set's two largest are
// found by exchanges between its own lanes whatever its size; the lanes hold
// the experts in order.
//
// What bounds it is the vector unit, not memory.  One MI355X, 32768 tokens of 256
// bfloat16 logits, 8 choices from 4 of 8 sets, random biases: 30 us to choose (its
// bytes would take 4), 11.4 to place; both together 41, with biases of zeros 66, without
// 62 (32-bit logits 39, 47 and 45).  With keys compared lane by lane at every choice, instead of sorted
// ones, choosing took 5 more.  5003 tokens of 60 32-bit logits, 6 choices: 13.3 and 4.7; 16 tokens of
// 64, chosen and placed in one launch: 6.4, the launch and one chain of latencies.
#pragma once

#include "route.hpp"

namespace gemmf32 {

struct BalanceArgs {
    RouteArgs route;         // (normalize as there)
    const float *bias;       // groups, or NULL
    int softmax, sets, kept;
    int lanes, each;         // lanes a set; experts a lane
    float scale;
};

constexpr int kBalanceMaxSets = 64;

// Tokens of a workgroup where there are up to kBalanceFewTokens of them (else
// kRouteTokens): a part for most CUs.
constexpr int kBalancePart = 32, kBalanceFewTokens = 8192;

// x moved between lanes by a DPP control.
template <int CTRL>
__device__ __forceinline__ double dpp64(double x)
{
    const u32x2 v = __builtin_bit_cast(u32x2, x);
    const u32x2 r = {(unsigned)__builtin_amdgcn_update_dpp(0, (int)v.x, CTRL, 0xf, 0xf, true),
                     (unsigned)__builtin_amdgcn_update_dpp(0, (int)v.y, CTRL, 0xf, 0xf, true)};
    return __builtin_bit_cast(double, r);
}

template <int CTRL>
__device__ __forceinline__ float mx_lane_f(float x)
{
    return __uint_as_float(mx_lane<CTRL>(__float_as_uint(x)));
}

// From the other half of 2 D lanes whose halves of D hold one value each (below
// 4 lanes: lane by lane).
template <int D>
__device__ __forceinline__ double other_half(double x)
{
    if constexpr (D == 1) return dpp64<0xb1>(x);
    else if constexpr (D == 2) return dpp64<0x4e>(x);
    else if constexpr (D == 4) return dpp64<0x141>(x);
    else if constexpr (D == 8) return dpp64<0x140>(x);
    else return __shfl_xor(x, D);
}

template <int D>
__device__ __forceinline__ float other_half(float x)
{
    if constexpr (D == 1) return mx_lane_f<0xb1>(x);
    else if constexpr (D == 2) return mx_lane_f<0x4e>(x);
    else if constexpr (D == 4) return mx_lane_f<0x141>(x);
    else if constexpr (D == 8) return mx_lane_f<0x140>(x);
    else return __shfl_xor(x, D);
}

__device__ __forceinline__ float larger(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ double larger(double a, double b) { return fmax(a, b); }
__device__ __forceinline__ float smaller(float a, float b) { return fminf(a, b); }
__device__ __forceinline__ double smaller(double a, double b) { return fmin(a, b); }

template <int LANES, class K>
__device__ __forceinline__ K lanes_max(K x)
{
    x = larger(x, other_half<1>(x));
    x = larger(x, other_half<2>(x));
    x = larger(x, other_half<4>(x));
    x = larger(x, other_half<8>(x));
    if constexpr (LANES == 64) {
        x = larger(x, other_half<16>(x));
        x = larger(x, other_half<32>(x));
    }
    return x;
}

template <int LANES, class K>
__device__ __forceinline__ K lanes_sum(K x)
{
    x += other_half<1>(x);
    x += other_half<2>(x);
    x += other_half<4>(x);
    x += other_half<8>(x);
    if constexpr (LANES == 64) {
        x += other_half<16>(x);
        x += other_half<32>(x);
    }
    return x;
}

// The two largest of a set, as its lanes join.
template <class K>
struct Two {
    K first, second;

    __device__ __forceinline__ void add(K x)
    {
        second = larger(second, smaller(first, x));
        first = larger(first, x);
    }
    template <int D>
    __device__ __forceinline__ void join()
    {
        const K f = other_half<D>(first), s = other_half<D>(second);
        second = larger(smaller(first, f), larger(second, s));
        first = larger(first, f);
    }
};

__device__ __forceinline__ double sigmoid64(double x) { return 1.0 / (1.0 + exp(-x)); }

// How many sets of the token come before this lane's: those in other lanes of
// the row, N lanes on and further.
template <int N, class K>
__device__ __forceinline__ int sets_before(K value, int set, int lanes)
{
    int n = 0;
    if constexpr (N < 16) {
        if (N % lanes == 0) {
            K v;
            if constexpr (sizeof(K) == 8) v = dpp64<0x120 + N>(value);
            else v = mx_lane_f<0x120 + N>(value);
            const int u = __builtin_amdgcn_update_dpp(0, set, 0x120 + N, 0xf, 0xf, true);
            n = v > value || (v == value && u < set) ? 1 : 0;
        }
        n += sets_before<N + 1>(value, set, lanes);
    }
    return n;
}

// The lane's keys.  x: its logits, `count` of them from
// expert e0 on; top: the token's largest (softmax).  Returns twice the error that a
// 32-bit score may have.
//
// Errors of 32-bit keys.  sigmoid: e = 2^(-x log2 e) is off by (1.5 |x| + 2)
// 2^-24 of itself, the sum and the reciprocal add 1.5 2^-23: the score's error is
// below 2^-21 (|x| s (1 - s) stays below 0.3).  softmax: e^(x - top) as much, the sum of
// up to 32 of them a lane and of 6 lane by lane 38 2^-24 more: below 2^-18 of the
// score, which is at most 1 / sum.  The bias adds a rounding, 2^-24 of the key.
template <int LANES, int V>
__device__ __forceinline__ float balance_keys(const BalanceArgs &b, const float (&x)[V], float top, int e0, int count,
                                              float (&c)[V])
{
    float near = 0x1p-20f;
    if (b.softmax) {
        float sum = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            c[i] = __builtin_amdgcn_exp2f((x[i] - top) * 1.44269504088896341f);
            sum += x[i] == x[i] ? c[i] : 0.0f;
        }
        sum = lanes_sum<LANES>(sum);
        const float each = __builtin_amdgcn_rcpf(sum);
        near = 0x1p-17f * each;
#pragma unroll
        for (int i = 0; i < V; ++i) c[i] *= each;
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) c[i] = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x[i] * -1.44269504088896341f));
    }
    // (Opaque: the biases would else be held in registers for all tokens.)
    int eb = e0;
    asm volatile("" : "+v"(eb));
    if (b.bias) {
        if constexpr (V % 8 == 0) {
            // (One by one, each with its bound: 36.6 us instead of 30 for 32768 tokens of 256.)
#pragma unroll
            for (int i = 0; i < V; i += 8) {
                float v[8];
                load8(b.bias + eb + i, count - i, v);
#pragma unroll
                for (int j = 0; j < 8; ++j) c[i + j] += v[j];
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) c[i] += i < count ? b.bias[eb + i] : 0.0f;
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = x[i] > -__builtin_inff() && c[i] == c[i] ? c[i] : -__builtin_inff();
    return near;
}

// The same in 64 bits, one after the other: each takes a logit's place in the
// registers.
template <int LANES, int V>
__device__ __forceinline__ float balance_keys(const BalanceArgs &b, const float (&x)[V], float top, int e0, int count,
                                              double (&c)[V])
{
    double sum = 1.0;
    if (b.softmax) {
        sum = 0.0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            sum += x[i] == x[i] ? exp((double)x[i] - (double)top) : 0.0;
            __builtin_amdgcn_sched_barrier(0);
        }
        sum = lanes_sum<LANES>(sum);
    }
    int eb = e0;
    asm volatile("" : "+v"(eb));
#pragma unroll
    for (int i = 0; i < V; ++i) {
        double s = b.softmax ? exp((double)x[i] - (double)top) / sum : sigmoid64((double)x[i]);
        if (b.bias) s += (double)(i < count ? b.bias[eb + i] : 0.0f);
        c[i] = x[i] > -__builtin_inff() && s == s ? s : -__builtin_inf();
        __builtin_amdgcn_sched_barrier(0);
    }
    return 0.0f;
}

// How many sets of the token come before this lane's, whose two largest keys are
// `two`, joined over its lanes.
template <class K, int LANES>
__device__ __forceinline__ int balance_sets(const BalanceArgs &b, Two<K> &two, int set, K &value)
{
    const K none = -__builtin_inff();
    if (b.lanes > 1) two.template join<1>();
    if (b.lanes > 2) two.template join<2>();
    if (b.lanes > 4) two.template join<4>();
    if (b.lanes > 8) two.template join<8>();
    if constexpr (LANES == 64) {
        if (b.lanes > 16) two.template join<16>();
        if (b.lanes > 32) two.template join<32>();
    }
    value = two.second > none ? two.first + two.second : two.first;
    if constexpr (LANES == 16) return sets_before<1>(value, set, b.lanes);
    int before = 0;
    for (int u = 0; u < b.sets; ++u) {
        const K v = __shfl(value, u * b.lanes);
        before += v > value || (v == value && u < set) ? 1 : 0;
    }
    return before;
}

// The lane of the token's that holds its largest, among those with `hit`.
template <int LANES>
__device__ __forceinline__ int first_lane(bool hit, int group)
{
    const unsigned long long lanes = __ballot(hit);
    if constexpr (LANES == 16) return __builtin_ctz((unsigned)(lanes >> (16 * group)) & 0xffffu);
    else return __builtin_ctzll(lanes);
}

template <int LANES>
__device__ __forceinline__ int lanes_max_int(int x)
{
    x = max(x, (int)mx_lane<0xb1>((unsigned)x));
    x = max(x, (int)mx_lane<0x4e>((unsigned)x));
    x = max(x, (int)mx_lane<0x141>((unsigned)x));
    x = max(x, (int)mx_lane<0x140>((unsigned)x));
    if constexpr (LANES == 64) {
        x = max(x, __shfl_xor(x, 16));
        x = max(x, __shfl_xor(x, 32));
    }
    return x;
}

__device__ __forceinline__ void order(int &a, int &b)
{
    const int most = max(a, b);
    b = min(a, b);
    a = most;
}

// Eight in falling order: nineteen comparisons, and twelve of two sorted runs,
// the second turned round.
__device__ __forceinline__ void sort8(int *p)
{
    order(p[0], p[2]), order(p[1], p[3]), order(p[4], p[6]), order(p[5], p[7]);
    order(p[0], p[4]), order(p[1], p[5]), order(p[2], p[6]), order(p[3], p[7]);
    order(p[0], p[1]), order(p[2], p[3]), order(p[4], p[5]), order(p[6], p[7]);
    order(p[2], p[4]), order(p[3], p[5]), order(p[1], p[4]), order(p[3], p[6]);
    order(p[1], p[2]), order(p[3], p[4]), order(p[5], p[6]);
}

__device__ __forceinline__ void merge8(int *p)
{
    order(p[0], p[4]), order(p[1], p[5]), order(p[2], p[6]), order(p[3], p[7]);
    order(p[0], p[2]), order(p[1], p[3]), order(p[4], p[6]), order(p[5], p[7]);
    order(p[0], p[1]), order(p[2], p[3]), order(p[4], p[5]), order(p[6], p[7]);
}

// A key and its place in the lane as one number in the keys' order: the key's bits
// but the last four, and 15 - i.  Dropping them takes a key down, by up to 15 units in
// its last place: below 2^-19 of what is left.  So of two, the larger one's packed key
// less the smaller one's is at most 2^-19 of the latter more than the keys' difference.
constexpr int kNoKey = (int)0x80000000, kLeastKey = (int)0x80800000;

__device__ __forceinline__ int packed_key(float c, int i)
{
    const int u = __float_as_int(c);
    return c > -__builtin_inff() ? ((u ^ (u >> 31 & 0x7fffffff)) & ~15) | (15 - i) : kNoKey;
}

__device__ __forceinline__ float unpacked_key(int p)
{
    const int s = p & ~15;
    return p < kLeastKey ? -__builtin_inff() : __int_as_float(s ^ (s >> 31 & 0x7fffffff));
}

// One token's choice, its experts to `mine`, for up to eight choices or up to eight
// experts a lane: every lane sorts its keys once (minima and maxima of integers, no
// comparison waits for another lane) and keeps the eight largest and the ninth, and
// a choice takes the largest of the lanes' first.  False: keys or sets whose order
// decides are nearer than their errors.
template <int LANES, int V>
__device__ __forceinline__ bool balance_pick_packed(const BalanceArgs &b, const float (&x)[V], float top, int sub, int group,
                                                    int set, int e0, int count, int *mine)
{
    static_assert(V <= 16, "places of four bits");
    constexpr int KEPT = V < 8 ? V : 8;
    int q[KEPT + 1];
    float near;
    {
        float c[V];
        near = balance_keys<LANES, V>(b, x, top, e0, count, c);
        int p[V < 8 ? 8 : V];
#pragma unroll
        for (int i = 0; i < (V < 8 ? 8 : V); ++i) p[i] = i < V ? packed_key(c[i < V ? i : 0], i) : kNoKey;
        sort8(p);
        q[KEPT] = kNoKey;
        if constexpr (V == 16) {
            sort8(p + 8);
            int rest = kNoKey;
#pragma unroll
            for (int i = 0; i < 8; ++i) rest = max(rest, min(p[i], p[15 - i]));
#pragma unroll
            for (int i = 0; i < 8; ++i) p[i] = max(p[i], p[15 - i]);
            merge8(p);
            q[KEPT] = rest;
        }
#pragma unroll
        for (int i = 0; i < KEPT; ++i) q[i] = p[i];
    }
    bool sure = true;
    const float none = -__builtin_inff();
    if (b.kept < b.sets) {
        Two<float> two{unpacked_key(q[0]), unpacked_key(q[1])};
        float value;
        const int before = balance_sets<float, LANES>(b, two, set, value);
        const bool out = before >= b.kept;
        const float least = -lanes_max<LANES>(out ? none : -value), most = lanes_max<LANES>(out ? value : none);
        const float size = lanes_max<LANES>(fabsf(two.first > none ? two.first : 0.0f) + fabsf(two.second > none ? two.second : 0.0f));
        sure = most == none || least - most > 2.0f * near + 0x1.2p-19f * size;      // (with the sums' rounding)
        if (out)
#pragma unroll
            for (int i = 0; i <= KEPT; ++i) q[i] = kNoKey;
    }
    float last = none;
    for (int j = 0;; ++j) {
        const int m = lanes_max_int<LANES>(q[0]);
        const bool used = m >= kLeastKey;
        const float key = unpacked_key(m);
        if (j > 0) sure = sure && (!used || last - key > near + 0x1.1p-19f * fabsf(key));
        last = key;
        if (j == b.route.choices) break;
        if (sub == first_lane<LANES>(q[0] == m, group)) {
            mine[j] = used ? e0 + 15 - (m & 15) : -1;
#pragma unroll
            for (int i = 0; i < KEPT; ++i) q[i] = q[i + 1];
            q[KEPT] = kNoKey;
        }
    }
    return sure;
}

// The same for any number of choices, key by key.  K: float or double, which is
// always sure.
template <class K, int LANES, int V>
__device__ __forceinline__ bool balance_pick(const BalanceArgs &b, const float (&x)[V], float top, int sub, int group, int set,
                                             int e0, int count, int *mine)
{
    constexpr bool kWide = sizeof(K) == 8;
    const K none = -__builtin_inff();
    K c[V];
    const float near = balance_keys<LANES, V>(b, x, top, e0, count, c);
    bool sure = true;
    if (b.kept < b.sets) {
        Two<K> two{none, none};
#pragma unroll
        for (int i = 0; i < V; ++i) two.add(c[i]);
        K value;
        const int before = balance_sets<K, LANES>(b, two, set, value);
        const bool out = before >= b.kept;
        if constexpr (!kWide) {
            const float least = -lanes_max<LANES>(out ? none : -value), most = lanes_max<LANES>(out ? value : none);
            // (By the keys' size, not the sums': keys of both signs cancel, their roundings do not.)
            const float size = lanes_max<LANES>(fabsf(two.first > none ? two.first : 0.0f) + fabsf(two.second > none ? two.second : 0.0f));
            sure = most == none || least - most > 2.0f * near + 0x1p-21f * size;
        }
        if (out)
#pragma unroll
            for (int i = 0; i < V; ++i) c[i] = none;
    }
    K last = none;
    for (int j = 0;; ++j) {
        K best = c[0];
        int at = 0;
#pragma unroll
        for (int i = 1; i < V; ++i) {
            const bool more = c[i] > best;
            best = more ? c[i] : best;
            at = more ? i : at;
        }
        const K m = lanes_max<LANES>(best);
        const bool used = m > none;
        if constexpr (!kWide) {
            if (j > 0) sure = sure && (!used || last - m > near + 0x1p-22f * (fabsf(last) + fabsf(m)));
            last = m;
        }
        if (j == b.route.choices) break;
        if (sub == first_lane<LANES>(best == m, group)) {
            mine[j] = used ? e0 + at : -1;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i == at) c[i] = none;
        }
        if (kWide && j + 1 == b.route.choices) break;     // (what comes next only bounds errors)
    }
    return sure;
}

// `count` logits from p on, -inf past them.
template <class E, int V>
__device__ __forceinline__ void balance_load(const E *p, int count, float (&x)[V])
{
    if constexpr (V % 8 == 0) {
#pragma unroll
        for (int i = 0; i < V; i += 8) {
            float v[8];
            load8(p + i, count - i, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[i + j] = i + j < count ? v[j] : -__builtin_inff();
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = i < count ? to_f32(p[i]) : -__builtin_inff();
    }
}

// Chooses for the workgroup's TOKENS tokens and counts the experts in LDS.
// `found` (LDS): `choices` experts for every LANES lanes.
template <class E, int LANES, int V, int THREADS, int TOKENS>
__device__ __forceinline__ void balance_choose(const BalanceArgs &b, int first, int *counts, int *found)
{
    const RouteArgs &a = b.route;
    constexpr int PER = 64 / LANES;                       // tokens a wavefront
    const int lane = threadIdx.x & 63, sub = lane % LANES, group = lane / LANES;
    const int last = min(first + TOKENS, a.tokens);
    const int size = a.groups / b.sets;                   // experts of a set
    const int set = sub / b.lanes, inner = sub % b.lanes * b.each;
    const int e0 = set * size + inner;
    const int count = set < b.sets ? max(0, min(b.each, size - inner)) : 0;
    int *const mine = found + (threadIdx.x / LANES) * a.choices;
    for (int t0 = first + (threadIdx.x >> 6) * PER; t0 < last; t0 += THREADS / LANES) {
        const int token = t0 + group;
        const bool live = token < last;
        const E *const row = reinterpret_cast<const E *>(a.logits) + (long long)(live ? token : last - 1) * a.ld;
        float x[V];
        balance_load<E, V>(row + e0, count, x);
        float top = 0.0f;
        if (b.softmax) {
            top = -__builtin_inff();
#pragma unroll
            for (int i = 0; i < V; ++i) top = fmaxf(top, x[i]);
            top = lanes_max<LANES>(top);
            top = top > -__builtin_inff() ? top : 0.0f;
        }
        bool sure;
        if constexpr (V > 16) sure = balance_pick<float, LANES, V>(b, x, top, sub, group, set, e0, count, mine);
        else if (V <= 8 || a.choices <= 8) sure = balance_pick_packed<LANES, V>(b, x, top, sub, group, set, e0, count, mine);
        else sure = balance_pick<float, LANES, V>(b, x, top, sub, group, set, e0, count, mine);
        if (__ballot(!sure)) balance_pick<double, LANES, V>(b, x, top, sub, group, set, e0, count, mine);
        // (Opaque, and the logits loaded again: what follows from these would be held in
        // registers through the choice.)
        int again = live ? token : last - 1;
        float scale = b.scale;
        asm volatile("" : "+v"(again), "+v"(scale));
        const E *const logits = reinterpret_cast<const E *>(a.logits) + (long long)again * a.ld;
        double sum = 1.0;
        if (b.softmax && !a.normalize) {
            sum = 0.0;
            balance_load<E, V>(logits + e0, count, x);
#pragma unroll
            for (int i = 0; i < V; ++i) sum += x[i] == x[i] ? exp((double)x[i] - (double)top) : 0.0;
            sum = lanes_sum<LANES>(sum);
        }
        wave_sync();
        // A lane a slot (two past LANES choices); their scores again.
        double w[2] = {};
        int e[2] = {-1, -1};
#pragma unroll
        for (int q = 0; q < 2; ++q)
            if (sub + LANES * q < a.choices) {
                e[q] = mine[sub + LANES * q];
                if (e[q] >= 0) {
                    const double v = (double)to_f32(logits[e[q]]);
                    w[q] = b.softmax ? exp(v - (double)top) / sum : sigmoid64(v);
                }
            }
        const double total = a.normalize ? lanes_sum<LANES>(w[0] + w[1]) : 1.0;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int j = sub + LANES * q;
            if (live && j < a.choices) {
                const long long s = (long long)token * a.choices + j;
                a.weights[s] = w[q] > 0.0 ? (float)(w[q] / total * (double)scale) : 0.0f;
                a.experts[s] = e[q];
                if (e[q] >= 0) atomicAdd(counts + e[q], 1);
            }
        }
        wave_sync();
    }
}

// LDS words for the choices found.
constexpr int balance_found_words(int lanes, int threads, int choices) { return threads / lanes * choices; }

// Every token in one workgroup: choose, count, place.
template <class E, int LANES, int V>
__global__ __launch_bounds__(kRouteThreads) void balance_one_kernel(BalanceArgs b)
{
    extern __shared__ int lds[];
    const RouteArgs &a = b.route;
    int *const base = lds, *const carry = lds + a.groups, *const held = lds + a.groups + 2;
    for (int e = threadIdx.x; e < a.groups; e += kRouteThreads) base[e] = 0;
    __syncthreads();
    balance_choose<E, LANES, V, kRouteThreads, kRouteTokens>(b, 0, base, held);
    // The chosen experts are read back by other lanes of this workgroup.
    __threadfence_block();
    __syncthreads();
    route_offsets(a, base, carry, true);
    if (a.groups <= 512) route_place<kRouteWaves>(a, 0, base, held);
    else route_place<kRouteFewWaves>(a, 0, base, held);
}

// First of two launches: choose and count.
template <class E, int LANES, int V, int THREADS, int TOKENS>
__global__ __launch_bounds__(THREADS) void balance_choose_kernel(BalanceArgs b)
{
    extern __shared__ int lds[];
    const RouteArgs &a = b.route;
    for (int e = threadIdx.x; e < a.groups; e += THREADS) lds[e] = 0;
    __syncthreads();
    balance_choose<E, LANES, V, THREADS, TOKENS>(b, blockIdx.x * TOKENS, lds, lds + a.groups);
    __syncthreads();
    for (int e = threadIdx.x; e < a.groups; e += THREADS) a.counts[(long long)blockIdx.x * a.groups + e] = lds[e];
}

// Second, of parts that route_place_kernel does not have.
template <int TOKENS>
__global__ __launch_bounds__(kRouteThreads) void balance_place_kernel(RouteArgs a)
{
    extern __shared__ int lds[];
    route_place_part<TOKENS>(a, lds);
}

// Floats of a token's row: whole 16-byte pieces, rows on different banks.
__device__ __host__ constexpr int balance_grad_row(int groups) { return (groups + 3) / 4 * 4 + 4; }

// A token's gradient is put together in LDS: what every expert has
// (0, or softmax's share), then the chosen ones' on top, a lane a slot; then it is
// stored 16 bytes a lane.  Bound by memory: 32768 tokens of 256 bfloat16 logits, 8
// choices: 6.8 us, 5 TB/s read and written.
template <class E>
__global__ __launch_bounds__(kGradThreads) void balance_grad_kernel(BalanceArgs b)
{
    extern __shared__ float all[];
    const RouteArgs &a = b.route;
    const int sub = threadIdx.x & 15;
    const int token = blockIdx.x * (kGradThreads / 16) + (threadIdx.x >> 4);
    if (token >= a.tokens) return;
    const int row = balance_grad_row(a.groups);
    float *const mine = all + (threadIdx.x >> 4) * row;
    const long long s0 = (long long)token * a.choices;
    const E *const logits = reinterpret_cast<const E *>(a.logits) + (long long)token * a.ld;
    float w[2] = {}, g[2] = {};
    int e[2] = {-1, -1};
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int j = sub + 16 * q;
        if (j < a.choices) {
            e[q] = a.experts[s0 + j];
            if (e[q] < 0 || e[q] >= a.groups) e[q] = -1;
            w[q] = e[q] >= 0 ? a.weights[s0 + j] : 0.0f;
            g[q] = e[q] >= 0 ? a.grad[s0 + j] : 0.0f;
        }
    }
    const float dot = row_sum(w[0] * g[0] + w[1] * g[1]);        // scale times the mean gradient
    if (b.softmax && !a.normalize) {
        float top = -__builtin_inff(), sum = 0.0f;
        for (int i = sub; i < a.groups; i += 16) {
            const float v = to_f32(logits[i]);
            mine[i] = v;
            top = fmaxf(top, v);
        }
        top = row_max(top);
        top = top > -__builtin_inff() ? top : 0.0f;
        for (int i = sub; i < a.groups; i += 16) {
            const float v = mine[i], p = v == v ? expf(v - top) : 0.0f;
            mine[i] = p;
            sum += p;
        }
        sum = row_sum(sum);
        const float each = sum > 0.0f ? -dot / sum : 0.0f;
        for (int i = sub; i < a.groups; i += 16) mine[i] *= each;
    } else {
        for (int i = sub * 4; i < row; i += 64) *reinterpret_cast<f32x4 *>(mine + i) = f32x4{};
    }
    wave_sync();
    const float mean = a.normalize ? dot / b.scale : 0.0f;
#pragma unroll
    for (int q = 0; q < 2; ++q)
        if (e[q] >= 0) {
            float d = w[q] * (g[q] - mean);
            // 1 - s = sigmoid(-x), without the difference of two near ones.
            if (!b.softmax) d /= 1.0f + expf(to_f32(logits[e[q]]));
            mine[e[q]] += d;
        }
    wave_sync();
    E *const p = reinterpret_cast<E *>(a.dlogits) + (long long)token * a.ldd;
    constexpr int N = 16 / sizeof(E);                       // elements of a 16-byte store
    struct __attribute__((packed, aligned(sizeof(E)))) Some {
        E e[N];
    };
    for (int i = sub * N; i < a.groups; i += 16 * N) {
        if (i + N <= a.groups) {
            Some t;
#pragma unroll
            for (int j = 0; j < N; ++j) t.e[j] = (E)mine[i + j];
            *reinterpret_cast<Some *>(p + i) = t;
        } else {
            for (int j = i; j < a.groups; ++j) p[j] = (E)mine[j];
        }
    }
}

}  // namespace gemmf32
