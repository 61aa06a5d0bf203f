// Routing tokens to experts: softmax over the experts' logits, the k largest,
// and the chosen (token, choice) slots sorted by expert.
//
//   choose   the `choices` largest logits of a token, equal ones by the lower
//            expert; an expert at -inf (or NaN) is never chosen, and a slot
//            that finds none gets expert -1 and weight 0.
//            weight_j = exp(x_j - max) / sum of exp(x - max) over the chosen
//            (normalize) or over all experts.
//   sort     order: slot numbers token * choices + j, stably sorted by
//            expert; offsets[e] .. offsets[e + 1] are expert e's places.  The
//            places after the last expert's hold -1.
//   grad     d logits = w (g - sum_j w_j g_j) over the experts that the
//            softmax sums over, g the slots' gradients at the chosen ones.
//
// A token is held by 16 lanes, each V neighbouring experts: four tokens a
// wavefront.  A choice is V compares, four maxima over the lanes (row
// rotations, no LDS), a ballot and V compares to strike the chosen one out.
// The lanes hold the experts in order, so the lowest lane with the largest
// value holds the lowest expert.  The chosen ones go to LDS, and the softmax is
// taken once, a lane a slot.
//
// The sort is a counting sort in two launches (one where a single workgroup
// holds every token): workgroups of kRouteTokens tokens count their experts;
// then each workgroup adds up the counts of the workgroups before it (from
// the L2 cache) and places its own slots, 64 at a time, by the lanes that hold
// the same expert.  No atomics on memory: the order is the same in every run.
// The counts that are read grow with the square of the tokens, (tokens / 128)^2 x
// experts: choose + place of 128 experts, 8 choices take 18.5 us for 32768 tokens,
// 35 for twice as many, then 77, 198 and 596 for 524288.
//
// Bound by latency: 16 wavefronts a workgroup, so that the loads and the
// chains of dependent operations of many tokens overlap.  32768 tokens, 128
// experts, 8 choices, bfloat16, choose + place + grad: 11.5 + 7.7 + 6.4 us (with
// 4 wavefronts a workgroup and the lanes' values exchanged through LDS 33 + 37 +
// 6.9; with logit and expert packed into one word, half the operations of a
// choice, 11.4 + 8.4: not what bounds it).  16 tokens, 64 experts: 4.1 us.
#pragma once

#include "mx4.hpp"

namespace gemmf32 {

constexpr int kRouteTokens = 128;      // tokens of a workgroup
constexpr int kRouteThreads = 1024;
constexpr int kRouteWaves = kRouteThreads / 64;
constexpr int kRouteFewWaves = 4;      // of them place, where the counts of all would not fit LDS
constexpr int kRouteMaxExperts = 1024;
constexpr int kRouteMaxChoices = 32;

struct RouteArgs {
    const void *logits;
    long long ld;            // elements from token to token
    float *weights;          // (tokens, choices)
    int *experts;            // (tokens, choices)
    int *offsets;            // groups + 1
    int *order;              // tokens * choices
    int *counts;             // (workgroups, groups): workspace
    int tokens, groups, choices, normalize;
    // gradient
    const float *grad;       // (tokens, choices)
    void *dlogits;           // (tokens, groups)
    long long ldd;
};

// x from the lane N places on in the row of 16.
template <int N>
__device__ __forceinline__ float row_rotate(float x)
{
    return __builtin_bit_cast(
        float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), 0x120 + N, 0xf, 0xf, true));
}

__device__ __forceinline__ float row_max(float x)
{
    x = fmaxf(x, row_rotate<8>(x));
    x = fmaxf(x, row_rotate<4>(x));
    x = fmaxf(x, row_rotate<2>(x));
    return fmaxf(x, row_rotate<1>(x));
}

__device__ __forceinline__ float row_sum(float x)
{
    x += row_rotate<8>(x);
    x += row_rotate<4>(x);
    x += row_rotate<2>(x);
    return x + row_rotate<1>(x);
}

// The V logits of a lane; absent experts, and NaN, are -inf.
template <class E, int V>
__device__ __forceinline__ void route_load(const RouteArgs &a, int token, int sub, float (&x)[V])
{
    const E *p = reinterpret_cast<const E *>(a.logits) + (long long)token * a.ld + sub * V;
    const int left = a.groups - sub * V;
    if constexpr (V % 8 == 0) {
#pragma unroll
        for (int b = 0; b < V; b += 8) {
            float v[8];
            load8(p + b, left - b, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[b + i] = b + i < left && v[i] == v[i] ? v[i] : -__builtin_inff();
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float v = i < left ? to_f32(p[i]) : -__builtin_inff();
            x[i] = v == v ? v : -__builtin_inff();
        }
    }
}

// What a choice found: the logit, and its expert or -1.
struct Choice {
    float logit;
    int expert;
};

// Chooses for the workgroup's tokens and counts the experts in LDS.  `found`
// (LDS): `choices` entries for every 16 lanes.
template <class E, int V>
__device__ __forceinline__ void route_choose(const RouteArgs &a, int first, int *counts, Choice *found)
{
    const int lane = threadIdx.x & 63, sub = lane & 15, group = lane >> 4;
    const int last = min(first + kRouteTokens, a.tokens);
    Choice *const mine = found + (threadIdx.x >> 4) * a.choices;
    for (int t0 = first + (threadIdx.x >> 6) * 4; t0 < last; t0 += kRouteThreads / 16) {
        const int token = t0 + group;
        const bool live = token < last;
        float x[V];
        route_load<E, V>(a, live ? token : last - 1, sub, x);
        float all = 0.0f, top = 0.0f;
        for (int j = 0; j < a.choices; ++j) {
            float best = x[0];
            int at = 0;
#pragma unroll
            for (int i = 1; i < V; ++i) {
                const bool more = x[i] > best;
                best = more ? x[i] : best;
                at = more ? i : at;
            }
            const float m = row_max(best);
            const bool used = m > -__builtin_inff();
            if (j == 0) {
                top = used ? m : 0.0f;
                if (!a.normalize) {
#pragma unroll
                    for (int i = 0; i < V; ++i) all += expf(x[i] - top);
                    all = row_sum(all);
                }
            }
            const unsigned long long hit = __ballot(best == m);
            const int who = __builtin_ctz((unsigned)(hit >> (16 * group)) & 0xffffu);
            if (sub == who) {
                mine[j] = Choice{m, used ? sub * V + at : -1};
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (i == at) x[i] = -__builtin_inff();
            }
        }
        wave_sync();
        // A lane a slot (two past sixteen choices).
        float w[2] = {};
        int e[2] = {-1, -1};
#pragma unroll
        for (int q = 0; q < 2; ++q)
            if (sub + 16 * q < a.choices) {
                const Choice c = mine[sub + 16 * q];
                e[q] = c.expert;
                w[q] = c.expert < 0 ? 0.0f : expf(c.logit - top);
            }
        const float total = a.normalize ? row_sum(w[0] + w[1]) : all;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int j = sub + 16 * q;
            if (live && j < a.choices) {
                const long long s = (long long)token * a.choices + j;
                a.weights[s] = e[q] < 0 ? 0.0f : w[q] / total;
                a.experts[s] = e[q];
                if (e[q] >= 0) atomicAdd(counts + e[q], 1);
            }
        }
        wave_sync();
    }
}

// Places the workgroup's slots.  `base` (LDS): where its slots of each
// expert begin; `held` (LDS): the wavefronts' own counts.  W wavefronts place.
template <int W>
__device__ __forceinline__ void route_place(const RouteArgs &a, int first, int *base, int *held)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = a.choices, last = min(first + kRouteTokens, a.tokens);
    constexpr int kPart = kRouteTokens / W;
    // A wavefront's slots, in order: those of its part of the tokens.
    const int s0 = min(first + wave * kPart, last) * c, s1 = wave < W ? min(first + (wave + 1) * kPart, last) * c : s0;
    int *const mine = held + (wave < W ? wave : 0) * a.groups;
    for (int e = threadIdx.x; e < W * a.groups; e += kRouteThreads) held[e] = 0;
    __syncthreads();
    for (int s = s0 + lane; s < s1; s += 64) {
        const int e = a.experts[s];
        if (e >= 0) atomicAdd(mine + e, 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.groups; e += kRouteThreads) {
        int at = base[e];
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const int n = held[w * a.groups + e];
            held[w * a.groups + e] = at;
            at += n;
        }
    }
    __syncthreads();
    for (int s = s0; s < s1; s += 64) {
        const int slot = s + lane;
        const int e = slot < s1 ? a.experts[slot] : -1;
        // The lanes that hold this lane's expert.
        unsigned long long same = __ballot(e >= 0);
        for (int bit = 0; (1 << bit) < a.groups; ++bit) {
            const unsigned long long ones = __ballot((e >> bit) & 1);
            same &= (e >> bit) & 1 ? ones : ~ones;
        }
        const int before = __popcll(same & ((1ull << lane) - 1));
        int at = 0;
        if (e >= 0) at = mine[e] + before;
        wave_sync();
        if (e >= 0) {
            a.order[at] = slot;
            if (before == 0) mine[e] = at + __popcll(same);
        }
        wave_sync();
    }
}

// LDS words of the kernels below: a count an expert, the placing wavefronts'
// counts, or the choices found, and one more word.
constexpr int route_waves(int groups) { return groups <= 512 ? kRouteWaves : kRouteFewWaves; }
constexpr int route_found_words(int choices) { return kRouteThreads / 16 * choices * 2; }
constexpr int route_place_words(int groups) { return route_waves(groups) * groups; }

// Exclusive sum over the experts of `totals` (LDS), into offsets, and -1 in
// the places that no slot takes (in the last workgroup).
__device__ __forceinline__ void route_offsets(const RouteArgs &a, int *totals, int *carry, bool write)
{
    // One wavefront, 64 experts at a time.
    if (threadIdx.x < 64) {
        const int lane = threadIdx.x;
        int run = 0;
        for (int b = 0; b < a.groups; b += 64) {
            const int n = b + lane < a.groups ? totals[b + lane] : 0;
            const int s = wave_inclusive_sum(n);
            if (b + lane < a.groups) {
                totals[b + lane] = run + s - n;
                if (write) a.offsets[b + lane] = run + s - n;
            }
            run += __shfl(s, 63);
        }
        if (lane == 0) {
            if (write) a.offsets[a.groups] = run;
            *carry = run;
        }
    }
    __syncthreads();
    if (write)
        for (int s = *carry + threadIdx.x; s < a.tokens * a.choices; s += kRouteThreads) a.order[s] = -1;
}

// Every token in one workgroup: choose, count, place.
template <class E, int V>
__global__ __launch_bounds__(kRouteThreads) void route_one_kernel(RouteArgs a)
{
    extern __shared__ int lds[];
    int *const base = lds, *const carry = lds + a.groups, *const held = lds + (a.groups + 2) / 2 * 2;
    for (int e = threadIdx.x; e < a.groups; e += kRouteThreads) base[e] = 0;
    __syncthreads();
    route_choose<E, V>(a, 0, base, reinterpret_cast<Choice *>(held));
    // The chosen experts are read back by other lanes of this workgroup.
    __threadfence_block();
    __syncthreads();
    route_offsets(a, base, carry, true);
    if (a.groups <= 512) route_place<kRouteWaves>(a, 0, base, held);
    else route_place<kRouteFewWaves>(a, 0, base, held);
}

// First of two launches: choose and count.
template <class E, int V>
__global__ __launch_bounds__(kRouteThreads) void route_choose_kernel(RouteArgs a)
{
    extern __shared__ int lds[];
    for (int e = threadIdx.x; e < a.groups; e += kRouteThreads) lds[e] = 0;
    __syncthreads();
    route_choose<E, V>(a, blockIdx.x * kRouteTokens, lds, reinterpret_cast<Choice *>(lds + (a.groups + 1) / 2 * 2));
    __syncthreads();
    for (int e = threadIdx.x; e < a.groups; e += kRouteThreads) a.counts[(long long)blockIdx.x * a.groups + e] = lds[e];
}

// Second: where each workgroup's slots of an expert begin, and their places.
__global__ __launch_bounds__(kRouteThreads) void route_place_kernel(RouteArgs a);

constexpr int kGradThreads = 256;

template <class E, int V>
__global__ __launch_bounds__(kGradThreads) void route_grad_kernel(RouteArgs a)
{
    // What each slot adds to its expert's gradient, for the 16 lanes that
    // hold the token.
    __shared__ Choice adds[kGradThreads / 16][kRouteMaxChoices];
    const int sub = threadIdx.x & 15;
    const int token = blockIdx.x * (kGradThreads / 16) + (threadIdx.x >> 4);
    if (token >= a.tokens) return;
    Choice *const mine = adds[threadIdx.x >> 4];
    const long long s0 = (long long)token * a.choices;
    // The slots' weights and gradients, a lane one slot (two past sixteen
    // choices); unused slots count nothing.
    float w[2] = {}, g[2] = {};
    int e[2] = {-1, -1};
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int j = sub + 16 * q;
        if (j < a.choices) {
            e[q] = a.experts[s0 + j];
            w[q] = a.weights[s0 + j];
            g[q] = e[q] >= 0 ? a.grad[s0 + j] : 0.0f;
        }
    }
    const float dot = row_sum(w[0] * g[0] + w[1] * g[1]);
#pragma unroll
    for (int q = 0; q < 2; ++q)
        if (sub + 16 * q < a.choices)
            mine[sub + 16 * q] = Choice{a.normalize ? w[q] * (g[q] - dot) : w[q] * g[q], e[q]};
    float d[V];
    if (a.normalize) {
#pragma unroll
        for (int i = 0; i < V; ++i) d[i] = 0.0f;
    } else {
        float x[V], top = -__builtin_inff(), sum = 0.0f;
        route_load<E, V>(a, token, sub, x);
#pragma unroll
        for (int i = 0; i < V; ++i) top = fmaxf(top, x[i]);
        top = row_max(top);
        top = top > -__builtin_inff() ? top : 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            x[i] = expf(x[i] - top);
            sum += x[i];
        }
        sum = row_sum(sum);
        const float each = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) d[i] = -x[i] * each * dot;
    }
    wave_sync();
    for (int j = 0; j < a.choices; ++j) {
        const Choice c = mine[j];
        const int i0 = c.expert - sub * V;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (c.expert >= 0 && i == i0) d[i] += c.logit;
    }
    E *p = reinterpret_cast<E *>(a.dlogits) + (long long)token * a.ldd + sub * V;
    const int left = a.groups - sub * V;
    if (V == 8 && left >= 8) {
        struct __attribute__((packed, aligned(sizeof(E)))) Some {
            E e[V];
        } t;
#pragma unroll
        for (int i = 0; i < V; ++i) t.e[i] = (E)d[i];
        *reinterpret_cast<Some *>(p) = t;
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i < left) p[i] = (E)d[i];
    }
}

}  // namespace gemmf32
