// Kernel translation unit: the routing kernels and their launches.
#include "expert_launch.hpp"
#include "route.hpp"

namespace gemmf32 {

__global__ __launch_bounds__(kRouteThreads) void route_place_kernel(RouteArgs a)
{
    extern __shared__ int lds[];
    int *const base = lds, *const held = lds + a.groups, *const carry = lds + 5 * a.groups;
    int *const totals = held;   // until the places are counted
    const int parts = gridDim.x;
    // Threads share an expert where there are more threads than experts:
    // part p adds up every (threads / experts)-th workgroup's counts.
    const int share = max(1, kRouteThreads / a.groups);
    for (int e = threadIdx.x; e < a.groups; e += kRouteThreads) base[e] = totals[e] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < a.groups * share; i += kRouteThreads) {
        const int e = i % a.groups;
        int before = 0, all = 0;
        for (int b = i / a.groups; b < parts; b += share) {
            const int n = a.counts[(long long)b * a.groups + e];
            all += n;
            before += b < (int)blockIdx.x ? n : 0;
        }
        atomicAdd(base + e, before);
        atomicAdd(totals + e, all);
    }
    __syncthreads();
    route_offsets(a, totals, carry, blockIdx.x == gridDim.x - 1);
    for (int e = threadIdx.x; e < a.groups; e += kRouteThreads) base[e] += totals[e];
    __syncthreads();
    route_place(a, blockIdx.x * kRouteTokens, base, held);
}

namespace {

template <class E, int V>
void launch_v(const RouteArgs &a, bool grad, hipStream_t s)
{
    const int lds = route_lds_words(a.groups) * 4;
    if (grad) {
        route_grad_kernel<E, V><<<(a.tokens + 15) / 16, kRouteThreads, 0, s>>>(a);
    } else if (a.tokens <= kRouteTokens) {
        route_one_kernel<E, V><<<1, kRouteThreads, lds, s>>>(a);
    } else {
        const int parts = (a.tokens + kRouteTokens - 1) / kRouteTokens;
        route_choose_kernel<E, V><<<parts, kRouteThreads, a.groups * 4, s>>>(a);
        route_place_kernel<<<parts, kRouteThreads, lds, s>>>(a);
    }
}

// The fewest experts a lane that hold them all.
template <class E>
void launch_e(const RouteArgs &a, bool grad, hipStream_t s)
{
    if (a.groups <= 16) launch_v<E, 1>(a, grad, s);
    else if (a.groups <= 32) launch_v<E, 2>(a, grad, s);
    else if (a.groups <= 64) launch_v<E, 4>(a, grad, s);
    else if (a.groups <= 128) launch_v<E, 8>(a, grad, s);
    else if (a.groups <= 256) launch_v<E, 16>(a, grad, s);
    else if (a.groups <= 512) launch_v<E, 32>(a, grad, s);
    else launch_v<E, 64>(a, grad, s);
}

}  // namespace

void launch_route(const RouteArgs &a, bool bf16, bool grad, hipStream_t s)
{
    bf16 ? launch_e<__bf16>(a, grad, s) : launch_e<float>(a, grad, s);
}

}  // namespace gemmf32
