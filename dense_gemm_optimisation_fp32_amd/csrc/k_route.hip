// Kernel translation unit: the routing kernels and their launches.
#include "expert_launch.hpp"
#include "route.hpp"

namespace gemmf32 {

__global__ __launch_bounds__(kRouteThreads) void route_place_kernel(RouteArgs a)
{
    extern __shared__ int lds[];
    int *const base = lds, *const carry = lds + a.groups, *const held = lds + (a.groups + 2) / 2 * 2;
    int *const totals = held;   // until the places are counted
    const int parts = gridDim.x;
    // Threads share an expert where there are more threads than experts, each
    // every share-th workgroup's counts, eight loads at a time.
    const int share = max(1, kRouteThreads / a.groups);
    for (int e = threadIdx.x; e < a.groups; e += kRouteThreads) base[e] = totals[e] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < a.groups * share; i += kRouteThreads) {
        const int e = i % a.groups;
        int before = 0, all = 0;
        for (int b0 = i / a.groups; b0 < parts; b0 += 8 * share) {
            int n[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int b = b0 + u * share;
                n[u] = b < parts ? a.counts[(long long)b * a.groups + e] : 0;
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                all += n[u];
                before += b0 + u * share < (int)blockIdx.x ? n[u] : 0;
            }
        }
        atomicAdd(base + e, before);
        atomicAdd(totals + e, all);
    }
    __syncthreads();
    route_offsets(a, totals, carry, blockIdx.x == gridDim.x - 1);
    for (int e = threadIdx.x; e < a.groups; e += kRouteThreads) base[e] += totals[e];
    __syncthreads();
    if (a.groups <= 512) route_place<kRouteWaves>(a, blockIdx.x * kRouteTokens, base, held);
    else route_place<kRouteFewWaves>(a, blockIdx.x * kRouteTokens, base, held);
}

namespace {

template <class E, int V>
int launch_v(const RouteArgs &a, bool grad, hipStream_t s)
{
    const int found = route_found_words(a.choices), place = route_place_words(a.groups);
    if (grad) return launch(route_grad_kernel<E, V>, (a.tokens + 15ll) / 16, kGradThreads, 0, s, a);
    if (a.tokens <= kRouteTokens)
        return launch(route_one_kernel<E, V>, 1, kRouteThreads, (a.groups + 2 + (found > place ? found : place)) * 4, s, a);
    const long long parts = (a.tokens + kRouteTokens - 1ll) / kRouteTokens;
    const int st = launch(route_choose_kernel<E, V>, parts, kRouteThreads, (a.groups + 1 + found) * 4, s, a);
    if (st != GEMM_F32_SUCCESS) return st;
    return launch(route_place_kernel, parts, kRouteThreads, (a.groups + 2 + place) * 4, s, a);
}

// The fewest experts a lane that hold them all.
template <class E>
int launch_e(const RouteArgs &a, bool grad, hipStream_t s)
{
    if (a.groups <= 16) return launch_v<E, 1>(a, grad, s);
    if (a.groups <= 32) return launch_v<E, 2>(a, grad, s);
    if (a.groups <= 64) return launch_v<E, 4>(a, grad, s);
    if (a.groups <= 128) return launch_v<E, 8>(a, grad, s);
    if (a.groups <= 256) return launch_v<E, 16>(a, grad, s);
    if (a.groups <= 512) return launch_v<E, 32>(a, grad, s);
    return launch_v<E, 64>(a, grad, s);
}

}  // namespace

int launch_route(const RouteArgs &a, bool bf16, bool grad, hipStream_t s)
{
    return bf16 ? launch_e<__bf16>(a, grad, s) : launch_e<float>(a, grad, s);
}

}  // namespace gemmf32
