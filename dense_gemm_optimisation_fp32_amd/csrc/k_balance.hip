// Kernel translation unit: balanced routing and its launches.
#include "balance.hpp"
#include "expert_launch.hpp"

namespace gemmf32 {

namespace {

template <class E, int LANES, int V>
int launch_choose(const BalanceArgs &b, hipStream_t s)
{
    const RouteArgs &a = b.route;
    // Half the threads where a lane's keys would not fit the registers of all.
    constexpr int THREADS = V > 16 ? 512 : kRouteThreads;
    const int found = balance_found_words(LANES, THREADS, a.choices), place = route_place_words(a.groups);
    // One launch, of one workgroup, as long as it holds all tokens, for it needs no
    // workspace.  Measured, us, 8 choices, one launch / two (parts of 32 tokens): 64 experts, 16
    // tokens 6.8 / 8.5, 64 9.7 / 10.4, 96 11.6 / 10.4, 128 15.0 / 10.4; 256 experts, 16 tokens
    // 10.9 / 16.1, 48 24 / 27, 64 30 / 27, 128 57 / 27; 512 experts 16 9.8 / 14.4, 64 25.7 / 24.6,
    // 128 49 / 27.
    if constexpr (V <= 16)
        if (a.tokens <= kRouteTokens)
            return launch(balance_one_kernel<E, LANES, V>, 1, kRouteThreads,
                          (a.groups + 2 + (found > place ? found : place)) * 4, s, b);
    if (a.tokens <= kBalanceFewTokens) {
        constexpr int FEW = kBalancePart * LANES < 512 ? kBalancePart * LANES : 512;
        const long long parts = (a.tokens + kBalancePart - 1ll) / kBalancePart;
        const int st = launch(balance_choose_kernel<E, LANES, V, FEW, kBalancePart>, parts, FEW,
                              (a.groups + balance_found_words(LANES, FEW, a.choices)) * 4, s, b);
        if (st != GEMM_F32_SUCCESS) return st;
        return launch(balance_place_kernel<kBalancePart>, parts, kRouteThreads, (a.groups + 2 + place) * 4, s, a);
    }
    const long long parts = (a.tokens + kRouteTokens - 1ll) / kRouteTokens;
    const int st = launch(balance_choose_kernel<E, LANES, V, THREADS, kRouteTokens>, parts, THREADS, (a.groups + found) * 4, s, b);
    if (st != GEMM_F32_SUCCESS) return st;
    return launch(route_place_kernel, parts, kRouteThreads, (a.groups + 2 + place) * 4, s, a);
}

// Lanes of a set: the largest power of two that leaves every set its own.
int lanes_of(int sets, int all)
{
    int n = 1;
    while (2 * n * sets <= all) n *= 2;
    return n;
}

template <class E>
int launch_choose_e(BalanceArgs b, hipStream_t s)
{
    const int size = b.route.groups / b.sets;
    if (b.sets <= 16) {
        b.lanes = lanes_of(b.sets, 16);
        b.each = (size + b.lanes - 1) / b.lanes;
        if (b.each <= 1) return launch_choose<E, 16, 1>(b, s);
        if (b.each <= 2) return launch_choose<E, 16, 2>(b, s);
        if (b.each <= 4) return launch_choose<E, 16, 4>(b, s);
        if (b.each <= 8) return launch_choose<E, 16, 8>(b, s);
        // (Few tokens: a wavefront each, in one workgroup.)
        if (b.each <= 16 && b.route.tokens > kRouteTokens) return launch_choose<E, 16, 16>(b, s);
    }
    b.lanes = lanes_of(b.sets, 64);
    b.each = (size + b.lanes - 1) / b.lanes;
    if (b.each <= 8) return launch_choose<E, 64, 8>(b, s);
    if (b.each <= 16) return launch_choose<E, 64, 16>(b, s);
    return launch_choose<E, 64, 32>(b, s);
}

template <class E>
int launch_grad_e(const BalanceArgs &b, hipStream_t s)
{
    return launch(balance_grad_kernel<E>, (b.route.tokens + 15ll) / 16, kGradThreads,
                  (size_t)16 * balance_grad_row(b.route.groups) * 4, s, b);
}

}  // namespace

int launch_balance(const BalanceArgs &b, bool bf16, bool grad, hipStream_t s)
{
    if (grad) return bf16 ? launch_grad_e<__bf16>(b, s) : launch_grad_e<float>(b, s);
    return bf16 ? launch_choose_e<__bf16>(b, s) : launch_choose_e<float>(b, s);
}

}  // namespace gemmf32
