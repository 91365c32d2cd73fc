// splitk_route.cu -- the router's choice: each token's `top` largest logits and
// their softmax shares, and the logits' gradient.
//
// A warp takes a token, V logits to a lane (logit 32 i + lane).  Each is turned into a
// whole number that rises with it, so that a choice is a maximum: `top` times the
// largest is taken (the lowest index of equal ones) and struck out.  -inf has the
// number 0 and is never taken.  The first choice is the row's maximum m, so the shares
// follow without another pass: s_j = exp(l_j - m) / sum exp(l - m), the sum over all G
// or over the chosen.
//
// To find and strike out one of V logits in each lane costs about 5 V comparisons and
// selections a choice, at half the rate of other operations.  So where there are a few
// choices of many logits, the lanes' maxima are taken first: the top-th largest of
// them is a bound that at least `top` logits reach and few others.  Those that reach it
// are moved to a lane each, in the order of their indexes, and a lane counts how many
// are before its own (8192 tokens, 256 experts, top 8: 5.4 us, by choices alone 10.8).
//
// Gradient, with p = softmax over all G (or over the chosen; p = 0 elsewhere) and
// c = sum_j p_{e_j} d_j:   dl_i = p_i (sum_{j: e_j = i} d_j - c).
//
// Bound by latency: neither memory (12 to 14% of its rate at 8192 tokens of 256 F32) nor
// the issue of instructions (68% for the choice, 57% for the gradient) is used up; what a
// token waits for is `top` warp-wide maxima one behind another and the trees of its sums.

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ptx.cuh"
#include "rows.cuh"
#include "splitk_internal.h"

namespace splitk {
namespace {

constexpr int kRouteThreads = 256;

// A number that rises with the logit; -inf has 0, and a NaN the largest.  (x + 0: -0 is
// +0, the two zeros are equal, and any NaN is the positive one.)
constexpr uint32_t kBelow = 0x007fffffu;   // what -inf would have
__device__ __forceinline__ uint32_t key_of(float x)
{
    const uint32_t u = __float_as_uint(__fadd_rn(x, 0.f));
    return (u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u)) - kBelow;
}
__device__ __forceinline__ float logit_of(uint32_t k)
{
    const uint32_t u = k + kBelow;
    return __uint_as_float(u >> 31 ? u ^ 0x80000000u : ~u);
}

__device__ __forceinline__ float sum_of(float x)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}

// The largest key of a warp and the lowest index that has it.
__device__ __forceinline__ void best_of(uint32_t &key, int &at)
{
    const uint32_t k = __reduce_max_sync(0xffffffffu, key);
    at = static_cast<int>(__reduce_min_sync(0xffffffffu, key == k ? static_cast<uint32_t>(at) : 0xffffffffu));
    key = k;
}

// Choices that the bound is worth finding for (8192 tokens of 256 F32, by choices and with
// the bound: top 2 4.3 and 4.5 us, 3 4.7 and 4.7, 4 5.6 and 4.9, 16 13.2 and 7.4, 17 13.6 and
// 8.0, 24 18.4 and 20.9, 32 23.6 and 26.5; of 64 experts 3.2 and 3.8 for 4, 5.8 and 6.2 for 16;
// of 1024 14 and 14 for 3, 43 and 19 for 16, 79 and 100 for 32).
constexpr int kFewest = 4, kMost = 16;

// Lane j keeps the j-th choice.
template <typename T, int V>
__global__ void __launch_bounds__(kRouteThreads) route_kernel(const T *logits, int *experts, float *shares, int64_t M, int G,
                                                              int top, int chosen_only)
{
    __shared__ uint2 reached[kRouteThreads / 32][32];
    ptx::launch_dependents();
    ptx::grid_dependency_wait();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int64_t m = static_cast<int64_t>(blockIdx.x) * (kRouteThreads / 32) + warp;
    if (m >= M) return;
    const T *const row = logits + m * G;
    float x[V];
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = i * 32 + lane < G ? static_cast<float>(row[i * 32 + lane]) : -INFINITY;
    uint32_t key[V], own = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        key[i] = key_of(x[i]);
        own = max(own, key[i]);
    }
    uint32_t one = own;     // the lane's logit where it has one alone
    int one_at = lane;
    // Logits that have lanes of their own; more than 32: none have.  (8192 tokens, 16
    // experts, top 2: 2.7 us by choices, 5.2 by counting.)
    int count = V == 1 && 4 * top >= G ? G : 33;
    uint32_t first = 0;
    if (V > 1 && top >= kFewest && top <= kMost) {
        uint32_t bound = 0, left = own;
        for (int j = 0; j < top; ++j) {
            bound = __reduce_max_sync(0xffffffffu, left);
            if (j == 0) first = bound;
            if (left == bound) left = 0;   // (equal ones at once: the bound is lower then)
        }
        if (bound == 0) bound = 1;
        count = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const uint32_t there = __ballot_sync(0xffffffffu, key[i] >= bound);
            const int at = count + __popc(there & ((1u << lane) - 1u));
            if (key[i] >= bound && at < 32) reached[warp][at] = make_uint2(key[i], static_cast<uint32_t>(i * 32 + lane));
            count += __popc(there);
        }
        __syncwarp();
        if (count <= 32) {   // else many are equal
            const uint2 r = lane < count ? reached[warp][lane] : make_uint2(0u, 0u);
            one = r.x, one_at = static_cast<int>(r.y);
        }
    } else {
        first = __reduce_max_sync(0xffffffffu, own);
    }
    const float most = first ? logit_of(first) : 0.f;
    float total = 0.f;
    if (!chosen_only) {
#pragma unroll
        for (int i = 0; i < V; ++i) total += expf(x[i] - most);
        total = sum_of(total);
    }
    // the lane's choice: its place among the token's, its expert and number
    int place = lane, chosen = -1;
    uint32_t k_chosen = 0;
    if (count <= 32) {
        place = 0;
        for (int i = 0; i < count; ++i) {
            const uint32_t k = __shfl_sync(0xffffffffu, one, i);
            place += i < lane ? k >= one : k > one;
        }
        if (one) chosen = one_at, k_chosen = one;
        else place = lane < count ? place : lane;
    } else {
        for (int j = 0; j < top; ++j) {
            uint32_t k = 0;
            int at = lane;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (key[i] > k) k = key[i], at = i * 32 + lane;
            best_of(k, at);
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i * 32 + lane == at) key[i] = 0;
            if (lane == j && k) chosen = at, k_chosen = k;
        }
    }
    const bool mine = place < top;
    const float part = mine && k_chosen ? expf(logit_of(k_chosen) - most) : 0.f;
    if (chosen_only) total = sum_of(part);
    if (mine) {
        experts[m * top + place] = chosen;
        shares[m * top + place] = chosen < 0 ? 0.f : part / total;
    }
}

template <typename T, int V>
__global__ void __launch_bounds__(kRouteThreads) route_grad_kernel(const T *logits, const int *experts, const float *dshares,
                                                                   T *dlogits, int64_t M, int G, int top, int chosen_only)
{
    ptx::launch_dependents();
    ptx::grid_dependency_wait();
    const int lane = threadIdx.x % 32;
    const int64_t m = static_cast<int64_t>(blockIdx.x) * (kRouteThreads / 32) + threadIdx.x / 32;
    if (m >= M) return;
    const T *const row = logits + m * G;
    T *const out = dlogits + m * G;
    // the lane's choice: its expert, logit and gradient
    int e = -1;
    float d = 0.f, l = -INFINITY;
    if (lane < top) {
        e = experts[m * top + lane];
        if (static_cast<unsigned>(e) < static_cast<unsigned>(G)) {
            d = dshares[m * top + lane];
            l = static_cast<float>(row[e]);
        } else {
            e = -1;
        }
    }
    float v[V];
    float most = l;
    if (!chosen_only) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            v[i] = i * 32 + lane < G ? static_cast<float>(row[i * 32 + lane]) : -INFINITY;
            most = fmaxf(most, v[i]);
        }
    }
#pragma unroll
    for (int s = 16; s; s >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, s));
    if (most == -INFINITY) most = 0.f;   // no expert at all: every exp is 0
    float total = 0.f;
    const float mine = e < 0 ? 0.f : expf(l - most);
    if (chosen_only) {
        total = mine;
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            v[i] = expf(v[i] - most);
            total += v[i];
        }
    }
    total = sum_of(total);
    const float inv = total == 0.f ? 0.f : 1.f / total, p = mine * inv;
    // an expert that is there twice has both gradients, and both shares where the
    // sum is over the chosen (added in the choices' order by each of its lanes)
    float both = 0.f;
    int times = 0;
    for (int j = 0; j < top; ++j) {
        const int other = __shfl_sync(0xffffffffu, e, j);
        const float theirs = __shfl_sync(0xffffffffu, d, j);
        if (other == e) both += theirs, ++times;
    }
    const float c = sum_of(p * d);
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (i * 32 + lane < G) out[i * 32 + lane] = static_cast<T>(chosen_only ? 0.f : -(v[i] * inv) * c);
    __syncwarp();
    if (e >= 0) out[e] = static_cast<T>(p * (both - (chosen_only ? static_cast<float>(times) * c : c)));
}

template <typename T, int V>
cudaError_t launch(const RouteProblem &p, cudaStream_t stream)
{
    cudaLaunchAttribute attr;
    const unsigned grid = static_cast<unsigned>((p.M * 32 + kRouteThreads - 1) / kRouteThreads);
    const cudaLaunchConfig_t cfg = config(grid, kRouteThreads, stream, &attr);
    const T *const logits = static_cast<const T *>(p.logits);
    const int G = static_cast<int>(p.G), top = static_cast<int>(p.top);
    if (p.dlogits)
        return note_error(cudaLaunchKernelEx(&cfg, route_grad_kernel<T, V>, logits, static_cast<const int *>(p.experts),
                                             static_cast<const float *>(p.shares), static_cast<T *>(p.dlogits), p.M, G, top,
                                             p.chosen_only),
                          "route_grad_kernel launch");
    return note_error(cudaLaunchKernelEx(&cfg, route_kernel<T, V>, logits, p.experts, p.shares, p.M, G, top, p.chosen_only),
                      "route_kernel launch");
}

template <typename T>
cudaError_t launch_type(const RouteProblem &p, cudaStream_t stream)
{
    if (p.G <= 32) return launch<T, 1>(p, stream);
    if (p.G <= 64) return launch<T, 2>(p, stream);
    if (p.G <= 128) return launch<T, 4>(p, stream);
    if (p.G <= 256) return launch<T, 8>(p, stream);
    if (p.G <= 512) return launch<T, 16>(p, stream);
    return launch<T, 32>(p, stream);
}

}  // namespace

cudaError_t launch_route(const RouteProblem &p, cudaStream_t stream)
{
    return p.dtype == 0 ? launch_type<float>(p, stream) : p.dtype == 1 ? launch_type<__half>(p, stream)
                                                                        : launch_type<__nv_bfloat16>(p, stream);
}

}  // namespace splitk
