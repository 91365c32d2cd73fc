// splitk_route.cu -- the router's choice: each token's `top` largest logits and
// their softmax shares, and the logits' gradient.
//
// A token's logits l_0..l_{G-1} stay in the registers of W lanes, V to a lane
// (logit i W + lane).  Each is turned into a whole number that rises with it, so
// that a choice is a maximum: `top` times the largest is taken (the lowest index
// of equal ones) and struck out.  -inf has the number 0 and is never taken.  The
// first choice is the row's maximum m, so the shares follow without another pass:
// s_j = exp(l_j - m) / sum exp(l - m), the sum over all G or over the chosen.
//
// Gradient, with p = softmax over all G (or over the chosen; p = 0 elsewhere) and
// c = sum_j p_{e_j} d_j:   dl_i = p_i (sum_{j: e_j = i} d_j - c).
//
// Bound by instructions more than by memory: a choice costs about 3 V + 20 of a
// warp (a shuffle tree of W lanes), and there are `top` of them.

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ptx.cuh"
#include "rows.cuh"
#include "splitk_internal.h"

namespace splitk {
namespace {

constexpr int kRouteThreads = 256;

// A number that rises with the logit; -inf has 0, and NaN the largest.  (-0 + 0 is
// +0: the two zeros are equal.)
__device__ __forceinline__ uint32_t key_of(float x)
{
    if (isnan(x)) return 0xffffffffu;
    const uint32_t u = __float_as_uint(x + 0.f);
    const uint32_t k = u ^ (u >> 31 ? 0xffffffffu : 0x80000000u);
    return k == 0x007fffffu ? 0u : k;   // -inf
}
__device__ __forceinline__ float logit_of(uint32_t k)
{
    if (k == 0) return -INFINITY;
    return __uint_as_float(k ^ (k >> 31 ? 0x80000000u : 0xffffffffu));
}

template <int W>
__device__ __forceinline__ float sum_of(float x)
{
#pragma unroll
    for (int d = W / 2; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}

// The largest key of the W lanes and the lowest index that has it.
template <int W>
__device__ __forceinline__ void best_of(uint32_t &key, int &at)
{
    if constexpr (W == 32) {
        const uint32_t k = __reduce_max_sync(0xffffffffu, key);
        at = static_cast<int>(__reduce_min_sync(0xffffffffu, key == k ? static_cast<uint32_t>(at) : 0xffffffffu));
        key = k;
    } else {
#pragma unroll
        for (int d = W / 2; d; d >>= 1) {
            const uint32_t k = __shfl_xor_sync(0xffffffffu, key, d);
            const int i = __shfl_xor_sync(0xffffffffu, at, d);
            if (k > key || (k == key && i < at)) key = k, at = i;
        }
    }
}

// W lanes a token, at least `top` of them: lane j keeps the j-th choice.
template <typename T, int W, int V>
__global__ void __launch_bounds__(kRouteThreads) route_kernel(const T *logits, int *experts, float *shares, int64_t M, int G,
                                                              int top, int chosen_only)
{
    ptx::launch_dependents();
    ptx::grid_dependency_wait();
    const int lane = threadIdx.x % W;
    const int64_t m = (static_cast<int64_t>(blockIdx.x) * kRouteThreads + threadIdx.x) / W;
    const bool live = m < M;   // whole warps go through the shuffles
    const T *const row = logits + (live ? m : 0) * G;
    uint32_t key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = live && i * W + lane < G ? key_of(static_cast<float>(row[i * W + lane])) : 0u;
    float most = 0.f, total = 0.f, mine = 0.f;
    int chosen = -1, last = -1;
    for (int j = 0; j < top; ++j) {
        uint32_t k = 0;
        int at = lane;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (i * W + lane == last) key[i] = 0;
            if (key[i] > k) k = key[i], at = i * W + lane;
        }
        best_of<W>(k, at);
        if (j == 0) {
            most = k ? logit_of(k) : 0.f;
            if (!chosen_only) {
                float part = 0.f;
#pragma unroll
                for (int i = 0; i < V; ++i) part += expf(logit_of(key[i]) - most);
                total = sum_of<W>(part);
            }
        }
        last = at;
        if (lane == j && k) chosen = at, mine = expf(logit_of(k) - most);
    }
    if (chosen_only) total = sum_of<W>(mine);
    if (live && lane < top) {
        experts[m * top + lane] = chosen;
        shares[m * top + lane] = chosen < 0 ? 0.f : mine / total;
    }
}

template <typename T, int W, int V>
__global__ void __launch_bounds__(kRouteThreads) route_grad_kernel(const T *logits, const int *experts, const float *dshares,
                                                                   T *dlogits, int64_t M, int G, int top, int chosen_only)
{
    ptx::launch_dependents();
    ptx::grid_dependency_wait();
    const int lane = threadIdx.x % W;
    const int64_t m = (static_cast<int64_t>(blockIdx.x) * kRouteThreads + threadIdx.x) / W;
    const bool live = m < M;
    const T *const row = logits + (live ? m : 0) * G;
    T *const out = dlogits + (live ? m : 0) * G;
    // the lane's choice: its expert, logit and gradient
    int e = -1;
    float d = 0.f, l = -INFINITY;
    if (live && lane < top) {
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
            v[i] = live && i * W + lane < G ? static_cast<float>(row[i * W + lane]) : -INFINITY;
            most = fmaxf(most, v[i]);
        }
    }
#pragma unroll
    for (int s = W / 2; s; s >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, s));
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
    total = sum_of<W>(total);
    const float inv = total == 0.f ? 0.f : 1.f / total, p = mine * inv;
    // an expert that is there twice has both gradients, and both shares where the
    // sum is over the chosen (added in the choices' order by each of its lanes)
    float both = 0.f;
    int times = 0;
    for (int j = 0; j < top; ++j) {
        const int other = __shfl_sync(0xffffffffu, e, j, W);
        const float theirs = __shfl_sync(0xffffffffu, d, j, W);
        if (other == e) both += theirs, ++times;
    }
    const float c = sum_of<W>(p * d);
    if (live) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i * W + lane < G) out[i * W + lane] = static_cast<T>(chosen_only ? 0.f : -(v[i] * inv) * c);
    }
    __syncwarp();
    if (e >= 0) out[e] = static_cast<T>(p * (both - (chosen_only ? static_cast<float>(times) * c : c)));
}

template <typename T, int W, int V>
cudaError_t launch(const RouteProblem &p, cudaStream_t stream)
{
    cudaLaunchAttribute attr;
    const unsigned grid = static_cast<unsigned>((p.M * W + kRouteThreads - 1) / kRouteThreads);
    const cudaLaunchConfig_t cfg = config(grid, kRouteThreads, stream, &attr);
    const T *const logits = static_cast<const T *>(p.logits);
    const int G = static_cast<int>(p.G), top = static_cast<int>(p.top);
    if (p.dlogits)
        return note_error(cudaLaunchKernelEx(&cfg, route_grad_kernel<T, W, V>, logits, static_cast<const int *>(p.experts),
                                             static_cast<const float *>(p.shares), static_cast<T *>(p.dlogits), p.M, G, top,
                                             p.chosen_only),
                          "route_grad_kernel launch");
    return note_error(cudaLaunchKernelEx(&cfg, route_kernel<T, W, V>, logits, p.experts, p.shares, p.M, G, top, p.chosen_only),
                      "route_kernel launch");
}

template <typename T>
cudaError_t launch_type(const RouteProblem &p, cudaStream_t stream)
{
    if (p.G <= 32) return launch<T, 32, 1>(p, stream);
    if (p.G <= 128) return launch<T, 32, 4>(p, stream);
    if (p.G <= 256) return launch<T, 32, 8>(p, stream);
    if (p.G <= 512) return launch<T, 32, 16>(p, stream);
    return launch<T, 32, 32>(p, stream);
}

}  // namespace

cudaError_t launch_route(const RouteProblem &p, cudaStream_t stream)
{
    return p.dtype == 0 ? launch_type<float>(p, stream) : p.dtype == 1 ? launch_type<__half>(p, stream)
                                                                        : launch_type<__nv_bfloat16>(p, stream);
}

}  // namespace splitk
