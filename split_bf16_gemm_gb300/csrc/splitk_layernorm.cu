// splitk_layernorm.cu -- layer norm (with the residual's addition before it) and
// its gradients.
//
// Forward: h = x + residual, rounded once to the inputs' type (the `sum` that the
// next layer adds to; the norm is of what is kept); u = mean h, v = mean (h - u)^2,
// r = 1 / sqrt(v + eps); y = (h - u) r w + b.  A row stays in registers over both
// sums.  The mean is found twice, the second time as the mean of h - u, which
// takes its rounding out of a row whose values are large against their spread.
//
// Backward, with x = (h - u) r and g = dy w:
//   dh = r (g - mean g - x mean (g x)) (+ the sum's own gradient)
//   dw = sum over the rows of dy x,  db = sum over the rows of dy
// Blocks take rows in turn; a thread keeps the same columns for all its rows and
// their dw and db in registers.  A second launch adds the blocks' parts in order.
//
// Rows longer than the registers of a block hold are read twice, and their dw and
// db are sums of a launch of their own.  Bound by memory.

#include <math.h>

#include <type_traits>

#include "ptx.cuh"
#include "rows.cuh"
#include "splitk_internal.h"

namespace splitk {
namespace {

struct NormArgs {
    const void *x, *residual, *weight, *bias;
    void *sum, *y;
    float *mean, *rstd;
    int64_t M;
    int K, vecs;
    float eps;
};

// The sum over a block's threads, the same in each.  `part` is free again after the
// next barrier.
template <int THREADS, int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float *part)
{
    constexpr int kWarps = THREADS / 32;
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int d = 16; d; d >>= 1) v[n] += __shfl_xor_sync(0xffffffffu, v[n], d);
    if (threadIdx.x % 32 == 0) {
#pragma unroll
        for (int n = 0; n < N; ++n) part[n * kWarps + threadIdx.x / 32] = v[n];
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n) {
        v[n] = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) v[n] += part[n * kWarps + w];
    }
}

// Whether F32 holds the squares that v + eps is made of.
__device__ __forceinline__ bool in_range(float v) { return v >= 0x1p-80f && v <= 0x1p120f; }

// One row a block.  LONG: any row length, VPT vectors in registers at a time.
template <typename T, int THREADS, int VPT, bool LONG>
__global__ void __launch_bounds__(THREADS) layernorm_kernel(const NormArgs a)
{
    constexpr int kWarps = THREADS / 32;
    __shared__ float part[4][2 * kWarps];
    ptx::launch_dependents();
    ptx::grid_dependency_wait();
    const int64_t row = blockIdx.x;
    const size_t at = static_cast<size_t>(row) * a.K;
    const T *const x = static_cast<const T *>(a.x) + at;
    const T *const res = a.residual ? static_cast<const T *>(a.residual) + at : nullptr;
    T *const sum = a.sum ? static_cast<T *>(a.sum) + at : nullptr;
    T *const y = static_cast<T *>(a.y) + at;
    float h[VPT][kVec];
    const int turns = LONG ? (a.vecs + THREADS * VPT - 1) / (THREADS * VPT) : 1;

    // h of the turn's vectors; `again`: a later reading of a long row, from `sum`
    // where there is one (x or the residual may be the same memory)
    auto load = [&](int turn, bool again) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = (turn * VPT + i) * THREADS + threadIdx.x;
#pragma unroll
            for (int j = 0; j < kVec; ++j) h[i][j] = 0.f;
            if (v >= a.vecs) continue;
            Pack<T> p = *reinterpret_cast<const Pack<T> *>((again && sum ? sum : x) + static_cast<size_t>(v) * kVec);
            unpack(p, h[i]);
            if (res && !(again && sum)) {
                float r[kVec];
                unpack(*reinterpret_cast<const Pack<T> *>(res + static_cast<size_t>(v) * kVec), r);
#pragma unroll
                for (int j = 0; j < kVec; ++j) h[i][j] += r[j];
                pack(h[i], p);
                unpack(p, h[i]);
            }
            if (sum && !again) *reinterpret_cast<Pack<T> *>(sum + static_cast<size_t>(v) * kVec) = p;
        }
    };
    // mean and 1 / sqrt of the row times `scale`, (h - mean) times `wide` in the squares
    float mean, rest, rstd;
    auto moments = [&](float scale, float wide, float *p, bool again) {
        float s[1] = {0.f};
        for (int turn = 0; turn < turns; ++turn) {
            if (LONG || !again) load(turn, again);
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int j = 0; j < kVec; ++j) s[0] += h[i][j] * scale;
        }
        block_sum<THREADS>(s, p);
        mean = s[0] / static_cast<float>(a.K);
        float q[2] = {0.f, 0.f};
        for (int turn = 0; turn < turns; ++turn) {
            if (LONG) load(turn, true);
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                if ((turn * VPT + i) * THREADS + static_cast<int>(threadIdx.x) >= a.vecs) continue;
#pragma unroll
                for (int j = 0; j < kVec; ++j) {
                    const float d = fmaf(h[i][j], scale, -mean) * wide;
                    q[0] += d;
                    q[1] = fmaf(d, d, q[1]);
                }
            }
        }
        block_sum<THREADS>(q, p + 2 * kWarps);
        rest = q[0] / static_cast<float>(a.K);
        float var = q[1] / static_cast<float>(a.K) - rest * rest;
        var = (var < 0.f ? 0.f : var) + a.eps * (scale * wide) * (scale * wide);   // (keeps a NaN)
        rstd = rsqrtf(var);
        return var;
    };
    float scale = 1.f, wide = 1.f;
    const float var = moments(1.f, 1.f, part[0], false);
    if (__builtin_expect(!in_range(var), false)) {
        // deviations whose squares F32 does not hold: the row times a power of two,
        // which the norm cancels
        if (var < 1.f) wide = 0x1p100f;
        else scale = 0x1p-80f;
        moments(scale, wide, part[2], true);
    }
    for (int turn = 0; turn < turns; ++turn) {
        if (LONG) load(turn, true);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = (turn * VPT + i) * THREADS + threadIdx.x;
            if (v >= a.vecs) continue;
            float w[kVec], b[kVec] = {};
            unpack(*reinterpret_cast<const Pack<T> *>(static_cast<const T *>(a.weight) + static_cast<size_t>(v) * kVec), w);
            if (a.bias) unpack(*reinterpret_cast<const Pack<T> *>(static_cast<const T *>(a.bias) + static_cast<size_t>(v) * kVec), b);
            float o[kVec];
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                const float d = fmaf(h[i][j], scale, -mean) * wide - rest;
                o[j] = fmaf(d * rstd, w[j], b[j]);
            }
            Pack<T> p;
            pack(o, p);
            *reinterpret_cast<Pack<T> *>(y + static_cast<size_t>(v) * kVec) = p;
        }
    }
    if (threadIdx.x == 0) {
        if (a.mean) a.mean[row] = (mean + rest / wide) / scale;
        if (a.rstd) a.rstd[row] = rstd * (scale * wide);
    }
}

struct NormGradArgs {
    const void *dy, *h, *weight, *dsum;
    const float *mean, *rstd;
    void *dx;
    float *parts;        // [blocks][2][K]: dw, then db
    int64_t M;
    int K, vecs;
};

// (h - mean) rstd; by halves, as the difference may leave F32's range
__device__ __forceinline__ float normal_of(float h, float half_mean, float rstd2) { return fmaf(0.5f, h, -half_mean) * rstd2; }

// Rows blockIdx.x, + gridDim.x, ...; a thread's columns are the same for all of them.
template <typename T, int THREADS, int VPT>
__global__ void __launch_bounds__(THREADS) layernorm_grad_kernel(const NormGradArgs a)
{
    constexpr int kWarps = THREADS / 32;
    __shared__ float part[2][2 * kWarps];
    ptx::launch_dependents();
    ptx::grid_dependency_wait();
    float dw[VPT][kVec] = {}, db[VPT][kVec] = {};
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x, turn ^= 1) {
        const size_t at = static_cast<size_t>(row) * a.K;
        const float half_mean = 0.5f * a.mean[row], rstd = a.rstd[row], rstd2 = 2.f * rstd;
        float g[VPT][kVec], x[VPT][kVec], s[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = i * THREADS + threadIdx.x;
            if (v >= a.vecs) continue;
            const size_t k = static_cast<size_t>(v) * kVec;
            float w[kVec];
            unpack(*reinterpret_cast<const Pack<T> *>(static_cast<const T *>(a.dy) + at + k), g[i]);
            unpack(*reinterpret_cast<const Pack<T> *>(static_cast<const T *>(a.h) + at + k), x[i]);
            unpack(*reinterpret_cast<const Pack<T> *>(static_cast<const T *>(a.weight) + k), w);
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                x[i][j] = normal_of(x[i][j], half_mean, rstd2);
                dw[i][j] = fmaf(g[i][j], x[i][j], dw[i][j]);
                db[i][j] += g[i][j];
                g[i][j] *= w[j];
                s[0] += g[i][j];
                s[1] = fmaf(g[i][j], x[i][j], s[1]);
            }
        }
        block_sum<THREADS>(s, part[turn]);
        const float mg = s[0] / static_cast<float>(a.K), mgx = s[1] / static_cast<float>(a.K);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = i * THREADS + threadIdx.x;
            if (v >= a.vecs) continue;
            const size_t k = static_cast<size_t>(v) * kVec;
            float o[kVec] = {};
            if (a.dsum) unpack(*reinterpret_cast<const Pack<T> *>(static_cast<const T *>(a.dsum) + at + k), o);
#pragma unroll
            for (int j = 0; j < kVec; ++j) o[j] = fmaf(rstd, g[i][j] - mg - x[i][j] * mgx, o[j]);
            Pack<T> p;
            pack(o, p);
            *reinterpret_cast<Pack<T> *>(static_cast<T *>(a.dx) + at + k) = p;
        }
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int v = i * THREADS + threadIdx.x;
        if (v >= a.vecs) continue;
        float *const to = a.parts + static_cast<size_t>(blockIdx.x) * 2 * a.K + static_cast<size_t>(v) * kVec;
        Pack<float> p;
        pack(dw[i], p);
        *reinterpret_cast<Pack<float> *>(to) = p;
        pack(db[i], p);
        *reinterpret_cast<Pack<float> *>(to + a.K) = p;
    }
}

// A row of any length, read twice: its dx.
template <typename T, int THREADS>
__global__ void __launch_bounds__(THREADS) layernorm_grad_long_kernel(const NormGradArgs a)
{
    __shared__ float part[2 * THREADS / 32];
    ptx::launch_dependents();
    ptx::grid_dependency_wait();
    const int64_t row = blockIdx.x;
    const size_t at = static_cast<size_t>(row) * a.K;
    const float half_mean = 0.5f * a.mean[row], rstd = a.rstd[row], rstd2 = 2.f * rstd;
    float s[2] = {0.f, 0.f};
    float g[kVec], x[kVec];
    auto load = [&](int v) {
        const size_t k = static_cast<size_t>(v) * kVec;
        float w[kVec];
        unpack(*reinterpret_cast<const Pack<T> *>(static_cast<const T *>(a.dy) + at + k), g);
        unpack(*reinterpret_cast<const Pack<T> *>(static_cast<const T *>(a.h) + at + k), x);
        unpack(*reinterpret_cast<const Pack<T> *>(static_cast<const T *>(a.weight) + k), w);
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            x[j] = normal_of(x[j], half_mean, rstd2);
            g[j] *= w[j];
        }
    };
    for (int v = threadIdx.x; v < a.vecs; v += THREADS) {
        load(v);
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            s[0] += g[j];
            s[1] = fmaf(g[j], x[j], s[1]);
        }
    }
    block_sum<THREADS>(s, part);
    const float mg = s[0] / static_cast<float>(a.K), mgx = s[1] / static_cast<float>(a.K);
    for (int v = threadIdx.x; v < a.vecs; v += THREADS) {
        load(v);
        const size_t k = static_cast<size_t>(v) * kVec;
        float o[kVec] = {};
        if (a.dsum) unpack(*reinterpret_cast<const Pack<T> *>(static_cast<const T *>(a.dsum) + at + k), o);
#pragma unroll
        for (int j = 0; j < kVec; ++j) o[j] = fmaf(rstd, g[j] - mg - x[j] * mgx, o[j]);
        Pack<T> p;
        pack(o, p);
        *reinterpret_cast<Pack<T> *>(static_cast<T *>(a.dx) + at + k) = p;
    }
}

// dw and db of long rows: a vector of columns to a thread, rows blockIdx.y, + gridDim.y, ...
template <typename T, int THREADS>
__global__ void __launch_bounds__(THREADS) layernorm_grad_columns_kernel(const NormGradArgs a)
{
    ptx::launch_dependents();
    ptx::grid_dependency_wait();
    const int v = blockIdx.x * THREADS + threadIdx.x;
    if (v >= a.vecs) return;
    const size_t k = static_cast<size_t>(v) * kVec;
    float dw[kVec] = {}, db[kVec] = {};
    for (int64_t row = blockIdx.y; row < a.M; row += gridDim.y) {
        const size_t at = static_cast<size_t>(row) * a.K + k;
        const float half_mean = 0.5f * a.mean[row], rstd2 = 2.f * a.rstd[row];
        float g[kVec], x[kVec];
        unpack(*reinterpret_cast<const Pack<T> *>(static_cast<const T *>(a.dy) + at), g);
        unpack(*reinterpret_cast<const Pack<T> *>(static_cast<const T *>(a.h) + at), x);
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            dw[j] = fmaf(g[j], normal_of(x[j], half_mean, rstd2), dw[j]);
            db[j] += g[j];
        }
    }
    float *const to = a.parts + static_cast<size_t>(blockIdx.y) * 2 * a.K + k;
    Pack<float> p;
    pack(dw, p);
    *reinterpret_cast<Pack<float> *>(to) = p;
    pack(db, p);
    *reinterpret_cast<Pack<float> *>(to + a.K) = p;
}

constexpr int kSumThreads = 256, kSumLanes = 32, kSumSlices = kSumThreads / kSumLanes;

// out[c] = sum over the blocks' parts, slices of them side by side, then the slices in
// order.  A block takes 32 columns, columns from K on are db's.
__global__ void __launch_bounds__(kSumThreads) layernorm_sum_kernel(const float *parts, float *dw, float *db, int blocks, int K)
{
    __shared__ float part[kSumSlices][kSumLanes];
    ptx::launch_dependents();
    ptx::grid_dependency_wait();
    const int lane = threadIdx.x % kSumLanes, slice = threadIdx.x / kSumLanes;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * kSumLanes + lane;
    float sum = 0.f;
    if (c < 2 * static_cast<int64_t>(K)) {
#pragma unroll 8
        for (int b = slice; b < blocks; b += kSumSlices) sum += parts[static_cast<size_t>(b) * 2 * K + c];
    }
    part[slice][lane] = sum;
    __syncthreads();
    if (slice == 0 && c < 2 * static_cast<int64_t>(K)) {
#pragma unroll
        for (int s = 1; s < kSumSlices; ++s) sum += part[s][lane];
        if (c < K) dw[c] = sum;
        else if (db) db[c - K] = sum;
    }
}

constexpr int kLongVecs = 2048;   // vectors of the longest row that a block's registers hold
constexpr int kMostParts = 304;   // two blocks to each of 152 SMs

template <typename T, int THREADS, int VPT, bool LONG = false>
cudaError_t launch_norm(const NormArgs &a, cudaStream_t stream)
{
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = config(static_cast<unsigned>(a.M), THREADS, stream, &attr);
    return note_error(cudaLaunchKernelEx(&cfg, layernorm_kernel<T, THREADS, VPT, LONG>, a), "layernorm_kernel launch");
}

template <typename T>
cudaError_t launch_norm_type(const NormArgs &a, cudaStream_t stream)
{
    if (a.vecs <= 128) return launch_norm<T, 128, 1>(a, stream);
    if (a.vecs <= 256) return launch_norm<T, 256, 1>(a, stream);
    if (a.vecs <= 512) return launch_norm<T, 256, 2>(a, stream);
    if (a.vecs <= 1024) return launch_norm<T, 256, 4>(a, stream);
    if (a.vecs <= kLongVecs) return launch_norm<T, 512, 4>(a, stream);
    return launch_norm<T, 512, 4, true>(a, stream);
}

template <typename T, int THREADS, int VPT>
cudaError_t launch_grad(const NormGradArgs &a, int blocks, cudaStream_t stream)
{
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = config(static_cast<unsigned>(blocks), THREADS, stream, &attr);
    return note_error(cudaLaunchKernelEx(&cfg, layernorm_grad_kernel<T, THREADS, VPT>, a), "layernorm_grad_kernel launch");
}

template <typename T>
cudaError_t launch_grad_type(const NormGradArgs &a, int blocks, cudaStream_t stream)
{
    if (a.vecs <= 128) return launch_grad<T, 128, 1>(a, blocks, stream);
    if (a.vecs <= 256) return launch_grad<T, 256, 1>(a, blocks, stream);
    if (a.vecs <= 512) return launch_grad<T, 256, 2>(a, blocks, stream);
    if (a.vecs <= 1024) return launch_grad<T, 512, 2>(a, blocks, stream);
    if (a.vecs <= kLongVecs) return launch_grad<T, 512, 4>(a, blocks, stream);
    constexpr int kThreads = 512;
    cudaLaunchAttribute attr;
    cudaLaunchConfig_t cfg = config(static_cast<unsigned>(a.M), kThreads, stream, &attr);
    // dw and db first: dx may be dy
    cfg.gridDim = dim3(static_cast<unsigned>((a.vecs + kThreads - 1) / kThreads), static_cast<unsigned>(blocks), 1);
    cudaError_t e = note_error(cudaLaunchKernelEx(&cfg, layernorm_grad_columns_kernel<T, kThreads>, a), "layernorm_grad_columns_kernel launch");
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(static_cast<unsigned>(a.M), 1, 1);
    return note_error(cudaLaunchKernelEx(&cfg, layernorm_grad_long_kernel<T, kThreads>, a), "layernorm_grad_long_kernel launch");
}

}  // namespace

cudaError_t launch_layernorm(const LayerNormProblem &p, cudaStream_t stream)
{
    const NormArgs a = {p.x, p.residual, p.weight, p.bias, p.sum, p.y, p.mean, p.rstd, p.M, static_cast<int>(p.K),
                        static_cast<int>(p.K / kVec), p.eps};
    return p.dtype == 0 ? launch_norm_type<float>(a, stream) : p.dtype == 1 ? launch_norm_type<__half>(a, stream)
                                                                             : launch_norm_type<__nv_bfloat16>(a, stream);
}

int64_t layernorm_grad_parts(int64_t M, int64_t K)
{
    // Long rows have columns enough for the threads: few parts.
    const int64_t most = K / kVec <= kLongVecs ? kMostParts : 16;
    return M < most ? M : most;
}

cudaError_t launch_layernorm_grad(const LayerNormGradProblem &p, cudaStream_t stream)
{
    const int blocks = static_cast<int>(layernorm_grad_parts(p.M, p.K)), K = static_cast<int>(p.K);
    const NormGradArgs a = {p.dy, p.h, p.weight, p.dsum, p.mean, p.rstd, p.dx, p.parts, p.M, K, K / kVec};
    if (blocks) {
        const cudaError_t e = p.dtype == 0   ? launch_grad_type<float>(a, blocks, stream)
                              : p.dtype == 1 ? launch_grad_type<__half>(a, blocks, stream)
                                             : launch_grad_type<__nv_bfloat16>(a, blocks, stream);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg =
        config(static_cast<unsigned>((2 * static_cast<int64_t>(K) + kSumLanes - 1) / kSumLanes), kSumThreads, stream, &attr);
    return note_error(cudaLaunchKernelEx(&cfg, layernorm_sum_kernel, static_cast<const float *>(p.parts), p.dweight, p.dbias, blocks, K),
                      "layernorm_sum_kernel launch");
}

}  // namespace splitk
