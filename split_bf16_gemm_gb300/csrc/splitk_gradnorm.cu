// splitk_gradnorm.cu -- the norm of all gradients of a model, and the gradients
// scaled to a largest norm.
//
//   norm = sqrt(sum over all tensors and values of g^2)
//   out  = g f,  f = min(1, max_norm / norm), rounded once
//
// The tensors are cut into chunks of 8192 values (2048 where there are few) that a
// grid's blocks take in turn.  A thread squares 32 (8) values of a chunk in F32 and adds
// that to a sum of two F32 numbers, the second of which holds what the first's
// roundings lose.  A block writes one part, a number and a power of two; further launches
// add to it, and keep what that loses beside it.  Parts are added in the same order every
// time.  F64 is kept out of the way: this chip does two F64 operations a clock and SM (9
// tensors of 1.3 M values 18 us with the parts, the root and the quotient in F64, 6.4
// without).  Squares that F32 does not hold (of gradients beyond 2^43 or all below 2^-40)
// are taken again of the values times a power of two.
// The scaling goes through the chunks backwards, so that it finds the last ones of the
// sum in L2.
//
// The tensors' addresses go into the kernels as parameters: no copy to the device
// before the launch, nothing to keep for a captured graph.  Bound by memory: the
// gradients read once for the norm, read again and written for the scaling.

#include <math.h>

#include "ptx.cuh"
#include "rows.cuh"
#include "splitk_internal.h"

namespace splitk {
namespace {

constexpr int kThreads = 256;
constexpr int kFewParts = 4 * 152;                      // blocks for few values
constexpr int chunk_of(int vecs) { return kThreads * vecs * kVec; }   // values, `vecs` vectors to a thread

template <int N>
struct Table {
    const void *g[N];
    void *out[N];
    int64_t size[N];
    int first[N + 1];         // chunks before the tensor
    uint8_t dtype[N];
    int count;
};

// A sum of two F32 numbers: what `hi`'s additions lose is in `lo` (D. Knuth, "The Art
// of Computer Programming", volume 2, 4.2.2, theorem B).
struct Sum {
    float hi, lo;
};
__device__ __forceinline__ void add(Sum &s, float x)
{
    const float t = s.hi + x, y = t - s.hi;
    s.lo += (s.hi - (t - y)) + (x - y);
    s.hi = t;
}

__device__ __forceinline__ float value(const Sum &s) { return isfinite(s.hi) ? s.hi + s.lo : s.hi; }

// m 2^e
struct Part {
    float m;
    int e;
};
constexpr int kNothing = -1023;   // e of a 0
// (m in [1, 2), or 0, an infinity or NaN)
__device__ __forceinline__ Part part_of(float v)
{
    const int bits = __float_as_int(v), e = bits >> 23 & 255;
    if (e == 0) return {0.f, kNothing};                            // (no sum is that small)
    if (e == 255) return {v, 1023};
    return {__int_as_float((bits & 0x7fffff) | 0x3f800000), e - 127};
}
__device__ __forceinline__ Part part_of(double v)
{
    const int64_t bits = __double_as_longlong(v);
    const int e = static_cast<int>(bits >> 52) & 2047;
    if (e == 0) return {0.f, kNothing};                            // (no square is that small)
    if (e == 2047) return {static_cast<float>(v), 1023};
    return {static_cast<float>(__longlong_as_double((bits & 0xfffffffffffffll) | 0x3ff0000000000000ll)), e - 1023};
}

// 2^e, 0 below F32's range
__device__ __forceinline__ float power(int e) { return e < -126 ? 0.f : __int_as_float((e + 127) << 23); }

struct Shared {
    int e[kThreads / 32];
    Sum s[kThreads / 32];
};

// The block's sum of the threads' numbers, the same in every thread: 2^e times the Sum.
__device__ __forceinline__ Sum block_sum(const Part &p, int &e, Shared &shared)
{
    const int warp = threadIdx.x / 32;
    const int most = __reduce_max_sync(0xffffffffu, p.e);
    if (threadIdx.x % 32 == 0) shared.e[warp] = most;
    __syncthreads();
    e = shared.e[0];
#pragma unroll
    for (int w = 1; w < kThreads / 32; ++w) e = max(e, shared.e[w]);
    Sum s = {p.m * power(p.e - e), 0.f};
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        const Sum o = {__shfl_xor_sync(0xffffffffu, s.hi, d), __shfl_xor_sync(0xffffffffu, s.lo, d)};
        add(s, o.hi);
        s.lo += o.lo;
    }
    if (threadIdx.x % 32 == 0) shared.s[warp] = s;
    __syncthreads();
    s = shared.s[0];
#pragma unroll
    for (int w = 1; w < kThreads / 32; ++w) {
        add(s, shared.s[w].hi);
        s.lo += shared.s[w].lo;
    }
    return s;
}

// Adds the squares of a thread's values of a chunk that starts at g, n values of the
// tensor left there; `far` takes those that F32 does not hold.
template <int kVecs, typename T>
__device__ __forceinline__ void squares(const T *g, int64_t n, Sum &total, double &far)
{
    float x[kVecs][kVec];
    if (n >= chunk_of(kVecs)) {
        Pack<T> p[kVecs];
#pragma unroll
        for (int i = 0; i < kVecs; ++i) p[i] = *reinterpret_cast<const Pack<T> *>(g + (i * kThreads + threadIdx.x) * kVec);
#pragma unroll
        for (int i = 0; i < kVecs; ++i) unpack(p[i], x[i]);
    } else {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int at = (i * kThreads + threadIdx.x) * kVec;
            if (at + kVec <= n) {
                unpack(*reinterpret_cast<const Pack<T> *>(g + at), x[i]);
            } else {
#pragma unroll
                for (int j = 0; j < kVec; ++j) x[i][j] = at + j < n ? static_cast<float>(g[at + j]) : 0.f;
            }
        }
    }
    float s[kVecs] = {};
#pragma unroll
    for (int j = 0; j < kVec; ++j)
#pragma unroll
        for (int i = 0; i < kVecs; ++i) s[i] = fmaf(x[i][j], x[i][j], s[i]);
    float sum = s[0];
#pragma unroll
    for (int i = 1; i < kVecs; ++i) sum += s[i];
    if (__builtin_expect(sum >= 0x1p-80f && sum <= 0x1p90f, true)) {   // (2^27 of them and more are below 2^127)
        add(total, sum);
        return;
    }
    if (sum == 0.f) {   // zeros, or all below 2^-75: F32 squares none of them
        bool zeros = true;
#pragma unroll
        for (int i = 0; i < kVecs; ++i)
#pragma unroll
            for (int j = 0; j < kVec; ++j) zeros &= x[i][j] == 0.f;
        if (zeros) return;
    }
    const float scale = sum < 1.f ? 0x1p100f : 0x1p-80f;
    float again = 0.f;
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
#pragma unroll
        for (int j = 0; j < kVec; ++j) again = fmaf(x[i][j] * scale, x[i][j] * scale, again);
    far += static_cast<double>(again) * (sum < 1.f ? 0x1p-200 : 0x1p160);
}

template <int kVecs, typename T>
__device__ __forceinline__ void scaled(const T *g, T *out, int64_t n, float f)
{
    if (n >= chunk_of(kVecs)) {
        Pack<T> p[kVecs];
#pragma unroll
        for (int i = 0; i < kVecs; ++i) p[i] = *reinterpret_cast<const Pack<T> *>(g + (i * kThreads + threadIdx.x) * kVec);
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            float x[kVec];
            unpack(p[i], x);
#pragma unroll
            for (int j = 0; j < kVec; ++j) x[j] *= f;
            pack(x, p[i]);
            *reinterpret_cast<Pack<T> *>(out + (i * kThreads + threadIdx.x) * kVec) = p[i];
        }
        return;
    }
    for (int at = threadIdx.x; at < n; at += kThreads) out[at] = static_cast<T>(static_cast<float>(g[at]) * f);
}

// The tensor that chunk c is of.
template <int N>
__device__ __forceinline__ int tensor_of(const Table<N> &t, int c)
{
    int lo = 0, hi = t.count - 1;   // the last with first[] <= c
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (t.first[mid] <= c) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// `lows`: behind the parts what their additions lose, where there are launches that add to
// them (else nullptr; `more`: this is one).
template <int N, int kVecs>
__global__ void __launch_bounds__(kThreads) norm_kernel(const __grid_constant__ Table<N> t, Part *parts, float *lows, int more)
{
    __shared__ Shared shared;
    ptx::launch_dependents();
    ptx::grid_dependency_wait();
    Sum sum = {0.f, 0.f};
    double far = 0.;
    int at = tensor_of(t, blockIdx.x);
    for (int c = blockIdx.x; c < t.first[t.count]; c += gridDim.x) {
        while (c >= t.first[at + 1]) ++at;
        const int64_t from = static_cast<int64_t>(c - t.first[at]) * chunk_of(kVecs), n = t.size[at] - from;
        if (t.dtype[at] == 0) squares<kVecs>(static_cast<const float *>(t.g[at]) + from, n, sum, far);
        else if (t.dtype[at] == 1) squares<kVecs>(static_cast<const __half *>(t.g[at]) + from, n, sum, far);
        else squares<kVecs>(static_cast<const __nv_bfloat16 *>(t.g[at]) + from, n, sum, far);
    }
    Part mine = part_of(value(sum));
    if (__builtin_expect(far != 0., false)) mine = part_of(far + static_cast<double>(value(sum)));
    int e;
    const Sum s = block_sum(mine, e, shared);
    if (threadIdx.x == 0) {
        Part p = {value(s), e};
        if (lows) {
            Sum both = {0.f, 0.f};
            if (more) {
                const Part q = parts[blockIdx.x];
                p.e = max(e, q.e);
                const float down = power(q.e - p.e);
                both = {q.m * down, lows[blockIdx.x] * down};
                add(both, p.m * power(e - p.e));
                p.m = both.hi;
            }
            lows[blockIdx.x] = both.lo;
        }
        parts[blockIdx.x] = p;
    }
}

// The norm from the blocks' parts, as root * 2^half, in every thread.  MORE: several
// launches made them.
template <bool MORE>
__device__ __forceinline__ float norm_of(const Part *parts, const float *lows, int blocks, int &half, Shared &shared)
{
    constexpr int kAtOnce = (kFewParts + kThreads - 1) / kThreads;   // loads in flight
    Part mine = {0.f, kNothing};
    Sum s = {0.f, 0.f};
    for (int from = 0; from < blocks; from += kAtOnce * kThreads) {
        Part p[kAtOnce];
        int most = mine.e;
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const int at = from + i * kThreads + static_cast<int>(threadIdx.x);
            p[i] = at < blocks ? parts[at] : Part{0.f, kNothing};
            most = max(most, p[i].e);
        }
        const float down = power(mine.e - most);
        s.hi *= down, s.lo *= down;
        mine.e = most;
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) add(s, p[i].m * power(p[i].e - most));
        if (MORE) {
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                const int at = from + i * kThreads + static_cast<int>(threadIdx.x);
                if (at < blocks) s.lo += lows[at] * power(p[i].e - most);
            }
        }
    }
    mine.m = value(s);
    int e;
    s = block_sum(mine, e, shared);
    const int odd = e & 1;
    half = (e - odd) / 2;
    return sqrtf(value(s) * (odd ? 2.f : 1.f));
}

__device__ __forceinline__ float norm_value(float root, int half)
{
    return half > 120 ? root * power(120) * power(min(half - 120, 127)) : half < -120 ? root * power(-120) * power(half + 120) : root * power(half);
}

// min(1, max_norm / norm), by halves of the power: neither has to be in F32's range
__device__ __forceinline__ float factor_of(float root, int half, float max_norm)
{
    const int some = -half / 2;
    const float q = max_norm / root * power(some) * power(-half - some);
    return isnan(root) ? root : root != 0.f && q < 1.f ? q : 1.f;
}

// The norm, and (factor != nullptr) the factor.
template <bool MORE>
__global__ void __launch_bounds__(kThreads) finish_kernel(const Part *parts, const float *lows, int blocks, float *norm, float max_norm,
                                                          float *factor)
{
    __shared__ Shared shared;
    ptx::launch_dependents();
    ptx::grid_dependency_wait();
    int half;
    const float root = norm_of<MORE>(parts, lows, blocks, half, shared);
    if (threadIdx.x == 0) {
        *norm = norm_value(root, half);
        if (factor) *factor = factor_of(root, half, max_norm);
    }
}

// FINISHED: the factor is there, and a block takes one chunk; else every block finds the
// norm, the first writes it, and blocks take chunks in turn.
template <int N, int kVecs, bool FINISHED, bool MORE>
__global__ void __launch_bounds__(kThreads) clip_kernel(const __grid_constant__ Table<N> t, const Part *parts, const float *lows,
                                                        int blocks, float max_norm, float *norm, const float *factor)
{
    __shared__ Shared shared;
    ptx::launch_dependents();
    ptx::grid_dependency_wait();
    float f;
    if constexpr (FINISHED) {
        f = *factor;
    } else {
        int half;
        const float root = norm_of<MORE>(parts, lows, blocks, half, shared);
        if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = norm_value(root, half);
        f = factor_of(root, half, max_norm);
    }
    const int last = t.first[t.count] - 1 - static_cast<int>(blockIdx.x);
    int at = tensor_of(t, last);
    for (int c = last; c >= 0; c -= gridDim.x) {
        while (c < t.first[at]) --at;
        if (f == 1.f && t.out[at] == t.g[at]) continue;   // in place, and nothing to change
        const int64_t from = static_cast<int64_t>(c - t.first[at]) * chunk_of(kVecs), left = t.size[at] - from;
        if (t.dtype[at] == 0) scaled<kVecs>(static_cast<const float *>(t.g[at]) + from, static_cast<float *>(t.out[at]) + from, left, f);
        else if (t.dtype[at] == 1) scaled<kVecs>(static_cast<const __half *>(t.g[at]) + from, static_cast<__half *>(t.out[at]) + from, left, f);
        else scaled<kVecs>(static_cast<const __nv_bfloat16 *>(t.g[at]) + from, static_cast<__nv_bfloat16 *>(t.out[at]) + from, left, f);
    }
}

constexpr int kMostTensors = 512;   // of one launch

// The factor's place behind the parts, and behind that what their additions lose where
// several launches make them.
float *factor_at(void *parts) { return reinterpret_cast<float *>(static_cast<Part *>(parts) + kGradNormParts); }
bool several(const GradNormProblem &p) { return p.count > kMostTensors; }
float *lows_of(const GradNormProblem &p) { return several(p) ? factor_at(p.parts) + 2 : nullptr; }

int64_t chunks_of(int64_t n, int vecs) { return (n + chunk_of(vecs) - 1) / chunk_of(vecs); }

template <int N, int kVecs, bool MORE = false>
cudaError_t launch(const GradNormProblem &p, int64_t begin, int64_t end, int blocks, bool clip, cudaStream_t stream)
{
    Table<N> t;
    t.count = static_cast<int>(end - begin);
    t.first[0] = 0;
    for (int i = 0; i < t.count; ++i) {
        t.g[i] = p.grads[begin + i];
        t.out[i] = p.out ? p.out[begin + i] : nullptr;
        t.size[i] = p.sizes[begin + i];
        t.dtype[i] = static_cast<uint8_t>(p.dtypes[begin + i]);
        t.first[i + 1] = t.first[i] + static_cast<int>(chunks_of(t.size[i], kVecs));
    }
    Part *const parts = static_cast<Part *>(p.parts);
    cudaLaunchAttribute attr;
    cudaLaunchConfig_t cfg = config(static_cast<unsigned>(blocks), kThreads, stream, &attr);
    if (!clip) return note_error(cudaLaunchKernelEx(&cfg, norm_kernel<N, kVecs>, t, parts, lows_of(p), begin ? 1 : 0), "norm_kernel launch");
    constexpr bool kFinished = kVecs > 1;
    if (kFinished) cfg.gridDim.x = static_cast<unsigned>(t.first[t.count] ? t.first[t.count] : 1);
    return note_error(cudaLaunchKernelEx(&cfg, clip_kernel<N, kVecs, kFinished, MORE>, t, static_cast<const Part *>(parts),
                                         static_cast<const float *>(lows_of(p)), blocks, p.max_norm,
                                         begin == 0 ? p.norm : static_cast<float *>(nullptr), static_cast<const float *>(factor_at(p.parts))),
                      "clip_kernel launch");
}

}  // namespace

// At most kMostTensors tensors to a launch; a few take the kernel with the short table.
cudaError_t launch_grad_norm(const GradNormProblem &p, cudaStream_t stream)
{
    constexpr int kFew = 32;
    auto most_of = [&](int vecs) {
        int64_t most = 1;
        for (int64_t begin = 0; begin < p.count; begin += kMostTensors) {
            int64_t chunks = 0;
            for (int64_t i = begin; i < p.count && i < begin + kMostTensors; ++i) chunks += chunks_of(p.sizes[i], vecs);
            most = most > chunks ? most : chunks;
        }
        return most;
    };
    // Chunks of 8192 values keep 4 loads in flight, and more blocks than the device holds
    // even out what each meets: 2.0 GB in 290 tensors 909 us with 24 blocks to an SM, 954
    // with 8.  A block to a chunk then scales, after a launch that finds the factor for
    // them all.  Few values: chunks of 2048, and no launch between (clipping with and
    // without it, F32: 1 M values 7.8 and 7.4 us, 2 M 8.0 and 11.3, 4 M 10.6 and 15.4, 8 M 17.0
    // and 17.4, 32 M 67 and 66; the norm alone 4.3 and 3.6, 5.9 and 4.7 of 4 M, 7.6 and 6.3 of 8).
    int64_t most = most_of(4);
    const bool few = most <= 512;
    if (few) most = most_of(1);
    const int64_t limit = few ? kFewParts : kGradNormParts;
    const int blocks = static_cast<int>(most < limit ? most : limit);
    auto all = [&](bool clip) {
        int64_t begin = 0;
        do {   // (no tensors: one launch that finds nothing)
            const int64_t end = begin + kMostTensors < p.count ? begin + kMostTensors : p.count;
            const auto go = several(p) ? few ? launch<kMostTensors, 1, true> : launch<kMostTensors, 4, true>
                            : few ? end - begin <= kFew ? launch<kFew, 1> : launch<kMostTensors, 1>
                            : end - begin <= kFew ? launch<kFew, 4> : launch<kMostTensors, 4>;
            const cudaError_t e = go(p, begin, end, blocks, clip, stream);
            if (e != cudaSuccess) return e;
            begin = end;
        } while (begin < p.count);
        return cudaSuccess;
    };
    const cudaError_t e = all(false);
    if (e != cudaSuccess) return e;
    if (!p.out || !few) {
        cudaLaunchAttribute attr;
        const cudaLaunchConfig_t cfg = config(1, kThreads, stream, &attr);
        const cudaError_t f = note_error(cudaLaunchKernelEx(&cfg, several(p) ? finish_kernel<true> : finish_kernel<false>, static_cast<const Part *>(p.parts),
                                                            static_cast<const float *>(lows_of(p)), blocks, p.norm, p.max_norm,
                                                            p.out ? factor_at(p.parts) : static_cast<float *>(nullptr)),
                                         "finish_kernel launch");
        if (f != cudaSuccess || !p.out) return f;
    }
    return all(true);
}

}  // namespace splitk
