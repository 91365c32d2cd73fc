// splitk_fp8.cu -- what makes 8-bit operands: rows (with the residual's
// addition and the root-mean-square norm before, or as they are) and weights.
//
// Rows: h = x + residual, rounded once to the inputs' type (the `sum` that the
// next layer adds to; the norm is of what is kept); y = h w / sqrt(mean h^2 +
// eps) in F32; each 128 consecutive y share the scale s = max(max|y| / 448,
// 2^-126), and q = E4M3(y / s), to nearest even.  448 is E4M3's largest value;
// the floor keeps y / s defined for a block of zeros and s out of the
// subnormals.  Rows whose squares F32 does not hold are scaled (row_again).  A NaN or an infinity in a block gives it a NaN or infinite
// scale and NaN products, never finite ones.
//
// A row is read once: its values stay in registers (8 to a 16-byte load of
// 16-bit inputs) between the sum of squares and the output.  Rows longer than
// the registers of a block hold are read twice.  Bound by memory: e + 1 to 4e +
// 1 bytes a value for e-byte inputs.  GB300: 8192 rows of 8192 BF16 with a
// residual 72 us, 6.6 TB/s (0.98 of the measured copy rate); one row of 2048
// 1.7 us in a graph.

#include <cuda_fp8.h>

#include <type_traits>

#include "ptx.cuh"
#include "rows.cuh"
#include "splitk_internal.h"

namespace splitk {
namespace {

constexpr float kE4m3Max = 448.f;
constexpr float kScaleFloor = 1.17549435082228751e-38f;   // 2^-126
constexpr int kBlockVecs = 128 / kVec;                     // threads that share a scale

// max that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ uint32_t to_e4m3(float a, float b, float c, float d)
{
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3),
                   hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

__device__ __forceinline__ uint2 to_e4m3(const float (&v)[kVec])
{
    return make_uint2(to_e4m3(v[0], v[1], v[2], v[3]), to_e4m3(v[4], v[5], v[6], v[7]));
}

// The scale of a block whose largest magnitude is m: m / 448, rounded once (the
// product with the rounded reciprocal alone is a unit off for 55% of the m), by the
// correction that divide() takes; an infinity stays one.
__device__ __forceinline__ float scale_of(float m)
{
    constexpr float kInv = 1.f / kE4m3Max;
    const float q0 = m * kInv;
    const float s = isinf(m) ? m : fmaf(fmaf(-kE4m3Max, q0, m), kInv, q0);
    return max_nan(s, kScaleFloor);
}

// The quotients of a block's values and its scale s, each rounded once: q0 =
// y (1/s), then Markstein's correction q = q0 + (y - s q0) (1/s) (P. Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor",
// 1990).  Three operations a value: the norm of 8192 x 8192 BF16 with a residual
// took 73 us, with a division 84, uncorrected 72.  An infinite scale gives 0 for
// finite values and NaN for the infinity, as a division does.
template <int N>
__device__ __forceinline__ void divide(float (&y)[N], float s)
{
    const float inv = 1.f / s, d = isinf(s) ? 0.f : s;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const float q0 = y[j] * inv;
        y[j] = fmaf(fmaf(-d, q0, y[j]), inv, q0);
    }
}

struct RowsArgs {
    const void *x, *residual, *weight;
    void *sum, *y;
    uint8_t *q;
    float *scales;
    int64_t M;
    int K, vecs, blocks;       // values, 16-byte groups of 8, scales of a row
    float eps;
};

// A barrier of the TPR threads of a row.  (The numbers are constants: a block that
// may use any of the 16 takes them all, and fewer blocks fit on an SM: 8192 rows of
// 1024 BF16 15.8 us, with constants 12.9.)
template <int TPR>
__device__ __forceinline__ void row_sync()
{
    static_assert(TPR == 32 || TPR == 128 || TPR >= 256, "one row a block, or two");
    if constexpr (TPR == 32)
        __syncwarp();
    else if constexpr (TPR >= 256)
        __syncthreads();
    else if (threadIdx.x < TPR)
        asm volatile("bar.sync 1, 128;" ::: "memory");
    else
        asm volatile("bar.sync 2, 128;" ::: "memory");
}

// The norm of a row whose squares F32 does not hold, once more by its TPR threads:
// the row times `scale`, a power of two, which the norm cancels.  Values of 2^53
// and more come under 2^48 (the squares of 2^22 of them add to less than 2^118),
// values under 2^-40 under 2^60, with squares from 2^-98 up.  Its sum is written.
// A block of 128 to a warp, four values to a lane: few registers, so that the
// kernel keeps its own.
template <typename T, int TPR>
__device__ __forceinline__ void row_again(const RowsArgs &a, int64_t row, float *part, float scale)
{
    constexpr int kWarps = TPR / 32;
    const int t = threadIdx.x % TPR;
    row_sync<TPR>();   // what the row's threads wrote is there for its others, and the parts are read
    const size_t at = static_cast<size_t>(row) * a.K;
    const T *const x = static_cast<const T *>(a.sum ? a.sum : a.x) + at;
    const T *const res = a.residual && !a.sum ? static_cast<const T *>(a.residual) + at : nullptr;
    auto load = [&](int k, float (&h)[4]) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            h[j] = static_cast<float>(x[k + j]);
            if (res) h[j] = static_cast<float>(static_cast<T>(h[j] + static_cast<float>(res[k + j])));
            h[j] *= scale;
        }
    };
    float h[4], sq = 0.f;
    for (int k = 4 * t; k < a.K; k += 4 * TPR) {
        load(k, h);
#pragma unroll
        for (int j = 0; j < 4; ++j) sq = fmaf(h[j], h[j], sq);
    }
    __syncwarp();
#pragma unroll
    for (int d = 16; d; d >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, d);
    if constexpr (kWarps > 1) {
        if (t % 32 == 0) part[t / 32] = sq;
        row_sync<TPR>();
        sq = 0.f;
        for (int i = 0; i < kWarps; ++i) sq += part[i];
    }
    const float rstd = rsqrtf(sq / static_cast<float>(a.K) + a.eps * scale * scale);
    for (int b = t / 32; b < a.blocks; b += kWarps) {
        const int k = b * 128 + t % 32 * 4;
        const bool in = k < a.K;
        float m = 0.f;
        if (in) {
            load(k, h);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                h[j] = h[j] * rstd * static_cast<float>(static_cast<const T *>(a.weight)[k + j]);
                m = max_nan(m, fabsf(h[j]));
            }
        }
        __syncwarp();
#pragma unroll
        for (int d = 16; d; d >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, d));
        const float s = scale_of(m);
        if (in) {
            if (a.y) {
#pragma unroll
                for (int j = 0; j < 4; ++j) static_cast<T *>(a.y)[at + k + j] = static_cast<T>(h[j]);
            }
            divide(h, s);
            *reinterpret_cast<uint32_t *>(a.q + at + k) = to_e4m3(h[0], h[1], h[2], h[3]);
            if (t % 32 == 0) a.scales[static_cast<size_t>(row) * a.blocks + b] = s;
        }
    }
}

// Blocks of an SM whose registers the compiler keeps to: 32 a thread with one
// vector, 40 with two of 16 bits, as without row_again (1024 rows of 2048 BF16 3.8 us,
// with 36 registers 4.2); 0 leaves it to the compiler.
template <typename T, int TPR, int VPT>
constexpr int rows_per_sm()
{
    return TPR > 256 || TPR < 128 ? 0 : VPT == 1 ? 8 : VPT == 2 && sizeof(T) == 2 ? 6 : 0;
}

// Rows per block: kThreads / TPR, TPR threads each, VPT vectors a thread.
// LONG: any row length, one block a row, VPT vectors in registers at a time.
template <typename T, int TPR, int VPT, bool LONG>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR, rows_per_sm<T, TPR, VPT>()) rows_kernel(const RowsArgs a)
{
    constexpr int kThreads = TPR < 256 ? 256 : TPR, kRows = kThreads / TPR, kWarps = TPR / 32;
    __shared__ float part[kThreads / 32];
    const int t = threadIdx.x % TPR, in_block = threadIdx.x / TPR;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + in_block;
    ptx::launch_dependents();
    ptx::grid_dependency_wait();
    const bool live = row < a.M;
    const size_t at = static_cast<size_t>(live ? row : 0) * a.K;
    const T *const x = static_cast<const T *>(a.x) + at;
    const T *const res = a.residual ? static_cast<const T *>(a.residual) + at : nullptr;
    T *const sum = a.sum ? static_cast<T *>(a.sum) + at : nullptr;
    const T *const weight = static_cast<const T *>(a.weight);
    float h[VPT][kVec];
    float sq = 0.f;
    const int turns = LONG ? (a.vecs + TPR * VPT - 1) / (TPR * VPT) : 1;

    // h of the turn's vectors; `again`: the second reading of a long row, from
    // `sum` where there is one (x or the residual may be the same memory)
    auto load = [&](int turn, bool again) {
        Pack<T> px[VPT], pr[VPT];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = (turn * VPT + i) * TPR + t;
            if (live && v < a.vecs) {
                px[i] = *reinterpret_cast<const Pack<T> *>((again && sum ? sum : x) + static_cast<size_t>(v) * kVec);
                if (res && !(again && sum)) pr[i] = *reinterpret_cast<const Pack<T> *>(res + static_cast<size_t>(v) * kVec);
            }
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = (turn * VPT + i) * TPR + t;
            if (live && v < a.vecs) {
                unpack(px[i], h[i]);
                if (res && !(again && sum)) {
                    float r[kVec];
                    unpack(pr[i], r);
#pragma unroll
                    for (int j = 0; j < kVec; ++j) h[i][j] += r[j];
                    Pack<T> p;
                    pack(h[i], p);
                    unpack(p, h[i]);
                    if (sum && !again) *reinterpret_cast<Pack<T> *>(sum + static_cast<size_t>(v) * kVec) = p;
                } else if (sum && !again) {
                    *reinterpret_cast<Pack<T> *>(sum + static_cast<size_t>(v) * kVec) = px[i];
                }
            } else {
#pragma unroll
                for (int j = 0; j < kVec; ++j) h[i][j] = 0.f;
            }
        }
    };

    float rstd = 1.f, mean = 1.f;
    for (int turn = 0; turn < turns; ++turn) {
        load(turn, false);
        if (weight) {
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int j = 0; j < kVec; ++j) sq = fmaf(h[i][j], h[i][j], sq);
        }
    }
    if (weight) {
#pragma unroll
        for (int d = 16; d; d >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, d);
        if constexpr (kWarps > 1) {
            if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = sq;
            __syncthreads();
            sq = 0.f;
#pragma unroll
            for (int i = 0; i < kWarps; ++i) sq += part[in_block * kWarps + i];
        }
        mean = sq / static_cast<float>(a.K) + a.eps;
        rstd = rsqrtf(mean);
    }
    for (int turn = 0; turn < turns; ++turn) {
        if (LONG) load(turn, true);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = (turn * VPT + i) * TPR + t;
            const bool in = live && v < a.vecs;
            if (weight && in) {
                float w[kVec];
                unpack(*reinterpret_cast<const Pack<T> *>(weight + static_cast<size_t>(v) * kVec), w);
#pragma unroll
                for (int j = 0; j < kVec; ++j) h[i][j] = h[i][j] * rstd * w[j];
            }
            float m = 0.f;
#pragma unroll
            for (int j = 0; j < kVec; ++j) m = max_nan(m, fabsf(h[i][j]));
            // the 16 threads of a scale are consecutive lanes of one warp
#pragma unroll
            for (int d = kBlockVecs / 2; d; d >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, d));
            const float s = scale_of(m);
            if (in) {
                if (a.y) {
                    Pack<T> p;
                    pack(h[i], p);
                    *reinterpret_cast<Pack<T> *>(static_cast<T *>(a.y) + at + static_cast<size_t>(v) * kVec) = p;
                }
                divide(h[i], s);
                *reinterpret_cast<uint2 *>(a.q + at + static_cast<size_t>(v) * kVec) = to_e4m3(h[i]);
                if (v % kBlockVecs == 0) a.scales[static_cast<size_t>(row) * a.blocks + v / kBlockVecs] = s;
            }
        }
    }
    // Squares out of range (F16's never are).  Here at the end, and from memory
    // again, it costs ordinary rows least: 8192 rows of 4096 BF16 38.8 us, without it
    // 37.7, with the scaled row in registers before the weights are loaded 39.7.
    if constexpr (!std::is_same_v<T, __half>) {
        if (__builtin_expect(live && (isinf(mean) || mean < 0x1p-80f), false)) {
            row_again<T, TPR>(a, row, part + in_block * kWarps, isinf(mean) ? 0x1p-80f : 0x1p100f);
        }
    }
}

// One block of 256 threads for each 128 x 128 block of a weight: thread t
// takes 8 consecutive values of rows t / 16, t / 16 + 16, ...
template <typename T>
__global__ void __launch_bounds__(256) prepare_fp8_kernel(const T *B, uint8_t *q, float *scales, int N, int K, int n_blocks,
                                                          int k_blocks)
{
    __shared__ float part[8];
    ptx::launch_dependents();
    ptx::grid_dependency_wait();
    const int64_t id = blockIdx.x;                       // (g * n_blocks + nb) * k_blocks + kb
    const int kb = static_cast<int>(id % k_blocks);
    const int64_t gn = id / k_blocks;
    const int nb = static_cast<int>(gn % n_blocks);
    const int64_t g = gn / n_blocks;
    const int k = kb * 128 + (threadIdx.x % 16) * kVec, r0 = threadIdx.x / 16;
    const size_t at = (static_cast<size_t>(g) * N + nb * 128) * K + k;
    const int rows = min(128, N - nb * 128);
    float h[8][kVec];
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = r0 + 16 * i;
        if (r < rows && k < K) {
            unpack(*reinterpret_cast<const Pack<T> *>(B + at + static_cast<size_t>(r) * K), h[i]);
#pragma unroll
            for (int j = 0; j < kVec; ++j) m = max_nan(m, fabsf(h[i][j]));
        }
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, d));
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max_nan(m, part[i]);
    const float s = scale_of(m);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = r0 + 16 * i;
        if (r < rows && k < K) {
            divide(h[i], s);
            *reinterpret_cast<uint2 *>(q + at + static_cast<size_t>(r) * K) = to_e4m3(h[i]);
        }
    }
    if (threadIdx.x == 0) scales[id] = s;
}

template <typename T, int TPR, int VPT, bool LONG = false>
cudaError_t launch_rows(const RowsArgs &a, cudaStream_t stream)
{
    constexpr int kThreads = TPR < 256 ? 256 : TPR, kRows = kThreads / TPR;
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = config(static_cast<unsigned>((a.M + kRows - 1) / kRows), kThreads, stream, &attr);
    return note_error(cudaLaunchKernelEx(&cfg, rows_kernel<T, TPR, VPT, LONG>, a), "rows_kernel launch");
}

template <typename T>
cudaError_t launch_rows_type(const RowsArgs &a, cudaStream_t stream)
{
    // Few rows: as many threads a row as it has vectors, for latency (8 rows
    // of 8192: 2.9 us, with 256 threads 4.6).
    if (a.M <= 64 && a.vecs > 256 && a.vecs <= 512) return launch_rows<T, 512, 1>(a, stream);
    if (a.M <= 64 && a.vecs > 512 && a.vecs <= 1024) return launch_rows<T, 512, 2>(a, stream);
    // Else 256 threads with the vectors that the row needs, fewer for short
    // rows (1024 rows of 2048: 3.8 us, with 128 threads 4.5; 4096 F32 rows of
    // 4096: 35 us, with 128 threads of 4 vectors 44).
    if (a.vecs <= 64) return launch_rows<T, 32, 2>(a, stream);
    if (a.vecs <= 128) return launch_rows<T, 128, 1>(a, stream);
    if (a.vecs <= 256) return launch_rows<T, 256, 1>(a, stream);
    if (a.vecs <= 512) return launch_rows<T, 256, 2>(a, stream);
    if (a.vecs <= 768) return launch_rows<T, 256, 3>(a, stream);
    if (a.vecs <= 1024) return launch_rows<T, 256, 4>(a, stream);
    if (a.vecs <= 1536) return launch_rows<T, 512, 3>(a, stream);
    if (a.vecs <= 2048) return launch_rows<T, 512, 4>(a, stream);
    return launch_rows<T, 512, 4, true>(a, stream);
}

}  // namespace

cudaError_t launch_rows_fp8(const RowsProblem &p, cudaStream_t stream)
{
    RowsArgs a = {p.x, p.residual, p.weight, p.sum, p.y, static_cast<uint8_t *>(p.q), p.scales, p.M,
                  static_cast<int>(p.K), static_cast<int>(p.K / kVec), static_cast<int>((p.K + 127) / 128), p.eps};
    return p.dtype == 0 ? launch_rows_type<float>(a, stream)
           : p.dtype == 1 ? launch_rows_type<__half>(a, stream)
                          : launch_rows_type<__nv_bfloat16>(a, stream);
}

cudaError_t launch_prepare_fp8(const void *B, void *q, float *scales, int64_t G, int64_t N, int64_t K, int dtype,
                               cudaStream_t stream)
{
    const int nb = static_cast<int>((N + 127) / 128), kb = static_cast<int>((K + 127) / 128);
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = config(static_cast<unsigned>(G * nb * kb), 256, stream, &attr);
    uint8_t *const o = static_cast<uint8_t *>(q);
    const int n = static_cast<int>(N), k = static_cast<int>(K);
    const cudaError_t e =
        dtype == 0   ? cudaLaunchKernelEx(&cfg, prepare_fp8_kernel<float>, static_cast<const float *>(B), o, scales, n, k, nb, kb)
        : dtype == 1 ? cudaLaunchKernelEx(&cfg, prepare_fp8_kernel<__half>, static_cast<const __half *>(B), o, scales, n, k, nb, kb)
                     : cudaLaunchKernelEx(&cfg, prepare_fp8_kernel<__nv_bfloat16>, static_cast<const __nv_bfloat16 *>(B), o, scales, n, k, nb, kb);
    return note_error(e, "prepare_fp8_kernel launch");
}

}  // namespace splitk
