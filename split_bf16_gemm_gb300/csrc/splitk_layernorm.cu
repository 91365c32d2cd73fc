// splitk_layernorm.cu -- layer norm (with the residual's addition before it) and
// its gradients.
//
// Forward: h = x + residual, rounded once to the inputs' type (the `sum` that the
// next layer adds to; the norm is of what is kept); u = mean h, v = mean (h - u)^2,
// r = 1 / sqrt(v + eps); y = (h - u) r w + b.  A row stays in registers over both
// sums.  The mean is found twice, the second time as the mean of h - u, which
// takes its rounding out of a row whose values are large against their spread (where
// that rounding is beyond the spread itself, the row is done again about a better mean).
//
// Backward, with x = (h - u) r and g = dy w:
//   dh = r (g - mean g - x mean (g x)) (+ the sum's own gradient)
//   dw = sum over the rows of dy x,  db = sum over the rows of dy
// Blocks take rows in turn; a thread keeps the same columns for all its rows and
// their dw and db in registers.  A second launch adds the blocks' parts in order.
//
// Rows longer than 8192 have dw and db from a launch of their own, which reads dy and h
// once more, and rows longer than 16384 are read twice for dx.  The norm reads rows longer
// than 16384 (32768 of 16 bits) three times: for the mean, the deviations and y.  GB300: 8192 x 8192 BF16 with the residual 80 us, 6.7 TB/s
// (the copy rate), one row of 2048 1.8 us in a graph.

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

template <typename T>
__device__ __forceinline__ void unpack(const Pack<T> &p, float2 (&v)[kVec / 2])
{
    float f[kVec];
    unpack(p, f);
#pragma unroll
    for (int j = 0; j < kVec / 2; ++j) v[j] = make_float2(f[2 * j], f[2 * j + 1]);
}
template <typename T>
__device__ __forceinline__ Pack<T> packed(const float2 (&v)[kVec / 2])
{
    float f[kVec];
#pragma unroll
    for (int j = 0; j < kVec / 2; ++j) f[2 * j] = v[j].x, f[2 * j + 1] = v[j].y;
    Pack<T> p;
    pack(f, p);
    return p;
}

// The sums of x and of y over a warp: of x in lanes 0-15, of y in lanes 16-31, 5
// exchanges for both (exchanges and shared memory's copies share a pipe).
__device__ __forceinline__ float lanes_sum(float2 v)
{
    const bool upper = threadIdx.x & 16;
    float s = (upper ? v.y : v.x) + __shfl_xor_sync(0xffffffffu, upper ? v.x : v.y, 16);
#pragma unroll
    for (int d = 8; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    return s;
}
// The sums over a row's threads (a block, or a warp), the same in each.  `part` is free again after the
// next barrier.
template <int THREADS>
__device__ __forceinline__ float2 block_sum(float2 v, float2 *part)
{
    constexpr int kWarps = THREADS / 32;
    const int lane = threadIdx.x % 32;
    const float s = lanes_sum(v);
    if constexpr (kWarps == 1) return make_float2(__shfl_sync(0xffffffffu, s, 0), __shfl_sync(0xffffffffu, s, 16));
    if (lane % 16 == 0) reinterpret_cast<float *>(part + threadIdx.x / 32)[lane / 16] = s;
    __syncthreads();
    v = make_float2(0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v = __fadd2_rn(v, part[w]);
    return v;
}

// The variances (with eps, and without) whose squares F32 holds as they are.
constexpr float kLeast = 0x1p-80f, kMost = 0x1p120f;

constexpr int kRowThreads = 256;   // of a block with a row to a warp

// Blocks of 16-bit rows to an SM, so that rows done again take no registers from the
// others: 30000 rows of 2048 F16 79 us with 8, with the 6 that came unasked 86; 16384 of
// 4096 78.6, with 5 82; 4096 of 16384 BF16 80, with one of 512 threads 105.  (0: as it comes.)
template <typename T, int THREADS, int VPT, bool LONG>
constexpr int norm_blocks()
{
    if (sizeof(T) != 2 || LONG || THREADS < 256) return 0;
    return VPT == 1 ? 8 : VPT == 2 ? 6 : VPT == 4 ? 1024 / THREADS : 0;
}

// THREADS a row, one row a block, or one a warp.  LONG: any row length, VPT vectors in
// registers at a time.
template <typename T, int THREADS, int VPT, bool LONG>
__global__ void __launch_bounds__(THREADS == 32 ? kRowThreads : THREADS, norm_blocks<T, THREADS, VPT, LONG>()) layernorm_kernel(const NormArgs a)
{
    constexpr int kWarps = THREADS / 32, kPairs = kVec / 2;
    __shared__ float2 part[4][kWarps];
    ptx::launch_dependents();
    ptx::grid_dependency_wait();
    const int t = THREADS == 32 ? threadIdx.x % 32 : threadIdx.x;
    const int64_t row = THREADS == 32 ? static_cast<int64_t>(blockIdx.x) * (kRowThreads / 32) + threadIdx.x / 32 : blockIdx.x;
    if (THREADS == 32 && row >= a.M) return;
    const size_t at = static_cast<size_t>(row) * a.vecs;
    const Pack<T> *const x = static_cast<const Pack<T> *>(a.x) + at;
    const Pack<T> *const res = a.residual ? static_cast<const Pack<T> *>(a.residual) + at : nullptr;
    Pack<T> *const sum = a.sum ? static_cast<Pack<T> *>(a.sum) + at : nullptr;
    float2 h[VPT][kPairs];
    const int turns = LONG ? (a.vecs + THREADS * VPT - 1) / (THREADS * VPT) : 1;
    const float inv = 1.f / static_cast<float>(a.K);

    // h of the turn's vectors; `again`: a later reading of a long row, from `sum`
    // where there is one (x or the residual may be the same memory)
    auto load = [&](int turn, bool again) {
        Pack<T> px[VPT], pr[VPT];
        const bool add = res && !(again && sum);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = (turn * VPT + i) * THREADS + t;
            if (v >= a.vecs) continue;
            px[i] = (again && sum ? sum : x)[v];
            if (add) pr[i] = res[v];
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = (turn * VPT + i) * THREADS + t;
#pragma unroll
            for (int j = 0; j < kPairs; ++j) h[i][j] = make_float2(0.f, 0.f);
            if (v >= a.vecs) continue;
            unpack(px[i], h[i]);
            if (add) {
                float2 r[kPairs];
                unpack(pr[i], r);
#pragma unroll
                for (int j = 0; j < kPairs; ++j) h[i][j] = __fadd2_rn(h[i][j], r[j]);
                px[i] = packed<T>(h[i]);
                unpack(px[i], h[i]);
            }
            if (sum && !again) sum[v] = px[i];
        }
    };
    // Mean (and the mean of what is left of it, `rest`) and the root.  scaled: of the
    // row times `scale`, the deviations times `wide`, a value at a time (pairs of factors
    // take registers: 60000 rows of 1000 BF16 78 us with them, 71 without).
    float mean, rest, rstd, scale = 1.f, wide = 1.f;
    auto deviation = [&](const bool scaled, float2 v) {
        return scaled ? make_float2(fmaf(v.x, scale, -mean) * wide, fmaf(v.y, scale, -mean) * wide)
                      : __fadd2_rn(v, make_float2(-mean, -mean));
    };
    auto find_mean = [&](const bool scaled, float2 *p) {
        float2 s = {0.f, 0.f};
        for (int turn = 0; turn < turns; ++turn) {
            if (LONG || !scaled) load(turn, scaled);
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int j = 0; j < kPairs; ++j)
                    s = scaled ? make_float2(fmaf(h[i][j].x, scale, s.x), fmaf(h[i][j].y, scale, s.y)) : __fadd2_rn(s, h[i][j]);
        }
        mean = block_sum<THREADS>(make_float2(s.x + s.y, 0.f), p).x * inv;
    };
    // The variance
    auto spread = [&](const bool scaled, float2 *p) {
        float2 s = {0.f, 0.f}, q = {0.f, 0.f};
        for (int turn = 0; turn < turns; ++turn) {
            if (LONG) load(turn, true);
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                if ((turn * VPT + i) * THREADS + t >= a.vecs) continue;
#pragma unroll
                for (int j = 0; j < kPairs; ++j) {
                    const float2 d = deviation(scaled, h[i][j]);
                    s = __fadd2_rn(s, d);
                    q = __ffma2_rn(d, d, q);
                }
            }
        }
        const float2 sums = block_sum<THREADS>(make_float2(s.x + s.y, q.x + q.y), p);
        rest = sums.x * inv;
        const float var = sums.y * inv - rest * rest;
        return var < 0.f ? 0.f : var;   // (keeps a NaN)
    };
    auto outputs = [&](const bool scaled) {
        const float2 less = make_float2(-rest, -rest), r = make_float2(rstd, rstd);
        for (int turn = 0; turn < turns; ++turn) {
            if (LONG) load(turn, true);
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int v = (turn * VPT + i) * THREADS + t;
                if (v >= a.vecs) continue;
                float2 w[kPairs], b[kPairs] = {};
                unpack(static_cast<const Pack<T> *>(a.weight)[v], w);
                if (a.bias) unpack(static_cast<const Pack<T> *>(a.bias)[v], b);
#pragma unroll
                for (int j = 0; j < kPairs; ++j) {
                    const float2 d = deviation(scaled, h[i][j]);
                    const float2 n = scaled ? make_float2((d.x - rest) * rstd, (d.y - rest) * rstd) : __fmul2_rn(__fadd2_rn(d, less), r);
                    b[j] = __ffma2_rn(n, w[j], b[j]);
                }
                (static_cast<Pack<T> *>(a.y) + at)[v] = packed<T>(b);
            }
        }
    };
    find_mean(false, part[0]);
    float v = spread(false, part[1]);
    const float var = v + a.eps;
    rstd = rsqrtf(var);
    if (__builtin_expect(var >= kLeast && v <= kMost && rest * rest <= var, true)) {
        outputs(false);
    } else {
        // Squares that F32 does not hold: the row times 2^-80, or the deviations times
        // 2^90, which the norm cancels.  (The squares of 2^22 values whose variance is
        // below 2^-80 then add up to 2^122 at most, and 2^-149's is 2^-118.)  Or values
        // that lie closer together than their mean's rounding (equal ones, above all: what
        // is left of that rounding is no variance): the mean is corrected until what is
        // left of it is below the root of the variance, mostly once.
        mean += rest;
        if (var < kLeast) {
            wide = 0x1p90f;
        } else if (!(v <= kMost)) {
            scale = 0x1p-80f;
            find_mean(true, part[0]);
        }
        // (A loop for 1024 threads: 2048 rows of 32768 BF16 93 us, with none 96; fewer threads
        // take more registers with one.)
#pragma unroll(THREADS == 1024 ? 1 : 2)
        for (int again = 0; again < 2; ++again) {
            if (again) mean += rest / wide;
            v = spread(true, part[2 + again]);
            rstd = v + a.eps * (scale * wide) * (scale * wide);
            if (!(rest * rest > rstd)) break;
        }
        // (Equal values leave eps alone, and F32 does not hold that times 2^-160.)
        const bool equal = v == 0.f && scale != 1.f;
        rstd = rsqrtf(equal ? a.eps : rstd);
        outputs(true);
        if (equal) wide = 1.f / scale;
    }
    if (t == 0) {
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


// ---- rows in shared memory ahead of their sums

constexpr int kSmCount = 152;

// A thread takes pieces of 16 bytes of a row, piece q at (thread + q row threads).
template <typename T>
constexpr int piece_values()
{
    return static_cast<int>(16 / sizeof(T));
}

// Rows in flight for each thread: what 192 KB of shared memory hold of dy, h and dsum.
constexpr size_t kRingBytes = 192 * 1024;
constexpr int ring_stages(int threads, int pieces) { return static_cast<int>(kRingBytes / (3 * 16 * threads * pieces)); }

__device__ __forceinline__ void copy_ahead(uint4 *dst, const uint8_t *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ptx::smem_addr(dst)), "l"(reinterpret_cast<uint64_t>(src)) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copies_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

__device__ __forceinline__ void pairs(const uint4 &p, float2 (&v)[2], float)
{
    v[0] = make_float2(__uint_as_float(p.x), __uint_as_float(p.y));
    v[1] = make_float2(__uint_as_float(p.z), __uint_as_float(p.w));
}
template <typename T>
__device__ __forceinline__ void pairs(const uint4 &p, float2 (&v)[4], T)
{
    unpack(Pack<T>{p}, v);
}
__device__ __forceinline__ uint4 piece(const float2 (&v)[2], float)
{
    return make_uint4(__float_as_uint(v[0].x), __float_as_uint(v[0].y), __float_as_uint(v[1].x), __float_as_uint(v[1].y));
}
template <typename T>
__device__ __forceinline__ uint4 piece(const float2 (&v)[4], T)
{
    return packed<T>(v).a;
}

// `threads` a row: whole warps, or 8 or 16 lanes (SMALL); groups of them take rows in
// turn.  A thread copies its own pieces of the next rows into its own places of shared
// memory, and reads them again when it comes to the row: no barrier but the row's sum.
// SUMS: dw and db of the thread's columns stay in its registers; else dx alone is made.
//
// 16 values a thread, 32 without SUMS: what a row costs besides its values (the sum's
// exchanges and barrier, addresses, factors) is most of the instructions with 8 (8192
// rows of 5120 BF16 71 us, with 16 67), and spills cost more than they save (640
// threads: 89).  Bound by memory where rows stand side by side (16384 x 4096 BF16 87 us,
// 0.92 of the copy rate), else by the wait for each row's sum (8192 x 8192 BF16 90 us,
// 0.89; 8192 x 5120 67, 0.75).
template <typename T, int THREADS, int PIECES, bool SUMS, bool SMALL>
__global__ void __launch_bounds__(THREADS, 1) layernorm_grad_ring_kernel(const NormGradArgs a, const int threads)
{
    constexpr int kStages = ring_stages(THREADS, PIECES), kValues = piece_values<T>(), kPairs = kValues / 2, kTensor = PIECES * THREADS;
    constexpr int kWarps = THREADS / 32, kOwn = SUMS ? PIECES : 1;
    extern __shared__ __align__(16) uint8_t ring_raw[];
    __shared__ float2 part[2][kWarps];
    uint4 *const ring = reinterpret_cast<uint4 *>(ring_raw) + threadIdx.x;   // [stage][tensor][piece][thread]
    ptx::launch_dependents();
    ptx::grid_dependency_wait();
    const int groups = static_cast<int>(blockDim.x) / threads, group = threadIdx.x / threads, v = threadIdx.x % threads;
    const int lane = threadIdx.x % 32, warps = threads / 32, pieces = a.K / kValues;
    auto in = [&](int q) { return v + q * threads < pieces; };
    // rows are counted in 32 bits (M <= 2^22), their addresses by a running offset; every
    // thread goes through the same number of turns
    const int M = static_cast<int>(a.M), step = static_cast<int>(gridDim.x) * groups, first = static_cast<int>(blockIdx.x) * groups + group;
    const size_t stride = static_cast<size_t>(step) * pieces * 16;
    size_t at = (static_cast<size_t>(first) * pieces + v) * 16;
    float2 w[PIECES][kPairs] = {};
#pragma unroll
    for (int q = 0; q < PIECES; ++q)
        if (in(q)) pairs(static_cast<const uint4 *>(a.weight)[v + q * threads], w[q], T{});
    auto ahead = [&](bool there, size_t from, int stage) {
        uint4 *const to = ring + stage * 3 * kTensor;
#pragma unroll
        for (int q = 0; q < PIECES; ++q) {
            if (!in(q) || !there) continue;
            const size_t f = from + static_cast<size_t>(q * threads) * 16;
            copy_ahead(to + q * THREADS, static_cast<const uint8_t *>(a.dy) + f);
            copy_ahead(to + q * THREADS + kTensor, static_cast<const uint8_t *>(a.h) + f);
            if (a.dsum) copy_ahead(to + q * THREADS + 2 * kTensor, static_cast<const uint8_t *>(a.dsum) + f);
        }
        copies_commit();
    };
#pragma unroll
    for (int s = 0; s < kStages; ++s) ahead(first + s * step < M, at + s * stride, s);
    float2 dw[kOwn][kPairs] = {}, db[kOwn][kPairs] = {};
    float mean = 0.f, rstd = 0.f;
    if (first < M) mean = a.mean[first], rstd = a.rstd[first];
    int stage = 0, turn = 0;
    const float inv = 1.f / static_cast<float>(a.K);
    const int blocks_first = static_cast<int>(blockIdx.x) * groups;
    for (int row0 = blocks_first, row = first; row0 < M; row0 += step, row += step, at += stride, turn ^= 1) {
        const bool live = row < M;
        copies_wait<kStages - 1>();
        const float2 half = {0.5f, 0.5f}, off = {-0.5f * mean, -0.5f * mean}, r = {rstd, rstd}, r2 = {2.f * rstd, 2.f * rstd};
        if (row + step < M) mean = a.mean[row + step], rstd = a.rstd[row + step];
        const uint4 *const from = ring + stage * 3 * kTensor;
        float2 g[PIECES][kPairs], x[PIECES][kPairs], s0 = {0.f, 0.f}, s1 = {0.f, 0.f};
#pragma unroll
        for (int q = 0; q < PIECES; ++q) {
            if (!in(q) || !live) continue;
            pairs(from[q * THREADS], g[q], T{});
            pairs(from[q * THREADS + kTensor], x[q], T{});
#pragma unroll
            for (int j = 0; j < kPairs; ++j) {
                x[q][j] = __fmul2_rn(__ffma2_rn(half, x[q][j], off), r2);   // normal_of
                if constexpr (SUMS) {
                    dw[q][j] = __ffma2_rn(g[q][j], x[q][j], dw[q][j]);
                    db[q][j] = __fadd2_rn(db[q][j], g[q][j]);
                }
                g[q][j] = __fmul2_rn(g[q][j], w[q][j]);
                s0 = __fadd2_rn(s0, g[q][j]);
                s1 = __ffma2_rn(g[q][j], x[q][j], s1);
            }
        }
        float2 s = make_float2(s0.x + s0.y, s1.x + s1.y);
        if constexpr (SMALL) {
            __syncwarp();
            for (int d = threads / 2; d; d >>= 1) {
                s.x += __shfl_xor_sync(0xffffffffu, s.x, d);
                s.y += __shfl_xor_sync(0xffffffffu, s.y, d);
            }
        } else {
            __syncwarp();
            float t = lanes_sum(s);
            if (warps > 1) {
                float2 *const mine = part[turn] + group * warps;
                if (lane % 16 == 0) reinterpret_cast<float *>(mine + v / 32)[lane / 16] = t;
                asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(threads) : "memory");
                t = lanes_sum(lane < warps ? mine[lane] : make_float2(0.f, 0.f));
            }
            s = make_float2(__shfl_sync(0xffffffffu, t, 0), __shfl_sync(0xffffffffu, t, 16));
        }
        const float2 mg = {-s.x * inv, -s.x * inv}, mgx = {-s.y * inv, -s.y * inv};
#pragma unroll
        for (int q = 0; q < PIECES; ++q) {
            if (!in(q) || !live) continue;
            float2 o[kPairs] = {};
            if (a.dsum) pairs(from[q * THREADS + 2 * kTensor], o, T{});
#pragma unroll
            for (int j = 0; j < kPairs; ++j) o[j] = __ffma2_rn(r, __ffma2_rn(x[q][j], mgx, __fadd2_rn(g[q][j], mg)), o[j]);
            *reinterpret_cast<uint4 *>(static_cast<uint8_t *>(a.dx) + at + static_cast<size_t>(q * threads) * 16) = piece(o, T{});
        }
        ahead(row + kStages * step < M, at + kStages * stride, stage);
        stage = stage + 1 == kStages ? 0 : stage + 1;
    }
    copies_wait<0>();
    if constexpr (SUMS) {
        // Column k of dw, then of db: the groups' through shared memory, in their order.
        const int width = threads * PIECES * kValues;
        float *const to = a.parts + static_cast<size_t>(blockIdx.x) * 2 * a.K, *const sums = reinterpret_cast<float *>(ring_raw);
        const bool single = groups == 1;
        float *const mine = single ? to : sums + group * 2 * width;   // [group][2][width]
        const int db_at = single ? a.K : width;
        if (!single) __syncthreads();
#pragma unroll
        for (int q = 0; q < PIECES; ++q) {
            if (single && !in(q)) continue;
            const int k = (v + q * threads) * kValues;
#pragma unroll
            for (int j = 0; j < kPairs; j += 2) {
                *reinterpret_cast<float4 *>(mine + k + 2 * j) = make_float4(dw[q][j].x, dw[q][j].y, dw[q][j + 1].x, dw[q][j + 1].y);
                *reinterpret_cast<float4 *>(mine + db_at + k + 2 * j) = make_float4(db[q][j].x, db[q][j].y, db[q][j + 1].x, db[q][j + 1].y);
            }
        }
        if (single) return;
        __syncthreads();
        for (int c = threadIdx.x; c < 2 * width; c += static_cast<int>(blockDim.x)) {
            float sum = 0.f;
#pragma unroll 4
            for (int i = 0; i < groups; ++i) sum += sums[i * 2 * width + c];
            const int which = c >= width, k = c - which * width;
            if (k < a.K) to[which * a.K + k] = sum;
        }
    }
}

// A row of any length, read twice: its dx.
template <typename T, int THREADS>
__global__ void __launch_bounds__(THREADS) layernorm_grad_long_kernel(const NormGradArgs a)
{
    __shared__ float2 part[THREADS / 32];
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
    const float2 t = block_sum<THREADS>(make_float2(s[0], s[1]), part);
    const float mg = t.x / static_cast<float>(a.K), mgx = t.y / static_cast<float>(a.K);
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
        constexpr int kAtOnce = 8;   // loads in flight
        int b = slice;
        for (; b + (kAtOnce - 1) * kSumSlices < blocks; b += kAtOnce * kSumSlices) {
            float x[kAtOnce];
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) x[i] = parts[static_cast<size_t>(b + i * kSumSlices) * 2 * K + c];
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) sum += x[i];
        }
        float x[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce - 1; ++i)
            x[i] = b + i * kSumSlices < blocks ? parts[static_cast<size_t>(b + i * kSumSlices) * 2 * K + c] : 0.f;
#pragma unroll
        for (int i = 0; i < kAtOnce - 1; ++i) sum += x[i];
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
constexpr int kRingVecs = 1024;   // the same for the ring with dw and db
constexpr int kColumnThreads = 512;

// How the ring takes rows of `vecs` vectors: two a thread, rows side by side.
struct RingShape {
    int threads;   // of a row: 8 or 16 lanes, or whole warps
    int rows;      // side by side
};
RingShape ring_shape(int64_t vecs)
{
    const int64_t n = (vecs + 1) / 2;
    const int threads = n <= 8 ? 8 : n <= 16 ? 16 : static_cast<int>((n + 31) / 32 * 32);
    return {threads, 512 / threads};
}

template <typename T, int THREADS, int VPT, bool LONG = false>
cudaError_t launch_norm(const NormArgs &a, cudaStream_t stream)
{
    cudaLaunchAttribute attr;
    constexpr int kThreads = THREADS == 32 ? kRowThreads : THREADS, kRows = kThreads / THREADS;
    const cudaLaunchConfig_t cfg = config(static_cast<unsigned>((a.M + kRows - 1) / kRows), kThreads, stream, &attr);
    return note_error(cudaLaunchKernelEx(&cfg, layernorm_kernel<T, THREADS, VPT, LONG>, a), "layernorm_kernel launch");
}

// Measured with the residual, BF16, in us, the other shapes beside it (threads x vectors):
// 100000 x 256 35 (128 x 1 102), 60000 x 512 37 (128 x 1 63; one of 64 rows 2.1 and 1.7), 60000 x
// 1024 71 (32 x 4 73, 64 x 2 72; 64 rows 1.7, 3.0, 2.0), 30000 x 2048 75 (128 x 2 71, 64 x 4 72; 64
// rows 1.9, 2.0, 2.7), 20000 x 2560 67 (512 x 1 91, 128 x 4 60), 16384 x 4096 78 (91, 79), 12000 x
// 6144 86 (512 x 2 97, 1024 x 1 159), 8192 x 8192 79 (512 x 2 80, 1024 x 1 120), 4096 x 16384 80
// (1024 x 2 120).
template <typename T>
cudaError_t launch_norm_type(const NormArgs &a, cudaStream_t stream)
{
    if (a.vecs <= 32) return launch_norm<T, 32, 1>(a, stream);
    if (a.vecs <= 64) return launch_norm<T, 32, 2>(a, stream);
    if (a.vecs <= 128) return launch_norm<T, 128, 1>(a, stream);
    if (a.vecs <= 256) return launch_norm<T, 256, 1>(a, stream);
    if (a.vecs <= 512) return launch_norm<T, 256, 2>(a, stream);
    if (a.vecs <= 768) return launch_norm<T, 256, 3>(a, stream);
    if (a.vecs <= 1024) return launch_norm<T, 256, 4>(a, stream);
    if (a.vecs <= kLongVecs) return launch_norm<T, 512, 4>(a, stream);
    if constexpr (sizeof(T) == 2)
        if (a.vecs <= 2 * kLongVecs) return launch_norm<T, 1024, 4>(a, stream);
    return launch_norm<T, 512, 4, true>(a, stream);
}

template <typename T, int THREADS, int VECS, bool SUMS, bool SMALL>
cudaError_t launch_ring(const NormGradArgs &a, int blocks, RingShape shape, cudaStream_t stream)
{
    auto *const kernel = layernorm_grad_ring_kernel<T, THREADS, VECS * kVec / piece_values<T>(), SUMS, SMALL>;
    const cudaError_t e = note_error(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kRingBytes)),
                                     "layernorm_grad_ring_kernel shared memory");
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr;
    cudaLaunchConfig_t cfg = config(static_cast<unsigned>(blocks), static_cast<unsigned>(shape.rows * shape.threads), stream, &attr);
    cfg.dynamicSmemBytes = kRingBytes;
    return note_error(cudaLaunchKernelEx(&cfg, kernel, a, shape.threads), "layernorm_grad_ring_kernel launch");
}

template <typename T>
cudaError_t launch_grad_type(const NormGradArgs &a, int blocks, cudaStream_t stream)
{
    if (a.vecs <= kRingVecs) {
        const RingShape shape = ring_shape(a.vecs);
        if (shape.threads < 32) return launch_ring<T, 512, 2, true, true>(a, blocks, shape, stream);
        return launch_ring<T, 512, 2, true, false>(a, blocks, shape, stream);
    }
    constexpr int kThreads = kColumnThreads;
    cudaLaunchAttribute attr;
    cudaLaunchConfig_t cfg = config(static_cast<unsigned>(a.M), kThreads, stream, &attr);
    // dw and db first: dx may be dy
    cfg.gridDim = dim3(static_cast<unsigned>((a.vecs + kThreads - 1) / kThreads), static_cast<unsigned>(blocks), 1);
    cudaError_t e = note_error(cudaLaunchKernelEx(&cfg, layernorm_grad_columns_kernel<T, kThreads>, a), "layernorm_grad_columns_kernel launch");
    if (e != cudaSuccess) return e;
    if (a.vecs <= 2 * kRingVecs)
        return launch_ring<T, 512, 4, false, false>(a, static_cast<int>(a.M < kSmCount ? a.M : kSmCount), {512, 1}, stream);
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
    // A block to an SM, and of four turns and more as few as take the same number (4096
    // rows of 1024 BF16: 128 blocks 11.5 us, 152 blocks 13.4; 333 rows of 5120 F16, three
    // turns: 111 blocks and the norm before them 17.0, 152 blocks 16.0).  Long rows have
    // columns for many blocks of kColumnThreads, and fewer parts the longer they are.
    const int64_t vecs = K / kVec, rows = vecs <= kRingVecs ? ring_shape(vecs).rows : 1;
    const int64_t across = (vecs + kColumnThreads - 1) / kColumnThreads, tiles = (M + rows - 1) / rows;
    const int64_t most = vecs <= kRingVecs ? kSmCount : across >= 40 ? 8 : across <= 5 ? 64 : 320 / across, turns = (tiles + most - 1) / most;
    return turns >= 4 ? (tiles + turns - 1) / turns : tiles < most ? tiles : most;
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
