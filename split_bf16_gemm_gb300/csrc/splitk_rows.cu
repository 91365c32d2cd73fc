// splitk_rows.cu -- rows sorted by expert and back.
//
// Entry i = m top + j says that token m goes to expert experts[i]; one outside
// [0, G) goes nowhere.  The sort is stable: run g holds g's entries in rising
// order, offsets[g] = how many entries have a lower expert, slots[i] the entry's
// row (-1: nowhere), source[r] the row's entry (-1 behind the last run).
//
// sort_kernel: one thread-block cluster sorts all entries by counting.  Every warp
// takes consecutive entries; it counts them by expert (lanes with the same expert
// find one another, one of them adds), the warps' counts become sums over the
// warps, the blocks' over the cluster through distributed shared memory, the
// experts' a scan; then each warp goes over its entries once more and knows every
// entry's row.  One launch, no workspace, no atomics on memory: the same bits
// every time.
//
// dispatch_kernel: a token's row is read once and written to each of its rows.
// For few entries (sorted_here) every block finds the rows of its own tokens by
// itself, comparing their entries with all others, and one more block makes the
// offsets: one launch instead of two.
//
// combine_kernel: out[m] = sum_j shares[m,j] rows[slots[m,j]] in F32, j rising,
// rounded once; combine_grad_kernel: drows[slots[m,j]] = shares[m,j] dout[m] and
// dshares[m,j] = sum_k dout[m,k] rows[slots[m,j],k], dout read once for all j.
//
// All but the sort are bound by memory.

#include "ptx.cuh"
#include "rows.cuh"
#include "splitk_internal.h"

namespace splitk {
namespace {

constexpr int kThreads = 256;

// ------------------------------------------------------------------ sort

constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32;
constexpr int kSortCluster = 8;
constexpr int kMaxGroups = 1024;   // SPLITK_MAX_GROUPS: an expert to a thread

__device__ __forceinline__ void cluster_arrive_release()
{
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}

__device__ __forceinline__ int load_peer(uint32_t addr, uint32_t rank)
{
    int v;
    asm volatile(
        "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.s32 %0, [a];\n}\n"
        : "=r"(v)
        : "r"(addr), "r"(rank)
        : "memory");
    return v;
}

// counts: [kSortWarps][G] of each warp, [G] of the block (its peers read them), [G]
// first rows of the block's entries.  T entries, `each` (a multiple of 32) to a warp.
__global__ void __launch_bounds__(kSortThreads) sort_kernel(const int *experts, int *offsets, int *slots, int *source, int T, int G,
                                                            int each, int blocks)
{
    extern __shared__ int counts[];
    __shared__ int part[kSortWarps];
    int *const block_counts = counts + kSortWarps * G, *const bases = block_counts + G;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int rank = static_cast<int>(blockIdx.x);
    for (int i = threadIdx.x; i < kSortWarps * G; i += kSortThreads) counts[i] = 0;
    ptx::grid_dependency_wait();
    // after the wait: what the next grid reads besides this sort's outputs is there when it starts
    ptx::launch_dependents();
    __syncthreads();
    int *const mine = counts + warp * G;
    const int64_t first = static_cast<int64_t>(rank * kSortWarps + warp) * each;
    const int begin = static_cast<int>(first < T ? first : T), end = static_cast<int>(first + each < T ? first + each : T);
    auto expert_of = [&](int i) {
        const int e = i < end ? experts[i] : -1;
        return static_cast<unsigned>(e) < static_cast<unsigned>(G) ? e : -1;
    };
    for (int i = begin; i < end; i += 32) {
        const int e = expert_of(i + lane);
        const uint32_t same = __match_any_sync(0xffffffffu, e);
        if (e >= 0 && lane == __ffs(same) - 1) mine[e] += __popc(same);
        __syncwarp();
    }
    __syncthreads();
    // a warp's counts become those of the warps before it
    const int g = threadIdx.x;
    int sum = 0;
    if (g < G) {
#pragma unroll 8
        for (int w = 0; w < kSortWarps; ++w) {
            const int c = counts[w * G + g];
            counts[w * G + g] = sum;
            sum += c;
        }
        block_counts[g] = sum;
    }
    int before = 0, all = sum;
    __syncwarp();
    if (blocks > 1) {
        cluster_arrive_release();
        ptx::cluster_wait();
        if (g < G) {
            all = 0;
            const uint32_t at = ptx::smem_addr(block_counts + g);
            for (int r = 0; r < blocks; ++r) {
                const int c = load_peer(at, static_cast<uint32_t>(r));
                if (r < rank) before += c;
                all += c;
            }
        }
        __syncwarp();
        cluster_arrive_release();   // no block leaves while its counts may be read
    }
    // the experts' first rows
    int scan = all;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int x = __shfl_up_sync(0xffffffffu, scan, d);
        if (lane >= d) scan += x;
    }
    if (lane == 31) part[warp] = scan;
    __syncthreads();
    int lower = 0, total = 0;
    for (int w = 0; w < kSortWarps; ++w) {
        if (w < warp) lower += part[w];
        total += part[w];
    }
    const int start = lower + scan - all;
    if (g < G) {
        bases[g] = start + before;
        if (rank == 0) offsets[g] = start;
    }
    if (rank == 0 && g == 0) offsets[G] = total;
    __syncthreads();
    for (int i = begin; i < end; i += 32) {
        const int e = expert_of(i + lane);
        const uint32_t same = __match_any_sync(0xffffffffu, e);
        int at = -1;
        if (e >= 0) {
            const int rank_here = __popc(same & ((1u << lane) - 1u));
            at = bases[e] + mine[e] + rank_here;
            if (source) source[at] = i + lane;
        }
        if (i + lane < end) slots[i + lane] = at;
        __syncwarp();
        if (e >= 0 && lane == __ffs(same) - 1) mine[e] += __popc(same);
        __syncwarp();
    }
    if (source)
        for (int r = total + rank * kSortThreads + static_cast<int>(threadIdx.x); r < T; r += blocks * kSortThreads) source[r] = -1;
    __syncwarp();
    if (blocks > 1) ptx::cluster_wait();
}

// ------------------------------------------------------------------ rows to their experts

struct DispatchArgs {
    const int *experts;      // sorted_here: [M,top]
    const uint4 *x;          // [M, vecs] 16-byte vectors
    const float *scales;     // [M, blocks] or nullptr
    int *offsets, *slots, *source;
    uint4 *rows;
    float *row_scales;
    int M, top, G, vecs, blocks;
};

constexpr int kHere = 1024;                    // most entries that every block sorts by itself
constexpr int kMaxTop = 32;

// The block's token: where its entries go, by comparison with every entry.
__device__ __forceinline__ void places_of(const DispatchArgs &a, int m, int *place)
{
    const int T = a.M * a.top;
    for (int j = threadIdx.x; j < a.top; j += kThreads) place[j] = 0;
    __syncthreads();
    int e[kHere / kThreads];
#pragma unroll
    for (int i = 0; i < kHere / kThreads; ++i) {
        const int t = i * kThreads + static_cast<int>(threadIdx.x);
        e[i] = t < T ? a.experts[t] : -1;
    }
    for (int j = 0; j < a.top; ++j) {
        const int at = m * a.top + j, mine = a.experts[at];
        int lower = 0;
#pragma unroll
        for (int i = 0; i < kHere / kThreads; ++i) {
            const int t = i * kThreads + static_cast<int>(threadIdx.x);
            lower += e[i] >= 0 && (e[i] < mine || (e[i] == mine && t < at));
        }
        lower = __reduce_add_sync(0xffffffffu, lower);
        if (threadIdx.x % 32 == 0 && lower) atomicAdd(&place[j], lower);   // (whole numbers: any order)
    }
    __syncthreads();
    if (threadIdx.x < a.top) {
        const int at = m * a.top + static_cast<int>(threadIdx.x);
        const bool in = static_cast<unsigned>(a.experts[at]) < static_cast<unsigned>(a.G);
        if (!in) place[threadIdx.x] = -1;
        a.slots[at] = place[threadIdx.x];
        if (in && a.source) a.source[place[threadIdx.x]] = at;
    }
    __syncthreads();
}

// The last block of a launch that sorts: offsets, and the end of `source`.
__device__ __forceinline__ void offsets_of(const DispatchArgs &a, int *counts)
{
    const int T = a.M * a.top;
    for (int g = threadIdx.x; g <= a.G; g += kThreads) counts[g] = 0;
    __syncthreads();
    for (int t = threadIdx.x; t < T; t += kThreads) {
        const int e = a.experts[t];
        if (static_cast<unsigned>(e) < static_cast<unsigned>(a.G)) atomicAdd(&counts[e], 1);
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        int before = 0;
        for (int g0 = 0; g0 <= a.G; g0 += 32) {
            const int g = g0 + static_cast<int>(threadIdx.x);
            const int c = g < a.G ? counts[g] : 0;
            int scan = c;
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const int x = __shfl_up_sync(0xffffffffu, scan, d);
                if (static_cast<int>(threadIdx.x) >= d) scan += x;
            }
            if (g <= a.G) a.offsets[g] = before + scan - c;
            before += __shfl_sync(0xffffffffu, scan, 31);
        }
        if (threadIdx.x == 0) counts[0] = before;
    }
    __syncthreads();
    if (a.source)
        for (int r = counts[0] + static_cast<int>(threadIdx.x); r < T; r += kThreads) a.source[r] = -1;
}

// A token to each block of x, split over the blocks of y along the row.
template <bool HERE>
__global__ void __launch_bounds__(kThreads) dispatch_kernel(const DispatchArgs a)
{
    __shared__ int place[HERE ? 1032 : kMaxTop];   // (HERE: G + 1 counts of the last block)
    if constexpr (HERE) ptx::launch_dependents();
    ptx::grid_dependency_wait();
    if constexpr (!HERE) ptx::launch_dependents();
    const int m = static_cast<int>(blockIdx.x);
    if (HERE && m == a.M) {
        offsets_of(a, place);
        return;
    }
    if constexpr (HERE) {
        places_of(a, m, place);
    } else {
        if (threadIdx.x < a.top) place[threadIdx.x] = a.slots[static_cast<int64_t>(m) * a.top + threadIdx.x];
        __syncthreads();
    }
    const uint4 *const x = a.x + static_cast<int64_t>(m) * a.vecs;
    for (int v = threadIdx.x; v < a.vecs; v += kThreads) {
        const uint4 p = x[v];
        for (int j = 0; j < a.top; ++j)
            if (place[j] >= 0) a.rows[static_cast<int64_t>(place[j]) * a.vecs + v] = p;
    }
    if (a.scales)
        for (int b = threadIdx.x; b < a.blocks; b += kThreads) {
            const float s = a.scales[static_cast<int64_t>(m) * a.blocks + b];
            for (int j = 0; j < a.top; ++j)
                if (place[j] >= 0) a.row_scales[static_cast<int64_t>(place[j]) * a.blocks + b] = s;
        }
}

// ------------------------------------------------------------------ and back

struct CombineArgs {
    const void *rows, *dout;
    const int *slots;
    const float *shares;     // or nullptr: ones
    void *out, *drows;
    float *dshares;
    int64_t M;
    int top, vecs, T;
};

// TPR threads a token.
template <typename T, typename O, int TPR>
__global__ void __launch_bounds__(kThreads) combine_kernel(const CombineArgs a)
{
    ptx::launch_dependents();
    ptx::grid_dependency_wait();
    const int64_t m = static_cast<int64_t>(blockIdx.x) * (kThreads / TPR) + threadIdx.x / TPR;
    if (m >= a.M) return;
    const int *const slots = a.slots + m * a.top;
    const Pack<T> *const rows = static_cast<const Pack<T> *>(a.rows);
    Pack<O> *const out = static_cast<Pack<O> *>(a.out) + m * a.vecs;
    for (int v = threadIdx.x % TPR; v < a.vecs; v += TPR) {
        float sum[kVec] = {};
#pragma unroll 4
        for (int j = 0; j < a.top; ++j) {
            const int r = slots[j];
            if (static_cast<unsigned>(r) < static_cast<unsigned>(a.T)) {
                const float s = a.shares ? a.shares[m * a.top + j] : 1.f;
                float x[kVec];
                unpack(rows[static_cast<int64_t>(r) * a.vecs + v], x);
#pragma unroll
                for (int i = 0; i < kVec; ++i) sum[i] = fmaf(s, x[i], sum[i]);
            }
        }
        Pack<O> p;
        pack(sum, p);
        out[v] = p;
    }
}

// One token a block.
template <typename T>
__global__ void __launch_bounds__(kThreads) combine_grad_kernel(const CombineArgs a)
{
    constexpr int kGroup = 4;   // rows at once
    __shared__ float part[kGroup][kThreads / 32];
    ptx::launch_dependents();
    ptx::grid_dependency_wait();
    const int64_t m = blockIdx.x;
    const Pack<T> *const rows = static_cast<const Pack<T> *>(a.rows), *const dout = static_cast<const Pack<T> *>(a.dout) + m * a.vecs;
    Pack<T> *const drows = static_cast<Pack<T> *>(a.drows);
    for (int j0 = 0; j0 < a.top; j0 += kGroup) {
        int r[kGroup];
        float s[kGroup], dot[kGroup] = {};
#pragma unroll
        for (int j = 0; j < kGroup; ++j) {
            r[j] = j0 + j < a.top ? a.slots[m * a.top + j0 + j] : -1;
            if (static_cast<unsigned>(r[j]) >= static_cast<unsigned>(a.T)) r[j] = -1;
            s[j] = r[j] >= 0 && a.shares ? a.shares[m * a.top + j0 + j] : 1.f;
        }
        for (int v = threadIdx.x; v < a.vecs; v += kThreads) {
            float d[kVec];
            unpack(dout[v], d);
            Pack<T> x[kGroup];
            if (rows) {
#pragma unroll
                for (int j = 0; j < kGroup; ++j)
                    if (r[j] >= 0) x[j] = rows[static_cast<int64_t>(r[j]) * a.vecs + v];
            }
#pragma unroll
            for (int j = 0; j < kGroup; ++j) {
                if (r[j] < 0) continue;
                float y[kVec];
                if (rows) {
                    unpack(x[j], y);
#pragma unroll
                    for (int i = 0; i < kVec; ++i) dot[j] = fmaf(d[i], y[i], dot[j]);
                }
                if (drows) {
#pragma unroll
                    for (int i = 0; i < kVec; ++i) y[i] = s[j] * d[i];
                    Pack<T> p;
                    pack(y, p);
                    drows[static_cast<int64_t>(r[j]) * a.vecs + v] = p;
                }
            }
        }
        if (a.dshares) {
#pragma unroll
            for (int j = 0; j < kGroup; ++j) {
#pragma unroll
                for (int d = 16; d; d >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], d);
                if (threadIdx.x % 32 == 0) part[j][threadIdx.x / 32] = dot[j];
            }
            __syncthreads();
            if (threadIdx.x < kGroup && j0 + static_cast<int>(threadIdx.x) < a.top) {
                float sum = 0.f;
#pragma unroll
                for (int w = 0; w < kThreads / 32; ++w) sum += part[threadIdx.x][w];
                a.dshares[m * a.top + j0 + threadIdx.x] = sum;
            }
            __syncthreads();
        }
    }
}

template <typename T, typename O>
cudaError_t launch_combine_types(const CombineArgs &a, cudaStream_t stream)
{
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = config(static_cast<unsigned>(a.M), kThreads, stream, &attr);
    return note_error(cudaLaunchKernelEx(&cfg, combine_kernel<T, O, kThreads>, a), "combine_kernel launch");
}

template <typename T>
cudaError_t launch_combine_type(const CombineArgs &a, int out_dtype, cudaStream_t stream)
{
    return out_dtype == 0   ? launch_combine_types<T, float>(a, stream)
           : out_dtype == 1 ? launch_combine_types<T, __half>(a, stream)
                            : launch_combine_types<T, __nv_bfloat16>(a, stream);
}

template <typename T>
cudaError_t launch_combine_grad_type(const CombineArgs &a, cudaStream_t stream)
{
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = config(static_cast<unsigned>(a.M), kThreads, stream, &attr);
    return note_error(cudaLaunchKernelEx(&cfg, combine_grad_kernel<T>, a), "combine_grad_kernel launch");
}

cudaError_t launch_sort(const DispatchProblem &p, cudaStream_t stream)
{
    const int T = static_cast<int>(p.M * p.top), G = static_cast<int>(p.G);
    int blocks = 1;
    while (blocks < kSortCluster && T > blocks * kSortThreads * 2) blocks *= 2;
    const int warps = blocks * kSortWarps;
    const int each = ((T + warps - 1) / warps + 31) / 32 * 32;
    const size_t smem = static_cast<size_t>(kSortWarps + 2) * G * sizeof(int);
    cudaError_t e = note_error(cudaFuncSetAttribute(sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                    (kSortWarps + 2) * kMaxGroups * static_cast<int>(sizeof(int))),
                               "sort_kernel shared memory");
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = config(static_cast<unsigned>(blocks), kSortThreads, stream, attr);
    cfg.dynamicSmemBytes = smem;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(blocks);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
    return note_error(cudaLaunchKernelEx(&cfg, sort_kernel, p.experts, p.offsets, p.slots, p.source, T, G, each, blocks),
                      "sort_kernel launch");
}

}  // namespace

cudaError_t launch_dispatch(const DispatchProblem &p, cudaStream_t stream)
{
    const DispatchArgs a = {p.experts,
                            static_cast<const uint4 *>(p.x),
                            p.scales,
                            p.offsets,
                            p.slots,
                            p.source,
                            static_cast<uint4 *>(p.rows),
                            p.row_scales,
                            static_cast<int>(p.M),
                            static_cast<int>(p.top),
                            static_cast<int>(p.G),
                            static_cast<int>(p.row_bytes / 16),
                            static_cast<int>(p.scale_blocks)};
    const bool here = p.x && p.M * p.top <= kHere;
    if (!here) {
        const cudaError_t e = launch_sort(p, stream);
        if (e != cudaSuccess || !p.x || p.M == 0) return e;
    }
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = config(static_cast<unsigned>(p.M + (here ? 1 : 0)), kThreads, stream, &attr);
    return note_error(here ? cudaLaunchKernelEx(&cfg, dispatch_kernel<true>, a) : cudaLaunchKernelEx(&cfg, dispatch_kernel<false>, a),
                      "dispatch_kernel launch");
}

cudaError_t launch_combine(const CombineProblem &p, cudaStream_t stream)
{
    const CombineArgs a = {p.rows, p.dout, p.slots, p.shares, p.out, p.drows, p.dshares, p.M, static_cast<int>(p.top),
                           static_cast<int>(p.K / kVec), static_cast<int>(p.M * p.top)};
    if (p.dout)
        return p.dtype == 0   ? launch_combine_grad_type<float>(a, stream)
               : p.dtype == 1 ? launch_combine_grad_type<__half>(a, stream)
                              : launch_combine_grad_type<__nv_bfloat16>(a, stream);
    return p.dtype == 0   ? launch_combine_type<float>(a, p.out_dtype, stream)
           : p.dtype == 1 ? launch_combine_type<__half>(a, p.out_dtype, stream)
                          : launch_combine_type<__nv_bfloat16>(a, p.out_dtype, stream);
}

}  // namespace splitk
