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
// entry's row.  One launch (and one that writes `source`, where it is asked for
// without rows and more than 16384 entries), no workspace, no atomics on memory: the
// same bits every time.
//
// dispatch_kernel: a token's row is read once and written to each of its rows.
// For up to 2048 entries every block finds the rows of its own tokens by
// itself, comparing their entries with all others, and one more block makes the
// offsets: one launch instead of two.
//
// combine_kernel: out[m] = sum_j shares[m,j] rows[slots[m,j]] in F32, j rising,
// rounded once; combine_grad_kernel: drows[slots[m,j]] = shares[m,j] dout[m] and
// dshares[m,j] = sum_k dout[m,k] rows[slots[m,j],k], dout read once for all j.
//
// All but the sort are bound by memory.

#include <atomic>

#include "ptx.cuh"
#include "rows.cuh"
#include "splitk_internal.h"

namespace splitk {
namespace {

constexpr int kThreads = 256;

// ------------------------------------------------------------------ sort

constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32;
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

// The lanes with the same e (>= 0, below 2^BITS) as this one.  A vote a bit: about 4
// BITS operations, where __match_any_sync's time goes by the number of different
// values (2^22 entries of 256 experts 1036 us with it).
template <int BITS>
__device__ __forceinline__ uint32_t same_as(int e)
{
    uint32_t same = __ballot_sync(0xffffffffu, e >= 0);
#pragma unroll
    for (int b = 0; b < BITS; ++b) {
        const bool set = e >> b & 1;
        const uint32_t with = __ballot_sync(0xffffffffu, set);
        same &= set ? with : ~with;
    }
    return same;
}

// counts: [kSortWarps][G] of each warp, [G] of the block (its peers read them), [G]
// first rows of the block's entries.  T entries, `each` (a multiple of 32) to a warp.
template <int BITS, int kBatch>
__global__ void __launch_bounds__(kSortThreads) sort_kernel(const int *experts, int *offsets, int *slots, int *source, int T, int G,
                                                            int each, int blocks, int rows_known)
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
    // kBatch entries a lane are loaded at once.  An entry's place among its warp's
    // entries of the same expert is known in the first pass already: it stays in a
    // register where the batch is all there is, else in `slots`.
    int e[kBatch], place[kBatch];
    const bool one = each <= 32 * kBatch;
    auto load = [&](int from) {
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int i = from + 32 * b + lane;
            e[b] = i < end ? experts[i] : -1;
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) e[b] = static_cast<unsigned>(e[b]) < static_cast<unsigned>(G) ? e[b] : -1;
    };
    for (int from = begin; from < end; from += 32 * kBatch) {
        load(from);
        uint32_t same[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) same[b] = same_as<BITS>(e[b]);
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int before = __popc(same[b] & ((1u << lane) - 1u)), n = e[b] >= 0 ? mine[e[b]] : 0;
            place[b] = n + before;
            __syncwarp();
            if (e[b] >= 0 && before == 0) mine[e[b]] = n + __popc(same[b]);
            __syncwarp();
        }
        if (!one) {
#pragma unroll
            for (int b = 0; b < kBatch; ++b)
                if (from + 32 * b + lane < end) slots[from + 32 * b + lane] = place[b];
        }
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
    for (int from = begin; from < end; from += 32 * kBatch) {
        if (!one) {
            load(from);
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                const int i = from + 32 * b + lane;
                if (i < end) place[b] = slots[i];
            }
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int i = from + 32 * b + lane;
            if (i >= end) continue;
            const int at = e[b] >= 0 ? bases[e[b]] + mine[e[b]] + place[b] : -1;
            if (source && !rows_known && at >= 0) source[at] = i;
            slots[i] = at;
        }
    }
    if (source)
        for (int r = total + rank * kSortThreads + static_cast<int>(threadIdx.x); r < T; r += blocks * kSortThreads) source[r] = -1;
    __syncwarp();
    if (blocks > 1) ptx::cluster_wait();
}

__global__ void __launch_bounds__(kThreads) source_kernel(const int *slots, int *source, int T)
{
    ptx::launch_dependents();
    ptx::grid_dependency_wait();
    const int i = static_cast<int>(blockIdx.x) * kThreads + static_cast<int>(threadIdx.x), r = i < T ? slots[i] : -1;
    if (r >= 0) source[r] = i;
}

// ------------------------------------------------------------------ rows to their experts

struct DispatchArgs {
    const int *experts;      // [M,top]
    const uint4 *x;          // [M, vecs] 16-byte vectors
    const float *scales;     // [M, blocks] or nullptr
    int *offsets, *slots, *source;
    uint4 *rows;
    float *row_scales;
    int M, top, G, vecs, blocks;
};

// Most entries that every block sorts by itself (rows of 2048 BF16, by themselves and
// behind a sort: 1024 entries 3.5 and 5.0 us, 2048 as 512 tokens 5.1 and 6.2, as 256 tokens of
// 256 experts 6.8 and 6.5).
constexpr int kHere = 2048;
constexpr int kMaxTop = 32;   // SPLITK_MAX_TOP

// The block's token: where its entries go, by comparison with every entry, E of them
// in each thread.
template <int E>
__device__ __forceinline__ void places_of(const DispatchArgs &a, int m, int *place)
{
    __shared__ int own[kMaxTop], part[kMaxTop][kThreads / 32];
    const int T = a.M * a.top, lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    int e[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const int t = i * kThreads + static_cast<int>(threadIdx.x);
        e[i] = t < T ? a.experts[t] : -1;
    }
    if (static_cast<int>(threadIdx.x) < a.top) own[threadIdx.x] = a.experts[m * a.top + threadIdx.x];
    __syncthreads();
#pragma unroll 4
    for (int j = 0; j < a.top; ++j) {
        const int at = m * a.top + j, mine = own[j];
        int lower = 0;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int t = i * kThreads + static_cast<int>(threadIdx.x);
            lower += e[i] >= 0 && (e[i] < mine || (e[i] == mine && t < at));
        }
        lower = __reduce_add_sync(0xffffffffu, lower);
        if (lane == 0) part[j][warp] = lower;
    }
    __syncthreads();
    if (static_cast<int>(threadIdx.x) < a.top) {
        const int at = m * a.top + static_cast<int>(threadIdx.x), mine = own[threadIdx.x];
        int lower = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) lower += part[threadIdx.x][w];
        if (static_cast<unsigned>(mine) >= static_cast<unsigned>(a.G)) lower = -1;
        place[threadIdx.x] = lower;
        a.slots[at] = lower;
        if (a.source && lower >= 0) a.source[lower] = at;
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
    // four consecutive experts to a thread
    constexpr int kEach = kMaxGroups / kThreads;
    __shared__ int sums[kThreads / 32];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    int c[kEach], mine = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int g = kEach * static_cast<int>(threadIdx.x) + i;
        c[i] = g < a.G ? counts[g] : 0;
        mine += c[i];
    }
    int scan = mine;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int x = __shfl_up_sync(0xffffffffu, scan, d);
        if (lane >= d) scan += x;
    }
    if (lane == 31) sums[warp] = scan;
    __syncthreads();
    int before = scan - mine, total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += sums[w];
        total += sums[w];
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int g = kEach * static_cast<int>(threadIdx.x) + i;
        if (g < a.G) a.offsets[g] = before;
        before += c[i];
    }
    if (threadIdx.x == 0) a.offsets[a.G] = total;
    if (a.source)
        for (int r = total + static_cast<int>(threadIdx.x); r < T; r += kThreads) a.source[r] = -1;
}

// A token to a block.  E > 0: the launch sorts too, up to 256 E entries.
template <int E>
__global__ void __launch_bounds__(kThreads) dispatch_kernel(const DispatchArgs a)
{
    constexpr bool HERE = E > 0;
    __shared__ int place[HERE ? kMaxGroups + 1 : kMaxTop];   // (HERE: the last block's counts)
    const int m = static_cast<int>(blockIdx.x);
    if constexpr (HERE) {
        ptx::launch_dependents();
        ptx::grid_dependency_wait();
        if (m == a.M) {
            offsets_of(a, place);
            return;
        }
    }
    // Vectors on their way while the rows are found.  (After a sort: it lets this launch
    // start when what was before the sort is done, so x is there; read from L2, as this
    // SM's L1 may hold what x was before that.)
    const uint4 *const x = a.x + static_cast<int64_t>(m) * a.vecs;
    constexpr int kAhead = 2;
    uint4 p[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        if (static_cast<int>(threadIdx.x) + i * kThreads < a.vecs) p[i] = __ldcg(x + threadIdx.x + i * kThreads);
    if constexpr (!HERE) {
        ptx::grid_dependency_wait();
        ptx::launch_dependents();
    }
    if constexpr (HERE) {
        places_of<E>(a, m, place);
    } else {
        if (threadIdx.x < a.top) {
            const int at = m * a.top + static_cast<int>(threadIdx.x), r = a.slots[at];
            place[threadIdx.x] = r;
            if (a.source && r >= 0) a.source[r] = at;
        }
        __syncthreads();
    }
    for (int v0 = threadIdx.x; v0 < a.vecs; v0 += kAhead * kThreads) {
        if (v0 >= kAhead * kThreads) {
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                if (v0 + i * kThreads < a.vecs) p[i] = x[v0 + i * kThreads];
        }
        for (int j = 0; j < a.top; ++j) {
            if (place[j] < 0) continue;
            uint4 *const to = a.rows + static_cast<int64_t>(place[j]) * a.vecs;
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                if (v0 + i * kThreads < a.vecs) to[v0 + i * kThreads] = p[i];
        }
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

// A vector that nothing reads again soon: the first to leave the caches (both ways and
// the gradient of the size below: 184 us, without 188).
template <typename P>
__device__ __forceinline__ P read_once(const P *p)
{
    P r;
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(P) / 16); ++i) reinterpret_cast<uint4 *>(&r)[i] = __ldcs(reinterpret_cast<const uint4 *>(p) + i);
    return r;
}

// Rows that a thread has in flight at once (8192 tokens of 2048 BF16, top 8, both ways
// and the gradient: 188 us, with 2 or 8 of them 193 and 201: fewer loads, or fewer
// blocks for their registers).
constexpr int kAtOnce = 4;

// `warps` warps a token along the row, blocks of y behind one another.
template <typename T, typename O>
__global__ void __launch_bounds__(kThreads) combine_kernel(const CombineArgs a, int warps)
{
    constexpr int J = kAtOnce;
    ptx::launch_dependents();
    ptx::grid_dependency_wait();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, tokens = static_cast<int>(blockDim.x) / 32 / warps;
    const int64_t m = static_cast<int64_t>(blockIdx.x) * tokens + warp / warps;
    const int v = (static_cast<int>(blockIdx.y) * warps + warp % warps) * 32 + lane;
    if (m >= a.M || v >= a.vecs) return;
    const Pack<T> *const rows = static_cast<const Pack<T> *>(a.rows) + v;
    float sum[kVec] = {};
    for (int j0 = 0; j0 < a.top; j0 += J) {
        int r[J];
        float s[J];
        Pack<T> x[J];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            r[j] = j0 + j < a.top ? a.slots[m * a.top + j0 + j] : -1;
            s[j] = a.shares && j0 + j < a.top ? a.shares[m * a.top + j0 + j] : 1.f;
        }
#pragma unroll
        for (int j = 0; j < J; ++j)
            if (static_cast<unsigned>(r[j]) < static_cast<unsigned>(a.T)) x[j] = read_once(rows + static_cast<int64_t>(r[j]) * a.vecs);
#pragma unroll
        for (int j = 0; j < J; ++j) {
            if (static_cast<unsigned>(r[j]) >= static_cast<unsigned>(a.T)) continue;
            float y[kVec];
            unpack(x[j], y);
#pragma unroll
            for (int i = 0; i < kVec; ++i) sum[i] = fmaf(s[j], y[i], sum[i]);
        }
    }
    Pack<O> p;
    pack(sum, p);
    static_cast<Pack<O> *>(a.out)[m * a.vecs + v] = p;
}

constexpr int kGradThreads = 512;

// One token a block.
template <typename T>
__global__ void __launch_bounds__(kGradThreads) combine_grad_kernel(const CombineArgs a)
{
    constexpr int kGroup = kAtOnce;
    __shared__ float part[kGroup][kGradThreads / 32];
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
        for (int v = threadIdx.x; v < a.vecs; v += static_cast<int>(blockDim.x)) {
            float d[kVec];
            unpack(dout[v], d);
            Pack<T> x[kGroup];
            if (rows) {
#pragma unroll
                for (int j = 0; j < kGroup; ++j)
                    if (r[j] >= 0) x[j] = read_once(rows + static_cast<int64_t>(r[j]) * a.vecs + v);
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
                for (int w = 0; w < static_cast<int>(blockDim.x) / 32; ++w) sum += part[threadIdx.x][w];
                a.dshares[m * a.top + j0 + threadIdx.x] = sum;
            }
            __syncthreads();
        }
    }
}

template <typename T, typename O>
cudaError_t launch_combine_types(const CombineArgs &a, cudaStream_t stream)
{
    // A token's warps in blocks of up to 8, evenly; several short rows to a block.
    const int units = (a.vecs + 31) / 32, splits = (units + 7) / 8, warps = (units + splits - 1) / splits, tokens = warps < 4 ? 8 / warps : 1;
    cudaLaunchAttribute attr;
    cudaLaunchConfig_t cfg = config(static_cast<unsigned>((a.M + tokens - 1) / tokens), static_cast<unsigned>(32 * warps * tokens), stream, &attr);
    cfg.gridDim.y = static_cast<unsigned>(splits);
    return note_error(cudaLaunchKernelEx(&cfg, combine_kernel<T, O>, a, warps), "combine_kernel launch");
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
    // Small blocks, so that their sums' barriers meet less often at once (8192 tokens of
    // 2048 BF16, top 8: 85 us, with 8 warps 93); few tokens take all the warps they can (16
    // and 4 warps: 304 tokens 4.5 and 5.9 us, 600 6.6 and 8.6, 1003 10.9 and 10.3, 2000 21 and
    // 19; rows of 1544, top 3: 152 tokens 2.2 and 2.6, 600 3.6 and 4.0, 1003 4.7 and 4.9).
    const int units = (a.vecs + 31) / 32, most = a.M <= 2 * 152 ? kGradThreads / 32 : 4, turns = (units + most - 1) / most;
    const cudaLaunchConfig_t cfg = config(static_cast<unsigned>(a.M), static_cast<unsigned>((units + turns - 1) / turns * 32), stream, &attr);
    return note_error(cudaLaunchKernelEx(&cfg, combine_grad_kernel<T>, a), "combine_grad_kernel launch");
}

template <typename F>
cudaError_t allow_smem(F *kernel)
{
    return note_error(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           (kSortWarps + 2) * kMaxGroups * static_cast<int>(sizeof(int))),
                      "sort_kernel shared memory");
}

void cluster_of(int blocks, cudaLaunchConfig_t *cfg)
{
    cudaLaunchAttribute &a = cfg->attrs[cfg->numAttrs++];
    a.id = cudaLaunchAttributeClusterDimension;
    a.val.clusterDim.x = static_cast<unsigned>(blocks);
    a.val.clusterDim.y = 1;
    a.val.clusterDim.z = 1;
}

// Whether this device runs clusters of 16 blocks of the sort (more than the portable
// 8), asked once a device.
bool wide_clusters()
{
    constexpr int kDevices = 64;
    static std::atomic<int> known[kDevices];   // 0 not asked, 1 no, 2 yes
    int device = 0;
    if (cudaGetDevice(&device) != cudaSuccess || device < 0 || device >= kDevices) return false;
    int k = known[device].load(std::memory_order_relaxed);
    if (k == 0) {
        auto *const kernel = sort_kernel<10, 8>;
        int clusters = 0;
        cudaLaunchAttribute attr[2];
        cudaLaunchConfig_t cfg = config(16, kSortThreads, nullptr, attr);
        cfg.dynamicSmemBytes = static_cast<size_t>(kSortWarps + 2) * kMaxGroups * sizeof(int);
        cluster_of(16, &cfg);
        const bool yes = allow_smem(kernel) == cudaSuccess &&
                         cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
                         cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg) == cudaSuccess && clusters > 0;
        if (!yes) cudaGetLastError();
        k = yes ? 2 : 1;
        known[device].store(k, std::memory_order_relaxed);
    }
    return k == 2;
}

template <int BITS>
auto sort_for(int each)
{
    return each <= 32 ? sort_kernel<BITS, 1> : each <= 64 ? sort_kernel<BITS, 2> : each <= 128 ? sort_kernel<BITS, 4> : sort_kernel<BITS, 8>;
}

cudaError_t launch_sort(const DispatchProblem &p, cudaStream_t stream)
{
    const int T = static_cast<int>(p.M * p.top), G = static_cast<int>(p.G);
    // 65536 entries of 256 experts: 16 blocks 6.7 us, 8 blocks 8.6; 8192: 8 blocks 4.2, 1
    // block 11; up to 1024 one block is 0.6 us faster than 8.
    const int blocks = T <= kSortThreads ? 1 : T > 16 * kSortThreads && wide_clusters() ? 16 : 8;
    const int warps = blocks * kSortWarps;
    const int each = ((T + warps - 1) / warps + 31) / 32 * 32;
    const size_t smem = static_cast<size_t>(kSortWarps + 2) * G * sizeof(int);
    auto *const kernel = G <= 16 ? sort_for<4>(each) : G <= 64 ? sort_for<6>(each) : G <= 256 ? sort_for<8>(each) : sort_for<10>(each);
    cudaError_t e = cudaSuccess;
    if (smem > 40 * 1024) e = allow_smem(kernel);   // (48 KB without, static shared memory included)
    if (e == cudaSuccess && blocks > 8)
        e = note_error(cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1), "sort_kernel cluster size");
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = config(static_cast<unsigned>(blocks), kSortThreads, stream, attr);
    cfg.dynamicSmemBytes = smem;
    cluster_of(blocks, &cfg);
    // Rows on their way have their entries written by their own blocks (and those of a
    // large sort by a grid): 4-byte stores to 32 places a warp hold a cluster up (65536
    // entries: 8.6 us without them, 12.3 with).
    const bool later = p.source && (p.x || T > 16 * kSortThreads);
    e = note_error(cudaLaunchKernelEx(&cfg, kernel, p.experts, p.offsets, p.slots, p.source, T, G, each, blocks, later ? 1 : 0), "sort_kernel launch");
    if (e != cudaSuccess || !later || p.x) return e;
    cudaLaunchAttribute more;
    const cudaLaunchConfig_t grid = config(static_cast<unsigned>((T + kThreads - 1) / kThreads), kThreads, stream, &more);
    return note_error(cudaLaunchKernelEx(&grid, source_kernel, static_cast<const int *>(p.slots), p.source, T), "source_kernel launch");
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
    const int64_t T = p.M * p.top;
    auto *const kernel = !here ? dispatch_kernel<0> : T <= kThreads ? dispatch_kernel<1> : T <= 2 * kThreads ? dispatch_kernel<2>
                         : T <= 4 * kThreads ? dispatch_kernel<4> : dispatch_kernel<8>;
    return note_error(cudaLaunchKernelEx(&cfg, kernel, a), "dispatch_kernel launch");
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
