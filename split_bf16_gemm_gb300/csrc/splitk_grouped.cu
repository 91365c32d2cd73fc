// splitk_grouped.cu -- 8-bit products with a scale for each block of 128, and
// products grouped by expert, on the 5th-generation tensor cores.
//
// One kernel computes, for ragged runs of rows (run g is rows offsets[g] ..
// offsets[g+1]-1; one run of all rows for the plain product):
//   kFp8   out[t,n]  = sum_kb sa[t,kb] sb[g,n/128,kb] sum_{k in kb} A[t,k] B[g,n,k]
//   kNk    out[t,n]  = sum_k A[t,k] B[g,n,k]
//   kKn    out[t,n]  = sum_k A[t,k] W[g,k,n]
//   kDw    dB[g,n,k] = sum_{t in run g} D[t,n] A[t,k]
//
// Every tile is 128 tensor-memory lanes by up to TC columns.  The lanes are
// the weight's rows n (kDw: the columns k of A) and the columns are tokens
// (kDw: the columns n of D), because the token count of a run is the ragged
// and often small extent: the MMA's N can be any multiple of 16, so a run of
// 5 tokens costs 16 columns and not a 128-row tile.  A run's columns are
// split evenly over its tiles.  Output rows are contiguous along the lanes.
//
// 384 threads:
//   warp 0     TMA producer (one lane): k-blocks of 128 bytes (128 8-bit or
//              64 16-bit values) of 128 lanes and of the tile's columns;
//   warp 1     MMA issuer (one lane);
//   warp 2     kFp8: the products sa * sb of each k-block's columns, into a
//              ring in shared memory; kDw: zeroes the rows past the run's end
//              in the last k-block (they belong to the next run);
//   warps 4-11 tensor memory -> registers -> output: lane quarter w % 4,
//              column half w / 4 - 1.
// kFp8 with many rows (ROWS, TC >= 128) exchanges the roles: the lanes are
// tokens and the columns weights, so that a thread's scale is one factor.
// kFp8: F32 scales cannot be applied inside the MMA, so each k-block's product
// goes to an accumulator of its own (a ring of them in tensor memory), and the
// last eight warps add it, times the scale, to F32 sums in registers while
// the next block multiplies.
//
// Long K with few tiles: the S blocks of a cluster each take 1/S of the
// k-blocks and add their F32 sums through distributed shared memory in rank
// order, so the result does not depend on timing.
//
// Every wait has a time limit.  A wait that runs out sets the device status
// word and a flag that ends the block's other waits; the loads in flight are
// awaited, the MMAs too, before tensor memory is freed.

#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <type_traits>

#include "ptx_grouped.cuh"
#include "splitk_internal.h"

namespace splitk {
namespace {

__device__ unsigned g_grouped_status;

constexpr uint64_t kWaitLimitNs = 1000000000ull;   // 1 s
constexpr int kThreads = 384;
constexpr int kEpilogueWarps = 8;
constexpr int kRoleWarps = 4;                       // of which the last is idle: registers move by four warps
constexpr int kLanes = 128;
constexpr uint32_t kLaneBytes = kLanes * 128;       // one k-block of the lane operand
constexpr int kMaxRing = 12;
constexpr int kScaleRing = 8;
constexpr int kUnit = 8;   // k-blocks (512 values of K) between additions in registers

enum Form { kFp8, kNk, kKn, kDw };

// TC: columns of a tile.  256 is a pair of blocks (cta_group::2) whose tile is
// 256 lanes, 128 to a block, by 256 columns, half of whose operand each block
// loads: 32 KB a k-block and block for four times the products of the 32 KB
// that a 128 x 128 tile takes.
template <int TC>
struct Shape {
    static constexpr bool kPair = TC == 256;
    static constexpr int kBlocks = kPair ? 2 : 1;
    static constexpr int kAcc = TC <= 64 ? 4 : 2;                 // accumulators in tensor memory
    static constexpr int kTmemCols = kAcc * TC;
    static constexpr int kLoadCols = TC / kBlocks;                // columns a block loads
    static constexpr uint32_t kColBytes = kLoadCols * 128;
    static constexpr uint32_t kStage = kLaneBytes + kColBytes;
    static constexpr int kTileLanes = kLanes * kBlocks;
    // Thread blocks of an SM.  A tile of 32 columns keeps neither the loads nor
    // the tensor cores busy by itself; two blocks share an SM's memory.
    static constexpr int kPerSm = TC == 32 ? 2 : 1;
    static constexpr size_t kSmem = kPerSm == 2 ? 112 * 1024 : kSmemLimit;
    // kFp8, a warp's part of the columns (half the tile's): read as fragments
    // of 8 columns, of which a thread holds two.  The scales of thread t % 4 =
    // p stand together, p's 4 words further round the banks than the last's.
    static constexpr int kHalf = TC / 2;
    static constexpr int kScalePitch = kHalf / 4 + 4;
    static constexpr int kScaleSlot = TC >= 128 ? TC : 2 * 4 * kScalePitch;   // ROWS: lanes by weight blocks
    static constexpr int kFragCols = kHalf < 32 ? kHalf : 32;     // columns of one tensor-memory load
    // staged rows of 64 bytes, padded by 16: 32 lanes of a column in 16 bits,
    // or (ROWS) a piece of a lane's columns; ROWS with 16-bit outputs: boxes of
    // 32 lanes by 64 columns, as a TMA store takes them
    static constexpr uint32_t kStageRow = 80;
    static constexpr uint32_t kStageWarp = TC >= 128 ? kHalf / 64 * 4096 : kFragCols * kStageRow;
};

struct GroupedArgs {
    const int *offsets;        // [G+1] on the device, or nullptr: one run of T rows
    const float *sa, *sb;      // kFp8
    void *out;
    int T, G;
    int lanes, cols;           // extent of the lanes; of the columns for kDw (else the run's length)
    int kblocks;               // of the contracted extent (not kDw)
    int out_type;              // splitk_dtype
    int bf16;
    int splits;                // cluster size along K
    int stages;
    int store_boxes;           // ROWS: 16-bit rows that start on 16 bytes
    uint32_t sum_off, scale_off, stage_off, table_off;   // byte offsets in shared memory after the stage ring
};

struct Maps {
    CUtensorMap lane, col, col_part;   // col_part: a quarter of col's rows
    CUtensorMap out;                   // ROWS, with store_boxes
};

struct Tile {
    int g;
    int lane0, cols, width;    // first lane; live columns, and rounded up to the MMA's N
    int col0;                  // first column: a token, or a column of D
    int kb0, nkb;              // this block's k-blocks
    int tok0, tok_n;           // kDw: the run
    int rows;                  // ROWS: live lanes of this block
};

// kBlock: an arrival of this block or of its loads.  Of the other block of a
// pair: kRelaxed, which guards tensor memory alone, and kAcquire, shared memory
// that the other block wrote.
enum Order { kBlock, kRelaxed, kAcquire };

template <Order ORDER = kBlock>
__device__ __forceinline__ bool bounded_wait(uint32_t bar, uint32_t parity, volatile unsigned *abort)
{
    auto ready = [&] {
        return ORDER == kRelaxed   ? ptx::mbar_try_wait_cluster_relaxed(bar, parity)
               : ORDER == kAcquire ? ptx::mbar_try_wait_cluster(bar, parity)
                                   : ptx::mbar_try_wait(bar, parity);
    };
    uint64_t t0 = 0;
    for (uint32_t i = 1;; ++i) {
        if (ready()) return true;
        if ((i & 63u) == 0) {              // the timer is slow to read: not on short waits
            const uint64_t now = ptx::globaltimer_ns();
            if (t0 == 0) t0 = now;
            if (*abort || now - t0 > kWaitLimitNs) {
                *abort = 1u;
                atomicOr(&g_grouped_status, 1u);
                return false;
            }
        }
    }
}

// The same for a whole warp: every lane goes one way.
template <Order ORDER = kBlock>
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile unsigned *abort)
{
    return __all_sync(0xffffffffu, bounded_wait<ORDER>(bar, parity, abort)) != 0;
}

template <typename T>
__device__ __forceinline__ T rounded(float v);
template <>
__device__ __forceinline__ float rounded<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half rounded<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 rounded<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Two values rounded to 16 bits, the first in the low half.
template <typename T>
__device__ __forceinline__ uint32_t pair16(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pair16<__half>(float lo, float hi)
{
    const __half2 y = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&y);
}
template <>
__device__ __forceinline__ uint32_t pair16<__nv_bfloat16>(float lo, float hi)
{
    const __nv_bfloat162 y = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&y);
}

// The first `live` of N values to rows `pitch` elements apart.  No branch
// inside: with two warps to a scheduler a branch's latency is not hidden (the
// stores of a 256 x 256 tile took 17,500 cycles with the type and the bound
// tested for each value).
template <typename T, int N, typename Value>
__device__ __forceinline__ void store_column(T *p, size_t pitch, int live, Value value)
{
    if (live >= N) {
#pragma unroll
        for (int j = 0; j < N; ++j, p += pitch) *p = rounded<T>(value(j));
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j, p += pitch)
            if (j < live) *p = rounded<T>(value(j));
    }
}

template <int N, typename Value>
__device__ __forceinline__ void store_values(void *out, int type, size_t at, size_t pitch, int live, Value value)
{
    if (live <= 0) return;
    if (type == 0)
        store_column<float, N>(static_cast<float *>(out) + at, pitch, live, value);
    else if (type == 1)
        store_column<__half, N>(static_cast<__half *>(out) + at, pitch, live, value);
    else
        store_column<__nv_bfloat16, N>(static_cast<__nv_bfloat16 *>(out) + at, pitch, live, value);
}

template <int FORM, int TC, bool SUMS>
__global__ void __launch_bounds__(kThreads, Shape<TC>::kPerSm)
    grouped_kernel(const __grid_constant__ Maps maps, const GroupedArgs args)
{
    static_assert(SUMS || FORM != kFp8, "8-bit operands need the F32 sums in registers");
    using Sh = Shape<TC>;
    constexpr bool FP8 = FORM == kFp8, DW = FORM == kDw;
    constexpr bool LMN = FORM == kKn || FORM == kDw;   // lane operand contiguous along its lanes
    constexpr bool PAIR = Sh::kPair;
    constexpr bool ROWS = FP8 && TC >= 128;            // lanes are tokens, columns weights
    constexpr int KB = FP8 ? 128 : 64;
    constexpr int UNIT = FP8 ? 1 : SUMS ? kUnit : 1 << 30;   // k-blocks summed in one accumulator
    constexpr int HALF = TC / 2;                       // columns of an epilogue warp
    constexpr int CHUNK = HALF < 32 ? HALF : 32;       // columns of one tensor-memory load
    static_assert(!DW || TC % 64 == 0, "the columns of kDw come in boxes of 64");

    extern __shared__ uint8_t dsmem[];
    __shared__ __align__(8) uint64_t bars[3 * kMaxRing + 2 * Sh::kAcc + 2 * kScaleRing + 1];
    __shared__ uint32_t tmem_slot;
    __shared__ unsigned abort_s;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t raw = ptx::smem_addr(dsmem);
    const uint32_t ring = (raw + 1023u) & ~1023u;
    uint8_t *const base = dsmem + (ring - raw);
    // splits > 1: [TC][128], ROWS [128][TC + 1]
    float *const sum_buf = reinterpret_cast<float *>(base + args.sum_off);
    float *const scale_buf = reinterpret_cast<float *>(base + args.scale_off);   // [kScaleRing][kScaleSlot]
    int *const offs = reinterpret_cast<int *>(base + args.table_off);            // [G+1]
    int *const pref = offs + args.G + 1;                                         // [G+1]: tiles before run g
    const uint32_t bar0 = ptx::smem_addr(&bars[0]);
    auto full_bar = [&](int i) { return bar0 + 8u * i; };
    auto empty_bar = [&](int i) { return bar0 + 8u * (kMaxRing + i); };
    auto acc_full = [&](int i) { return bar0 + 8u * (2 * kMaxRing + i); };
    auto acc_empty = [&](int i) { return bar0 + 8u * (2 * kMaxRing + Sh::kAcc + i); };
    auto scale_full = [&](int i) { return bar0 + 8u * (2 * kMaxRing + 2 * Sh::kAcc + i); };
    auto scale_empty = [&](int i) { return bar0 + 8u * (2 * kMaxRing + 2 * Sh::kAcc + kScaleRing + i); };
    auto tail_bar = [&](int i) { return bar0 + 8u * (2 * kMaxRing + 2 * Sh::kAcc + 2 * kScaleRing + i); };   // kDw
    const uint32_t drain_bar = tail_bar(kMaxRing);
    const int peer = PAIR ? static_cast<int>(blockIdx.x) & 1 : 0;   // 0: the block that issues the pair's MMAs
    auto release_acc = [&](uint32_t bar) {
        if constexpr (PAIR)
            ptx::mbar_arrive_cluster_relaxed(ptx::mapa(bar, 0));
        else
            ptx::mbar_arrive(bar);
    };
    auto cluster_sync = [&]() {
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        ptx::cluster_wait();
    };
    const int stages = args.stages, S = args.splits;

    const int lane_tiles = (args.lanes + Sh::kTileLanes - 1) / Sh::kTileLanes;
    if (tid == 0) {
        if (args.offsets == nullptr) {               // one run of all rows
            offs[0] = 0, offs[1] = args.T;
            pref[0] = 0, pref[1] = lane_tiles * ((args.T + TC - 1) / TC);
        }
        ptx::prefetch_tensormap(&maps.lane);
        ptx::prefetch_tensormap(&maps.col);
        for (int i = 0; i < stages; ++i) {
            // kDw: one arrival a block, by its producer or, where it repairs
            // the stage first, by its warp 2
            ptx::mbar_init(full_bar(i), DW ? Sh::kBlocks : 1);
            ptx::mbar_init(empty_bar(i), 1);
            ptx::mbar_init(tail_bar(i), 1);
        }
        for (int i = 0; i < Sh::kAcc; ++i) {
            ptx::mbar_init(acc_full(i), 1);
            ptx::mbar_init(acc_empty(i), kEpilogueWarps * Sh::kBlocks);
        }
        for (int i = 0; i < kScaleRing; ++i) {
            ptx::mbar_init(scale_full(i), 1);
            ptx::mbar_init(scale_empty(i), kEpilogueWarps);
        }
        ptx::mbar_init(drain_bar, 1);
        abort_s = 0;
        ptx::fence_mbar_init();
        ptx::fence_proxy_async_smem();
    }
    if (warp == 1) {
        if constexpr (PAIR) {
            ptx::tmem_alloc_pair(ptx::smem_addr(&tmem_slot), Sh::kTmemCols);
            ptx::tmem_relinquish_pair();
        } else {
            ptx::tmem_alloc(ptx::smem_addr(&tmem_slot), Sh::kTmemCols);
            ptx::tmem_relinquish();
        }
    }
    ptx::tc_fence_before_sync();
    __syncthreads();
    if constexpr (PAIR) cluster_sync();   // the other block's barriers are set up
    ptx::tc_fence_after_sync();
    const uint32_t tmem = tmem_slot;
    // the next launch's blocks may set up now (every block here holds its
    // tensor memory); they wait for this grid before they read anything
    // (with plain loads: what the grid before wrote is not constant while this
    // one runs)
    ptx::launch_dependents();
    ptx::grid_dependency_wait();

    // ---- the runs, made monotone and within [0, T] whatever the offsets
    // hold, and the number of tiles before each
    if (args.offsets != nullptr) {
        const bool staged = args.G > 32;               // more than one round of a warp: read all at once first
        if (staged) {
            for (int i = tid; i <= args.G; i += kThreads) offs[i] = min(max(args.offsets[i], 0), args.T);
            __syncthreads();
        }
        if (warp == 2) {
            auto offset = [&](int i) { return staged ? offs[i] : min(max(args.offsets[i], 0), args.T); };
            int most = offset(0), tiles = 0;
            const int begin0 = most;
            for (int b = 0; b < args.G; b += 32) {
                const int g = b + lane;
                int end = g < args.G ? offset(g + 1) : 0;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int o = __shfl_up_sync(0xffffffffu, end, d);
                    if (lane >= d) end = max(end, o);
                }
                end = max(end, most);
                int begin = __shfl_up_sync(0xffffffffu, end, 1);
                if (lane == 0) begin = most;
                const int ext = DW ? args.cols : end - begin;
                int n = g < args.G ? lane_tiles * ((ext + TC - 1) / TC) : 0;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int o = __shfl_up_sync(0xffffffffu, n, d);
                    if (lane >= d) n += o;
                }
                __syncwarp();
                if (g < args.G) {
                    offs[g + 1] = end;
                    pref[g + 1] = tiles + n;
                }
                most = __shfl_sync(0xffffffffu, end, 31);
                tiles += __shfl_sync(0xffffffffu, n, 31);
            }
            if (lane == 0) offs[0] = begin0, pref[0] = 0;
        }
        __syncthreads();
    }
    const int total = pref[args.G];
    const int rank = S > 1 ? static_cast<int>(blockIdx.x) % S : 0;
    const int group = PAIR ? 2 : S;                   // blocks at work on a tile
    const int first = static_cast<int>(blockIdx.x) / group, step = static_cast<int>(gridDim.x) / group;

    // Tile w of run g.  Within a run, bands of up to 16 column tiles are
    // walked column tile first, so that the blocks at work at one time share
    // both operands' rows in L2.
    auto locate = [&](int w, int &g, Tile &t) {
        while (w >= pref[g + 1]) ++g;
        const int begin = offs[g], run = offs[g + 1] - begin;
        const int ext = DW ? args.cols : run;
        const int ct = (ext + TC - 1) / TC;
        constexpr int kBand = 16;
        const int r = w - pref[g];
        const int band = r / (kBand * lane_tiles);
        const int rb = r - band * kBand * lane_tiles;
        const int bw = min(kBand, ct - band * kBand);
        const int li = rb / bw, ci = band * kBand + rb - li * bw;
        constexpr int kRound = (DW ? 64 : 16) * Sh::kBlocks;
        const int each = ((ext + ct - 1) / ct + kRound - 1) / kRound * kRound;
        t.g = g;
        t.lane0 = li * Sh::kTileLanes + peer * kLanes;
        t.cols = min(each, ext - ci * each);
        t.width = (t.cols + kRound - 1) / kRound * kRound;
        t.tok0 = begin;
        t.tok_n = run;
        if constexpr (DW) {
            t.col0 = ci * each;
            t.kb0 = 0;
            t.nkb = (run + KB - 1) / KB;
        } else {
            t.col0 = begin + ci * each;
            if constexpr (ROWS) {
                t.col0 = li * TC;                      // whole blocks of 128: a scale for each warp's columns
                t.cols = min(TC, args.lanes - t.col0);
                t.width = (t.cols + 31) / 32 * 32;
                t.lane0 = begin + ci * Sh::kTileLanes + peer * kLanes;
                t.rows = min(kLanes, begin + run - t.lane0);
            }
            const int lo = rank * args.kblocks / S, hi = (rank + 1) * args.kblocks / S;
            t.kb0 = lo;
            t.nkb = hi - lo;
        }
    };

    // 384 threads start with 168 registers each.  The sums of a 256-column tile
    // need more in warps 4-11: 4 * 32 * 88 + 8 * 32 * 208 = 384 * 168
    // (fewer in warps 0-3 spill their loops: 136 against 112 us then, at M4096 N8192 K4096).
    constexpr bool kMoveRegs = SUMS && TC == 256;
    if (kMoveRegs && warp < kRoleWarps) ptx::regs_down<88>();
    if (warp == 0) {
        // ---- producer
        int g = 0, slot = 0;
        uint32_t ph = 0;
        int issued = 0;
        bool dead = false;
        const uint64_t once = ptx::l2_policy_evict_normal(), again = ptx::l2_policy_evict_last();
        const uint32_t full0 = PAIR ? ptx::mapa(full_bar(0), 0) : full_bar(0);   // the issuing block's
        for (int w = first; w < total; w += step) {
            Tile t;
            locate(w, g, t);
            if (!dead) {
                constexpr int kPart = Sh::kLoadCols / 4;
                const int load_cols = t.width / Sh::kBlocks;             // this block's part of the columns
                const int col = t.col0 + peer * load_cols;
                const int parts = DW ? load_cols / 64 : (load_cols + kPart - 1) / kPart;
                const bool whole = !DW && parts > 2;
                const uint32_t bytes = kLaneBytes + (DW ? static_cast<uint32_t>(parts) * 8192u
                                                     : whole ? Sh::kColBytes
                                                             : static_cast<uint32_t>(parts) * kPart * 128u);
                auto load2 = [&](uint32_t dst, const CUtensorMap *map, uint32_t bar, int x, int y, uint64_t policy) {
                    if constexpr (PAIR)
                        ptx::tma_load_2d_pair(dst, map, bar, x, y, policy);
                    else
                        ptx::tma_load_2d(dst, map, bar, x, y, policy);
                };
                auto load3 = [&](uint32_t dst, uint32_t bar, int x, int y, const CUtensorMap *map) {
                    if constexpr (PAIR)
                        ptx::tma_load_3d_pair(dst, map, bar, x, y, t.g, once);
                    else
                        ptx::tma_load_3d(dst, map, bar, x, y, t.g, once);
                };
                for (int i = 0; i < t.nkb; ++i) {
                    if (!warp_wait(empty_bar(slot), ph ^ 1u, &abort_s)) {
                        dead = true;
                        break;
                    }
                    // one lane issues; the whole warp walks the loop, so that
                    // slots and coordinates stay in uniform registers
                    if (ptx::elect_one()) {
                        const uint32_t sl = ring + slot * Sh::kStage, sc = sl + kLaneBytes;
                        const int kx = (t.kb0 + i) * KB;
                        uint32_t bar = full0 + 8u * slot;
                        const bool tail = DW && t.tok_n - kx < KB && (t.tok_n - kx) % 16 != 0;
                        if (tail) {                              // to this block's warp 2 first
                            bar = tail_bar(slot);
                            ptx::mbar_arrive_expect_tx(bar, bytes);
                            if constexpr (PAIR) bar = ptx::mapa(bar, peer);
                        } else if (peer == 0) {
                            ptx::mbar_arrive_expect_tx(full_bar(slot), bytes * Sh::kBlocks);
                            if (DW && PAIR) ptx::mbar_arrive(full_bar(slot));
                        }
                        if constexpr (DW) {
                            const int y = t.tok0 + kx;
                            load2(sl, &maps.lane, bar, t.lane0, y, once);
                            load2(sl + 8192u, &maps.lane, bar, t.lane0 + 64, y, once);
                            for (int j = 0; j < parts; ++j)
                                load2(sc + j * 8192u, &maps.col, bar, col + 64 * j, y, once);
                        } else {
                            if constexpr (LMN) {
                                load3(sl, bar, t.lane0, kx, &maps.lane);
                                load3(sl + 8192u, bar, t.lane0 + 64, kx, &maps.lane);
                            } else if constexpr (ROWS) {
                                load2(sl, &maps.col, bar, kx, t.lane0, again);
                            } else {
                                load3(sl, bar, kx, t.lane0, &maps.lane);
                            }
                            if constexpr (ROWS) {
                                if (whole)
                                    load3(sc, bar, kx, col, &maps.lane);
                                else
                                    for (int j = 0; j < parts; ++j)
                                        load3(sc + j * kPart * 128u, bar, kx, col + j * kPart, &maps.col_part);
                            } else if (whole) {
                                load2(sc, &maps.col, bar, kx, col, again);
                            } else {
                                for (int j = 0; j < parts; ++j)
                                    load2(sc + j * kPart * 128u, &maps.col_part, bar, kx, col + j * kPart,
                                          again);
                            }
                        }
                    }
                    __syncwarp();
                    ++issued;
                    if (++slot == stages) {
                        slot = 0;
                        ph ^= 1u;
                    }
                }
            }
            if (S > 1) {
                __syncwarp();
                cluster_sync();
                cluster_sync();
            }
        }
        if constexpr (PAIR) {
            // The issuing block's commits arrive on both blocks' empty barriers,
            // also for the stages that are not filled again: each block waits
            // for those too, as no arrival may reach a block that has left.
            int s = slot;
            uint32_t p = ph;
            for (int i = 0; i < stages && !dead; ++i) {   // (a stage never filled is free at once)
                if (!warp_wait(empty_bar(s), p ^ 1u, &abort_s)) dead = true;
                if (++s == stages) {
                    s = 0;
                    p ^= 1u;
                }
            }
        }
        if (PAIR && peer == 1 && dead) {
            // after a time-out nothing here counts this block's loads in
            // flight: long enough for them to land
            const uint64_t t0 = ptx::globaltimer_ns();
            while (ptx::globaltimer_ns() - t0 < 100000) {
            }
        }
        if (peer == 0) {
            // every load has landed before the block may leave (the issuing
            // block's barriers count the pair's)
            for (int i = 0; i < min(stages, issued); ++i) {
                if (--slot < 0) {
                    slot = stages - 1;
                    ph ^= 1u;
                }
                ptx::mbar_wait_bounded(full_bar(slot), ph, kWaitLimitNs);
            }
        }
    } else if (warp == 1) {
        // ---- MMA issuer
        int g = 0, slot = 0, buf = 0;
        uint32_t ph = 0, aph = 0;
        bool dead = false;
        // One thread issues every MMA with no other to hide its latency: the
        // descriptors are built once, and a slot or a K step is an addition to
        // the low word, whose address field (bytes >> 4) never carries out.
        const uint64_t a0 = LMN ? ptx::sdesc_mnmajor_sw128(ring, 8192u) : ptx::sdesc_kmajor_sw128(ring);
        const uint64_t b0 = DW ? ptx::sdesc_mnmajor_sw128(ring + kLaneBytes, 8192u)
                               : ptx::sdesc_kmajor_sw128(ring + kLaneBytes);
        const uint32_t a_lo = static_cast<uint32_t>(a0), a_hi = static_cast<uint32_t>(a0 >> 32);
        const uint32_t b_lo = static_cast<uint32_t>(b0), b_hi = static_cast<uint32_t>(b0 >> 32);
        for (int w = first; w < total; w += step) {
            Tile t;
            locate(w, g, t);
            if (!dead && peer == 0) {
                uint32_t idesc = (1u << 4) | (static_cast<uint32_t>(t.width >> 3) << 17) | ((Sh::kTileLanes >> 4) << 24);
                if (!FP8 && args.bf16) idesc |= (1u << 7) | (1u << 10);
                if (LMN) idesc |= 1u << 15;
                if (DW) idesc |= 1u << 16;
                for (int i = 0; i < t.nkb; ++i) {
                    const bool unit_start = i % UNIT == 0, unit_end = i % UNIT == UNIT - 1 || i == t.nkb - 1;
                    if (unit_start && !warp_wait<PAIR ? kRelaxed : kBlock>(acc_empty(buf), aph ^ 1u, &abort_s)) {
                        dead = true;
                        break;
                    }
                    // a run's last k-block may hold rows that the other block zeroed
                    if (!(DW && PAIR && i == t.nkb - 1 ? warp_wait<kAcquire>(full_bar(slot), ph, &abort_s)
                                                       : warp_wait(full_bar(slot), ph, &abort_s))) {
                        dead = true;
                        break;
                    }
                    int steps = 4;
                    if constexpr (DW) {
                        const int rem = t.tok_n - i * KB;
                        if (rem < KB) steps = (rem + 15) / 16;
                    }
                    ptx::tc_fence_after_sync();
                    if (ptx::elect_one()) {
                        const uint32_t at = static_cast<uint32_t>(slot) * (Sh::kStage >> 4);
                        const uint32_t d = tmem + static_cast<uint32_t>(buf * TC);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            if (DW && k >= steps) break;
                            const uint32_t accumulate = unit_start && k == 0 ? 0u : 1u;
                            const uint64_t a = ptx::desc64(a_lo + at + (LMN ? 128u : 2u) * k, a_hi);
                            const uint64_t b = ptx::desc64(b_lo + at + (DW ? 128u : 2u) * k, b_hi);
                            if constexpr (PAIR)
                                ptx::mma_pair<FP8>(d, a, b, idesc, accumulate);
                            else if constexpr (FP8)
                                ptx::mma_f8(d, a, b, idesc, accumulate);
                            else
                                ptx::mma_f16(d, a, b, idesc, accumulate);
                        }
                        if constexpr (PAIR)
                            ptx::mma_commit_pair(empty_bar(slot));
                        else
                            ptx::mma_commit(empty_bar(slot));
                        if (unit_end) {
                            if constexpr (PAIR)
                                ptx::mma_commit_pair(acc_full(buf));
                            else
                                ptx::mma_commit(acc_full(buf));
                        }
                    }
                    __syncwarp();
                    if (unit_end && ++buf == Sh::kAcc) {
                        buf = 0;
                        aph ^= 1u;
                    }
                    if (++slot == stages) {
                        slot = 0;
                        ph ^= 1u;
                    }
                }
            }
            if (S > 1) {
                __syncwarp();
                cluster_sync();
                cluster_sync();
            }
        }
        if (peer == 0) {
            // the lane that issued: a commit is for its own operations
            if (ptx::elect_one()) {
                if constexpr (PAIR)
                    ptx::mma_commit_own(drain_bar);   // the other block may be leaving
                else
                    ptx::mma_commit(drain_bar);
            }
            ptx::mbar_wait_bounded(drain_bar, 0, kWaitLimitNs);
        }
        __syncwarp();
    } else if (warp == 2) {
        // ---- kFp8: scales; kDw: the run's last rows
        int g = 0, slot = 0;
        uint32_t ph = 0;                                 // kDw: the phase of each slot's tail barrier, a bit each
        bool dead = false;
        for (int w = first; w < total; w += step) {
            Tile t;
            locate(w, g, t);
            if constexpr (ROWS) {
                // Four k-blocks of 128 tokens' scales at a time.  A token's
                // scales stand together, so that a warp's read touches 32
                // lines: this warp makes them once, 16 bytes wide where rows
                // allow it, for the eight that use them.
                const int nbs = (args.lanes + kLanes - 1) / kLanes, nb = t.col0 / kLanes;
                const float *const sb = args.sb + (static_cast<size_t>(t.g) * nbs + nb) * args.kblocks + t.kb0;
                const float *const sb2 = sb + (nb + 1 < nbs ? args.kblocks : 0);   // the second block of a pair's columns
                const bool wide = args.kblocks % 4 == 0 && t.kb0 % 4 == 0 && t.nkb % 4 == 0;
                const float *sa[4];
#pragma unroll
                for (int p = 0; p < 4; ++p)              // lanes without a token: any row
                    sa[p] = args.sa + static_cast<size_t>(t.rows > 0 ? t.lane0 + min(p * 32 + lane, t.rows - 1) : 0) *
                                          args.kblocks + t.kb0;
                auto read4 = [&](const float *at, int b, float (&to)[4]) {
                    if (wide) {
                        const float4 x = *reinterpret_cast<const float4 *>(at + b);
                        to[0] = x.x, to[1] = x.y, to[2] = x.z, to[3] = x.w;
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j) to[j] = at[min(b + j, t.nkb - 1)];
                    }
                };
                for (int b = 0; b < t.nkb && !dead; b += 4) {
                    // the ring holds eight k-blocks, more than these reads' latency
                    float now[4][4], f[4], f2[4] = {};
#pragma unroll
                    for (int p = 0; p < 4; ++p) read4(sa[p], b, now[p]);
                    read4(sb, b, f);
                    if (PAIR) read4(sb2, b, f2);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (b + j >= t.nkb || dead) break;
                        if (!warp_wait(scale_empty(slot), ph ^ 1u, &abort_s)) {
                            dead = true;
                            break;
                        }
#pragma unroll
                        for (int p = 0; p < 4; ++p) {
                            scale_buf[slot * Sh::kScaleSlot + p * 32 + lane] = now[p][j] * f[j];
                            if (PAIR) scale_buf[slot * Sh::kScaleSlot + kLanes + p * 32 + lane] = now[p][j] * f2[j];
                        }
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive(scale_full(slot));
                        if (++slot == kScaleRing) {
                            slot = 0;
                            ph ^= 1u;
                        }
                    }
                }
            } else if constexpr (FP8) {
                constexpr int PER = TC / 32, BATCH = 4;
                const int lane_blocks = (args.lanes + kLanes - 1) / kLanes;
                const float *const sb =
                    args.sb + (static_cast<size_t>(t.g) * lane_blocks + t.lane0 / kLanes) * args.kblocks + t.kb0;
                const float *sa[PER];
#pragma unroll
                for (int p = 0; p < PER; ++p) {
                    const int c = min(p * 32 + lane, t.cols - 1);   // columns past the tile's repeat its last
                    sa[p] = args.sa + static_cast<size_t>(t.col0 + c) * args.kblocks + t.kb0;
                }
                for (int b = 0; b < t.nkb && !dead; b += BATCH) {
                    // read together, multiplied when stored: the ring holds
                    // eight k-blocks, more than these reads' latency
                    float now[PER][BATCH], f[BATCH];
#pragma unroll
                    for (int j = 0; j < BATCH; ++j) {
                        const int kb = min(b + j, t.nkb - 1);
                        f[j] = sb[kb];
#pragma unroll
                        for (int p = 0; p < PER; ++p) now[p][j] = sa[p][kb];
                    }
#pragma unroll
                    for (int j = 0; j < BATCH; ++j) {
                        if (b + j >= t.nkb || dead) break;
                        if (!warp_wait(scale_empty(slot), ph ^ 1u, &abort_s)) {
                            dead = true;
                            break;
                        }
#pragma unroll
                        for (int p = 0; p < PER; ++p) {
                            const int c = p * 32 + lane, in = c % HALF;
                            scale_buf[slot * Sh::kScaleSlot + (c / HALF * 4 + in % 8 / 2) * Sh::kScalePitch + in / 8 * 2 +
                                      in % 2] = now[p][j] * f[j];
                        }
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive(scale_full(slot));
                        if (++slot == kScaleRing) {
                            slot = 0;
                            ph ^= 1u;
                        }
                    }
                }
            } else if constexpr (DW) {
                // a run's last k-block, where its rows end inside a step of 16
                const int rem = t.tok_n - (t.nkb - 1) * KB;
                if (t.nkb > 0 && rem % 16 && !dead) {
                    const int at = (slot + t.nkb - 1) % stages;
                    if (!warp_wait(tail_bar(at), (ph >> at) & 1u, &abort_s)) {
                        dead = true;
                    } else {
                        ph ^= 1u << at;
                        const int boxes = 2 + t.width / Sh::kBlocks / 64;   // [64 rows][128 bytes], lanes' then columns'
                        const int end = (rem + 15) / 16 * 16;               // of the MMA's step
                        const uint32_t sl = ring + at * Sh::kStage + static_cast<uint32_t>(lane & 7) * 16u;
                        for (int row = rem + (lane >> 3); row < end; row += 4)
                            for (int box = 0; box < boxes; ++box)
                                ptx::st_shared_v4(sl + box * 8192u + row * 128u, 0u, 0u, 0u, 0u);
                        ptx::fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            if constexpr (PAIR)
                                ptx::mbar_arrive_cluster(ptx::mapa(full_bar(at), 0));
                            else
                                ptx::mbar_arrive(full_bar(at));
                        }
                    }
                }
                slot = (slot + t.nkb) % stages;
            }
            if (S > 1) {
                __syncwarp();
                cluster_sync();
                cluster_sync();
            }
        }
    } else if (warp < kRoleWarps) {
        if (S > 1) {
            for (int w = first; w < total; w += step) {
                cluster_sync();
                cluster_sync();
            }
        }
    } else {
        // ---- epilogue
        if constexpr (kMoveRegs) ptx::regs_up<208>();
        const int quarter = warp & 3, half = (warp - kRoleWarps) >> 2;
        const int c_lo = half * HALF;
        const uint32_t lane_addr = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(c_lo);
        const int my = quarter * 32 + lane;             // the thread's lane of the tile
        int g = 0, buf = 0, slot = 0;
        uint32_t aph = 0, ph = 0;
        bool dead = false;
        for (int w = first; w < total; w += step) {
            Tile t;
            locate(w, g, t);
            const size_t pitch = static_cast<size_t>(args.lanes);
            const size_t out0 = (DW ? static_cast<size_t>(t.g) * args.cols + t.col0 : static_cast<size_t>(t.col0)) * pitch +
                                t.lane0 + my;
            const bool live = t.lane0 + my < args.lanes;
            // N finished values of the thread's lane, from column c on
            auto emit = [&](auto n, int c, auto value) {
                constexpr int N = decltype(n)::value;
                if (S > 1) {
#pragma unroll
                    for (int j = 0; j < N; ++j) sum_buf[(c + j) * kLanes + my] = value(j);
                } else {
                    store_values<N>(args.out, args.out_type, out0 + static_cast<size_t>(c) * pitch, pitch,
                                    live ? t.cols - c : 0, value);
                }
            };
            if constexpr (ROWS) {
                // A token to a thread: its scale times the weight block's is one
                // factor for the warp's 128 columns (the tile's columns are
                // whole weight blocks), and the sums of two columns share a
                // 64-bit register (fma.rn.f32x2).  Reading and adding 128
                // columns takes 8 warps 310 cycles by themselves and 570 beside
                // the MMAs, which take 512 a k-block; as fragments with a
                // scale for each column, 855 by themselves.
                uint64_t acc[HALF / 2];
#pragma unroll
                for (int j = 0; j < HALF / 2; ++j) acc[j] = 0;
                const int chunks = (min(HALF, max(0, t.width - c_lo)) + 15) / 16;
                const float *const factors = scale_buf + c_lo / kLanes * kLanes + my;
#pragma unroll 1
                for (int i = 0; i < t.nkb && !dead; ++i) {
                    bool ok = ptx::mbar_try_wait(acc_full(buf), aph) & ptx::mbar_try_wait(scale_full(slot), ph);
                    if (!__all_sync(0xffffffffu, ok)) {
                        ok = bounded_wait(acc_full(buf), aph, &abort_s) && bounded_wait(scale_full(slot), ph, &abort_s);
                        if (!__all_sync(0xffffffffu, ok)) {
                            dead = true;
                            break;
                        }
                    }
                    ptx::tc_fence_after_sync();
                    const float factor = factors[slot * Sh::kScaleSlot];
                    const uint64_t f2 = ptx::pack_b32x2(__float_as_uint(factor), __float_as_uint(factor));
                    const uint32_t from = lane_addr + static_cast<uint32_t>(buf * TC);
                    auto release = [&]() {
                        ptx::tc_fence_before_sync();
                        __syncwarp();
                        if (lane == 0) {
                            release_acc(acc_empty(buf));
                            ptx::mbar_arrive(scale_empty(slot));
                        }
                    };
                    uint32_t v[2][16];
                    auto add = [&](int c) {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            acc[c * 8 + j] = ptx::fma_f32x2(ptx::pack_b32x2(v[c & 1][2 * j], v[c & 1][2 * j + 1]), f2,
                                                            acc[c * 8 + j]);
                    };
                    if (chunks == HALF / 16) {                 // every column in use: no branch a load
                        ptx::tmem_ld_start_x16(from, v[0]);
#pragma unroll
                        for (int c = 0; c < HALF / 16; ++c) {
                            ptx::tmem_wait_x16(v[c & 1]);
                            if (c + 1 < HALF / 16)
                                ptx::tmem_ld_start_x16(from + (c + 1) * 16, v[(c + 1) & 1]);
                            else
                                release();
                            add(c);
                        }
                    } else {
#pragma unroll
                        for (int c = 0; c < HALF / 16; ++c) {
                            if (c < chunks) {
                                ptx::tmem_ld_start_x16(from + c * 16, v[c & 1]);
                                ptx::tmem_wait_x16(v[c & 1]);
                                add(c);
                            }
                        }
                        release();
                    }
                    if (++buf == Sh::kAcc) {
                        buf = 0;
                        aph ^= 1u;
                    }
                    if (++slot == kScaleRing) {
                        slot = 0;
                        ph ^= 1u;
                    }
                }
                auto value = [&](int j) {
                    return __uint_as_float(static_cast<uint32_t>(j & 1 ? acc[j / 2] >> 32 : acc[j / 2]));
                };
                const int cols = min(HALF, t.cols - c_lo);      // of the warp
                if (dead || cols <= 0) {
                } else if (S > 1) {
#pragma unroll
                    for (int j = 0; j < HALF; ++j) sum_buf[my * (TC + 1) + c_lo + j] = value(j);
                } else {
                    // 64 bytes of each row at a time through shared memory, so
                    // that a store writes whole sectors
                    const uint32_t warp_at = ptx::smem_addr(base + args.stage_off) +
                                             static_cast<uint32_t>(warp - kRoleWarps) * Sh::kStageWarp;
                    const uint32_t mine = warp_at + static_cast<uint32_t>(lane) * Sh::kStageRow;
                    auto staged = [&](auto *to) {
                        using T = std::remove_pointer_t<decltype(to)>;
                        constexpr int E = sizeof(T), V = 16 / E, PIECE = 64 / E;   // values of 16 and of 64 bytes
                        T *const out = to + static_cast<size_t>(t.lane0 + quarter * 32) * pitch + t.col0 + c_lo;
                        const bool wide = static_cast<uint32_t>(args.lanes) % V == 0;   // rows start on 16 bytes
                        // the last tile's boxes have been read
                        if (lane == 0) ptx::bulk_wait_read();
                        __syncwarp();
                        if constexpr (E == 2) {
                            if (args.store_boxes && quarter * 32 + 32 <= t.rows) {
                                // every row is the run's: whole boxes, which the
                                // TMA unit writes beside the next tile's sums
                                // (M4096 N8192 K4096: 109 us, stores by the
                                // warps 115; 16 runs of 8192 rows 79 and 85)
#pragma unroll
                                for (int c = 0; c < HALF; c += 8)
                                    ptx::st_shared_v4(warp_at + static_cast<uint32_t>(c / 64) * 4096u +
                                                          static_cast<uint32_t>(lane) * 128u +
                                                          static_cast<uint32_t>((c / 8 % 8) ^ (lane & 7)) * 16u,
                                                      pair16<T>(value(c), value(c + 1)), pair16<T>(value(c + 2), value(c + 3)),
                                                      pair16<T>(value(c + 4), value(c + 5)),
                                                      pair16<T>(value(c + 6), value(c + 7)));
                                ptx::fence_proxy_async_smem();
                                __syncwarp();
                                if (lane == 0) {
#pragma unroll
                                    for (int c = 0; c < HALF; c += 64)
                                        if (c < cols)
                                            ptx::tma_store_2d(&maps.out, warp_at + static_cast<uint32_t>(c / 64) * 4096u,
                                                              t.col0 + c_lo + c, t.lane0 + quarter * 32);
                                    ptx::bulk_commit();
                                }
                                return;
                            }
                        }
#pragma unroll
                        for (int c = 0; c < HALF; c += PIECE) {
                            __syncwarp();
#pragma unroll
                            for (int d = 0; d < PIECE; d += V) {
                                if constexpr (E == 4)
                                    ptx::st_shared_v4(mine + d * E, __float_as_uint(value(c + d)),
                                                      __float_as_uint(value(c + d + 1)), __float_as_uint(value(c + d + 2)),
                                                      __float_as_uint(value(c + d + 3)));
                                else
                                    ptx::st_shared_v4(mine + d * E, pair16<T>(value(c + d), value(c + d + 1)),
                                                      pair16<T>(value(c + d + 2), value(c + d + 3)),
                                                      pair16<T>(value(c + d + 4), value(c + d + 5)),
                                                      pair16<T>(value(c + d + 6), value(c + d + 7)));
                            }
                            __syncwarp();
                            if (wide) {
                                const int col = c + lane % 4 * V;
                                const bool in = col < cols;
#pragma unroll
                                for (int r = 0; r < 32; r += 8) {
                                    const int row = r + lane / 4;
                                    const float4 x = ptx::ld_shared_v4(warp_at + static_cast<uint32_t>(row) * Sh::kStageRow +
                                                                       static_cast<uint32_t>(lane % 4) * 16u);
                                    if (in && quarter * 32 + row < t.rows)
                                        *reinterpret_cast<float4 *>(out + static_cast<size_t>(row) * pitch + col) = x;
                                }
                            } else {
                                constexpr int AT_ONCE = 32 / PIECE;              // rows of a store
                                const int col = lane % PIECE, row0 = lane / PIECE;
                                const T *const from = reinterpret_cast<const T *>(
                                    base + args.stage_off + (warp - kRoleWarps) * Sh::kStageWarp) + col;
                                const int live_rows = c + col < cols ? t.rows - quarter * 32 : 0;
#pragma unroll 8
                                for (int r = row0; r < 32; r += AT_ONCE)
                                    if (r < live_rows)
                                        out[static_cast<size_t>(r) * pitch + c + col] = from[r * (Sh::kStageRow / E)];
                            }
                        }
                    };
                    if (args.out_type == 0)
                        staged(static_cast<float *>(args.out));
                    else if (args.out_type == 1)
                        staged(static_cast<__half *>(args.out));
                    else
                        staged(static_cast<__nv_bfloat16 *>(args.out));
                }
            } else if constexpr (FP8) {
                // F32 sums in fragments, two columns to a 64-bit register
                // (fma.rn.f32x2).  A thread of a fragment needs the scales of a
                // quarter of the columns, a quarter of the shared-memory reads of
                // a thread that holds a whole lane.
                constexpr int GC = Sh::kFragCols, GROUPS = HALF / GC, R = GC / 2;   // R registers a load
                const int p = lane & 3, r8 = lane >> 2;
                uint64_t acc[GROUPS][2][R / 2];
#pragma unroll
                for (int c = 0; c < GROUPS; ++c)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int j = 0; j < R / 2; ++j) acc[c][h][j] = 0;
                const int groups = (min(HALF, max(0, t.width - c_lo)) + GC - 1) / GC;
                for (int i = 0; i < t.nkb && !dead; ++i) {
                    bool ok = ptx::mbar_try_wait(acc_full(buf), aph) & ptx::mbar_try_wait(scale_full(slot), ph);
                    if (!__all_sync(0xffffffffu, ok)) {
                        ok = bounded_wait(acc_full(buf), aph, &abort_s) && bounded_wait(scale_full(slot), ph, &abort_s);
                        if (!__all_sync(0xffffffffu, ok)) {
                            dead = true;
                            break;
                        }
                    }
                    ptx::tc_fence_after_sync();
                    uint32_t v[2][R];
                    const uint32_t from = lane_addr + static_cast<uint32_t>(buf * TC);
                    const float *const sc = scale_buf + slot * Sh::kScaleSlot + (half * 4 + p) * Sh::kScalePitch;
                    // load n covers columns n / 2 * GC .. and lanes 16 (n % 2) ..
                    auto start = [&](int n) {
                        ptx::tmem_ld_start_frag(from + static_cast<uint32_t>(n / 2 * GC) + (static_cast<uint32_t>(n % 2 * 16) << 16),
                                                v[n % 2]);
                    };
                    auto add = [&](int n) {
                        const ulonglong2 *const s2 = reinterpret_cast<const ulonglong2 *>(sc + n / 2 * (GC / 4));
                        uint32_t(&now)[R] = v[n % 2];
                        uint64_t(&a)[R / 2] = acc[n / 2][n % 2];
#pragma unroll
                        for (int j = 0; j < GC / 16; ++j) {    // two groups of 8 columns
                            const ulonglong2 f = s2[j];
                            a[4 * j] = ptx::fma_f32x2(ptx::pack_b32x2(now[8 * j], now[8 * j + 1]), f.x, a[4 * j]);
                            a[4 * j + 1] = ptx::fma_f32x2(ptx::pack_b32x2(now[8 * j + 2], now[8 * j + 3]), f.x, a[4 * j + 1]);
                            a[4 * j + 2] = ptx::fma_f32x2(ptx::pack_b32x2(now[8 * j + 4], now[8 * j + 5]), f.y, a[4 * j + 2]);
                            a[4 * j + 3] = ptx::fma_f32x2(ptx::pack_b32x2(now[8 * j + 6], now[8 * j + 7]), f.y, a[4 * j + 3]);
                        }
                    };
                    auto release = [&]() {                      // the accumulator may be overwritten
                        ptx::tc_fence_before_sync();
                        __syncwarp();
                        if (lane == 0) release_acc(acc_empty(buf));
                    };
                    if (groups == GROUPS) {                    // every column in use: no branch a load
                        start(0);
#pragma unroll
                        for (int n = 0; n < 2 * GROUPS; ++n) {
                            ptx::tmem_wait(v[n % 2]);
                            if (n + 1 < 2 * GROUPS)
                                start(n + 1);
                            else
                                release();
                            add(n);
                        }
                    } else {
#pragma unroll
                        for (int c = 0; c < GROUPS; ++c) {
                            if (c < groups) {
                                start(2 * c);
                                start(2 * c + 1);
                                ptx::tmem_wait(v[0]);
                                ptx::tmem_wait(v[1]);
                                add(2 * c);
                                add(2 * c + 1);
                            }
                        }
                        release();
                    }
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(scale_empty(slot));
                    if (++buf == Sh::kAcc) {
                        buf = 0;
                        aph ^= 1u;
                    }
                    if (++slot == kScaleRing) {
                        slot = 0;
                        ph ^= 1u;
                    }
                }
                // value of group c, lane half h, 8-column group i, row pair rp, column b of the pair
                auto value = [&](int c, int h, int i, int rp, int b) {
                    const uint64_t x = acc[c][h][2 * i + rp];
                    return __uint_as_float(static_cast<uint32_t>(b ? x >> 32 : x));
                };
                const int row = quarter * 32 + r8;              // of the tile, plus 16 h + 8 rp
                if (dead) {
                } else if (S > 1) {
#pragma unroll
                    for (int c = 0; c < GROUPS; ++c)
#pragma unroll
                        for (int h = 0; h < 2; ++h)
#pragma unroll
                            for (int e = 0; e < R; ++e)         // i = e / 4, rp = e / 2 % 2, b = e % 2
                                sum_buf[(c_lo + c * GC + e / 4 * 8 + 2 * p + e % 2) * kLanes + row + 16 * h + e / 2 % 2 * 8] =
                                    value(c, h, e / 4, e / 2 % 2, e % 2);
                } else if (args.out_type != 0 && args.lanes % 8 == 0) {
                    // 16-bit outputs: 32 lanes by GC columns through shared
                    // memory (transposed on the way), then 64 bytes a row
                    const uint32_t mine = ptx::smem_addr(base + args.stage_off) +
                                          static_cast<uint32_t>(warp - kRoleWarps) * Sh::kStageWarp;
                    const int n = t.lane0 + quarter * 32 + (lane & 3) * 8;
                    auto staged = [&](auto *to) {
                        using T = std::remove_pointer_t<decltype(to)>;
                        T *const out = to + static_cast<size_t>(t.col0) * pitch + n;
                        auto pair = [&](int c, int h, int i, int rp) {
                            return pair16<T>(value(c, h, i, rp, 0), value(c, h, i, rp, 1));
                        };
#pragma unroll
                        for (int c = 0; c < GROUPS; ++c) {
                            if (c >= groups) break;
                            __syncwarp();
#pragma unroll
                            for (int i = 0; i < GC / 8; ++i)
                                ptx::stmatrix_x4_trans(mine + static_cast<uint32_t>(i * 8 + (lane & 7)) * Sh::kStageRow +
                                                           static_cast<uint32_t>(lane >> 3) * 16u,
                                                       pair(c, 0, i, 0), pair(c, 0, i, 1), pair(c, 1, i, 0), pair(c, 1, i, 1));
                            __syncwarp();
#pragma unroll
                            for (int i = 0; i < GC / 8; ++i) {
                                const int col = c_lo + c * GC + i * 8 + (lane >> 2);
                                const float4 x = ptx::ld_shared_v4(mine + static_cast<uint32_t>(i * 8 + (lane >> 2)) * Sh::kStageRow +
                                                                   static_cast<uint32_t>(lane & 3) * 16u);
                                if (col < t.cols && n < args.lanes)
                                    *reinterpret_cast<float4 *>(out + static_cast<size_t>(col) * pitch) = x;
                            }
                        }
                    };
                    if (args.out_type == 1)
                        staged(static_cast<__half *>(args.out));
                    else
                        staged(static_cast<__nv_bfloat16 *>(args.out));
                } else {
                    // F32 rows in pieces of 32 bytes; rows whose 16-bit length
                    // is no multiple of 16 bytes, value by value
                    auto direct = [&](auto *out) {
                        using T = std::remove_pointer_t<decltype(out)>;
                        T *at = out + static_cast<size_t>(t.col0 + c_lo + 2 * p) * pitch + t.lane0 + row;
                        const int cols = t.cols - c_lo - 2 * p, rows = args.lanes - t.lane0 - row;
#pragma unroll
                        for (int c = 0; c < GROUPS; ++c)
#pragma unroll
                            for (int i = 0; i < GC / 8; ++i, at += 8 * pitch)
#pragma unroll
                                for (int e = 0; e < 8; ++e) {   // b = e % 2, h = e / 4, rp = e / 2 % 2
                                    const int up = e / 4 * 16 + e / 2 % 2 * 8;
                                    if (c * GC + i * 8 + e % 2 < cols && up < rows)
                                        at[(e % 2 ? pitch : 0) + up] = rounded<T>(value(c, e / 4, i, e / 2 % 2, e % 2));
                                }
                    };
                    if (args.out_type == 0)
                        direct(static_cast<float *>(args.out));
                    else if (args.out_type == 1)
                        direct(static_cast<__half *>(args.out));
                    else
                        direct(static_cast<__nv_bfloat16 *>(args.out));
                }
            } else if constexpr (SUMS) {
                constexpr uint64_t kOnes = 0x3F8000003F800000ull;   // 1.f twice
                // F32 sums, two to a 64-bit register (fma.rn.f32x2)
                uint64_t acc[HALF / 2];
#pragma unroll
                for (int j = 0; j < HALF / 2; ++j) acc[j] = 0;
                const int chunks = min(HALF, max(0, t.width - c_lo)) / 16;
                for (int i = 0; i < t.nkb && !dead; i += UNIT) {
                    const bool ok = bounded_wait(acc_full(buf), aph, &abort_s);
                    if (!__all_sync(0xffffffffu, ok)) {
                        dead = true;
                        break;
                    }
                    ptx::tc_fence_after_sync();
                    // 16 columns load while the 16 before are added
                    uint32_t v[2][16];
                    const uint32_t from = lane_addr + static_cast<uint32_t>(buf * TC);
                    auto add = [&](int c) {
                        uint32_t(&now)[16] = v[c & 1];
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            acc[c * 8 + j] = ptx::fma_f32x2(ptx::pack_b32x2(now[2 * j], now[2 * j + 1]), kOnes, acc[c * 8 + j]);
                    };
                    if (chunks == HALF / 16) {                 // every column in use: no branch a chunk
                        ptx::tmem_ld_start_x16(from, v[0]);
#pragma unroll
                        for (int c = 0; c < HALF / 16; ++c) {
                            ptx::tmem_wait_x16(v[c & 1]);
                            if (c + 1 < HALF / 16) ptx::tmem_ld_start_x16(from + (c + 1) * 16, v[(c + 1) & 1]);
                            add(c);
                        }
                    } else {
#pragma unroll
                        for (int c = 0; c < HALF / 16; ++c) {
                            if (c < chunks) {
                                ptx::tmem_ld_start_x16(from + c * 16, v[c & 1]);
                                ptx::tmem_wait_x16(v[c & 1]);
                                add(c);
                            }
                        }
                    }
                    ptx::tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) {
                        release_acc(acc_empty(buf));
                    }
                    if (++buf == Sh::kAcc) {
                        buf = 0;
                        aph ^= 1u;
                    }
                }
                if (!dead) {
                    emit(std::integral_constant<int, HALF>(), c_lo, [&](int j) {
                        return __uint_as_float(static_cast<uint32_t>(j & 1 ? acc[j / 2] >> 32 : acc[j / 2]));
                    });
                }
            } else {
                const bool any = t.nkb > 0;             // kDw: a run without rows has zero gradients
                if (any && !dead && !warp_wait(acc_full(buf), aph, &abort_s)) dead = true;
                if (!dead) {
                    ptx::tc_fence_after_sync();
#pragma unroll 1
                    for (int c = 0; c < HALF; c += CHUNK) {
                        if (c_lo + c >= t.width) break;
                        uint32_t v[CHUNK];
                        if (any) {
                            if constexpr (CHUNK == 32)
                                ptx::tmem_ld_32x32b_x32(lane_addr + static_cast<uint32_t>(buf * TC + c), v);
                            else
                                ptx::tmem_ld_32x32b_x16(lane_addr + static_cast<uint32_t>(buf * TC + c), v);
                        } else {
#pragma unroll
                            for (int j = 0; j < CHUNK; ++j) v[j] = 0u;
                        }
                        emit(std::integral_constant<int, CHUNK>(), c_lo + c, [&](int j) { return __uint_as_float(v[j]); });
                    }
                    if (any) {
                        ptx::tc_fence_before_sync();
                        __syncwarp();
                        if (lane == 0) release_acc(acc_empty(buf));
                        if (++buf == Sh::kAcc) {
                            buf = 0;
                            aph ^= 1u;
                        }
                    }
                }
            }
            if (S > 1) {
                __syncwarp();
                cluster_sync();                        // every rank's sums stand in its shared memory
                // This block adds columns rank, rank + S, ... (ROWS: lanes), in
                // rank order, 16 reads of the blocks' memory in flight at a time.
                // A thread keeps to one place along the output's rows.
                const int lines = ROWS ? t.rows : t.cols, line_pitch = ROWS ? TC + 1 : kLanes;
                const bool on = ROWS ? my < t.cols : live;
                const size_t to = ROWS ? static_cast<size_t>(t.lane0) * pitch + t.col0 + my : out0;
                auto add_ranks = [&](auto splits) {
                    constexpr int R = decltype(splits)::value, AT_ONCE = 16 / R;
                    const uint32_t mine = ptx::smem_addr(sum_buf + my);
                    uint32_t at[R];
#pragma unroll
                    for (int r = 0; r < R; ++r) at[r] = ptx::mapa(mine, r);
                    for (int c0 = rank + R * half; c0 < lines; c0 += 2 * R * AT_ONCE) {
                        float x[AT_ONCE][R];
#pragma unroll
                        for (int j = 0; j < AT_ONCE; ++j) {
                            const uint32_t off = static_cast<uint32_t>(min(c0 + 2 * R * j, lines - 1) * line_pitch) * 4u;
#pragma unroll
                            for (int r = 0; r < R; ++r) x[j][r] = ptx::ld_cluster_f32(at[r] + off);
                        }
#pragma unroll
                        for (int j = 0; j < AT_ONCE; ++j) {
                            float sum = x[j][0];
#pragma unroll
                            for (int r = 1; r < R; ++r) sum += x[j][r];
                            const int c = c0 + 2 * R * j;
                            store_values<1>(args.out, args.out_type, to + static_cast<size_t>(c) * pitch, pitch,
                                            on && c < lines, [&](int) { return sum; });
                        }
                    }
                };
                if (S == 2)
                    add_ranks(std::integral_constant<int, 2>());
                else if (S == 4)
                    add_ranks(std::integral_constant<int, 4>());
                else
                    add_ranks(std::integral_constant<int, 8>());
                cluster_sync();                        // and may be overwritten
            }
        }
    }
    if (ROWS && warp >= kRoleWarps && lane == 0) ptx::bulk_wait();   // the outputs are written when the grid ends
    ptx::tc_fence_before_sync();
    __syncthreads();
    if constexpr (PAIR) cluster_sync();   // neither block's memory is in use by the other any more
    if (warp == 1) {
        ptx::tc_fence_after_sync();
        if constexpr (PAIR)
            ptx::tmem_dealloc_pair(tmem, Sh::kTmemCols);
        else
            ptx::tmem_dealloc(tmem, Sh::kTmemCols);
    }
}

// ------------------------------------------------------------------ host side

constexpr int kMaxDevices = 64;

std::atomic<bool> g_launched[kMaxDevices];   // a product of this file was launched (or captured)

std::atomic<int> g_plan_override{0};   // columns of a tile << 8 | splits, 0 for either: the model's choice

bool encode(CUtensorMap *map, CUtensorMapDataType type, int elem, int rank, const void *ptr, const uint64_t *dims,
            const uint32_t *box)
{
    auto fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encoder());
    if (!fn) {
        note_message("cuTensorMapEncodeTiled is not available from the driver", 0);
        return false;
    }
    cuuint64_t d[3], strides[2];
    cuuint32_t b[3], estr[3] = {1, 1, 1};
    uint64_t s = elem;
    for (int i = 0; i < rank; ++i) {
        d[i] = dims[i];
        b[i] = box[i];
        s *= dims[i];
        if (i + 1 < rank) strides[i] = s;
    }
    const CUresult r = fn(map, type, rank, const_cast<void *>(ptr), d, strides, b, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) note_message("cuTensorMapEncodeTiled (grouped operands) failed", static_cast<int>(r));
    return r == CUDA_SUCCESS;
}

template <int FORM, int TC, bool SUMS>
cudaError_t launch_tiles(const GroupedProblem &p, int splits, int64_t tiles, int dev, int sms, cudaStream_t stream)
{
    using Sh = Shape<TC>;
    constexpr bool FP8 = FORM == kFp8, DW = FORM == kDw;
    constexpr int KB = FP8 ? 128 : 64, elem = FP8 ? 1 : 2;
    const CUtensorMapDataType type = FP8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                         : p.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    Maps maps;
    // without rows (kDw writes its zeros all the same) nothing is loaded; the
    // maps describe memory that exists
    const void *const A = p.T ? p.A : p.out, *const D = p.T ? p.B : p.out;
    const uint64_t T = static_cast<uint64_t>(std::max<int64_t>(p.T, 1)), G = p.G, N = p.N, K = p.K;
    bool ok;
    if (DW) {
        const uint64_t da[2] = {K, T}, dd[2] = {N, T};
        const uint32_t box[2] = {64, 64};
        ok = encode(&maps.lane, type, elem, 2, A, da, box) && encode(&maps.col, type, elem, 2, D, dd, box);
        maps.col_part = maps.col;
    } else {
        const uint64_t da[2] = {K, T};
        const uint64_t dn[3] = {K, N, G}, dk[3] = {N, K, G};
        const uint32_t ba[2] = {KB, Sh::kLoadCols}, bp[2] = {KB, Sh::kLoadCols / 4}, bn[3] = {KB, kLanes, 1}, bk[3] = {64, 64, 1},
                       bq[3] = {KB, Sh::kLoadCols / 4, 1};
        ok = (FORM == kKn ? encode(&maps.lane, type, elem, 3, p.B, dk, bk)
                          : encode(&maps.lane, type, elem, 3, p.B, dn, bn)) &&
             encode(&maps.col, type, elem, 2, p.A, da, ba) &&
             (FP8 && TC >= 128 ? encode(&maps.col_part, type, elem, 3, p.B, dn, bq)
                               : encode(&maps.col_part, type, elem, 2, p.A, da, bp));
    }
    const bool boxes = FP8 && TC >= 128 && p.out_type != 0 && p.N % 8 == 0;
    if (ok && boxes) {
        const uint64_t dims[2] = {N, T};
        const uint32_t box[2] = {64, 32};
        ok = encode(&maps.out, p.out_type == 1 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, 2,
                    p.out, dims, box);
    }
    if (!ok) return cudaErrorInvalidValue;
    GroupedArgs a = {};
    a.store_boxes = boxes;
    a.offsets = p.offsets;
    a.sa = p.sa;
    a.sb = p.sb;
    a.out = p.out;
    a.T = static_cast<int>(p.T);
    a.G = static_cast<int>(p.G);
    a.lanes = static_cast<int>(DW ? p.K : p.N);
    a.cols = static_cast<int>(p.N);
    a.kblocks = static_cast<int>((p.K + KB - 1) / KB);
    a.out_type = p.out_type;
    a.bf16 = p.bf16;
    a.splits = splits;
    const uint32_t sums = splits > 1 ? ((TC + (FP8 && TC >= 128 ? 1 : 0)) * kLanes * 4 + 1023) / 1024 * 1024 : 0, scales = FP8 ? kScaleRing * Sh::kScaleSlot * 4 : 0,
                   staging = FP8 ? kEpilogueWarps * Sh::kStageWarp : 0;
    const uint32_t tables = (static_cast<uint32_t>(2 * (p.G + 1)) * 4 + 127) / 128 * 128;
    const uint32_t rest = sums + scales + staging + tables;
    const uint32_t room = static_cast<uint32_t>(Sh::kSmem) - 1024 - rest;
    a.stages = static_cast<int>(std::min<uint32_t>(kMaxRing, room / Sh::kStage));
    a.sum_off = a.stages * Sh::kStage;
    a.scale_off = a.sum_off + sums;
    a.stage_off = a.scale_off + scales;
    a.table_off = a.stage_off + staging;
    // enough shared memory that the blocks sharing an SM never ask for more
    // than its 512 tensor-memory columns (tmem_fits)
    const size_t smem = Sh::kSmem;
    static std::atomic<bool> ready[kMaxDevices];       // the attribute is set, per device
    if (dev >= kMaxDevices || !ready[dev].load(std::memory_order_relaxed)) {
        const void *fn = reinterpret_cast<const void *>(grouped_kernel<FORM, TC, SUMS>);
        const cudaError_t e =
            cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (e != cudaSuccess) return note_error(e, "cudaFuncSetAttribute(grouped_kernel)");
        if (dev < kMaxDevices) ready[dev].store(true, std::memory_order_relaxed);
    }
    cudaLaunchConfig_t cfg = {};
    const int cluster = Sh::kPair ? 2 : splits;
    const int64_t clusters = std::max<int64_t>(1, std::min<int64_t>(tiles, sms * Sh::kPerSm / cluster));
    cfg.gridDim = dim3(static_cast<unsigned>(clusters * cluster), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return note_error(cudaLaunchKernelEx(&cfg, grouped_kernel<FORM, TC, SUMS>, maps, a), "cudaLaunchKernelEx(grouped_kernel)");
}

// Products of a value that a 16-bit output may leave to one accumulator in
// tensor memory.  It cuts off what a step of 16 products adds below its last
// place: sums of one sign come out low by about 1.6 * 2^-24 a step on GB300, 8192
// products by 5e-5 (an eighth of F16's half unit, 2^-11), 131072 by 7.8e-4.
// Longer ones are added in registers every kUnit k-blocks, as for an F32 output
// (131072 products: 1e-5; 8192 rows, N 8192, K 16384: 1.23 ms, in one accumulator
// 1.17; the gradient of 8 runs of 16384 rows, N = K = 2048: 648 us and 640).
constexpr int64_t kOneAccumulator = 8192;

template <int FORM, int TC>
cudaError_t launch_form(const GroupedProblem &p, int splits, int64_t tiles, int dev, int sms, cudaStream_t stream)
{
    // (kDw: no run is longer than T)
    const int64_t products = FORM == kDw ? p.T : (p.K + splits - 1) / splits;
    if constexpr (FORM != kFp8)
        if (p.out_type != 0 && products <= kOneAccumulator) return launch_tiles<FORM, TC, false>(p, splits, tiles, dev, sms, stream);
    return launch_tiles<FORM, TC, true>(p, splits, tiles, dev, sms, stream);
}

}  // namespace

int64_t grouped_tiles(const GroupedProblem &p, int tc)
{
    const int64_t lanes = p.form == GroupedForm::kDw ? p.K : p.N, tl = tc == 256 ? 2 * kLanes : kLanes;
    const int64_t lane_tiles = (lanes + tl - 1) / tl;
    if (p.form == GroupedForm::kDw) return p.G * lane_tiles * ((p.N + tc - 1) / tc);
    // a run of c rows has ceil(c / tc) column tiles: at most T / tc of them full, and one more each
    return lane_tiles * (p.G == 1 ? (p.T + tc - 1) / tc : p.T / tc + std::min<int64_t>(p.G, p.T));
}

// The plan with the least time by a model of one launch:
//   waves * (k-blocks / splits) * us a k-block + waves * us to join the splits
// The microseconds are measured on GB300 with every SM at work (M 16 to 2048,
// N 1024 to 8192, K 2048 to 8192, and 8 to 24 runs) and hold all that a k-block
// costs there.  Set-up, a tile's stores and rows that straddle lines have no term:
// the model ranks plans, it is not the time (M4096 N8192 K4096 in 8 bits: 121 us
// here, 109 measured; the gradient of 8 runs of 8192 rows, N = K = 2048: 35 and 60).
// Runs of unknown lengths are taken to end half a tile past their last full one
// on average.
GroupedPlan plan_grouped(const GroupedProblem &p, int sms)
{
    struct Tiling {
        int tc;
        double us8, us16, join;
    };
    static constexpr Tiling kTilings[] = {   // 32: two blocks to an SM
        {32, 0.38, 0.30, 1.5}, {64, 0.285, 0.26, 2.}, {128, 0.33, 0.26, 2.5}, {256, 0.54, 0.31, 0.}};
    constexpr double kAlone = 0.8;           // of those figures, for a 32-column block alone on its SM
    const bool dw = p.form == GroupedForm::kDw, fp8 = p.form == GroupedForm::kFp8;
    const int64_t k = dw ? std::max<int64_t>(1, p.T / p.G) : p.K, kb = (k + (fp8 ? 127 : 63)) / (fp8 ? 128 : 64);
    const int asked = g_plan_override.load(std::memory_order_relaxed), only_tc = asked >> 8, only_splits = asked & 255;
    GroupedPlan best = {128, 1};
    double least = 0;
    for (const Tiling &t : kTilings) {
        if (dw && t.tc < 128) continue;
        if (only_tc != 0 && t.tc != only_tc && !(dw && only_tc < 128)) continue;
        const int64_t tl = t.tc == 256 ? 2 * kLanes : kLanes;
        const double lane_tiles = static_cast<double>(((dw ? p.K : p.N) + tl - 1) / tl);
        const double runs = static_cast<double>(std::min(p.G, p.T));
        const double col_tiles = dw ? static_cast<double>(p.G) * static_cast<double>((p.N + t.tc - 1) / t.tc)
                                 : p.G == 1 ? static_cast<double>((p.T + t.tc - 1) / t.tc)
                                            : std::max(runs, static_cast<double>(p.T) / t.tc + runs / 2);
        const double places = t.tc == 256 ? sms / 2 : t.tc == 32 ? sms * 2 : sms;
        int most = 1;   // a split of fewer than two k-blocks never pays
        while (most < 8 && !dw && t.tc != 256 && kb >= 4 * most) most *= 2;
        for (int splits = 1; splits <= most; splits *= 2) {
            if (only_splits != 0) {
                if (splits != std::min(only_splits, most)) continue;
            } else if (splits > 1 && lane_tiles * col_tiles * splits > places) {
                break;   // more blocks than places
            }
            const double waves = std::ceil(lane_tiles * col_tiles * splits / places);
            double rate = (fp8 ? t.us8 : t.us16) * (t.tc == 32 && lane_tiles * col_tiles * splits <= sms ? kAlone : 1.);
            // a pair's 16-bit time goes by the rows it loads: 128 lanes and half the columns a block
            // (set at 24 ragged runs of 1003 rows, N 1000, K 1544: 17 us in pairs, 23 in 64 columns)
            if (t.tc == 256 && !fp8 && !dw) rate *= 0.65 + 0.35 * std::min(1., static_cast<double>(p.T) / (runs * t.tc));
            const double us = waves * (static_cast<double>((kb + splits - 1) / splits) * rate + (splits > 1 ? t.join : 0.));
            if (least == 0 || us < least) {
                least = us;
                best = {t.tc, splits};
            }
        }
    }
    return best;
}

void set_grouped_override(int columns, int splits) { g_plan_override.store(columns << 8 | splits); }

template <int FORM>
cudaError_t launch_plan(const GroupedProblem &p, const GroupedPlan &plan, int64_t tiles, int dev, int sms, cudaStream_t stream)
{
    switch (plan.tc) {
    case 256: return launch_form<FORM, 256>(p, plan.splits, tiles, dev, sms, stream);
    case 128: return launch_form<FORM, 128>(p, plan.splits, tiles, dev, sms, stream);
    case 64:
        if constexpr (FORM != kDw) return launch_form<FORM, 64>(p, plan.splits, tiles, dev, sms, stream);
        break;
    case 32:
        if constexpr (FORM != kDw) return launch_form<FORM, 32>(p, plan.splits, tiles, dev, sms, stream);
        break;
    }
    return note_error(cudaErrorInvalidConfiguration, "columns of a tile");
}

cudaError_t launch_grouped(const GroupedProblem &p, cudaStream_t stream)
{
    static std::atomic<int> counts[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return note_error(e, "cudaGetDevice");
    int sms = dev < kMaxDevices ? counts[dev].load(std::memory_order_relaxed) : 0;
    if (sms == 0) {
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return note_error(e, "cudaDeviceGetAttribute(MultiProcessorCount)");
        if (dev < kMaxDevices) counts[dev].store(sms, std::memory_order_relaxed);
    }
    if (dev < kMaxDevices) g_launched[dev].store(true);
    const GroupedPlan plan = plan_grouped(p, sms);
    const int64_t tiles = grouped_tiles(p, plan.tc);
    switch (p.form) {
    case GroupedForm::kFp8: return launch_plan<kFp8>(p, plan, tiles, dev, sms, stream);
    case GroupedForm::kNk: return launch_plan<kNk>(p, plan, tiles, dev, sms, stream);
    case GroupedForm::kKn: return launch_plan<kKn>(p, plan, tiles, dev, sms, stream);
    default: return launch_plan<kDw>(p, plan, tiles, dev, sms, stream);
    }
}

cudaError_t read_and_clear_grouped_status(unsigned *status)
{
    const unsigned zero = 0;
    *status = 0;
    int dev = 0;
    // nothing launched, nothing to read: a copy is 5 us
    if (cudaGetDevice(&dev) == cudaSuccess && dev < kMaxDevices && !g_launched[dev].load()) return cudaSuccess;
    cudaError_t e = cudaMemcpyFromSymbol(status, g_grouped_status, sizeof *status);
    if (e == cudaSuccess && *status) e = cudaMemcpyToSymbol(g_grouped_status, &zero, sizeof zero);
    return note_error(e, "reading the grouped kernels' status word");
}

}  // namespace splitk
