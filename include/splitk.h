/*
 * splitk.h -- C ABI of libsplitk: split-K GEMM with prepared, transposed
 * weights, for NVIDIA GB300 (sm_103a).
 *
 * The operation (pages "Aligned shared rows for pipelined NAX on CUDA", section
 * "Contract and correctness", and "Wider consecutive-weight NAX GEMM", section
 * "Launch contract and correctness"):
 *
 *   A        row-major [M,K]          F32, F16 or BF16
 *   B        row-major [N,K]          same element type; the prepared weight,
 *                                     i.e. the transpose of a [K,N] weight
 *   split s  covers k in [s*kps, min((s+1)*kps, K))
 *   partials[s,m,n] = sum_{k in split s} A[m,k] * B[n,k]     F32, [splits,M,N]
 *   out[m,n]        = sum_{s=0}^{splits-1} partials[s,m,n]   F32, [M,N]
 *
 * The second line is the separate accumulation pass the pages run after the
 * partial pass ("an existing accumulation pass produces the final output").
 *
 * Contract enforced by every entry point before any device work:
 *   - M, K and k_per_split are positive multiples of 32; N is a positive
 *     multiple of 64;                                   else SPLITK_ERR_SHAPE
 *   - every split starts below K and the splits cover K, i.e.
 *     splits == ceil(K / k_per_split);                  else SPLITK_ERR_SPLIT
 *   - M, N, K <= SPLITK_MAX_DIM and splits <= SPLITK_MAX_SPLITS
 *     (implementation limits);                           else SPLITK_ERR_SHAPE
 *   - no pointer is NULL;                                else SPLITK_ERR_NULL
 *   - every pointer is 16-byte aligned;                  else SPLITK_ERR_ALIGN
 *   - output byte ranges overlap neither the input ranges nor each other
 *     (A and B may overlap each other: both are only read); else SPLITK_ERR_ALIAS
 *
 * Memory and ownership: every data pointer is a DEVICE pointer on the current
 * CUDA device, owned by the caller, except the host activations and results
 * of gemm_bt_host_batch.  The library allocates no device memory on any call
 * path and keeps no pointer to caller memory for use after a call returns.
 * (Each host thread caches, in host memory, the last tile plans and TMA
 * tensor maps it built; a cached map records an address and a shape and is
 * reused only by a later call with the same address and shape.)
 *
 * Asynchrony and errors: calls enqueue work on `stream` (a cudaStream_t, passed
 * as void*; NULL means the legacy default stream) and return without
 * synchronising.  A non-zero return means nothing was enqueued (validation
 * failed) or the launch itself failed (SPLITK_ERR_CUDA).  No exception and no
 * abort crosses the ABI.  Every wait inside a kernel has a time limit; a wait
 * that runs out sets a device status word, which splitk_get_device_status()
 * reads.  The compute entry points (gemm_splitk_bt, splitk_reduce, gemm_bt,
 * their [K,N] forms, gemm_bt_batch and gemm_bt_noalloc after its first call)
 * may be captured into a CUDA graph.
 *
 * Consecutive launches inside a graph: every launch is a programmatic
 * dependent of the one before it on its stream.  Eagerly, each launch waits
 * for the previous grid to finish before it reads its operands.  While a
 * stream is being captured, the library sees what the next launch depends on
 * (cudaStreamGetCaptureInfo); when that is exactly its own previous launch on
 * the stream, and the new launch reads (A and B; the partials, for the
 * reduce) no byte that any of its launches still able to run writes, the new
 * launch starts loading and multiplying at once and waits for the previous
 * grid only before its first store ("overlap"); if none of them reads or
 * writes what the new launch writes either, it also stores at once and
 * waits only before it finishes, so the grids still finish in launch order.
 * Such a fused launch may also give each thread block two consecutive chunks
 * of its split (all of them where a split has two), each in its own
 * accumulator, added inside the block (the owner adds a split's chunks in
 * pairs too), or, for large shapes with full splits, every chunk of every
 * split.
 * A call that may store early and has the same shape and plan as the launch
 * before it joins that launch instead of adding one: the launch's graph
 * node then computes both calls (up to 8), whose blocks may run in any
 * order; the first such call after a run's first launch may also switch
 * that launch to its own plan (compact, or whole-K).  Its results are
 * bitwise those of the same launch without overlap.
 * Launches that read what an
 * earlier one writes (a chain of GEMMs, the reduce after the partial pass),
 * launches after another kernel or a copy, and launches outside a capture
 * wait as usual.  The decision is made at capture time from the pointers
 * passed; a graph whose nodes are later given other buffers
 * (cudaGraphExecKernelNodeSetParams) must keep the same pattern of overlaps
 * between them, and the calls grouped into one node stay in that node.
 * splitk_set_overlap turns the grouping, or both, off for later captures.
 */
#ifndef SPLITK_H
#define SPLITK_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Element type of A and B.  Partials and the output are always F32. */
typedef enum {
    SPLITK_F32 = 0,
    SPLITK_F16 = 1,
    SPLITK_BF16 = 2
} splitk_dtype;

typedef enum {
    SPLITK_OK = 0,
    SPLITK_ERR_NULL = -1,           /* a required pointer is NULL */
    SPLITK_ERR_SHAPE = -2,          /* M,K,kps not positive multiples of 32, N of 64, or too large */
    SPLITK_ERR_SPLIT = -3,          /* splits != ceil(K/kps): a split starts at/after K or K is not covered */
    SPLITK_ERR_ALIAS = -4,          /* an output range overlaps an input or another output */
    SPLITK_ERR_ALIGN = -5,          /* a pointer is not 16-byte aligned */
    SPLITK_ERR_DTYPE = -6,          /* unknown element type */
    SPLITK_ERR_WORKSPACE = -7,      /* workspace smaller than the call's ..._workspace_bytes() */
    SPLITK_ERR_CUDA = -8,           /* a CUDA runtime call or launch failed */
    SPLITK_ERR_DEVICE_TIMEOUT = -9, /* a kernel's bounded wait ran out (see splitk_get_device_status) */
    SPLITK_ERR_CONFIG = -10         /* an invalid value (tile override, eps, max_norm, a mode) */
} splitk_status;

#define SPLITK_MAX_DIM (1 << 22)
#define SPLITK_MAX_SPLITS 4096
/* Runs (experts) of a grouped product. */
#define SPLITK_MAX_GROUPS 1024
/* Experts of one token. */
#define SPLITK_MAX_TOP 32
/* Tensors of one gradient norm, and values of one of them. */
#define SPLITK_MAX_TENSORS 65536
#define SPLITK_MAX_TENSOR_VALUES ((int64_t)1 << 34)
/* Size of the scratch array gemm_bt_noalloc keeps in device memory. */
#define SPLITK_NOALLOC_MAX_BYTES (32 << 20)

/* Checks the contract's shape and split rules only (no pointers, no device
 * work).  Returns SPLITK_OK, SPLITK_ERR_SHAPE or SPLITK_ERR_SPLIT; the shape
 * rule is checked first. */
int splitk_check_geometry(int64_t M, int64_t N, int64_t K, int64_t splits,
                          int64_t k_per_split);

/* The partial pass: partials[s,m,n] = sum over split s of A[m,k]*B[n,k].
 *   A         device, [M,K] row-major, element type `dtype`
 *   B         device, [N,K] row-major, element type `dtype`
 *   partials  device, [splits,M,N] row-major F32; fully overwritten
 * BF16/F16 operands run on the tensor cores (tcgen05, F32 accumulate in tensor
 * memory, native operands).  F32 operands run on the tensor cores too, each
 * product as three TF32 products: x = hi + lo, where hi is the F32 operand as
 * loaded, which the tensor cores read as TF32 by dropping its 13 low fraction
 * bits (its top 19 bits; measured on GB300: truncation, not rounding), and
 * lo = x - (x with those 13 bits cleared), exact in F32; hi*lo + lo*hi +
 * hi*hi, relative error per product about 2^-21.  Each element is a sum in
 * F32 whose order is fixed for a given shape. */
int gemm_splitk_bt(const void *A, const void *B, float *partials, int64_t M,
                   int64_t N, int64_t K, int64_t splits, int64_t k_per_split,
                   int dtype, void *stream);

/* Weight preparation (pages: "Wider consecutive-weight NAX GEMM", section
 * "Performance method" -- the transposed layout is prepared once, outside
 * timing, and kept resident): B[n,k] = W[k,n].
 *   W  device, [K,N] row-major, element type `dtype` (bits copied as they are)
 *   B  device, [N,K] row-major, same type; fully overwritten
 * K a positive multiple of 32 and N of 64 (the GEMM's contract for B),
 * 16-byte aligned pointers, no overlap; else SPLITK_ERR_SHAPE / _DTYPE /
 * _NULL / _ALIGN / _ALIAS before any device work. */
int splitk_prepare_bt(const void *W, void *B, int64_t K, int64_t N, int dtype,
                      void *stream);

/* The accumulation pass: out[i] = (((P[0][i] + P[1][i]) + P[2][i]) + ...) in
 * F32, in split order s = 0..splits-1.
 *   partials  device, [splits,M,N] F32, read only
 *   out       device, [M,N] F32; fully overwritten
 * Requires M, N >= 1, splits >= 1, 16-byte aligned pointers and no overlap
 * between the two ranges. */
int splitk_reduce(const float *partials, float *out, int64_t splits, int64_t M,
                  int64_t N, void *stream);

/* Bytes of device workspace gemm_bt needs: the F32 partials [splits,M,N],
 * splits*M*N*4 bytes.  The same size serves every value of `fused`.  Returns
 * 0 for a geometry that breaks the contract. */
size_t gemm_bt_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t splits,
                               int64_t k_per_split, int fused);

/* Zeroes a workspace (cudaMemsetAsync on `stream`).  gemm_bt needs no
 * particular workspace contents (every byte it reads it wrote in the same
 * call); this gives callers a defined starting state. */
int gemm_bt_workspace_init(void *workspace, size_t workspace_bytes, void *stream);

/* One call: the partial pass then the accumulation pass, on one stream.
 *   out        device, [M,N] F32; fully overwritten
 *   workspace  device, >= gemm_bt_workspace_bytes() bytes, caller-owned
 *              scratch; may not overlap A, B or out.
 *   fused      0: two kernels (gemm_splitk_bt, then splitk_reduce); the
 *                 workspace then holds the partials [splits,M,N] in its
 *                 first bytes;
 *              1: one kernel where the tile plan holds all of a tile's
 *                 splits in one resident thread-block cluster: the splits
 *                 are summed inside the launch, over distributed shared
 *                 memory, and the partials are not kept.  Where it cannot
 *                 (too many splits for one cluster, or more tiles than
 *                 resident clusters), the call runs the two kernels of 0,
 *                 which measured faster there than summing through global
 *                 memory.  splitk_describe_launch reports which;
 *              3: as 1, and the workspace also holds the partials afterwards.
 * For a given shape, `out` (and the partials, where kept) are bitwise the
 * same for every value of `fused`. */
int gemm_bt(const void *A, const void *B, float *out, void *workspace,
            size_t workspace_bytes, int64_t M, int64_t N, int64_t K,
            int64_t splits, int64_t k_per_split, int dtype, int fused,
            void *stream);

/* The same two operations with the weight in its own [K,N] layout, the other
 * layout the pages keep resident ("Wider consecutive-weight NAX GEMM",
 * section "Performance method": both layouts uploaded once); no preparation
 * step.
 *   W  device, [K,N] row-major, element type `dtype`; B[n,k] = W[k,n]
 * Every other argument, the contract and the checks are those of
 * gemm_splitk_bt and gemm_bt with B = W^T, and for BF16/F16 the results too
 * (bitwise): the tensor cores read W N-contiguous (MN-major operand).  F32
 * operands with W run exact F32 FMA on the CUDA cores (no fused variant: the
 * two-kernel path runs for every `fused`). */
int gemm_splitk_kn(const void *A, const void *W, float *partials, int64_t M,
                   int64_t N, int64_t K, int64_t splits, int64_t k_per_split,
                   int dtype, void *stream);
int gemm_kn(const void *A, const void *W, float *out, void *workspace,
            size_t workspace_bytes, int64_t M, int64_t N, int64_t K,
            int64_t splits, int64_t k_per_split, int dtype, int fused,
            void *stream);

/* gemm_bt for callers that cannot allocate device memory.  The paper has no
 * counterpart of this entry point; it exists for hosts that hand an operator
 * only its input and output buffers and forbid allocation while it runs (the
 * execute callback of an inference-runtime plugin, for one) and for loops
 * where cudaMalloc's implicit device synchronisation is not acceptable.
 *   A, B, out, M, N, K, splits, k_per_split, dtype, fused, stream
 *              as for gemm_bt; no workspace argument.
 * Instead of a caller workspace it uses a scratch array of
 * SPLITK_NOALLOC_MAX_BYTES (32 MiB) that the library keeps in device memory;
 * every GPU that loads the library holds that array until the process exits.
 * A shape whose gemm_bt_workspace_bytes() exceeds it is rejected with
 * SPLITK_ERR_WORKSPACE before any device work (splitk_last_error() gives the
 * sizes).  The call allocates nothing: no cudaMalloc, no cudaFree, no
 * allocating library routine.  Each call looks up the array's device
 * address on the current device (cudaGetSymbolAddress, a lookup that
 * allocates nothing); the first call on a device also loads the library's
 * device code there, so make that first call before any stream capture.
 * Every call on a device shares the one array and leaves its contents behind
 * (the partials).  Calls whose executions overlap on the GPU (on different
 * streams, say) race on the array and must not be issued. */
int gemm_bt_noalloc(const void *A, const void *B, float *out, int64_t M,
                    int64_t N, int64_t K, int64_t splits, int64_t k_per_split,
                    int dtype, int fused, void *stream);

/* `count` independent operations out_i = gemm_bt(A_i, B_i) of one shape on
 * device buffers, enqueued on `stream` in as few launches as the plan
 * allows.  The pages time eight complete operations per replay ("pack 8":
 * "Aligned shared rows for pipelined NAX on CUDA", section "Measurement
 * protocol"); outside a graph capture this call gives such a pack the
 * grouped launches a capture would.
 *   A, B, out   host arrays of `count` DEVICE pointers: activations [M,K],
 *               prepared weights [N,K] (entries may repeat, as may A's) and
 *               outputs [M,N] F32, each fully overwritten
 *   workspace   device, >= gemm_bt_workspace_bytes() bytes: scratch for the
 *               operations that run the two kernels, used one after another
 *   count       1 .. 65536
 *   fused       0 or 1 (as for gemm_bt; fused = 1 calls whose splits are
 *               summed inside the launch run up to 8 to a launch, BF16/F16
 *               with a compact plan; everything else one gemm_bt each)
 * Every result is bitwise that of gemm_bt(fused) on the same operands.
 * Returns as gemm_bt's validation would for each operation, plus
 * SPLITK_ERR_CONFIG for count outside [1, 65536] or fused not 0 or 1, and
 * SPLITK_ERR_ALIAS when an output overlaps another output, an input or the
 * workspace; nothing is enqueued unless every operation passes. */
int gemm_bt_batch(const void *const *A, const void *const *B, float *const *out,
                  int64_t count, void *workspace, size_t workspace_bytes,
                  int64_t M, int64_t N, int64_t K, int64_t splits,
                  int64_t k_per_split, int dtype, int fused, void *stream);

/* Device staging bytes gemm_bt_host_batch needs for `count` operations of
 * this shape: count A slots [M,K], count output slots [M,N] F32 and one
 * gemm_bt workspace.  Returns 0 for a rejected geometry or element type, or
 * count outside [1, 65536]. */
size_t gemm_bt_host_staging_bytes(int64_t count, int64_t M, int64_t N,
                                  int64_t K, int64_t splits,
                                  int64_t k_per_split, int dtype);

/* `count` operations out_i = gemm_bt(A_i, B_i) whose activations and results
 * live in HOST memory.  The pages time operands already on the device; this
 * entry point adds the copies a serving loop needs, pipelined so that they
 * overlap the kernels.
 *   A_host     host, [count,M,K] elements of `dtype`, operation i at
 *              i*M*K; read by the copy engine (page-locked memory lets the
 *              copies run asynchronously; any memory cudaMemcpyDefault
 *              accepts works)
 *   B          host array of `count` DEVICE pointers, each a prepared weight
 *              [N,K] (16-byte aligned; entries may repeat)
 *   out_host   host, [count,M,N] F32; fully overwritten once `stream`
 *              reaches the end of the call's work
 *   staging    device, >= gemm_bt_host_staging_bytes(), 16-byte aligned,
 *              overlapping no B
 *   fused      as for gemm_bt (0, 1 or 3)
 *   ops_per_copy  operations moved by one copy each way; 0 lets the library
 *              choose (at least 4 MiB of A per copy, at most half the batch)
 * Every operation is bitwise the gemm_bt result for its operands.  With
 * fused = 1, 16-bit operands and a shape whose splits are summed inside the
 * launch, the operations of a group run as one launch (up to 8 of them; the
 * same tiles and sums as one call each); otherwise one gemm_bt each.  The copy
 * in of group g+1 and the copy out of group g-1 run on two library streams
 * while group g computes on `stream`, and `stream` waits for the last copy
 * out, so synchronising `stream` completes the batch.  Host buffers must stay
 * valid until then.  The copy in waits for the end of the previous call on
 * the same staging (the library keeps one event per staging buffer, for the
 * 32 most recently used), or, for a staging it has not seen, for the work
 * already on `stream`: calls that alternate two staging buffers overlap one
 * batch's copy in with the previous batch's kernels.  On one stream a call's
 * kernels still follow the previous call's copy out (stream order); calls
 * that alternate two streams as well also overlap that copy out with the
 * next batch's kernels.  Between calls the
 * staging belongs to them: other work must not write it, and one staging is
 * used with one stream (its workspace part is used in stream order).
 * The first call on a device creates those two streams and four events (kept
 * until exit); a process-wide mutex serialises the enqueueing of concurrent
 * calls.  Returns as gemm_bt's validation would (plus SPLITK_ERR_CONFIG for
 * count outside [1, 65536] or ops_per_copy < 0, SPLITK_ERR_WORKSPACE for a
 * small staging, SPLITK_ERR_ALIAS when A_host and out_host overlap or the
 * staging overlaps a B or a host range) before enqueueing anything. */
int gemm_bt_host_batch(const void *A_host, const void *const *B,
                       float *out_host, int64_t count, void *staging,
                       size_t staging_bytes, int64_t M, int64_t N, int64_t K,
                       int64_t splits, int64_t k_per_split, int dtype,
                       int fused, int64_t ops_per_copy, void *stream);

/* Split count for a shape.  The pages sweep 1, 2, 4, 8 and 16 splits of fixed
 * shapes ("Aligned shared rows for pipelined NAX on CUDA", section
 * "Measurement protocol"; "Wider consecutive-weight NAX GEMM", section
 * "Performance method"); these two entry points pick among the same
 * candidates.  For a candidate n, k_per_split = ceil(K/n) rounded up to a
 * multiple of 32 and splits = ceil(K/k_per_split) (below n when K is short).
 *
 * splitk_choose_splits: the library's cost model of gemm_bt with `fused`
 * (the tile planner's estimate plus the reduce for the two-kernel path); no
 * device work.  Writes the cheapest legal (splits, k_per_split) and, when
 * model_us is not NULL, model_us[0..4] = the estimate in microseconds per
 * call for candidates 1, 2, 4, 8, 16 (-1 for an illegal one).  M and K positive
 * multiples of 32, N of 64 (else SPLITK_ERR_SHAPE), a known dtype
 * (SPLITK_ERR_DTYPE), fused in {0, 1, 3} (SPLITK_ERR_CONFIG), non-NULL
 * outputs (SPLITK_ERR_NULL). */
int splitk_choose_splits(int64_t M, int64_t N, int64_t K, int dtype, int fused,
                         int64_t *splits, int64_t *k_per_split,
                         double *model_us);

/* splitk_autotune_splits: measures each candidate on the caller's buffers
 * (A, B, out, workspace as for gemm_bt) and writes the fastest legal
 * (splits, k_per_split).  Per candidate: one untimed call, then a CUDA graph
 * of `reps` calls (1..1000) replayed three times between CUDA events on a
 * private stream that first waits for the work already on `stream`.
 * us[0..4], when not NULL, receive the microseconds per call of candidates
 * 1, 2, 4, 8, 16 (-1 where a candidate was not run: its workspace does not
 * fit `workspace_bytes`, or it repeats an earlier candidate's split count).
 * Every candidate's arguments are checked before anything is enqueued (the
 * statuses of gemm_bt; SPLITK_ERR_WORKSPACE if no candidate fits).  On
 * return the private stream has finished, `out` holds the chosen split's
 * result and `stream` is ordered after it.  The inputs are
 * read repeatedly, so they sit in L2 when they fit there: the timings rank
 * the candidates, they are not cold-cache figures.  Not capturable. */
int splitk_autotune_splits(const void *A, const void *B, float *out,
                           void *workspace, size_t workspace_bytes, int64_t M,
                           int64_t N, int64_t K, int dtype, int fused,
                           int reps, void *stream, int64_t *splits,
                           int64_t *k_per_split, float *us);

/* ---- 8-bit operands and rows grouped by expert
 *
 * 8-bit values are E4M3 (largest value 448, no infinities), stored one to a
 * byte.  Along K they share an F32 scale in blocks of 128, the last block
 * possibly short: the number that q stands for is q * scale.
 *   activations  q [M,K], scales [M, ceil(K/128)]: a scale for each 128
 *                values of a row
 *   weights      q [G,N,K], scales [G, ceil(N/128), ceil(K/128)]: a scale for
 *                each 128 x 128 block (edge blocks smaller)
 * Scales may be any F32 values (no power of two is assumed).  A product forms
 * the two scales that meet into one F32 factor first: beyond F32's range it is
 * infinite, and NaN against a sum of 0; below 2^-126 it is within 2^-150 (a
 * block of zeros, whose scale is 2^-126, gives 0 with any finite scale).
 *
 * Every tensor is dense and row-major; rows follow one another without
 * padding.  K is a positive multiple of 16 with 8-bit operands and of 8 with
 * 16-bit ones, whatever N and M (or T) are, unless said otherwise.  M (or T)
 * may be 0: nothing is written then, except by gemm_grouped_dw, and the
 * tensors without elements may be NULL.  M, T, N, K <=
 * SPLITK_MAX_DIM, G <= SPLITK_MAX_GROUPS, and what a call works through must
 * count below 2^31: ceil(N/128) * (T/32 + G) tiles of a product (M for T, G =
 * 1 where there are no runs), G * ceil(K/128) * ceil(N/32) of gemm_grouped_dw,
 * the scales of fp8_prepare_bt (else SPLITK_ERR_SHAPE).  Pointers are
 * 16-byte aligned (`offsets`: 4-byte), outputs overlap nothing (exceptions are
 * named), and out_dtype is SPLITK_F32, _F16 or _BF16, rounded once from the
 * F32 sum.  Checks come before any device work, in the order shape, dtype,
 * NULL, alignment, overlap, eps.  The calls take no workspace, may be captured,
 * and give the same bits for the same call every time. */

/* Residual addition, root-mean-square norm, 8-bit output:
 *   h = x + residual, rounded to `dtype` (h = x without a residual)
 *   y = h * weight / sqrt(mean_k h^2 + eps), in F32
 *   scales[m,b] = max(max_{k in b} |y[m,k]| / 448, 2^-126)
 *   q[m,k]      = y[m,k] / scales[m,b] to E4M3, to nearest even
 *   x, residual  device, [M,K] of `dtype` (SPLITK_F32, _F16, _BF16); residual
 *                may be NULL
 *   weight       device, [K] of `dtype`
 *   sum          device, [M,K] of `dtype` or NULL: receives h; may be exactly
 *                x or residual (in place)
 *   y            device, [M,K] of `dtype` or NULL: receives y, rounded once
 *   q, scales    device, as above
 * Finite rows of any size have their norm, also where the squares leave F32's
 * range.  A row that holds a NaN gets NaN scales and codes; one that holds an
 * infinity NaN in the infinity's block and zeros elsewhere (its mean is
 * infinite).  eps >= 0 (else SPLITK_ERR_CONFIG); with eps = 0 a row of zeros
 * is 0 / 0: NaN scales and codes. */
int rmsnorm_fp8(const void *x, const void *residual, const void *weight,
                void *sum, void *y, void *q, float *scales, int64_t M,
                int64_t K, float eps, int dtype, void *stream);

/* Activations x [M,K] of `dtype` to 8 bits, as rmsnorm_fp8 does with y = x. A
 * block that holds a NaN gets NaN scale and codes; one that holds an infinity
 * an infinite scale (and NaN for the infinity, 0 for the rest). */
int fp8_quantize(const void *x, void *q, float *scales, int64_t M, int64_t K,
                 int dtype, void *stream);

/* Weight preparation, once: B [G,N,K] of `dtype` to 8 bits with a scale for
 * each 128 x 128 block (max |B| / 448, at least 2^-126).  G = 1 for a single
 * weight. */
int fp8_prepare_bt(const void *B, void *Bq, float *scales, int64_t G,
                   int64_t N, int64_t K, int dtype, void *stream);

/* out[m,n] = sum_b a_scales[m,b] * b_scales[n/128,b] * sum_{k in b} A[m,k]*B[n,k]
 * with A [M,K] and B [N,K] in 8 bits.  The sum over a block runs on the
 * tensor cores; the scaled sum over blocks is in F32, the scales multiplied
 * first. */
int gemm_fp8_bt(const void *A, const float *a_scales, const void *B,
                const float *b_scales, void *out, int64_t M, int64_t N,
                int64_t K, int out_dtype, void *stream);

/* Products grouped by expert: the rows of A [T,K] stand sorted by expert, run
 * g being rows offsets[g] .. offsets[g+1]-1, and each run meets its own weight:
 *   out[t,n] = sum_k A[t,k] * B[g,n,k]        t in run g
 *   offsets  device, int32 [G+1], not decreasing, within [0,T]; runs may be
 *            empty.  It is read on the device: no synchronisation.  (Offsets
 *            that break the rule are clamped to it, so that no access leaves
 *            the tensors; the result is then that of the clamped runs.)
 *   out      device, [T,N]; rows before offsets[0] and from offsets[G] on are
 *            left as they are
 * gemm_grouped_fp8_bt: 8-bit operands with scales, as gemm_fp8_bt. */
int gemm_grouped_fp8_bt(const void *A, const float *a_scales, const void *B,
                        const float *b_scales, const int32_t *offsets,
                        void *out, int64_t T, int64_t G, int64_t N, int64_t K,
                        int out_dtype, void *stream);

/* 16-bit operands (dtype SPLITK_F16 or _BF16; else SPLITK_ERR_DTYPE), weights
 * B [G,N,K]. */
int gemm_grouped_bt(const void *A, const void *B, const int32_t *offsets,
                    void *out, int64_t T, int64_t G, int64_t N, int64_t K,
                    int dtype, int out_dtype, void *stream);

/* The same with weights W [G,K,N] (N a multiple of 8).  It is also the
 * gradient of gemm_grouped_bt's A: dA = gemm_grouped_kn(dOut, B) with N and K
 * exchanged. */
int gemm_grouped_kn(const void *A, const void *W, const int32_t *offsets,
                    void *out, int64_t T, int64_t G, int64_t N, int64_t K,
                    int dtype, int out_dtype, void *stream);

/* The gradient of gemm_grouped_bt's B:
 *   dB[g,n,k] = sum_{t in run g} D[t,n] * A[t,k]
 *   A   device, [T,K]; D device, [T,N], the output's gradient (N a multiple of
 *       8); both of `dtype`
 *   dB  device, [G,N,K] of out_dtype, fully overwritten: zeros for an empty
 *       run
 * (gemm_grouped_kn's W has the gradient dW[g,k,n]: the same call with A and D,
 * and N and K, exchanged.) */
int gemm_grouped_dw(const void *A, const void *D, const int32_t *offsets,
                    void *dB, int64_t T, int64_t G, int64_t N, int64_t K,
                    int dtype, int out_dtype, void *stream);

/* ---- Routing, and rows sorted by expert and back
 *
 * M tokens (M may be 0), each with `top` entries (1 .. SPLITK_MAX_TOP): entry
 * m * top + j is token m's j-th expert.  M * top <= SPLITK_MAX_DIM, the rows that
 * a grouped product takes.  Every tensor is dense and row-major.  The int32
 * tensors are 4-byte aligned, the others 16-byte; outputs overlap nothing
 * (exceptions are named).  Checks come before any device work, in the order
 * shape, dtype, NULL, alignment, overlap, values.  The calls take no workspace,
 * may be captured, and give the same bits for the same call every time. */

/* The router's choice: each token's `top` largest logits and their shares.
 *   logits   device, [M,G] of `dtype` (SPLITK_F32, _F16, _BF16), top <= G <=
 *            SPLITK_MAX_GROUPS; -inf masks an expert
 *   experts  device, int32 [M,top]: falling logits, the lowest index first among
 *            equal ones; -1 where a token has fewer experts above -inf
 *   shares   device, F32 [M,top]: exp(logit) / sum exp(logit), the sum over all
 *            G (chosen_only = 0) or over the token's experts (1); 0 for a -1
 * A NaN counts as larger than any number (and its experts are valid ones); a row
 * with a NaN or +inf among the logits that are summed has NaN shares. */
int moe_route(const void *logits, int32_t *experts, float *shares, int64_t M,
              int64_t G, int64_t top, int chosen_only, int dtype, void *stream);

/* The logits' gradient:
 *   dlogits[m,i] = p[i] * (sum_{j: experts[m,j] = i} dshares[m,j] - c),
 *   c = sum_j p[experts[m,j]] * dshares[m,j]
 * with p the row's softmax (chosen_only: over the token's experts, 0 elsewhere).
 *   logits, experts  as moe_route had and gave them; an entry outside [0,G) is
 *                    passed over, and an expert that is there twice counts twice
 *   dshares          device, F32 [M,top]
 *   dlogits          device, [M,G] of `dtype`, fully overwritten */
int moe_route_grad(const void *logits, const int32_t *experts,
                   const float *dshares, void *dlogits, int64_t M, int64_t G,
                   int64_t top, int chosen_only, int dtype, void *stream);

/* Entries sorted by expert, equal experts in the entries' order:
 *   experts  device, int32 [M,top]; an entry outside [0,G) goes nowhere
 *   offsets  device, int32 [G+1]: run g of a grouped product; offsets[0] = 0
 *   slots    device, int32 [M,top]: the entry's row, -1 for one that goes nowhere
 *   source   device, int32 [M*top] or NULL: the row's entry, -1 from offsets[G] on
 * With M = 0 the offsets are zeros. */
int moe_sort(const int32_t *experts, int32_t *offsets, int32_t *slots,
             int32_t *source, int64_t M, int64_t top, int64_t G, void *stream);

/* moe_sort, and the tokens' rows with it: rows[slots[m,j]] = x[m].
 *   x     device, [M,K] of `dtype`, K a positive multiple of 8
 *   rows  device, [M*top,K]; rows from offsets[G] on are left as they are
 * The gradient of x: moe_combine of the rows' gradients, without shares. */
int moe_dispatch(const int32_t *experts, const void *x, int32_t *offsets,
                 int32_t *slots, int32_t *source, void *rows, int64_t M,
                 int64_t top, int64_t G, int64_t K, int dtype, void *stream);

/* The same for rows in 8 bits with their scales: q [M,K] and scales
 * [M,ceil(K/128)] to rows [M*top,K] and row_scales [M*top,ceil(K/128)]; K a
 * positive multiple of 16. */
int moe_dispatch_fp8(const int32_t *experts, const void *q, const float *scales,
                     int32_t *offsets, int32_t *slots, int32_t *source,
                     void *rows, float *row_scales, int64_t M, int64_t top,
                     int64_t G, int64_t K, void *stream);

/* Rows back to their tokens, weighted:
 *   out[m] = sum_j shares[m,j] * rows[slots[m,j]]   in F32, j rising, rounded once
 *   rows    device, [M*top,K] of `dtype`, K a positive multiple of 8
 *   slots   device, int32 [M,top]; an entry outside [0,M*top) adds nothing
 *   shares  device, F32 [M,top], or NULL for ones
 *   out     device, [M,K] of out_dtype */
int moe_combine(const void *rows, const int32_t *slots, const float *shares,
                void *out, int64_t M, int64_t top, int64_t K, int dtype,
                int out_dtype, void *stream);

/* The gradients of moe_combine's rows and shares:
 *   drows[slots[m,j]] = shares[m,j] * dout[m]
 *   dshares[m,j]      = sum_k dout[m,k] * rows[slots[m,j],k]   (0 for a slot that
 *                       is none)
 *   dout     device, [M,K] of `dtype`
 *   rows     device, [M*top,K] of `dtype`; read for dshares alone (else may be NULL)
 *   drows    device, [M*top,K] of `dtype` or NULL; rows that no slot names are
 *            left as they are; may be exactly `rows` (in place)
 *   dshares  device, F32 [M,top] or NULL; one of the two is asked for (else
 *            SPLITK_ERR_NULL)
 * No two slots name the same row (moe_sort's never do). */
int moe_combine_grad(const void *dout, const void *rows, const int32_t *slots,
                     const float *shares, void *drows, float *dshares,
                     int64_t M, int64_t top, int64_t K, int dtype, void *stream);

/* ---- Layer norm
 *
 * Rows [M,K] (M may be 0), K a positive multiple of 8, M and K <= SPLITK_MAX_DIM,
 * element type SPLITK_F32, _F16 or _BF16; pointers 16-byte aligned.  The checks
 * and the rest as above; grad calls take a workspace, checked after the overlaps
 * (SPLITK_ERR_WORKSPACE). */

/* Residual addition and layer norm:
 *   h = x + residual, rounded to `dtype` (h = x without a residual)
 *   y = (h - mean) * rstd * weight + bias,  rstd = 1 / sqrt(mean_k (h - mean)^2 + eps)
 *   x, residual   device, [M,K]; residual may be NULL
 *   weight, bias  device, [K]; bias may be NULL
 *   sum           device, [M,K] or NULL: receives h; may be exactly x or residual
 *   y             device, [M,K], rounded once from F32
 *   mean, rstd    device, F32 [M] or NULL: what layernorm_grad takes
 * Finite rows of any size have their norm, also where the sum or the squares leave
 * F32's range; a row that holds a NaN or an infinity is NaN.  eps >= 0 (else
 * SPLITK_ERR_CONFIG); with eps = 0 a row of equal values is 0 / 0, and the rstd of
 * one whose deviations are below 2^-128 is infinite. */
int layernorm(const void *x, const void *residual, const void *weight,
              const void *bias, void *sum, void *y, float *mean, float *rstd,
              int64_t M, int64_t K, float eps, int dtype, void *stream);

/* Bytes of device workspace layernorm_grad needs; 0 for a rejected shape. */
size_t layernorm_grad_workspace_bytes(int64_t M, int64_t K);

/* Its gradients, with n = (h - mean) * rstd and g = dy * weight:
 *   dx      = rstd * (g - mean_k g - n * mean_k (g n)) + dsum
 *   dweight = sum_m dy * n,  dbias = sum_m dy
 *   dy          device, [M,K]
 *   h           device, [M,K]: the norm's input (`sum`, or x without a residual)
 *   mean, rstd  device, F32 [M], from layernorm (n is that of the rounded mean;
 *               rstd below 2^127)
 *   dsum        device, [M,K] or NULL: the gradient that reaches h besides
 *   dx          device, [M,K], rounded once: the gradient of x and of the
 *               residual; may be exactly dy or dsum
 *   dweight     device, F32 [K], fully overwritten (zeros with M = 0)
 *   dbias       device, F32 [K] or NULL, as dweight
 *   workspace   device, >= layernorm_grad_workspace_bytes(), needs no contents;
 *               calls that may run at the same time need one each */
int layernorm_grad(const void *dy, const void *h, const void *weight,
                   const float *mean, const float *rstd, const void *dsum,
                   void *dx, float *dweight, float *dbias, void *workspace,
                   size_t workspace_bytes, int64_t M, int64_t K, int dtype,
                   void *stream);

/* ---- The norm of all gradients
 *
 * `count` (0 .. SPLITK_MAX_TENSORS) dense tensors, given as host arrays that are
 * read before the call returns:
 *   grads   device pointers, 16-byte aligned; NULL where the size is 0
 *   sizes   values of each, 0 .. SPLITK_MAX_TENSOR_VALUES, any number
 *   dtypes  SPLITK_F32, _F16 or _BF16 of each
 *   norm    device, one F32 (4-byte aligned): sqrt of the sum of all squares
 *   workspace  device, >= grad_norm_workspace_bytes(), 16-byte aligned, needs no
 *              contents; calls that may run at the same time need one each
 * Finite gradients of any size have their norm (infinite where F32 does not hold
 * it).  A captured call keeps the tensors' addresses in its graph nodes.  Checks
 * come before any device work, in the order sizes, dtype, NULL, alignment, overlap,
 * workspace, max_norm; the same call gives the same bits every time. */
size_t grad_norm_workspace_bytes(void);
int grad_norm(const void *const *grads, const int64_t *sizes, const int *dtypes,
              int64_t count, float *norm, void *workspace,
              size_t workspace_bytes, void *stream);

/* The norm as above (of the gradients before scaling), and
 *   out[i] = grads[i] * min(1, max_norm / norm)   rounded once
 *   out  device pointers of the same sizes and types, or NULL for grads (in
 *        place; so may any single out[i]); no other overlap, and no tensor twice
 * With a NaN gradient every value becomes NaN, with an infinite one 0 (infinities
 * NaN).  Finite gradients are scaled to max_norm also where F32 does not hold their
 * norm (`norm` is infinite then).  max_norm finite and >= 0, else SPLITK_ERR_CONFIG. */
int grad_clip(void *const *grads, void *const *out, const int64_t *sizes,
              const int *dtypes, int64_t count, float max_norm, float *norm,
              void *workspace, size_t workspace_bytes, void *stream);

/* Reads and clears the device status word on the current device,
 * synchronising `stream` first.  Returns SPLITK_OK, SPLITK_ERR_DEVICE_TIMEOUT
 * (since the last call a kernel's bounded wait ran out, or a launch met a tile
 * configuration it cannot run; that launch's outputs are not valid) or
 * SPLITK_ERR_CUDA. */
int splitk_get_device_status(void *stream);

/* What the most recent SPLITK_ERR_CUDA on the calling host thread came from:
 * the failing call and CUDA's name and description of its error.  The string
 * is owned by the library and stays valid until the thread's next failure. */
const char *splitk_last_error(void);

/* A short, static description of a status code. */
const char *splitk_status_string(int status);

/* Tile-shape override for tuning: every later tensor-core launch uses tile
 * width `bn` (64, 128 or 256; must divide N, else the automatic choice is
 * kept), `chunks` thread blocks per split along K (1, 2, 4 or 8; fewer when
 * the shared memory of that many does not fit) and `kblocks_per_stage`
 * 64-wide k-blocks per pipeline stage (1, 2 or 4; more than 1 only when K and
 * k_per_split are multiples of 64).  Zero keeps the automatic choice for that
 * item.  Process-wide; not thread-safe against concurrent launches.  Returns
 * SPLITK_OK or SPLITK_ERR_CONFIG. */
int splitk_set_tile_override(int bn, int chunks, int kblocks_per_stage);

/* The same for gemm_fp8_bt and the grouped products: every later launch takes
 * tiles of `columns` columns (32, 64, 128 or 256, a pair of thread blocks;
 * gemm_grouped_dw has 128 and 256 and keeps its own choice for less) and
 * `splits` thread blocks along K (1, 2, 4 or 8; fewer where a split would have
 * less than two k-blocks, and one with 256 columns and for gemm_grouped_dw).
 * Zero keeps the automatic choice for that item.  Process-wide.  Returns
 * SPLITK_OK or SPLITK_ERR_CONFIG. */
int splitk_set_grouped_override(int columns, int splits);

/* Describes the launch gemm_bt would make, without launching: info[0..25] =
 * {path (0 tensor-core, 2 tensor-core 3xTF32 for F32), bn, chunks, chunk_len, stages,
 *  cluster_size (chunks, or splits * chunks), grid_x, grid_y, grid_z,
 *  dynamic_smem_bytes,
 *  fused_in_kernel (0/1), kernels_per_call, kblocks_per_stage,
 *  three_d_loads (0/1), split_sum (0 none, 2 inside the thread-block
 *  cluster; a fused call whose splits do not fit one resident cluster
 *  reports the two-kernel launch, fused_in_kernel 0), prefetchers (fused calls
 *  only: CTAs that fit beside a running launch and prefetch A and B into L2
 *  before the dependency wait), rows_first (1: grid x walks the 128-row tiles
 *  and grid y the column tiles, so grid_x and grid_y are swapped; chosen for
 *  launches of more than one wave with M < N whose B slab per split,
 *  N * k_per_split elements, is over 32 MB), tile_m (rows of A per thread
 *  block: 128, or 256 for BN 256 plans with one block per tile, no cluster
 *  chosen when it saves waves; grid_x or grid_y
 *  then counts 256-row tiles),
 *  compact (1: the call's tensor-core launch, captured into a graph, when it
 *  starts beside the launch before it or heads such a run, takes the compact
 *  layout: the same tiles, chunks and sums, a stage ring cut so that two or
 *  three thread blocks fit on an SM, the peers' shares received inside the
 *  ring; one-wave plans),
 *  compact_stages, compact_kblocks_per_stage, compact_dynamic_smem_bytes,
 *  compact_chunks_per_block (1, or two consecutive chunks of a split in one
 *  thread block, each in its own accumulator, added before the exchange:
 *  the same sums, since a split's chunks are added in pairs; or, more than
 *  chunks, every chunk of every split in one block of 128 x 128, no cluster and one block per SM, which
 *  adds each split's chunks and then the splits in the same order: fused
 *  16-bit calls whose splits are full and whose chunks tile them, where the
 *  compact plan would take more than half the SMs), compact_cluster_size,
 *  compact_grid_z,
 *  compact_bn (the compact plan's tile width, which may be wider than bn:
 *  the products of an output element do not depend on it)
 *  (0 when compact is 0).  The compact fields describe a call that starts
 *  beside the launch before it; the first call of a run launches without
 *  whole-K blocks, and the next call that takes them converts that launch
 *  and joins it}; `info` must hold 26 ints.
 * Returns a status as gemm_bt's validation would (pointers are not checked). */
int splitk_describe_launch(int64_t M, int64_t N, int64_t K, int64_t splits,
                           int64_t k_per_split, int dtype, int fused,
                           int *info);

/* Self-test of the bounded-wait machinery: launches one block that waits on a
 * barrier nothing ever completes, with a limit of `limit_ns` nanoseconds
 * (clamped to [1e3, 1e9]), synchronises `stream`, and returns what
 * splitk_get_device_status() then reads (SPLITK_ERR_DEVICE_TIMEOUT expected). */
int splitk_selftest_bounded_wait(int64_t limit_ns, void *stream);

/* Self-test of the tensor-core kernel's own time-out path: one fused launch
 * (arguments as for gemm_bt with fused = 1, no workspace; the shape must sum
 * its splits inside the launch, else SPLITK_ERR_CONFIG) whose wait for the
 * final accumulator gives up at once: the warps that wait for it test it
 * once, before the MMA issuer has finished, as a wait that ran out would.  The
 * kernel then records the time-out, still sends and awaits every cluster
 * message, waits for the MMAs (normal limit) before it frees its tensor
 * memory, and finishes; `out` is not valid.  Synchronises `stream` and
 * returns what splitk_get_device_status() reads (SPLITK_ERR_DEVICE_TIMEOUT
 * expected).  At that wait every TMA load of the launch has landed, and the
 * waits after it keep their normal limits, so no copy is in flight when a
 * block exits. */
int splitk_selftest_kernel_timeout(const void *A, const void *B, float *out,
                                   int64_t M, int64_t N, int64_t K,
                                   int64_t splits, int64_t k_per_split,
                                   int dtype, void *stream);

/* What the library does with consecutive independent calls inside a graph
 * capture (see the top of this header), for every later call of the
 * process: 2 (the default) overlap them and group them into one launch
 * where they can be; 1 overlap them only (one launch per call); 0 neither
 * (every launch waits for the one before).  Launches already captured keep
 * what was decided for them.  Returns SPLITK_OK or SPLITK_ERR_CONFIG. */
int splitk_set_overlap(int mode);

/* What the calling host thread's most recent tensor-core launch did:
 * info[0..10] = {overlap (0: it waited for the previous grid before loading;
 * 1: it loaded before that grid finished and waited before its first store;
 * 2: it also stored before, waiting only before it finished), compact (its
 * ring was cut so that two or three of its thread blocks fit on an SM,
 * taken for such launches and for the first of a capture, when a one-wave
 * plan allows it), capturing (the stream was being captured), bn, chunks,
 * stages, kblocks_per_stage, dynamic_smem_bytes, chunks_per_block (1, or
 * two consecutive chunks of a split, each in its own accumulator and added
 * inside the block: the same sums; more than chunks: every chunk of every
 * split, no cluster), cluster_size, group (the calls
 * the launch computes so far: 1, or more where the call joined the launch
 * of the calls before it)}.  `info` must hold 11 ints.  Diagnostic;
 * returns SPLITK_OK or SPLITK_ERR_NULL. */
int splitk_last_launch(int *info);

#ifdef __cplusplus
}
#endif

#endif /* SPLITK_H */
