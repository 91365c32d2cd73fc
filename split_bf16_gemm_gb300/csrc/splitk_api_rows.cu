// splitk_api_rows.cu -- the C ABI of routing, rows sorted by expert and back, layer
// norm and the gradient norm (declared in include/splitk.h).  As everywhere, the
// arguments are checked completely on the host before any CUDA call.

#include <algorithm>
#include <cmath>
#include <new>

#include "splitk.h"
#include "splitk_checks.h"
#include "splitk_internal.h"

namespace {

using splitk::blocks_of;
using splitk::cuda_status;
using splitk::elem_bytes;
using splitk::Extent;
using splitk::overlap;
using splitk::Range;
using splitk::range_of;
using splitk::validate_extents;

uint64_t bytes_of(int64_t n, int e) { return static_cast<uint64_t>(n) * static_cast<uint64_t>(e); }

// M tokens with `top` entries each, as many rows as the grouped products take.
bool entries_ok(int64_t M, int64_t top)
{
    return M >= 0 && M <= SPLITK_MAX_DIM && top > 0 && top <= SPLITK_MAX_TOP && M * top <= SPLITK_MAX_DIM;
}

bool groups_ok(int64_t G, int64_t top) { return G >= top && G <= SPLITK_MAX_GROUPS; }

bool length_ok(int64_t K, int64_t step) { return K > 0 && K <= SPLITK_MAX_DIM && K % step == 0; }

// moe_sort (no rows), moe_dispatch and moe_dispatch_fp8 (scales).
int dispatch(const int32_t *experts, const void *x, const float *scales, int32_t *offsets, int32_t *slots, int32_t *source,
             void *rows, float *row_scales, int64_t M, int64_t top, int64_t G, int64_t K, int e, bool with_rows, bool fp8,
             void *stream)
{
    const int64_t T = M * top, kb = fp8 ? blocks_of(K) : 0;
    Extent in[3] = {{experts, bytes_of(T, 4), 4}}, out[5] = {{offsets, bytes_of(G + 1, 4), 4}, {slots, bytes_of(T, 4), 4}};
    int n_in = 1, n_out = 2;
    if (source) out[n_out++] = {source, bytes_of(T, 4), 4};
    if (with_rows) {
        in[n_in++] = {x, bytes_of(M * K, e)};
        out[n_out++] = {rows, bytes_of(T * K, e)};
    }
    if (fp8) {
        in[n_in++] = {scales, bytes_of(M * kb, 4)};
        out[n_out++] = {row_scales, bytes_of(T * kb, 4)};
    }
    const int st = validate_extents(in, n_in, out, n_out);
    if (st != SPLITK_OK) return st;
    const splitk::DispatchProblem p = {experts, with_rows ? x : nullptr, scales, offsets, slots, source, rows, row_scales,
                                       M, top, G, with_rows ? K * e : 0, kb};
    return cuda_status(splitk::launch_dispatch(p, static_cast<cudaStream_t>(stream)));
}

// grad_norm and (clip) grad_clip.
int grad_norm_call(const void *const *grads, void *const *out, const int64_t *sizes, const int *dtypes, int64_t count,
                   float max_norm, float *norm, void *workspace, size_t workspace_bytes, bool clip, void *stream)
{
    if (count < 0 || count > SPLITK_MAX_TENSORS) return SPLITK_ERR_SHAPE;
    if (count && (!grads || !sizes || !dtypes)) return SPLITK_ERR_NULL;
    for (int64_t i = 0; i < count; ++i)
        if (sizes[i] < 0 || sizes[i] > SPLITK_MAX_TENSOR_VALUES) return SPLITK_ERR_SHAPE;
    for (int64_t i = 0; i < count; ++i)
        if (elem_bytes(dtypes[i]) == 0) return SPLITK_ERR_DTYPE;
    if (!norm || !workspace) return SPLITK_ERR_NULL;
    for (int64_t i = 0; i < count; ++i)
        if (sizes[i] && (!grads[i] || (clip && !out[i]))) return SPLITK_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(norm) % 4 || reinterpret_cast<uintptr_t>(workspace) % 16) return SPLITK_ERR_ALIGN;
    for (int64_t i = 0; i < count; ++i)
        if (reinterpret_cast<uintptr_t>(grads[i]) % 16 || (clip && reinterpret_cast<uintptr_t>(out[i]) % 16)) return SPLITK_ERR_ALIGN;
    // What is written, in order of address: disjoint, and met by no gradient but an
    // output's own.
    struct Written {
        Range r;
        int64_t of;   // tensor, or -1
    };
    const int64_t n = (clip ? count : 0) + 2;
    Written *const w = new (std::nothrow) Written[static_cast<size_t>(n)];
    if (!w) {
        splitk::note_message("host memory for the overlap check", 0);
        return SPLITK_ERR_CUDA;
    }
    const Range work = range_of(workspace, grad_norm_workspace_bytes()), scalar = range_of(norm, 4);
    int64_t m = 0;
    w[m++] = {work, -1};
    w[m++] = {scalar, -1};
    for (int64_t i = 0; clip && i < count; ++i)
        if (sizes[i]) w[m++] = {range_of(out[i], bytes_of(sizes[i], elem_bytes(dtypes[i]))), i};
    std::sort(w, w + m, [](const Written &a, const Written &b) { return a.r.lo < b.r.lo; });
    bool alias = false;
    for (int64_t i = 1; i < m; ++i) alias |= overlap(w[i - 1].r, w[i].r);
    for (int64_t i = 0; i < count && !alias; ++i) {
        if (!sizes[i]) continue;
        const Range r = range_of(grads[i], bytes_of(sizes[i], elem_bytes(dtypes[i])));
        // the first that ends behind the gradient's start (disjoint: sorted by end too)
        const Written *x = std::upper_bound(w, w + m, r.lo, [](uintptr_t lo, const Written &y) { return lo < y.r.hi; });
        for (; x != w + m && x->r.lo < r.hi; ++x) alias |= !(x->of == i && x->r.lo == r.lo);
    }
    delete[] w;
    if (alias) return SPLITK_ERR_ALIAS;
    if (workspace_bytes < grad_norm_workspace_bytes()) return SPLITK_ERR_WORKSPACE;
    if (clip && !(max_norm >= 0.f && std::isfinite(max_norm))) return SPLITK_ERR_CONFIG;
    const splitk::GradNormProblem p = {grads, clip ? out : nullptr, sizes, dtypes, count, max_norm, norm, workspace};
    return cuda_status(splitk::launch_grad_norm(p, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

int moe_route(const void *logits, int32_t *experts, float *shares, int64_t M, int64_t G, int64_t top, int chosen_only, int dtype,
              void *stream)
{
    if (!entries_ok(M, top) || !groups_ok(G, top)) return SPLITK_ERR_SHAPE;
    const int e = elem_bytes(dtype);
    if (e == 0) return SPLITK_ERR_DTYPE;
    const Extent in[1] = {{logits, bytes_of(M * G, e)}};
    const Extent out[2] = {{experts, bytes_of(M * top, 4), 4}, {shares, bytes_of(M * top, 4)}};
    const int st = validate_extents(in, 1, out, 2);
    if (st != SPLITK_OK) return st;
    if (chosen_only != 0 && chosen_only != 1) return SPLITK_ERR_CONFIG;
    if (M == 0) return SPLITK_OK;
    return cuda_status(splitk::launch_route({logits, experts, shares, nullptr, M, G, top, chosen_only, dtype},
                                            static_cast<cudaStream_t>(stream)));
}

int moe_route_grad(const void *logits, const int32_t *experts, const float *dshares, void *dlogits, int64_t M, int64_t G,
                   int64_t top, int chosen_only, int dtype, void *stream)
{
    if (!entries_ok(M, top) || !groups_ok(G, top)) return SPLITK_ERR_SHAPE;
    const int e = elem_bytes(dtype);
    if (e == 0) return SPLITK_ERR_DTYPE;
    const Extent in[3] = {{logits, bytes_of(M * G, e)}, {experts, bytes_of(M * top, 4), 4}, {dshares, bytes_of(M * top, 4)}};
    const Extent out[1] = {{dlogits, bytes_of(M * G, e)}};
    const int st = validate_extents(in, 3, out, 1);
    if (st != SPLITK_OK) return st;
    if (chosen_only != 0 && chosen_only != 1) return SPLITK_ERR_CONFIG;
    if (M == 0) return SPLITK_OK;
    return cuda_status(splitk::launch_route({logits, const_cast<int32_t *>(experts), const_cast<float *>(dshares), dlogits, M, G, top,
                                             chosen_only, dtype},
                                            static_cast<cudaStream_t>(stream)));
}

int moe_sort(const int32_t *experts, int32_t *offsets, int32_t *slots, int32_t *source, int64_t M, int64_t top, int64_t G,
             void *stream)
{
    if (!entries_ok(M, top) || G <= 0 || G > SPLITK_MAX_GROUPS) return SPLITK_ERR_SHAPE;
    return dispatch(experts, nullptr, nullptr, offsets, slots, source, nullptr, nullptr, M, top, G, 0, 0, false, false, stream);
}

int moe_dispatch(const int32_t *experts, const void *x, int32_t *offsets, int32_t *slots, int32_t *source, void *rows, int64_t M,
                 int64_t top, int64_t G, int64_t K, int dtype, void *stream)
{
    if (!entries_ok(M, top) || G <= 0 || G > SPLITK_MAX_GROUPS || !length_ok(K, 8)) return SPLITK_ERR_SHAPE;
    const int e = elem_bytes(dtype);
    if (e == 0) return SPLITK_ERR_DTYPE;
    return dispatch(experts, x, nullptr, offsets, slots, source, rows, nullptr, M, top, G, K, e, true, false, stream);
}

int moe_dispatch_fp8(const int32_t *experts, const void *q, const float *scales, int32_t *offsets, int32_t *slots, int32_t *source,
                     void *rows, float *row_scales, int64_t M, int64_t top, int64_t G, int64_t K, void *stream)
{
    if (!entries_ok(M, top) || G <= 0 || G > SPLITK_MAX_GROUPS || !length_ok(K, 16)) return SPLITK_ERR_SHAPE;
    return dispatch(experts, q, scales, offsets, slots, source, rows, row_scales, M, top, G, K, 1, true, true, stream);
}

int moe_combine(const void *rows, const int32_t *slots, const float *shares, void *out, int64_t M, int64_t top, int64_t K, int dtype,
                int out_dtype, void *stream)
{
    if (!entries_ok(M, top) || !length_ok(K, 8)) return SPLITK_ERR_SHAPE;
    const int e = elem_bytes(dtype), oe = elem_bytes(out_dtype);
    if (e == 0 || oe == 0) return SPLITK_ERR_DTYPE;
    Extent in[3] = {{rows, bytes_of(M * top * K, e)}, {slots, bytes_of(M * top, 4), 4}};
    int n_in = 2;
    if (shares) in[n_in++] = {shares, bytes_of(M * top, 4)};
    const Extent o[1] = {{out, bytes_of(M * K, oe)}};
    const int st = validate_extents(in, n_in, o, 1);
    if (st != SPLITK_OK) return st;
    if (M == 0) return SPLITK_OK;
    return cuda_status(splitk::launch_combine({rows, nullptr, slots, shares, out, nullptr, nullptr, M, top, K, dtype, out_dtype},
                                              static_cast<cudaStream_t>(stream)));
}

int moe_combine_grad(const void *dout, const void *rows, const int32_t *slots, const float *shares, void *drows, float *dshares,
                     int64_t M, int64_t top, int64_t K, int dtype, void *stream)
{
    if (!entries_ok(M, top) || !length_ok(K, 8)) return SPLITK_ERR_SHAPE;
    const int e = elem_bytes(dtype);
    if (e == 0) return SPLITK_ERR_DTYPE;
    if (M && !drows && !dshares) return SPLITK_ERR_NULL;
    Extent in[4], out[2];
    int n_in = 0, n_out = 0, in_place = -1;
    if (dshares || rows) in[n_in++] = {rows, bytes_of(M * top * K, e)};
    const int rows_first = n_in;                       // which drows may be
    in[n_in++] = {dout, bytes_of(M * K, e)};
    in[n_in++] = {slots, bytes_of(M * top, 4), 4};
    if (shares) in[n_in++] = {shares, bytes_of(M * top, 4)};
    if (drows) {
        in_place = n_out;
        out[n_out++] = {drows, bytes_of(M * top * K, e)};
    }
    if (dshares) out[n_out++] = {dshares, bytes_of(M * top, 4)};
    const int st = validate_extents(in, n_in, out, n_out, in_place, rows_first);
    if (st != SPLITK_OK) return st;
    if (M == 0) return SPLITK_OK;
    return cuda_status(splitk::launch_combine({dshares ? rows : nullptr, dout, slots, shares, nullptr, drows, dshares, M, top, K, dtype, dtype},
                                              static_cast<cudaStream_t>(stream)));
}

int layernorm(const void *x, const void *residual, const void *weight, const void *bias, void *sum, void *y, float *mean, float *rstd,
              int64_t M, int64_t K, float eps, int dtype, void *stream)
{
    if (M < 0 || M > SPLITK_MAX_DIM || !length_ok(K, 8)) return SPLITK_ERR_SHAPE;
    const int e = elem_bytes(dtype);
    if (e == 0) return SPLITK_ERR_DTYPE;
    const uint64_t bytes = bytes_of(M * K, e);
    Extent in[4] = {{x, bytes}}, out[4] = {{y, bytes}};
    int n_in = 1, n_out = 1, in_place = -1;
    if (residual) in[n_in++] = {residual, bytes};
    const int rows = n_in;                             // x and the residual, which `sum` may be
    in[n_in++] = {weight, bytes_of(K, e)};
    if (bias) in[n_in++] = {bias, bytes_of(K, e)};
    if (sum) {
        in_place = n_out;
        out[n_out++] = {sum, bytes};
    }
    if (mean) out[n_out++] = {mean, bytes_of(M, 4)};
    if (rstd) out[n_out++] = {rstd, bytes_of(M, 4)};
    const int st = validate_extents(in, n_in, out, n_out, in_place, rows);
    if (st != SPLITK_OK) return st;
    if (!(eps >= 0.f)) return SPLITK_ERR_CONFIG;
    if (M == 0) return SPLITK_OK;
    return cuda_status(splitk::launch_layernorm({x, residual, weight, bias, sum, y, mean, rstd, M, K, eps, dtype},
                                                static_cast<cudaStream_t>(stream)));
}

size_t layernorm_grad_workspace_bytes(int64_t M, int64_t K)
{
    if (M < 0 || M > SPLITK_MAX_DIM || !length_ok(K, 8)) return 0;
    return static_cast<size_t>(splitk::layernorm_grad_parts(M, K)) * 2 * static_cast<size_t>(K) * sizeof(float);
}

int layernorm_grad(const void *dy, const void *h, const void *weight, const float *mean, const float *rstd, const void *dsum, void *dx,
                   float *dweight, float *dbias, void *workspace, size_t workspace_bytes, int64_t M, int64_t K, int dtype,
                   void *stream)
{
    if (M < 0 || M > SPLITK_MAX_DIM || !length_ok(K, 8)) return SPLITK_ERR_SHAPE;
    const int e = elem_bytes(dtype);
    if (e == 0) return SPLITK_ERR_DTYPE;
    const uint64_t bytes = bytes_of(M * K, e);
    const size_t need = layernorm_grad_workspace_bytes(M, K);
    Extent in[6] = {{dy, bytes}}, out[4] = {{dx, bytes}, {dweight, bytes_of(K, 4)}};
    int n_in = 1, n_out = 2;
    if (dsum) in[n_in++] = {dsum, bytes};
    const int rows = n_in;                             // the gradients, either of which dx may be
    in[n_in++] = {h, bytes};
    in[n_in++] = {weight, bytes_of(K, e)};
    in[n_in++] = {mean, bytes_of(M, 4)};
    in[n_in++] = {rstd, bytes_of(M, 4)};
    if (dbias) out[n_out++] = {dbias, bytes_of(K, 4)};
    out[n_out++] = {workspace, need};
    const int st = validate_extents(in, n_in, out, n_out, 0, rows);
    if (st != SPLITK_OK) return st;
    if (workspace_bytes < need) return SPLITK_ERR_WORKSPACE;
    return cuda_status(splitk::launch_layernorm_grad(
        {dy, h, weight, dsum, mean, rstd, dx, dweight, dbias, static_cast<float *>(workspace), M, K, dtype}, static_cast<cudaStream_t>(stream)));
}

size_t grad_norm_workspace_bytes(void) { return (splitk::kGradNormParts + 1) * 8 + splitk::kGradNormParts * 4; }

int grad_norm(const void *const *grads, const int64_t *sizes, const int *dtypes, int64_t count, float *norm, void *workspace,
              size_t workspace_bytes, void *stream)
{
    return grad_norm_call(grads, nullptr, sizes, dtypes, count, 0.f, norm, workspace, workspace_bytes, false, stream);
}

int grad_clip(void *const *grads, void *const *out, const int64_t *sizes, const int *dtypes, int64_t count, float max_norm, float *norm,
              void *workspace, size_t workspace_bytes, void *stream)
{
    return grad_norm_call(grads, out ? out : grads, sizes, dtypes, count, max_norm, norm, workspace, workspace_bytes, true, stream);
}

}  // extern "C"
