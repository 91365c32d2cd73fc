// splitk_checks.h -- what the entry points check their arguments with.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "splitk.h"

namespace splitk {

constexpr int kFp8Block = 128;

inline int elem_bytes(int dtype)
{
    switch (dtype) {
    case SPLITK_F32: return 4;
    case SPLITK_F16: return 2;
    case SPLITK_BF16: return 2;
    default: return 0;
    }
}

struct Range {
    uintptr_t lo, hi;   // [lo, hi)
};

// (An empty range overlaps nothing.)
inline bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi && a.lo < a.hi && b.lo < b.hi; }

inline Range range_of(const void *p, uint64_t bytes)
{
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return Range{lo, lo + static_cast<uintptr_t>(bytes)};
}

inline int cuda_status(cudaError_t e) { return e == cudaSuccess ? SPLITK_OK : SPLITK_ERR_CUDA; }

struct Extent {
    const void *p;
    uint64_t bytes;
    uintptr_t align = 16;
};

// NULL and alignment of every pointer (a tensor without elements may be NULL),
// then each output against the inputs and the other outputs.  `in_place` (may
// be -1): the one output that may be exactly one of the first `in_place_of`
// inputs (same address and extent).
inline int validate_extents(const Extent *in, int n_in, const Extent *out, int n_out, int in_place = -1, int in_place_of = 0)
{
    for (int i = 0; i < n_in; ++i)
        if (!in[i].p && in[i].bytes) return SPLITK_ERR_NULL;
    for (int i = 0; i < n_out; ++i)
        if (!out[i].p && out[i].bytes) return SPLITK_ERR_NULL;
    for (int i = 0; i < n_in; ++i)
        if (reinterpret_cast<uintptr_t>(in[i].p) % in[i].align) return SPLITK_ERR_ALIGN;
    for (int i = 0; i < n_out; ++i)
        if (reinterpret_cast<uintptr_t>(out[i].p) % out[i].align) return SPLITK_ERR_ALIGN;
    for (int o = 0; o < n_out; ++o) {
        const Range r = range_of(out[o].p, out[o].bytes);
        for (int i = 0; i < n_in; ++i)
            if (overlap(r, range_of(in[i].p, in[i].bytes)) &&
                !(o == in_place && i < in_place_of && in[i].p == out[o].p && in[i].bytes == out[o].bytes))
                return SPLITK_ERR_ALIAS;
        for (int i = 0; i < o; ++i)
            if (overlap(r, range_of(out[i].p, out[i].bytes))) return SPLITK_ERR_ALIAS;
    }
    return SPLITK_OK;
}

inline int64_t blocks_of(int64_t n) { return (n + kFp8Block - 1) / kFp8Block; }

}  // namespace splitk
