// Host-side pieces that the C ABI's translation units of the language-model operators share:
// workspace regions, strides, overlaps, launch sizes and the status of a launch.  Internal.
#pragma once

#include <stdint.h>

#include "ss_check.h"
#include "ss_internal.h"
#include "ss_scan.h"

namespace {

constexpr size_t kBad = static_cast<size_t>(-1);

inline int64_t elem_size(ss_dtype dtype) { return dtype == SS_F32 ? 4 : 2; }
inline bool known(ss_dtype dtype) { return dtype == SS_F32 || dtype == SS_BF16; }

inline ss_status done(hipError_t e)
{
    if (e == hipSuccess) return SS_OK;
    ssk::note_hip_error(e);
    return SS_ERR_HIP;
}

// Regions of a workspace, each from a 256-byte boundary.
struct Regions {
    int64_t at = 0;
    bool ok = true;
    int64_t add(int64_t count, int64_t size)
    {
        int64_t bytes, from;
        if (!ok || !mul(count, size, &bytes) || __builtin_add_overflow(at, int64_t(255), &from)) {
            ok = false;
            return 0;
        }
        if (bytes == 0) return at;  // not there
        from &= ~int64_t(255);
        if (__builtin_add_overflow(from, bytes, &at)) ok = false;
        return from;
    }
};

// Bytes that `rows` rows of `cols` elements, ld elements apart, span.
inline bool strided_bytes(int64_t rows, int64_t cols, int64_t ld, int64_t es, int64_t* bytes)
{
    int64_t n;
    return mul(rows - 1, ld, &n) && !__builtin_add_overflow(n, cols, &n) && mul(n, es, bytes);
}

// Whether two tensors of the same rows, row length and stride (bytes) share an element.
// Column slices of one tensor interleave without sharing any.
inline bool strided_overlap(const void* p, const void* q, int64_t bytes, int64_t row, int64_t stride)
{
    if (!overlap(span(p, bytes), span(q, bytes))) return false;
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    const int64_t off = static_cast<int64_t>((a < b ? b - a : a - b) % static_cast<uintptr_t>(stride));
    return off < row || off + row > stride;
}

// Whether a launch fits: HIP takes fewer than 2^32 threads along a grid's axis.
inline bool launch_fits(int64_t blocks, int64_t threads) { return blocks <= int64_t(UINT32_MAX) / threads; }

inline ss_status check_workspace(void* workspace, size_t given, int64_t need, const Range* others, size_t count)
{
    if (need == 0) return SS_OK;
    if (!workspace || given < static_cast<size_t>(need)) return SS_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return SS_ERR_INVALID_ARG;
    const Range w = span(workspace, need);
    for (size_t i = 0; i < count; ++i)
        if (overlap(w, others[i])) return SS_ERR_INVALID_ARG;
    return SS_OK;
}

inline bool any_overlap(const Range* outputs, size_t n_out, const Range* inputs, size_t n_in)
{
    for (size_t i = 0; i < n_out; ++i) {
        for (size_t k = 0; k < n_in; ++k)
            if (overlap(outputs[i], inputs[k])) return true;
        for (size_t k = i + 1; k < n_out; ++k)
            if (overlap(outputs[i], outputs[k])) return true;
    }
    return false;
}

}  // namespace
