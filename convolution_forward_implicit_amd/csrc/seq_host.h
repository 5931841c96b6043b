// What the host sides of the sequence operators share: checks of the callers'
// tensors and workspaces, limits of a launch.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>

#include "../../include/convfwd.h"
#include "status.h"

namespace convfwd {

constexpr int64_t kMaxDim = int64_t(1) << 30;
constexpr double kMaxBytes = 9.0e18;
constexpr double kMaxThreads = 4294967296.0;     // a launch has fewer threads than this

inline bool one_launch(double workgroups, int threads) { return workgroups * threads < kMaxThreads; }

inline conv_status_t launched()
{
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? CONV_OK : fail(CONV_ERR_HIP, "kernel launch failed: %s", hipGetErrorString(e));
}

// A tensor as `rows` runs of `width` elements, `ld` apart.
struct Rows {
    const char *name;
    const void *p;
    int64_t rows, width, ld, esz;
};

inline bool share_memory(const Rows &a, const Rows &b)
{
    if (!a.p || !b.p || a.rows <= 0 || b.rows <= 0 || a.width <= 0 || b.width <= 0) return false;
    const int64_t a0 = (int64_t)(uintptr_t)a.p, b0 = (int64_t)(uintptr_t)b.p;
    const int64_t a1 = a0 + ((a.rows - 1) * a.ld + a.width) * a.esz, b1 = b0 + ((b.rows - 1) * b.ld + b.width) * b.esz;
    if (a1 <= b0 || b1 <= a0) return false;
    const int64_t step = a.ld * a.esz;
    if (step != b.ld * b.esz) return true;
    // equal strides: column ranges of one matrix, disjoint iff the runs are, modulo the stride
    int64_t d = (b0 - a0) % step;
    if (d < 0) d += step;
    return d < a.width * a.esz || d + b.width * b.esz > step;
}

// Every output against every input and the outputs before it.
inline conv_status_t check_overlap(const Rows *out, int nout, const Rows *in, int nin)
{
    for (int i = 0; i < nout; ++i) {
        for (int j = 0; j < nin; ++j)
            if (share_memory(out[i], in[j])) return fail(CONV_ERR_INVALID_ARG, "%s overlaps %s", out[i].name, in[j].name);
        for (int j = 0; j < i; ++j)
            if (share_memory(out[i], out[j]))
                return fail(CONV_ERR_INVALID_ARG, "%s overlaps %s", out[i].name, out[j].name);
    }
    return CONV_OK;
}

// Alignment of every tensor to its elements, and token strides that hold a row.
inline conv_status_t check_rows(const Rows *t, int n)
{
    for (int i = 0; i < n; ++i) {
        if (t[i].p && (uintptr_t)t[i].p % t[i].esz)
            return fail(CONV_ERR_INVALID_ARG, "%s is not aligned to its elements", t[i].name);
        if (t[i].ld < t[i].width)
            return fail(CONV_ERR_INVALID_ARG, "%s: %lld elements from token to token, a row has %lld", t[i].name,
                        (long long)t[i].ld, (long long)t[i].width);
        // a chunk of 64 tokens is addressed by 32-bit byte offsets
        if ((double)t[i].ld * t[i].esz * std::max<int64_t>(1, t[i].rows) > kMaxBytes ||
            (t[i].rows > 1 && t[i].ld * t[i].esz >= int64_t(1) << 25))
            return fail(CONV_ERR_UNSUPPORTED, "%s: %lld elements from token to token", t[i].name, (long long)t[i].ld);
    }
    return CONV_OK;
}

inline bool vector_rows(const Rows &t) { return !t.p || ((uintptr_t)t.p % 16 == 0 && t.ld * t.esz % 16 == 0); }

inline int64_t or_packed(int64_t ld, int64_t width) { return ld == 0 ? width : ld; }

// What a kernel gets as a tensor's stride.  One row has no next one, and its
// stride may be any: a small one keeps the 32-bit offsets of the rows that a
// tile has none of past the tensor's end (64 rows of 2^27 bytes wrap round).
inline int64_t stride(const Rows &t) { return t.rows > 1 ? t.ld : std::min<int64_t>(t.ld, 65536); }

inline conv_status_t check_workspace(const void *ws, int64_t bytes, int64_t need)
{
    if (need == 0) return CONV_OK;
    if (!ws) return fail(CONV_ERR_INVALID_ARG, "workspace is NULL");
    if (bytes < need)
        return fail(CONV_ERR_INVALID_ARG, "workspace has %lld bytes, the plan needs %lld", (long long)bytes, (long long)need);
    if ((uintptr_t)ws % 16) return fail(CONV_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
    return CONV_OK;
}

}  // namespace convfwd
