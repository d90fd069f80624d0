// checks.h -- host-side argument checks shared by the C-ABI files.
#pragma once

#include "twell.h"

#include <hip/hip_runtime.h>

namespace {

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int elem_size(int32_t vdtype) { return vdtype == TWELL_BF16 ? 2 : 4; }

inline bool aligned_to(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Rows of a call: row numbers and roundings of them stay below 2^31.
constexpr int32_t MOST_ROWS = 1 << 30;

inline bool known_dtype(int32_t dt) { return dt == TWELL_F32 || dt == TWELL_BF16; }

inline int check_mat(const void *p)
{
    if (!p)
        return TWELL_E_NULL;
    return aligned16(p) ? TWELL_OK : TWELL_E_ALIGN;
}

inline int hip_status(hipError_t e) { return e == hipSuccess ? TWELL_OK : TWELL_E_HIP; }

#define TWELL_TRY(expr)                  \
    do {                                 \
        const int _st = (expr);          \
        if (_st != TWELL_OK)             \
            return _st;                  \
    } while (0)

// A vector of elements of size es: NULL and alignment.
inline int check_vec(const void *p, size_t es)
{
    if (!p)
        return TWELL_E_NULL;
    return aligned_to(p, es) ? TWELL_OK : TWELL_E_ALIGN;
}

// Whether na bytes at a and nb bytes at b share any.
inline bool overlap(const void *a, int64_t na, const void *b, int64_t nb)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return na > 0 && nb > 0 && x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

inline size_t up256(size_t b) { return (b + 255) & ~(size_t)255; }

// The workspace argument against a layout's size.
inline int check_ws(const void *workspace, size_t workspace_bytes, size_t need)
{
    if (need == 0)
        return TWELL_OK;
    if (!workspace || workspace_bytes < need)
        return TWELL_E_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
        return TWELL_E_ALIGN;
    return TWELL_OK;
}

}  // namespace
