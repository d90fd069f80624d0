// checks.h -- host-side argument checks shared by the C-ABI files.
#pragma once

#include "twell.h"

#include <hip/hip_runtime.h>

namespace {

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int elem_size(int32_t vdtype) { return vdtype == TWELL_BF16 ? 2 : 4; }

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
