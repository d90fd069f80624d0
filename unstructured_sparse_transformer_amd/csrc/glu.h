// glu.h -- arguments of the dense gated product (host and device side).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "dense_gemm.h"

namespace twell {

enum GluAct { GLU_RELU = 0, GLU_SILU = 1, GLU_GELU = 2, GLU_GELU_TANH = 3 };

constexpr int GLU_FEW = 64;  // rows up to which the forward pass streams the weights

struct GluFwd {
    int T, d, F, act;
    DgTiles tiles;
    const void *x, *wg, *wu;
    void *h, *g, *u;  // g, u may be NULL
    float *part;      // [splits][g | u][T][F] partial sums
    int splits;       // of K, when the tiles alone leave CUs idle
};

struct MulPlan {
    int tile, splits;  // of a product: which of the tiles, and into how many parts K is split
    bool operator==(const MulPlan &o) const { return tile == o.tile && splits == o.splits; }
};

// The backward pass's workspace (dg and du first, then the splits' parts), and
// what it is laid out for.
struct GluWs {
    size_t part_dx, part_dw, bytes;
    MulPlan dx, dw;
    bool together;  // both products in one launch, with one tile
    bool dx_first;  // dx's workgroups first in it
};
GluWs glu_backward_ws(int T, int d, int F, int vdtype);

struct GluBwd {
    int T, d, F, act;
    const void *x, *wg, *wu, *g, *u, *dh;
    void *dx, *dwg, *dwu;  // NULL: not wanted
    void *dgu;             // the workspace: [T to a multiple of 64] rows of glu_pitch(F), a row's dg, then its du
    GluWs ws;
};

// Elements from one row of dgu to the next.  64 more than it holds: rows that
// are a power of two apart meet few of the memory channels when a tile reads
// the same columns of 256 of them (dx at the 2B-like layer: 425 us with the
// gap, 437 us without).
__host__ __device__ inline int64_t glu_pitch(int F) { return 2 * (int64_t)F + 64; }

size_t glu_forward_ws(int T, int d, int F, int vdtype);  // bytes
// The most bytes of any call with up to T rows.
size_t glu_forward_most_ws(int T, int d, int F, int vdtype);
size_t glu_backward_most_ws(int T, int d, int F, int vdtype);

hipError_t launch_glu(int vdtype, const GluFwd &a, hipStream_t s);
hipError_t launch_glu_backward(int vdtype, const GluBwd &a, hipStream_t s);

}  // namespace twell
