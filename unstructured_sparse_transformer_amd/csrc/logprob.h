// logprob.h -- arguments of the log probabilities from logits (host and device
// side).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace twell {

constexpr int LP_MOST_TOP = 64;  // alternatives of a row

struct LpSum;  // the sums of a part of a row

struct LpArgs {
    int T, V, k;
    int id64, bf16;
    float scale, scale2;  // of the logits; times log2(e)
    int64_t ld, ldd;      // elements between rows of logits, of dlogits
    const void *logits, *targets;
    // forward
    float *logp, *norm, *entropy, *top_logp;
    int32_t *top_idx;
    int segs, seg;        // segments of a row, and elements of one
    LpSum *part;          // [T][segs]
    uint64_t *keys;       // [T][segs][k]
    // backward
    const float *norm_in, *entropy_in, *dlogp, *dentropy;
    void *dlogits;
};

// Segments of a row, and the bytes of the workspace of a call and of any call with up to T rows.
void lp_segments(int T, int V, int bf16, int &segs, int &seg);
size_t lp_workspace(int T, int V, int bf16, int k);
size_t lp_most_workspace(int T, int V, int k);

hipError_t launch_logprob(const LpArgs &a, void *ws, hipStream_t s);
hipError_t launch_logprob_backward(const LpArgs &a, hipStream_t s);

}  // namespace twell
