// block_norm.h -- arguments of the block norms (host and device side).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace twell {

constexpr int BN_MAX_D = 8192;   // 1024 threads of 8 elements hold a row
constexpr int BN_BWD_THREADS = 256 * 768;  // threads of the backward pass

// A tensor whose element type is known at run time.
struct BnTensor {
    void *p;
    int bf16;
};

// Elements from one partial row to the next: whole pieces of 16 bytes.
__host__ __device__ inline int64_t bn_pitch(int d) { return (d + 3) & ~3; }

struct BnArgs {
    int T, d;
    int post;            // a norm after the block
    float eps, alpha;
    int gate_span;       // rows that share a gate row; 0 without a gate
    BnTensor res, y, gate, out, n;   // forward: out, n written; backward: out read as `res`
    BnTensor w_post, b_post, w_pre, b_pre;
    // backward
    BnTensor dout, dn, dres, dy, dgate;
    float *dw[4];        // dw_post, db_post, dw_pre, db_pre (or NULL)
    float *part;         // [6][groups][bn_pitch(d)]: the four vectors, then the gate rows cut at a group's first and last row
    int groups;          // row groups of the backward pass
    int rows;            // rows of a group
    int cuts;            // gate rows or group boundaries to look for cut gate rows at
};

hipError_t launch_block_norm(const BnArgs &a, bool layer, bool vec, hipStream_t s);
hipError_t launch_block_norm_backward(const BnArgs &a, bool layer, bool vec, hipStream_t s);
int block_norm_groups(int T, int d);  // row groups of the backward pass
int block_norm_rows(int T, int d);    // rows of each, none of them empty
int block_norm_most_groups(int T, int d);  // the most groups of any call with up to T rows

// Bytes of the partial rows of so many groups.
inline size_t block_norm_ws(int groups, int d) { return (size_t)6 * groups * bn_pitch(d) * sizeof(float); }

}  // namespace twell
