// adamw.h -- arguments of the multi-tensor AdamW step (host and device side).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace twell {

constexpr int AW_QBLOCK = 256;  // elements that share one scale of the 8-bit states
constexpr int AW_BATCH = 40;    // tensors per launch: their table travels in the kernel's arguments
constexpr int AW_THREADS = 256;
constexpr int AW_PASS = AW_THREADS * 8;  // elements a workgroup handles at once
constexpr int AW_PASSES = 4;             // passes of one workgroup, or 1 where that leaves CUs without one

enum : uint32_t { AW_P_BF16 = 1, AW_G_BF16 = 2, AW_VEC = 4 };

struct AwTensor {
    int64_t n;
    void *p;
    __bf16 *copy;  // or NULL
    const void *grad;
    void *m, *v;   // float or 8-bit codes
    float *m_scale, *v_scale;
    float decay;      // 1 - lr * weight decay
    uint32_t flags;
    uint32_t key;     // seed of this tensor's rounding noise
    int32_t chunk0;   // first workgroup
};

struct AwBatch {
    AwTensor t[AW_BATCH];
    int32_t count, passes;
    float beta1, omb1, beta2, omb2, eps;
    float size;  // lr / (1 - beta1^step)
    float root;  // 1 / sqrt(1 - beta2^step)
    const float *grad_scale;
};
static_assert(sizeof(AwBatch) <= 4096, "kernel arguments");

struct AwUnpack {
    struct {
        int64_t n;
        const uint8_t *m, *v;
        const float *m_scale, *v_scale;
        float *m_values, *v_values;
        int32_t chunk0;
        uint32_t vec;
    } t[AW_BATCH];
    int32_t count, passes;
};
static_assert(sizeof(AwUnpack) <= 4096, "kernel arguments");

hipError_t launch_adamw(const AwBatch &b, bool coded, int chunks, hipStream_t s);
hipError_t launch_adamw_unpack(const AwUnpack &b, int chunks, hipStream_t s);

}  // namespace twell
