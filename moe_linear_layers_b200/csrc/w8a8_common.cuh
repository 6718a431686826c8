// Shared by the INT8 x INT8 (W8A8) kernels: the problem, the rescale and the gated activation.
#pragma once

#include "q4_common.cuh"

namespace w8 {

// The kernels start while the previous one on the stream still runs (programmatic dependent launch) and read what it may
// write only behind their wait; those are plain loads, since a read-only (.nc) load promises that the data does not change
// while the kernel lives.
struct Problem {
    const int8_t* xq;        // [m][k]
    const float* scale_a;    // [m]
    const int8_t* w0;        // [n][k]: the weights, or the gate's
    const float* scale_0;    // [n]
    const int8_t* w1;        // gated: up's
    const float* scale_1;
    const float* bias;       // [n] or NULL (plain only)
    void* y;                 // [m][n]
    int m, n, k;
    int out_bf16;
    int act;                 // gated: Q8_ACT_*
    int32_t* status;
};

// acc is exact; fp32 rounds it once (to 2^-24), then each factor once
__device__ __forceinline__ float rescale(int acc, float sw, float sa) { return __fmul_rn(__fmul_rn((float)acc, sw), sa); }

// v / (1 + e^-z).  __expf is within 2 + 1.173 |z| ulp and __fdividef within 2: for z above 0 the exponential's part is small
// against 1; at z = -20, where the result is 2e-9 of v, it is 25 ulp (1.5e-6 of the result, far below a bf16 step).  z so
// negative that e^-z leaves fdividef's range (above 2^126) gives 0, off by less than |v| * 2^-126.
__device__ __forceinline__ float logistic_times(float v, float z) { return __fdividef(v, 1.0f + __expf(-z)); }

__device__ __forceinline__ float gated(float g, float u, int act)
{
    // 2 sqrt(2/pi) = 1.5957691..., times 0.044715 = 0.0713548...
    const float z = act == Q8_ACT_SILU ? g : g * fmaf(0.0713548163f * g, g, 1.5957691216f);
    return logistic_times(g, z) * u;
}

}  // namespace w8
