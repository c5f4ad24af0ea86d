// zq_mixer.cuh -- launch descriptions of the recurrent mixer's and the block
// edges' operators, and the gate's activation.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "zq.h"

namespace zq {

struct LinearAttnArgs {
    const float *q, *k, *v;
    long long q_stride, k_stride, v_stride;
    int T, B, Hk, Hv;          // T: rows (of a step: B)
    const float *g;            // may be null (no decay)
    long long g_stride;
    const int32_t *starts;     // [B + 1] rows of each sequence (null for a step)
    float *state;              // [n][Hv][Dk][Dv]
    int n;
    const int32_t *slots;      // [B]
    const int32_t *fresh;      // [B] or null
    float scale;
    float *out;
    long long out_stride;
    // zq_debug_linear_attn_expiry: the waits' limit (0: kWaitLimitNs), and the chunk (1 or 2, 0: none) whose queries and keys,
    // or whose values, are never all there
    unsigned int wait_us;
    int withhold_rows, withhold_values;
};
cudaError_t launch_linear_attn_step(const LinearAttnArgs &a, int Dk, int Dv, cudaStream_t st);
size_t linear_attn_workspace(int T, int B, int Hv, int Dk, int Dv);
// the cut of a call into segments, for starts in host memory (zq_debug_linear_segments)
void linear_segments(const LinearAttnArgs &a, int Dv, int32_t *out);
cudaError_t launch_linear_attn(const LinearAttnArgs &a, int Dk, int Dv, void *workspace, cudaStream_t st);

struct GatedNormArgs {
    const float *x;
    long long x_stride;
    int B, H;
    const float *gamma;        // [D] or null
    float eps;
    const float *gate;         // may be null
    long long gate_stride;
    int act;
    float *out;                // may be null
    long long out_stride;
    zq_q8_1 q8;                // qs may be null
};
cudaError_t launch_gated_norm(const GatedNormArgs &a, int D, cudaStream_t st);

struct ResidualNormArgs {
    const float *x, *y;
    long long x_stride, y_stride;
    int B, K;
    const float *gamma_post;   // [K] or null
    const float *gate;         // may be null
    long long gate_stride;     // 0: one row for all tokens
    int act;
    float scale;
    float *x_out;
    long long x_out_stride;
    const float *gamma;        // [K] or null
    float eps;
    float *out;                // may be null
    long long out_stride;
    zq_q8_1 q8;                // qs may be null
};
cudaError_t launch_residual_norm(const ResidualNormArgs &a, cudaStream_t st);

// 1 / (1 + exp(-g)) to about 2^-21 of itself: exp(-g) as 2^(-g log2 e), the
// product's rounding error put back as a factor (2^hi alone would be off by
// 2^-24 |g|), and two approximate units instead of an IEEE division.
__device__ __forceinline__ float sigmoid32(float g)
{
    const float hi = __fmul_rn(g, -0x1.715476p+0f);
    const float lo = __fmaf_rn(g, -0x1.4ae0cp-26f, __fmaf_rn(g, -0x1.715476p+0f, -hi));
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(hi));
    // |hi| >= 128: the power is 0 or infinity already, and hi itself may be
    if (fabsf(hi) < 128.0f) e = __fmaf_rn(e * lo, 0x1.62e43p-1f, e);
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return r;
}

// values times their gates (the choice is the call's, made once for all of them)
template <int E>
__device__ __forceinline__ void gate_values(float (&x)[E], const float (&g)[E], int act)
{
    if (act == ZQ_GATE_LINEAR) {
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] *= g[e];
    } else if (act == ZQ_GATE_SIGMOID) {
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] *= sigmoid32(g[e]);
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] *= g[e] * sigmoid32(g[e]);
    }
}

}  // namespace zq
