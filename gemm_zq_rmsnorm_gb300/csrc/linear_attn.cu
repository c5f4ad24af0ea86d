// linear_attn.cu -- linear attention with a decay for each head: the step of
// one token per sequence.  (Not the delta rule of MIInfer's recurrent layers, README,
// "Status", whose state has the same sizes.)
//
// S <- exp(g) S + k v^T,  o = scale * S^T q, for every value head h with the key
// head h / (Hv / Hk).
//
// A CTA owns 64 columns of one head's state, in registers: thread (r, c) holds
// rows r, r + 16, ... of the four columns 4 c, so that a row of the slice is two
// lines of memory.  The token's decay, key and value update the values where they
// are, and the products with the query are added up over the rows by shuffles and
// once through shared memory, in an order that the sizes alone give.
//
// HBM bound: every state is read and written once, and not read again before the
// next token, so it passes through L2 as streaming data.  What decides is how much of
// it an SM has on its way: four CTAs an SM (64 registers a thread, 128 KB of state)
// reach 57.7 us for 61 sequences of 48 heads of 128 x 128, 6.7 TB/s (0.98 of the measured
// copy rate); five with 48 registers 60.8, eight with slices of 32 columns 63.9, two
// with slices of 128 66.8.  One sequence 2.2 us: one round of loads.
#include "zq_async.cuh"
#include "zq_internal.cuh"
#include "zq_mixer.cuh"

namespace zq {
namespace {

constexpr int kStepThreads = 256;
constexpr int SL = 64;   // columns of a slice

template <int DK>
__global__ void __launch_bounds__(kStepThreads, 4) linear_attn_step_kernel(const __grid_constant__ LinearAttnArgs a, int Dv)
{
    constexpr int C = SL / 4;            // threads of a row
    constexpr int R = kStepThreads / C;  // rows of one pass
    constexpr int N = DK / R;            // rows of a thread
    __shared__ float4 part[kStepThreads / 32][C];
    pdl_wait();   // the projection's rows and the state come from earlier kernels
    pdl_launch_dependents();
    const int c = threadIdx.x % C, r = threadIdx.x / C, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int slices = Dv / SL;
    const int col0 = (int)(blockIdx.x % slices) * SL, item = blockIdx.x / slices;
    const int h = item % a.Hv, hk = h / (a.Hv / a.Hk);
    const long long b = item / a.Hv;
    const int slot = a.slots[b];
    const float g = a.g ? a.g[b * a.g_stride + h] : 0.0f;
    const float *q = a.q + b * a.q_stride + (long long)hk * DK + r;
    const float *k = a.k + b * a.k_stride + (long long)hk * DK + r;
    const float4 v = *reinterpret_cast<const float4 *>(a.v + b * a.v_stride + (long long)h * Dv + col0 + 4 * c);
    float kr[N], qr[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        kr[i] = k[i * R];
        qr[i] = q[i * R];
    }
    const bool kept = slot >= 0 && slot < a.n;
    float *sp = a.state + (((long long)slot * a.Hv + h) * DK + r) * Dv + col0 + 4 * c;
    float4 s[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
        s[i] = kept ? __ldcs(reinterpret_cast<const float4 *>(sp + (long long)i * R * Dv)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const float decay = expf(g);
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        s[i].x = __fmaf_rn(s[i].x, decay, kr[i] * v.x);
        s[i].y = __fmaf_rn(s[i].y, decay, kr[i] * v.y);
        s[i].z = __fmaf_rn(s[i].z, decay, kr[i] * v.z);
        s[i].w = __fmaf_rn(s[i].w, decay, kr[i] * v.w);
        o.x = __fmaf_rn(qr[i], s[i].x, o.x);
        o.y = __fmaf_rn(qr[i], s[i].y, o.y);
        o.z = __fmaf_rn(qr[i], s[i].z, o.z);
        o.w = __fmaf_rn(qr[i], s[i].w, o.w);
    }
    if (kept)
#pragma unroll
        for (int i = 0; i < N; ++i) __stcs(reinterpret_cast<float4 *>(sp + (long long)i * R * Dv), s[i]);
#pragma unroll
    for (int off = C; off < 32; off <<= 1) {
        o.x += __shfl_xor_sync(0xffffffffu, o.x, off);
        o.y += __shfl_xor_sync(0xffffffffu, o.y, off);
        o.z += __shfl_xor_sync(0xffffffffu, o.z, off);
        o.w += __shfl_xor_sync(0xffffffffu, o.w, off);
    }
    if (lane < C) part[warp][c] = o;
    __syncthreads();
    if (threadIdx.x < SL) {
        const float *p = reinterpret_cast<const float *>(part) + threadIdx.x;
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kStepThreads / 32; ++w) sum += p[w * SL];
        a.out[b * a.out_stride + (long long)h * Dv + col0 + threadIdx.x] = a.scale * sum;
    }
}

}  // namespace

cudaError_t launch_linear_attn_step(const LinearAttnArgs &a, int Dk, int Dv, cudaStream_t st)
{
    const dim3 grid((unsigned)((long long)a.B * a.Hv * (Dv / SL)));
    return launch_pdl(Dk == 64 ? linear_attn_step_kernel<64> : linear_attn_step_kernel<128>, grid, dim3(kStepThreads), 0, st, a, Dv);
}

}  // namespace zq
