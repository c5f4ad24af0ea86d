// linear_attn.cu -- linear attention with a decay for each head: the step of
// one token per sequence, and prompts of ragged lengths (MIInfer README,
// "Status": recurrent layers whose state is [heads][128][128] and whose output
// projection is the Q5_K one).
//
// S_t = exp(g_t) S_{t-1} + k_t v_t^T,  o_t = scale * S_t^T q_t, for every value
// head h with the key head h / (Hv / Hk).
//
// A CTA owns SL columns of one head's state, in registers: thread (r, c) holds
// rows r, r + R, ... of the four columns 4 c.  A row of the slice is one
// coalesced access.  The token's decay, key and value update the values where
// they are, and the products with the query are added up over the rows by
// shuffles and once through shared memory.
#include "zq_async.cuh"
#include "zq_internal.cuh"
#include "zq_mixer.cuh"

namespace zq {
namespace {

constexpr int kStepThreads = 256;

// One sequence, head and slice of SL columns: the rows t0 .. t1.
template <int DK, int SL>
__device__ __forceinline__ void recurrence(const LinearAttnArgs &a, int h, int col0, int Dv, long long slot, bool from_zero,
                                           int t0, int t1)
{
    constexpr int C = SL / 4;                 // threads of a row
    constexpr int R = kStepThreads / C;       // rows of one pass
    constexpr int N = DK / R;                 // rows of a thread
    __shared__ float4 part[kStepThreads / 32][C];
    const int c = threadIdx.x % C, r = threadIdx.x / C, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool kept = slot >= 0;
    float *sp = a.state + ((slot * a.Hv + h) * DK + r) * Dv + col0 + 4 * c;
    float4 s[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
        s[i] = kept && !from_zero ? *reinterpret_cast<const float4 *>(sp + (long long)i * R * Dv)
                                  : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const int hk = h / (a.Hv / a.Hk);
    for (int t = t0; t < t1; ++t) {
        const float *q = a.q + t * a.q_stride + (long long)hk * DK + r;
        const float *k = a.k + t * a.k_stride + (long long)hk * DK + r;
        const float4 v = *reinterpret_cast<const float4 *>(a.v + t * a.v_stride + (long long)h * Dv + col0 + 4 * c);
        const float decay = a.g ? expf(a.g[t * a.g_stride + h]) : 1.0f;
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float kr = k[i * R], qr = q[i * R];
            s[i].x = __fmaf_rn(s[i].x, decay, kr * v.x);
            s[i].y = __fmaf_rn(s[i].y, decay, kr * v.y);
            s[i].z = __fmaf_rn(s[i].z, decay, kr * v.z);
            s[i].w = __fmaf_rn(s[i].w, decay, kr * v.w);
            o.x = __fmaf_rn(qr, s[i].x, o.x);
            o.y = __fmaf_rn(qr, s[i].y, o.y);
            o.z = __fmaf_rn(qr, s[i].z, o.z);
            o.w = __fmaf_rn(qr, s[i].w, o.w);
        }
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
            a.out[t * a.out_stride + (long long)h * Dv + col0 + threadIdx.x] = a.scale * sum;
        }
        if (t + 1 < t1) __syncthreads();
    }
    if (kept)
#pragma unroll
        for (int i = 0; i < N; ++i) *reinterpret_cast<float4 *>(sp + (long long)i * R * Dv) = s[i];
}

template <int DK, int SL>
__global__ void __launch_bounds__(kStepThreads) linear_attn_step_kernel(const __grid_constant__ LinearAttnArgs a, int Dv)
{
    pdl_wait();   // the projection's rows and the state come from earlier kernels
    pdl_launch_dependents();
    const int slices = Dv / SL;
    const int slice = blockIdx.x % slices, item = blockIdx.x / slices;
    const int h = item % a.Hv, b = item / a.Hv;
    const int slot = a.slots[b];
    const bool kept = slot >= 0 && slot < a.n;
    recurrence<DK, SL>(a, h, slice * SL, Dv, kept ? slot : -1, false, b, b + 1);
}

template <int DK, int SL>
cudaError_t launch_slices(const LinearAttnArgs &a, int Dv, cudaStream_t st)
{
    const long long ctas = (long long)a.B * a.Hv * (Dv / SL);
    return launch_pdl(linear_attn_step_kernel<DK, SL>, dim3((unsigned)ctas), dim3(kStepThreads), 0, st, a, Dv);
}

}  // namespace

cudaError_t launch_linear_attn_step(const LinearAttnArgs &a, int Dk, int Dv, cudaStream_t st)
{
    if (Dk == 64) return Dv == 64 ? launch_slices<64, 64>(a, Dv, st) : launch_slices<64, 128>(a, Dv, st);
    return Dv == 64 ? launch_slices<128, 64>(a, Dv, st) : launch_slices<128, 128>(a, Dv, st);
}

}  // namespace zq
