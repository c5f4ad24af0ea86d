// gated_norm.cu -- what follows a block's mixer: RMSNorm of every head times
// the gate, packed to Q8_1 for the output projection (MIInfer README, "Status":
// the heads' RMS norms in one launch; ZINC docs "ROCm backend": activations
// packed to Q8 in the kernel that makes them).
//
// A head row of D values belongs to min(32, D / 4) lanes with four neighbouring
// values each (a second four, D / 2 further on, when D = 256), so eight lanes
// have a Q8_1 block: its largest value and code sum are three shuffles, and a
// warp's codes leave as one 128-byte row.
//
// HBM bound: 8 bytes a value read, 1.125 (codes) or 4 (fp32) written.
#include "zq_async.cuh"
#include "zq_internal.cuh"
#include "zq_mixer.cuh"
#include "zq_q8_1_pack.cuh"

namespace zq {
namespace {

constexpr int kThreads = 128;

template <int D>
__global__ void __launch_bounds__(kThreads) gated_norm_kernel(const __grid_constant__ GatedNormArgs a)
{
    constexpr int L = D / 4 < 32 ? D / 4 : 32;   // lanes of a row
    constexpr int V = D / (4 * L);               // float4 of a lane
    pdl_wait();   // x and the gate come from earlier kernels
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const long long rows = (long long)a.B * a.H;
    const long long row = ((long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * (32 / L) + lane / L;
    const bool live = row < rows;
    const long long at = live ? row : 0;
    const int b = (int)(at / a.H), h = (int)(at % a.H), col = 4 * (lane % L);
    const float *x = a.x + b * a.x_stride + h * D + col;
    float4 y[V], gt[V], gm[V];
#pragma unroll
    for (int i = 0; i < V; ++i) y[i] = *reinterpret_cast<const float4 *>(x + i * 128);
    if (a.gate)
#pragma unroll
        for (int i = 0; i < V; ++i)
            gt[i] = *reinterpret_cast<const float4 *>(a.gate + b * a.gate_stride + h * D + col + i * 128);
    if (a.gamma) {
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            gm[i] = *reinterpret_cast<const float4 *>(a.gamma + col + i * 128);
            ss = __fmaf_rn(y[i].x, y[i].x, ss);
            ss = __fmaf_rn(y[i].y, y[i].y, ss);
            ss = __fmaf_rn(y[i].z, y[i].z, ss);
            ss = __fmaf_rn(y[i].w, y[i].w, ss);
        }
#pragma unroll
        for (int off = L / 2; off >= 1; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
        const float r = rms_scale(ss, D, a.eps);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            y[i].x = y[i].x * r * gm[i].x;
            y[i].y = y[i].y * r * gm[i].y;
            y[i].z = y[i].z * r * gm[i].z;
            y[i].w = y[i].w * r * gm[i].w;
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        float e[4] = {y[i].x, y[i].y, y[i].z, y[i].w};
        if (a.gate) {
            const float g[4] = {gt[i].x, gt[i].y, gt[i].z, gt[i].w};
            gate_values(e, g, a.act);
        }
        if (a.out && live) *reinterpret_cast<float4 *>(a.out + b * a.out_stride + h * D + col + i * 128) = make_float4(e[0], e[1], e[2], e[3]);
        if (a.q8.qs) {
            const long long o = ((long long)b * a.H + h) * D + col + i * 128;
            uint32_t code[1];
            __half d, s;
            q8_1_pack_lanes<4>(e, code, d, s);
            if (live) {
                *reinterpret_cast<uint32_t *>(a.q8.qs + o) = code[0];
                if ((lane & 7) == 0) {
                    a.q8.d[o / 32] = __half_as_ushort(d);
                    a.q8.s[o / 32] = __half_as_ushort(s);
                }
            }
        }
    }
}

template <int D>
cudaError_t launch_one(const GatedNormArgs &a, cudaStream_t st)
{
    constexpr int per_cta = kThreads / 32 * (D / 4 < 32 ? 32 / (D / 4) : 1);
    const long long rows = (long long)a.B * a.H;
    return launch_pdl(gated_norm_kernel<D>, dim3((unsigned)((rows + per_cta - 1) / per_cta)), dim3(kThreads), 0, st, a);
}

}  // namespace

cudaError_t launch_gated_norm(const GatedNormArgs &a, int D, cudaStream_t st)
{
    switch (D) {
    case 64: return launch_one<64>(a, st);
    case 128: return launch_one<128>(a, st);
    default: return launch_one<256>(a, st);
    }
}

}  // namespace zq
