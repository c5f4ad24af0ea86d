// gated_norm.cu -- what follows a block's mixer: RMSNorm of every head times
// the gate, packed to Q8_1 for the output projection (MIInfer README, "Status":
// the heads' RMS norms in one launch; ZINC docs "ROCm backend": activations
// packed to Q8 in the kernel that makes them).
//
// A head row of D values belongs to D / 8 lanes with eight neighbouring values each,
// so four lanes have a Q8_1 block: its largest value and the sum of its codes are two
// shuffles.  (With four values a lane what a block costs once weighed twice as much:
// 4096 rows of 48 heads of 128 to codes took 61.8 us.)
//
// HBM bound when there are many: 8 bytes a value read, 1.125 (codes) or 4 (fp32)
// written.  4096 rows of 48 x 128: codes 38.9 us (5.9 TB/s, 87 % of the copy rate), fp32
// 43.6 (6.9 TB/s: the written rows stay in L2); one row 1.5 and 61 2.1, a load's way.
#include "zq_async.cuh"
#include "zq_internal.cuh"
#include "zq_mixer.cuh"
#include "zq_q8_1_pack.cuh"

namespace zq {
namespace {

constexpr int kThreads = 128;

// kSteps: row groups that a warp has on their way at once.
template <int D, int kSteps>
__global__ void __launch_bounds__(kThreads) gated_norm_kernel(const __grid_constant__ GatedNormArgs a)
{
    constexpr int L = D / 8, R = 32 / L;   // lanes of a row, rows of a warp
    pdl_wait();   // x and the gate come from earlier kernels
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, col = 8 * (lane % L);
    const unsigned rows = (unsigned)a.B * (unsigned)a.H;
    const unsigned first = ((blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * kSteps) * R + lane / L;
    auto load8 = [](const float *p, float (&x)[8]) {
        const float4 u = reinterpret_cast<const float4 *>(p)[0], v = reinterpret_cast<const float4 *>(p)[1];
        x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w;
        x[4] = v.x, x[5] = v.y, x[6] = v.z, x[7] = v.w;
    };
    float y[kSteps][8], gt[kSteps][8], gm[8];
    long long b[kSteps];
    int at[kSteps];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        const unsigned row = min(first + i * R, rows - 1), token = row / (unsigned)a.H;
        b[i] = token;
        at[i] = (int)(row - token * (unsigned)a.H) * D + col;
        load8(a.x + b[i] * a.x_stride + at[i], y[i]);
        if (a.gate) load8(a.gate + b[i] * a.gate_stride + at[i], gt[i]);
    }
    if (a.gamma) load8(a.gamma + col, gm);
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        const bool live = first + i * R < rows;
        if (a.gamma) {
            float ss = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = __fmaf_rn(y[i][e], y[i][e], ss);
#pragma unroll
            for (int off = L / 2; off >= 1; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
            const float r = rms_scale(ss, D, a.eps);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[i][e] = y[i][e] * r * gm[e];
        }
        if (a.gate) gate_values(y[i], gt[i], a.act);
        if (a.out && live) {
            float4 *o = reinterpret_cast<float4 *>(a.out + b[i] * a.out_stride + at[i]);
            o[0] = make_float4(y[i][0], y[i][1], y[i][2], y[i][3]);
            o[1] = make_float4(y[i][4], y[i][5], y[i][6], y[i][7]);
        }
        if (a.q8.qs) {
            uint32_t code[2];
            __half d, s;
            q8_1_pack_lanes<8>(y[i], code, d, s);
            if (live) {
                const long long o = b[i] * a.H * D + at[i];
                *reinterpret_cast<uint2 *>(a.q8.qs + o) = make_uint2(code[0], code[1]);
                if ((lane & 3) == 0) {
                    a.q8.d[o / 32] = __half_as_ushort(d);
                    a.q8.s[o / 32] = __half_as_ushort(s);
                }
            }
        }
    }
}

template <int D, int kSteps>
cudaError_t launch_steps(const GatedNormArgs &a, cudaStream_t st)
{
    constexpr int per_cta = kThreads / 32 * kSteps * (32 / (D / 8));
    const long long rows = (long long)a.B * a.H;
    return launch_pdl(gated_norm_kernel<D, kSteps>, dim3((unsigned)((rows + per_cta - 1) / per_cta)), dim3(kThreads), 0, st, a);
}

template <int D>
cudaError_t launch_one(const GatedNormArgs &a, cudaStream_t st)
{
    // Two row groups a warp pay when many warps follow one another and pack codes, whose
    // arithmetic then runs beside the second group's loads (one / two, us, codes of 128:
    // 4096 x 48 42.4 / 38.9, 1000 x 48 12.9 / 12.0; 400 x 48 5.1 / 5.3, 61 x 48 2.1 / 2.8).
    // fp32 rows gain nothing (4096 x 48 43.6 / 44.3).
    const long long values = (long long)a.B * a.H * D;
    return a.q8.qs && values >= 4000000 ? launch_steps<D, 2>(a, st) : launch_steps<D, 1>(a, st);
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
