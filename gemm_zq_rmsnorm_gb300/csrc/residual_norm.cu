// residual_norm.cu -- the edge between two blocks in one pass: the norm after a
// block, its gate and residual scale, the residual addition, and the norm before
// the next block packed to Q8_1 (ZINC docs "ROCm backend", "Build and verify":
// normalisation and Q8 packing in one per-token kernel).
//
// One CTA per token.  Four lanes share a 32-value block, eight neighbouring
// values each, so that a warp reads 1 KB of consecutive bytes; the whole row
// stays in registers between its two norms, and every value of x and y is read
// once.  The norm before the next block adds its squares up in the library's
// fixed order (the block's fma chain runs through its four lanes), so the codes
// are those of zq_rmsnorm_q8_1 on x_out, byte for byte.
//
// HBM bound: 8 bytes a value read (12 with a gate), 4 + 1.125 written.
#include "zq_async.cuh"
#include "zq_internal.cuh"
#include "zq_mixer.cuh"
#include "zq_q8_1_pack.cuh"

namespace zq {
namespace {

constexpr int kMaxK = 32768;

__device__ __forceinline__ void load8(const float *p, float (&x)[8])
{
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

__device__ __forceinline__ void store8(float *p, const float (&x)[8])
{
    reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

// Sum of squares of the row from its block sums p[nblk], in the library's order:
// 256 slots, then the pairwise tree.  The tree's levels 128, 64 and 32 are taken
// from the slots themselves; every warp does it for itself, so that one barrier
// is enough.
__device__ __forceinline__ float row_sumsq(const float *p, int nblk)
{
    const int lane = threadIdx.x & 31;
    auto slot = [&](int t) {
        float s = 0.0f;
        for (int b = t; b < nblk; b += 256) s = __fadd_rn(s, p[b]);
        return s;
    };
    auto pair = [&](int t) { return __fadd_rn(slot(t), slot(t + 128)); };
    auto four = [&](int t) { return __fadd_rn(pair(t), pair(t + 64)); };
    float v = __fadd_rn(four(lane), four(lane + 32));
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) v = __fadd_rn(v, __shfl_down_sync(0xffffffffu, v, off));
    return __shfl_sync(0xffffffffu, v, 0);
}

// p_b of the block that four lanes share: the fma chain over its squares in
// index order, through the lanes one after another.
__device__ __forceinline__ float block_chain(const float (&x)[8])
{
    const int j = threadIdx.x & 3;
    float part = 0.0f;
#pragma unroll
    for (int step = 0; step < 4; ++step) {
        const float before = __shfl_up_sync(0xffffffffu, part, 1, 4);
        if (step == j) {
            part = step ? before : 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) part = __fmaf_rn(x[e], x[e], part);
        }
    }
    return part;   // in lane 3 of the four
}

template <int P, int THREADS>
__global__ void __launch_bounds__(THREADS) residual_norm_kernel(const __grid_constant__ ResidualNormArgs a)
{
    __shared__ float p_s[2][kMaxK / 32];
    pdl_wait();   // x, y and the gate come from earlier kernels
    pdl_launch_dependents();
    const long long b = blockIdx.x;
    const int K = a.K, nblk = K >> 5, nthr = blockDim.x;
    float x[P][8], y[P][8];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int c = 8 * (threadIdx.x + i * nthr);
        if (c < K) {
            load8(a.y + b * a.y_stride + c, y[i]);
            load8(a.x + b * a.x_stride + c, x[i]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[i][e] = y[i][e] = 0.0f;
        }
    }
    if (a.gamma_post) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const float part = block_chain(y[i]);
            const int blk = (threadIdx.x + i * nthr) >> 2;
            if ((threadIdx.x & 3) == 3 && blk < nblk) p_s[0][blk] = part;
        }
        __syncthreads();
        const float r = rms_scale(row_sumsq(p_s[0], nblk), K, a.eps);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int c = 8 * (threadIdx.x + i * nthr);
            if (c < K) {
                float gm[8];
                load8(a.gamma_post + c, gm);
#pragma unroll
                for (int e = 0; e < 8; ++e) y[i][e] = y[i][e] * r * gm[e];
            }
        }
    }
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int c = 8 * (threadIdx.x + i * nthr);
        if (c < K) {
            if (a.gate) {
                float gt[8];
                load8(a.gate + b * a.gate_stride + c, gt);
#pragma unroll
                for (int e = 0; e < 8; ++e) y[i][e] = gated(y[i][e], gt[e], a.act);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) x[i][e] = __fmaf_rn(a.scale, y[i][e], x[i][e]);
            store8(a.x_out + b * a.x_out_stride + c, x[i]);
        }
    }
    if (!a.out && !a.q8.qs) return;
    float r = 1.0f;
    if (a.gamma) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const float part = block_chain(x[i]);
            const int blk = (threadIdx.x + i * nthr) >> 2;
            if ((threadIdx.x & 3) == 3 && blk < nblk) p_s[1][blk] = part;
        }
        __syncthreads();
        r = rms_scale(row_sumsq(p_s[1], nblk), K, a.eps);
    }
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int c = 8 * (threadIdx.x + i * nthr);
        const bool live = c < K;
        if (live && a.gamma) {
            float gm[8];
            load8(a.gamma + c, gm);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[i][e] = __fmul_rn(__fmul_rn(x[i][e], r), gm[e]);
        }
        if (live && a.out) store8(a.out + b * a.out_stride + c, x[i]);
        if (a.q8.qs) {
            uint32_t code[2];
            __half d, s;
            q8_1_pack_lanes<8>(x[i], code, d, s);
            if (live) {
                *reinterpret_cast<uint2 *>(a.q8.qs + b * K + c) = make_uint2(code[0], code[1]);
                if ((threadIdx.x & 3) == 0) {
                    a.q8.d[b * nblk + (c >> 5)] = __half_as_ushort(d);
                    a.q8.s[b * nblk + (c >> 5)] = __half_as_ushort(s);
                }
            }
        }
    }
}

}  // namespace

cudaError_t launch_residual_norm(const ResidualNormArgs &a, cudaStream_t st)
{
    const int eights = a.K / 8;
    auto threads = [&](int passes) { return dim3((unsigned)(((eights + passes - 1) / passes + 31) / 32 * 32)); };
    const dim3 grid((unsigned)a.B);
    if (eights <= 1024) return launch_pdl(residual_norm_kernel<1, 1024>, grid, threads(1), 0, st, a);
    if (eights <= 2048) return launch_pdl(residual_norm_kernel<2, 1024>, grid, threads(2), 0, st, a);
    return launch_pdl(residual_norm_kernel<4, 1024>, grid, threads(4), 0, st, a);
}

}  // namespace zq
