// residual_norm.cu -- the edge between two blocks in one pass: the norm after a
// block, its gate and residual scale, the residual addition, and the norm before
// the next block packed to Q8_1 (ZINC docs "ROCm backend", "Build and verify":
// normalisation and Q8 packing in one per-token kernel).
//
// One CTA for a token (or for several in turn).  Four lanes share a 32-value block,
// eight neighbouring values each, so that a warp reads 1 KB of consecutive bytes; the
// whole row stays in registers between its two norms, and every value of x and y is
// read once.  The norm before the next block adds its squares up in the library's
// fixed order (the block's fma chain runs through its four lanes), so the codes are
// those of zq_rmsnorm_q8_1 on x_out, byte for byte.
//
// HBM bound: 8 bytes a value read (12 with a gate), 4 + 1.125 written.  4096 x 5120
// with a norm after the block and a gate 62 us, 5.8 TB/s (0.85 of the measured copy
// rate; issue slots 54 % busy: about 60 instructions a value for the gate, the two
// norms and the packing); 61 tokens 3.7 us, one 3.6 (2.5 at 1024): two barriers and a
// chain of dependent loads.
#include <algorithm>
#include <atomic>

#include "zq_async.cuh"
#include "zq_internal.cuh"
#include "zq_kv.cuh"
#include "zq_mixer.cuh"
#include "zq_q8_1_pack.cuh"

namespace zq {
namespace {

constexpr int kMaxK = 32768, kMaxRowsK = 8192;

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

// Sum of squares of the row from its block sums p (zeros behind the last, up to
// 256), in the library's order: 256 slots, then the pairwise tree.  The tree's levels
// 128, 64 and 32 are taken from the slots themselves; every warp does it for itself,
// so that one barrier is enough.
__device__ __forceinline__ float row_sumsq(const float *p, int nblk)
{
    const int lane = threadIdx.x & 31;
    float slot[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) slot[i] = p[lane + 32 * i];
    for (int b0 = 256; b0 < nblk; b0 += 256)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (b0 + lane + 32 * i < nblk) slot[i] = __fadd_rn(slot[i], p[b0 + lane + 32 * i]);
#pragma unroll
    for (int off = 4; off >= 1; off >>= 1)
#pragma unroll
        for (int i = 0; i < off; ++i) slot[i] = __fadd_rn(slot[i], slot[i + off]);
    float v = slot[0];
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) v = __fadd_rn(v, __shfl_down_sync(0xffffffffu, v, off));
    return __shfl_sync(0xffffffffu, v, 0);
}

// p_b of the block that four lanes share: the fma chain over its squares in index
// order, through the lanes one after another.  Every lane goes on at every step from
// what the lane before it had; at the fourth step lane 3 has the chain of all.
__device__ __forceinline__ float block_chain(const float (&x)[8])
{
    float part = 0.0f;
#pragma unroll
    for (int step = 0; step < 4; ++step) {
        if (step) part = __shfl_up_sync(0xffffffffu, part, 1, 4);
#pragma unroll
        for (int e = 0; e < 8; ++e) part = __fmaf_rn(x[e], x[e], part);
    }
    return part;
}

// One token, its rows from `px`, `py`, `pg` (global or shared memory), by the whole
// CTA.  post_s: 32 sums, pre_s: block sums (zeros behind the last); taken: called once the rows are in registers,
// after the first barrier behind it.
template <int P, typename Taken>
__device__ __forceinline__ void one_token(const ResidualNormArgs &a, long long b, const float *px, const float *py,
                                          const float *pg, float *post_s, float *pre_s, Taken taken)
{
    const int K = a.K, nblk = K >> 5, nthr = blockDim.x;
    float x[P][8], y[P][8];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int c = 8 * (threadIdx.x + i * nthr);
        if (c < K) {
            load8(py + c, y[i]);
            load8(px + c, x[i]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[i][e] = y[i][e] = 0.0f;
        }
    }
    if (a.gamma_post) {
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < P; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = __fmaf_rn(y[i][e], y[i][e], ss);
        ss = warp_sum(ss);
        const int lane = threadIdx.x & 31;
        if (lane == 0) post_s[threadIdx.x >> 5] = ss;
        __syncthreads();
        const float r = rms_scale(warp_sum(lane < (nthr >> 5) ? post_s[lane] : 0.0f), K, a.eps);
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
                load8(pg + c, gt);
                gate_values(y[i], gt, a.act);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) x[i][e] = __fmaf_rn(a.scale, y[i][e], x[i][e]);
            store8(a.x_out + b * a.x_out_stride + c, x[i]);
        }
    }
    float r = 1.0f;
    const bool normed = a.gamma && (a.out || a.q8.qs);
    if (normed) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const float part = block_chain(x[i]);
            const int blk = (threadIdx.x + i * nthr) >> 2;
            if ((threadIdx.x & 3) == 3 && blk < nblk) pre_s[blk] = part;
        }
        __syncthreads();
        taken();
        r = rms_scale(row_sumsq(pre_s, nblk), K, a.eps);
    } else if (Taken::needed) {
        __syncthreads();
        taken();
    }
    if (!a.out && !a.q8.qs) return;
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

// A CTA for a token, its rows straight from memory: the shortest way for one.
struct NotTaken {
    static constexpr bool needed = false;
    __device__ __forceinline__ void operator()() const {}
};
template <int P, int THREADS>
__global__ void __launch_bounds__(THREADS) residual_norm_kernel(const __grid_constant__ ResidualNormArgs a)
{
    __shared__ float post_s[32], pre_s[kMaxK / 32];
    for (int i = (a.K >> 5) + threadIdx.x; i < 256; i += blockDim.x) pre_s[i] = 0.0f;
    pdl_wait();   // x, y and the gate come from earlier kernels
    pdl_launch_dependents();
    const long long b = blockIdx.x;
    one_token<P>(a, b, a.x + b * a.x_stride, a.y + b * a.y_stride, a.gate + b * a.gate_stride, post_s, pre_s, NotTaken{});
}

// Many tokens: as many CTAs as run at the same time take them in turn, and the next
// token's rows come to shared memory (bulk copies) while the CTA works on this one.
struct NextRows {
    static constexpr bool needed = true;
    const ResidualNormArgs &a;
    long long b;
    float *rows;
    uint64_t *bar;
    __device__ __forceinline__ void operator()() const
    {
        if (threadIdx.x || b >= a.B) return;
        const uint32_t bytes = a.K * 4;
        mbar_arrive_expect_tx(bar, a.gate ? 3 * bytes : 2 * bytes);
        bulk_g2s(rows, a.y + b * a.y_stride, bytes, bar);
        bulk_g2s(rows + a.K, a.x + b * a.x_stride, bytes, bar);
        if (a.gate) bulk_g2s(rows + 2 * a.K, a.gate + b * a.gate_stride, bytes, bar);
    }
};
template <int P, int THREADS>
__global__ void __launch_bounds__(THREADS) residual_norm_rows_kernel(const __grid_constant__ ResidualNormArgs a,
                                                                     unsigned int *status)
{
    extern __shared__ __align__(128) float rows[];   // y, x and gate
    __shared__ float post_s[2][32], pre_s[2][kMaxRowsK / 32];   // of tokens in turn
    __shared__ uint64_t bar;
    for (int i = (a.K >> 5) + threadIdx.x; i < 256; i += blockDim.x) pre_s[0][i] = pre_s[1][i] = 0.0f;
    if (threadIdx.x == 0) {
        mbar_init(&bar, 1);
        fence_mbar_init();
    }
    __syncthreads();
    pdl_wait();
    pdl_launch_dependents();
    NextRows{a, blockIdx.x, rows, &bar}();
    int turn = 0;
    for (long long b = blockIdx.x; b < a.B; b += gridDim.x, ++turn) {
        // after a wait that ran out (the status word says so) the CTA goes on with what is there
        if (!mbar_wait(&bar, turn & 1, status)) mbar_wait_for(&bar, turn & 1, nullptr, 1000000ull);
        one_token<P>(a, b, rows + a.K, rows, rows + 2 * a.K, post_s[turn & 1], pre_s[turn & 1],
                     NextRows{a, b + gridDim.x, rows, &bar});
    }
}

template <int P, int THREADS, int REGS>
cudaError_t launch_rows(const ResidualNormArgs &a, int threads, cudaStream_t st)
{
    static std::atomic<bool> ready[64];
    auto *kernel = residual_norm_rows_kernel<P, THREADS>;
    constexpr int kShared = 227 * 1024, kStatic = 6 * 1024;   // of an SM, of a CTA beside its rows
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (!ready[dev & 63].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kShared - kStatic);
        if (e != cudaSuccess) return e;
        ready[dev & 63].store(true, std::memory_order_release);
    }
    const int smem = a.K * 4 * (a.gate ? 3 : 2);
    const int per_sm = std::max(1, std::min({kShared / (smem + kStatic), 2048 / threads, 65536 / (REGS * threads)}));
    const long long ctas = (long long)per_sm * num_sms();
    return launch_pdl(kernel, dim3((unsigned)(a.B < ctas ? a.B : ctas)), dim3(threads), smem, st, a, device_status_word());
}

}  // namespace

cudaError_t launch_residual_norm(const ResidualNormArgs &a, cudaStream_t st)
{
    const int eights = a.K / 8;
    auto threads = [&](int passes) { return ((eights + passes - 1) / passes + 31) / 32 * 32; };
    // Rows in turn against a CTA each, us (inputs larger than L2, norm after the block).  With a gate, whose row is one more
    // to wait for: 1000 x 5120 23.2 and 22.5, 1750 x 5120 32.3 and 32.9, 4096 x 5120 62.3 and 69.7, 1250 x 8192 38.3 and
    // 38.7; but short rows leave such a CTA little to do beside its waits: 16000 x 1024 55.5 and 53.6, 40000 x 256 51.5 and
    // 42.6.  Without one: 2000 x 5120 32.3 and 30.1, 3000 x 5120 42.9 and 41.7, 4096 x 5120 53.8 and 54.1, 3000 x 8192 64.8
    // and 66.1; of up to 4096, where a CTA each has one piece a thread, 3000 x 4096 34.8 and 40.5, 10000 x 1024 28.2 and
    // 28.8, 40000 x 256 41.3 and 42.1.
    const long long values = (long long)a.B * a.K;
    const bool in_turn = a.gate ? a.K > 1024 && values >= 9000000 : values >= (a.K > 4096 ? 18000000 : 10000000);
    if (a.K <= kMaxRowsK && in_turn) return launch_rows<2, 512, 64>(a, threads(2), st);
    auto direct = [&](auto *kernel, int passes) { return launch_pdl(kernel, dim3((unsigned)a.B), dim3(threads(passes)), 0, st, a); };
    // Two pieces a thread let two CTAs run on an SM where they are wide enough for one to fill it: with one piece and with
    // two, us (inputs larger than L2, norm after the block), 400 rows of 5120 9.9 and 9.2, 1000 18.9 and 18.7, of 8192 400
    // rows 16.1 and 14.2, 1000 34.9 and 27.5; 512 of 5120 are 11.8 and 12.7 (they just fill one piece's waves), 61 3.7 and
    // 4.1, 400 of 1024 3.0 and 3.5.
    if (eights <= 1024)
        return a.B > 2 * num_sms() && a.K > 4096 ? direct(residual_norm_kernel<2, 512>, 2) : direct(residual_norm_kernel<1, 1024>, 1);
    if (eights <= 2048) return direct(residual_norm_kernel<2, 1024>, 2);
    return direct(residual_norm_kernel<4, 1024>, 4);
}

}  // namespace zq
