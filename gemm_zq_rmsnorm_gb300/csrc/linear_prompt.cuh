// linear_prompt.cuh -- what the two kernels of linear attention over prompts
// share: the cut of sequences into segments, the parts of a value, and a chunk's
// factors.
//
// In chunks of 64 tokens the recurrence is matrix products: with G_t the sum of g
// from the chunk's first token to t,
//   o_t = scale (exp(G_t) S^T q_t + sum_{s <= t} exp(G_t - G_s) (q_t . k_s) v_s),
//   S'  = exp(G_C) S + sum_s exp(G_C - G_s) k_s v_s^T.
//
// Every product is as exact as an fp32 one: a row x is taken as 2^e (hi + lo), two
// binary16 parts of the row scaled to [1, 2), and a product is hi hi + hi lo + lo
// hi (2^-22 of what bounds it; sums fp32, a chunk's sums added to the state outside
// the tensor core, whose accumulator truncates).  Weights exp(G_t - G_s) and the
// rows' powers of two meet in the exponent: with u_s = e_k + e_v - G_s (G in base
// two) and M_t the largest u of s <= t, the weight in the product is 2^(u_s - M_t)
// <= 1 and 2^(M_t + G_t) goes to the row, so that a token counts exactly where no
// larger one of its past drowns it, and the future does not matter at all.  G and u
// are sums in units of 2^-40.
#pragma once

#include <limits.h>

#include <cuda.h>
#include <cuda_fp16.h>

#include "zq_async.cuh"
#include "zq_internal.cuh"
#include "zq_mixer.cuh"
#include "zq_mma.cuh"

namespace zq {

constexpr int kChunk = 64;         // tokens of a chunk

struct PromptArgs {
    LinearAttnArgs a;
    int Dv;
    int length, segments;      // tokens of a segment (a multiple of kChunk; 0: sequences are not cut), segments at most
    float *local;              // [segments][Hv][Dk][Dv]: a segment's own state, then the one it starts from
    long long *decay;          // [segments][Hv]: its G
    unsigned int *status;
};

// the rows of sequence b, within the call's rows whatever the starts say
__device__ __forceinline__ void sequence_rows(const LinearAttnArgs &a, int b, int &r0, int &r1)
{
    r0 = min(max(a.starts[b], 0), a.T);
    r1 = min(max(a.starts[b + 1], r0), a.T);
}
__device__ __forceinline__ int segments_of(const PromptArgs &p, int b)
{
    int r0, r1;
    sequence_rows(p.a, b, r0, r1);
    return max(1, (r1 - r0 + p.length - 1) / p.length);
}

struct Segment {
    int seq, seg, last, row0, row1;   // seq < 0: there is none
};

// Segment number `at` of the call, by one warp.
__device__ __forceinline__ Segment find_segment(const PromptArgs &p, int at)
{
    const LinearAttnArgs &a = p.a;
    const int lane = threadIdx.x & 31;
    Segment s{-1, 0, 1, 0, 0};
    if (p.length == 0) {
        s.seq = at;
    } else {
        int base = 0;
        for (int b0 = 0; b0 < a.B && s.seq < 0; b0 += 32) {
            const int cnt = b0 + lane < a.B ? segments_of(p, b0 + lane) : 0;
            int sum = cnt;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, sum, d);
                if (lane >= d) sum += o;
            }
            const unsigned who = __ballot_sync(0xffffffffu, at >= base + sum - cnt && at < base + sum);
            if (who) {
                const int l = __ffs(who) - 1;
                s.seq = b0 + l;
                s.seg = at - base - __shfl_sync(0xffffffffu, sum - cnt, l);
                s.last = s.seg + 1 == __shfl_sync(0xffffffffu, cnt, l);
            }
            base += __shfl_sync(0xffffffffu, sum, 31);
        }
    }
    if (s.seq >= 0) {
        int r0, r1;
        sequence_rows(a, s.seq, r0, r1);
        s.row0 = r0 + s.seg * p.length;
        s.row1 = s.last ? r1 : s.row0 + p.length;
    }
    return s;
}

// ---------------------------------------------------------------- parts of values
// two scaled values to their binary16 parts
__device__ __forceinline__ void split2(float x, float y, uint32_t &hi, uint32_t &lo)
{
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(y), "f"(x));
    const float2 h = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(lo) : "f"(y - h.y), "f"(x - h.x));
}

__device__ __forceinline__ float exp2_fast(float x)
{
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x));
    return e;
}

// exponent of a row's largest magnitude (its bits), such that the row over 2^e lies below 4
__device__ __forceinline__ int row_exponent(uint32_t bits)
{
    const int e = (int)(bits >> 23) - 127;
    return e < -126 ? -126 : e > 126 ? 126 : e;
}
__device__ __forceinline__ float pow2(int e) { return __int_as_float((127 + e) << 23); }   // -126 <= e <= 127

__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// ---------------------------------------------------------------- a chunk's factors
constexpr long long kOne = 1LL << 40;          // units of G and u
constexpr long long kNothing = -(1LL << 60);   // u of a row of zeros

struct Factors {
    float uh[kChunk], ul[kChunk], mh[kChunk], ml[kChunk];   // u and M: whole and broken part
    float f1[kChunk], f2[kChunk], w[kChunk];                // the rows' factors, the tokens' weights in the state
    float keep, add;                                        // what the state, and what the chunk's sums are multiplied by
    long long G;
};

// 2^(x / kOne + e), the broken part's power to 2^-22
__device__ __forceinline__ float exp2_units(long long x, int e)
{
    const long long whole = (x >> 40) + e;
    const int n = (int)(whole < -252 ? -252 : whole > 252 ? 252 : whole);   // 2^-252 and 2^252 as two factors: 0, infinity
    const float part = (float)((uint32_t)(x >> 8)) * 0x1p-32f;
    return exp2_fast(part) * pow2(n >> 1) * pow2(n - (n >> 1));
}

// x log2 e in units of 2^-40, to 2^-33 of itself and half a unit: the significand times 2^32 log2 e, shifted
__device__ __forceinline__ long long log2_units(float x)
{
    // beyond +-200 the power is 0 or infinity; NaN is marked elsewhere
    x = fminf(fmaxf(x, -200.0f), 200.0f);
    const uint32_t bits = __float_as_uint(x) & 0x7fffffffu;
    const int shift = 142 - (int)(bits >> 23);   // 15 - e, at least 8
    const uint64_t product = (uint64_t)((bits & 0x7fffffu) | 0x800000u) * 6196328019ull;
    const long long r = shift > 62 ? 0 : (long long)((product + (1ull << (shift - 1))) >> shift);
    return x < 0.0f ? -r : r;
}

__device__ __forceinline__ long long clamp_units(long long G) { return min(max(G, -(1LL << 52)), 1LL << 52); }

// The factors of a chunk's rows, by one warp with two tokens a lane: their decays,
// exponents of key and value together (INT_MIN: one of them is zero) and of the query.
__device__ __forceinline__ void make_factors(Factors &s, const float (&g)[2], const int (&ekv)[2], const int (&eq)[2],
                                             float scale)
{
    const int lane = threadIdx.x & 31;
    const long long b = log2_units(g[1]);
    long long sum = log2_units(g[0]) + b;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += o;
    }
    const long long Gt[2] = {sum - b, sum};
    long long u[2], M[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) u[i] = ekv[i] == INT_MIN ? kNothing : ekv[i] * kOne - Gt[i];
    long long top = max(u[0], u[1]);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, top, d);
        if (lane >= d) top = max(top, o);
    }
    const long long before = __shfl_up_sync(0xffffffffu, top, 1);
    M[0] = lane ? max(before, u[0]) : u[0];
    M[1] = top;
    const long long last = __shfl_sync(0xffffffffu, top, 31), G = __shfl_sync(0xffffffffu, sum, 31);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int t = 2 * lane + i;
        s.uh[t] = (float)(int)(u[i] >> 40);
        s.ul[t] = (float)((uint32_t)(u[i] >> 8)) * 0x1p-32f;
        s.mh[t] = (float)(int)(M[i] >> 40);
        s.ml[t] = (float)((uint32_t)(M[i] >> 8)) * 0x1p-32f;
        s.f1[t] = scale * exp2_units(M[i] + Gt[i], eq[i]);
        s.f2[t] = scale * exp2_units(Gt[i], eq[i]);
        s.w[t] = exp2_units(u[i] - last, 0);
    }
    if (lane == 0) {
        s.keep = exp2_units(G, 0);
        s.add = exp2_units(G + last, 0);
        s.G = G;
    }
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// Two neighbouring rows of one operand: a lane has four values of each when a row
// is 128 wide, of one of them when it is 64.
template <int D>
struct Rows {
    static constexpr int N = D / 64;
    float4 x[N];
    __device__ __forceinline__ static int row(int i) { return N == 2 ? i : (threadIdx.x & 31) >> 4; }
    __device__ __forceinline__ static int lane() { return threadIdx.x & (D / 4 - 1); }
    // rows r and r + 1 of rows `stride` bytes apart, zeros from row n on
    __device__ __forceinline__ void load(const float *p, int stride, int r, int n)
    {
        const char *base = reinterpret_cast<const char *>(p + 4 * lane());
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int at = r + row(i);
            x[i] = at < n ? *reinterpret_cast<const float4 *>(base + (long long)at * stride)
                          : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
    }
    // from rows in shared memory, one after another
    __device__ __forceinline__ void load_shared(const float *p)
    {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = reinterpret_cast<const float4 *>(p + row(i) * D)[lane()];
    }
    // bits of the largest magnitude of both rows, in every lane; NANS: a NaN is the largest (else it is passed over)
    template <bool NANS = true>
    __device__ __forceinline__ void largest(uint32_t &first, uint32_t &second) const
    {
        uint32_t b[N];
#pragma unroll
        for (int i = 0; i < N; ++i)
            b[i] = NANS ? max(max(magnitude(x[i].x), magnitude(x[i].y)), max(magnitude(x[i].z), magnitude(x[i].w)))
                        : __float_as_uint(fmaxf(fmaxf(fabsf(x[i].x), fabsf(x[i].y)), fmaxf(fabsf(x[i].z), fabsf(x[i].w))));
        if constexpr (N == 2) {
            first = __reduce_max_sync(0xffffffffu, b[0]);
            second = __reduce_max_sync(0xffffffffu, b[1]);
        } else {
            const bool half = threadIdx.x & 16;
            first = __reduce_max_sync(0xffffffffu, half ? 0u : b[0]);
            second = __reduce_max_sync(0xffffffffu, half ? b[0] : 0u);
        }
    }
    // the rows over 2^e as binary16 parts at(row, 16-byte piece) bytes into hi and lo; fill: instead of them 1 zeros, 2 NaN
    template <typename At>
    __device__ __forceinline__ void store(__half *hi, __half *lo, int r, const int (&e)[2], const int (&fill)[2], At at) const
    {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int j = row(i);
            const float s = pow2(-(N == 2 ? e[i] : j ? e[1] : e[0]));
            const int f = N == 2 ? fill[i] : j ? fill[1] : fill[0];
            uint2 h, l;
            split2(x[i].x * s, x[i].y * s, h.x, l.x);
            split2(x[i].z * s, x[i].w * s, h.y, l.y);
            if (f) h = l = f == 1 ? make_uint2(0u, 0u) : make_uint2(0x7e007e00u, 0x7e007e00u);
            const uint32_t to = at(r + j, lane() >> 1) + ((lane() & 1) << 3);
            *reinterpret_cast<uint2 *>(reinterpret_cast<char *>(hi) + to) = h;
            *reinterpret_cast<uint2 *>(reinterpret_cast<char *>(lo) + to) = l;
        }
    }
};

// The kernel on the 5th-generation tensor cores (linear_prompt_tc.cu), 128 columns
// of a head a CTA: Dv a multiple of 128.  states: every segment's own state, but a
// sequence's last one's.
cudaError_t launch_linear_prompt_tc(const PromptArgs &p, int Dk, bool states, cudaStream_t st);

}  // namespace zq
