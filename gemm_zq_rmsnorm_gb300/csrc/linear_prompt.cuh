// linear_prompt.cuh -- what the two kernels of linear attention over prompts
// share: the cut of sequences into segments, the parts of a value, and a chunk's
// factors.
//
// In chunks of 64 tokens the recurrence is matrix products: with G_t the sum of g
// from the chunk's first token to t,
//   o_t = scale (exp(G_t) S^T q_t + sum_{s <= t} exp(G_t - G_s) (q_t . k_s) v_s),
//   S'  = exp(G_C) S + sum_s exp(G_C - G_s) k_s v_s^T.
//
// Every product is taken of two binary16 parts of each factor: a row x is 2^e (hi + lo),
// the parts being those of the row scaled to [2^14, 2^15), so that each value keeps 22 bits
// of its own unless it is 2^16 below the row's largest (then 2^-39 of that); a product is hi hi + hi lo + lo hi
// (2^-22 of itself; sums fp32, a chunk's sums added to the state outside the tensor core,
// whose accumulator truncates).  (Scaled to [1, 2), the low parts end at 2^-25 of the row's
// largest value: a channel 1000 times the others, which the other factor lacks, cost 8.7e-6
// of a score's root mean square.)  Weights exp(G_t - G_s) and the rows' powers of two meet
// in the exponent: with u_s = e_k + e_v - G_s (G in base two) and M_t the whole number above
// the largest u of s <= t, the weight in the product is 2^(u_s - M_t) <= 1 and 2^(M_t + G_t)
// goes to the row, so that a token counts exactly where no larger one of its past drowns
// it, and the future does not matter at all.  G is a sum in units of 2^-32.
#pragma once

#include <limits.h>

#include <cuda.h>
#include <cuda_fp16.h>

#include "zq_async.cuh"
#include "zq_internal.cuh"
#include "zq_mixer.cuh"

namespace zq {

constexpr int kChunk = 64;         // tokens of a chunk

struct PromptArgs {
    LinearAttnArgs a;
    int Dv;
    int length, segments;      // tokens of a segment (a multiple of kChunk; 0: sequences are not cut), segments at most
    int few;                   // few segments of a sequence: each makes the state that it starts from itself
    // [segments][Hv][Dk][Dv]: a segment's own state, then the one it starts from; few: its own state, and in the place of a
    // sequence's last segment what the sequence starts from
    float *local;
    long long *decay;          // [segments][Hv]: its G
    float scale;               // a.scale is scale 2^scale_exponent, scale below 1
    int scale_exponent;
    unsigned int *status;
};

// the rows of sequence b, within the call's rows whatever the starts say
__host__ __device__ __forceinline__ void sequence_rows(const LinearAttnArgs &a, int b, int &r0, int &r1)
{
    const int s0 = a.starts[b] < 0 ? 0 : a.starts[b], s1 = a.starts[b + 1];
    r0 = s0 < a.T ? s0 : a.T;
    r1 = s1 < r0 ? r0 : s1 < a.T ? s1 : a.T;
}
__host__ __device__ __forceinline__ int segments_of(const PromptArgs &p, int b)
{
    int r0, r1;
    sequence_rows(p.a, b, r0, r1);
    return r0 == r1 ? 1 : (r1 - r0 + p.length - 1) / p.length;
}
// How many of a sequence's n segments, the first of them number `base` of the call, there is room for: all of them, but
// where starts decrease there may be more segments than states in the workspace.
__host__ __device__ __forceinline__ int within_room(const PromptArgs &p, int base, int n)
{
    const int room = p.segments - base;
    return room < 0 ? 0 : n < room ? n : room;
}

struct Segment {
    int seq, seg, last, row0, row1;   // seq < 0: there is none
    int place, count;                 // its number of all segments, the sequence's segments
};

// Segment number `at` of the call, or of those that are not their sequence's last,
// by one warp.
__device__ __forceinline__ Segment find_segment(const PromptArgs &p, int at, bool but_last)
{
    const LinearAttnArgs &a = p.a;
    const int lane = threadIdx.x & 31;
    Segment s{-1, 0, 1, 0, 0, at, 1};
    if (p.length == 0) {
        s.seq = at;
    } else {
        int base = 0;
        for (int b0 = 0; b0 < a.B && s.seq < 0; b0 += 32) {
            const int cnt = b0 + lane < a.B ? segments_of(p, b0 + lane) - but_last : 0;
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
                s.count = __shfl_sync(0xffffffffu, cnt, l) + but_last;
                s.last = s.seg + 1 == s.count;
            }
            base += __shfl_sync(0xffffffffu, sum, 31);
        }
    }
    if (s.seq >= 0) {
        if (but_last) s.place += s.seq;   // a last segment of each sequence before
        int r0, r1;
        sequence_rows(a, s.seq, r0, r1);
        s.row0 = r0 + s.seg * p.length;
        s.row1 = s.last ? r1 : s.row0 + p.length;
    }
    return s;
}

// ---------------------------------------------------------------- parts of values
// two products, sums, and fused products and sums in one instruction
__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    float2 d;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmul.rn.f32x2 z, x, y;\n\t"
        "mov.b64 {%0, %1}, z;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 d;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tadd.rn.f32x2 z, x, y;\n\t"
        "mov.b64 {%0, %1}, z;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 z, x, y, z;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

// two scaled values to their binary16 parts
__device__ __forceinline__ void split2(float2 x, uint32_t &hi, uint32_t &lo)
{
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(x.y), "f"(x.x));
    const float2 rest = fma2(__half22float2(*reinterpret_cast<const __half2 *>(&hi)), make_float2(-1.0f, -1.0f), x);
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(lo) : "f"(rest.y), "f"(rest.x));
}

__device__ __forceinline__ float exp2_fast(float x)
{
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x));
    return e;
}

// exponent of a magnitude (its bits)
__device__ __forceinline__ int exponent_of(uint32_t bits) { return (int)(bits >> 23) - 127; }
// that of a row, from its largest magnitude: the row over 2^e lies below 2^15
__device__ __forceinline__ int row_exponent(uint32_t bits) { return max(exponent_of(bits) - 14, -126); }
__device__ __forceinline__ float pow2(int e) { return __int_as_float((127 + e) << 23); }   // -126 <= e <= 127

__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// ---------------------------------------------------------------- a chunk's factors
// G in units of 2^-32: a whole part in the high word, a broken one in the low word
constexpr int kNothing = -(1 << 20);           // whole part of u of a row of zeros
// Scores are below 2^37 and lose this many powers of two before they are parts below 2^15.  (By a product of their
// own: in the weights' exponent, whose sum is an fp32 number, they would cost it bits.)
constexpr int kRoom = 22;
constexpr int kReach = 40;                     // the sums of a chunk reach at most this far above a state's exponent

struct alignas(16) Factors {                   // (arrays of tokens are read four values at a time)
    float uh[kChunk], ul[kChunk], m[kChunk];   // u, whole and broken part; M
    int gw[kChunk];                            // G, whole and broken part
    float gb[kChunk];
    float f1[kChunk], f2[kChunk];              // the rows' factors
    float part[kChunk];                        // the rows' factors where fp32 does not hold them: f2 = part 2^n,
    int n[kChunk];                             // f1 = part 2^(n + M + kRoom)
    int wide;                                  // a row needs these (make_factors)
    // OUT: what a state in registers is multiplied by, when its exponent is low .. low + range; the sums' factor is then
    // gpart 2^(low + kReach - exponent)
    struct alignas(16) Update {
        float keep, gpart;
        int low;
        unsigned range;
    } update;
    int grow, reach;                           // keep is gpart 2^grow, the sums' factor gpart 2^reach
    float keep, add;                           // !OUT: what the state, and what the chunk's sums are multiplied by
    long long scale;                           // !OUT: the power of two (in units) that the state counts in
    long long G;
};

// values of two neighbouring tokens
template <typename T>
__device__ __forceinline__ void store2(T *p, T a, T b)
{
    struct alignas(8) Two { T a, b; };
    *reinterpret_cast<Two *>(p) = {a, b};
}

__device__ __forceinline__ int whole(long long x) { return (int)(x >> 32); }
__device__ __forceinline__ float broken(long long x) { return (float)(uint32_t)x * 0x1p-32f; }

// x 2^n; 0 below the normal numbers' powers
__device__ __forceinline__ float times_pow2(float x, int n)
{
    const float y = x * pow2(max(-126, min(127, n)));
    return n < -126 ? 0.0f : n > 127 ? y * pow2(min(127, n - 127)) : y;
}
// 2^(n + part), the part's power to 2^-22
__device__ __forceinline__ float exp2_parts(int n, float part) { return times_pow2(exp2_fast(part), n); }
__device__ __forceinline__ float exp2_units(long long x) { return exp2_parts(whole(x), broken(x)); }

// x 2^units + y, for powers of any size: a large x stays a number below them
__device__ __forceinline__ float decayed(float x, long long units, float y)
{
    const int n = whole(units);
    const float part = exp2_fast(broken(units));
    return n >= -126 && n < 127 ? __fmaf_rn(part * pow2(n), x, y) : ldexpf(x, n) * part + y;
}

// x log2 e in units, to 2^-33 of itself and half a unit: the significand times 2^32 log2 e, shifted
__device__ __forceinline__ long long log2_units(float x)
{
    // e^-600 empties any state for any query, and the other end is infinity; NaN is marked elsewhere
    x = fminf(fmaxf(x, -600.0f), 600.0f);
    const uint32_t bits = __float_as_uint(x) & 0x7fffffffu;
    const int shift = min(63, 150 - (int)(bits >> 23));   // 23 - e, at least 14
    const uint64_t product = (uint64_t)((bits & 0x7fffffu) | 0x800000u) * 6196328019ull;
    const long long r = (long long)((product + (1ull << (shift - 1))) >> shift);
    return x < 0.0f ? -r : r;
}

__device__ __forceinline__ long long clamp_units(long long G) { return min(max(G, -(1LL << 44)), 1LL << 44); }
// the least power that a state counts in (its values are zero)
constexpr long long kNoScale = -(1LL << 53);

// G of a chunk's tokens from their decays, by one warp with two tokens a lane.
__device__ __forceinline__ void sum_decays(const float (&g)[2], long long (&G)[2])
{
    const int lane = threadIdx.x & 31;
    const long long b = log2_units(g[1]);
    long long sum = log2_units(g[0]) + b;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += o;
    }
    G[0] = sum - b;
    G[1] = sum;
}

// What a chunk's weights are made of, by the same warp: from G and the exponents of key and
// value together (INT_MIN: one of them is zero).  M need only be near the largest u: it is
// the whole number above it.  w: the tokens' weights in the state.  OUT: with M of every row.  !OUT: the state counts in
// 2^counts, which follows its decays and the chunk's sums, whichever is larger, so that no
// decay of many chunks empties the registers; one of its two factors is 1.
template <bool OUT>
__device__ __forceinline__ void make_weights(Factors &s, const long long (&G)[2], const int (&ekv)[2], float (&w)[2],
                                             long long &counts)
{
    const int lane = threadIdx.x & 31;
    int uw[2], M[2];
    float ub[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uw[i] = ekv[i] == INT_MIN ? kNothing : ekv[i] + whole(-G[i]);
        ub[i] = broken(-G[i]);
    }
    int top = max(uw[0], uw[1]), last;
    if (OUT) {
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, top, d);
            if (lane >= d) top = max(top, o);
        }
        const int before = __shfl_up_sync(0xffffffffu, top, 1);
        M[0] = (lane ? max(before, uw[0]) : uw[0]) + 1;
        M[1] = top + 1;
        last = __shfl_sync(0xffffffffu, M[1], 31);
    } else {
        last = __reduce_max_sync(0xffffffffu, top) + 1;
    }
    if (OUT) {
        store2(s.uh + 2 * lane, (float)uw[0], (float)uw[1]);
        store2(s.ul + 2 * lane, ub[0], ub[1]);
        store2(s.m + 2 * lane, (float)M[0], (float)M[1]);
        store2(s.gw + 2 * lane, whole(G[0]), whole(G[1]));
        store2(s.gb + 2 * lane, broken(G[0]), broken(G[1]));
    }
    w[0] = exp2_parts(uw[0] - last, ub[0]);
    w[1] = exp2_parts(uw[1] - last, ub[1]);
    if (lane == 31) {
        if (OUT) {
            // The state stays in its scale unless the sums are far above it, or far below (a state of zeros), or the decay
            // would empty the registers although the state (2^8 and more there) still counts beside the sums (near 2^28).
            const int grow = whole(G[1]), reach = grow + last;
            s.update = {exp2_units(G[1]), exp2_fast(broken(G[1])), grow > 90 ? INT_MAX / 2 : reach - kReach,
                        (unsigned)(grow < -90 ? min(150, -grow) : 150)};
            s.grow = grow;
            s.reach = reach;
        } else {
            const long long state = max(counts + G[1], kNoScale), sums = G[1] + ((long long)last << 32);
            counts = min(max(state, sums), -kNoScale);
            s.keep = exp2_units(state - counts);
            s.add = exp2_units(sums - counts);
            s.scale = counts;
        }
        s.G = G[1];
    }
}

// The factors of a chunk's rows of the output, by another warp, from what those have left
// and the largest magnitudes of the queries; the call's scale is scale 2^scale_exponent.
//
// wide: a row's factors are not all numbers that fp32 holds, although what they belong to
// may be (a query of 2^100 for tokens of 2^-110; a large state after decays of 2^-150): a
// power above 2^100, f1 below the normal numbers, or f2 below them where its term still
// counts.  That term is at most 2^(57 + n) for a state whose exponent is at most 20, and
// counts from 2^-149 and from 2^-40 of the row's own tokens (near 2^(20 + x), x the power of f1) on.
__device__ __forceinline__ void make_factors(Factors &s, const uint32_t *mq, float scale, int scale_exponent)
{
    const int lane = threadIdx.x & 31;
    bool wide = false;
    float part[2], f1[2], f2[2];
    int n[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int t = 2 * lane + i;
        // (zeros need no factor)
        n[i] = s.gw[t] + scale_exponent + (mq[t] ? row_exponent(mq[t]) : 0);
        const int x = n[i] + (int)s.m[t] + kRoom;
        part[i] = scale * exp2_fast(s.gb[t]);
        // (pow2(-127) is 0)
        f1[i] = part[i] * pow2(max(-127, min(127, x)));
        f2[i] = part[i] * pow2(max(-127, min(127, n[i])));
        wide |= max(n[i], x) > 100 || (x < -126 && x > -300) || (n[i] < -126 && n[i] + 57 >= max(-149, x - 20));
    }
    store2(s.f1 + 2 * lane, f1[0], f1[1]);
    store2(s.f2 + 2 * lane, f2[0], f2[1]);
    store2(s.part + 2 * lane, part[0], part[1]);
    store2(s.n + 2 * lane, n[0], n[1]);
    wide = __any_sync(0xffffffffu, wide);
    if (lane == 0) s.wide = wide;
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
    // the rows over 2^e as binary16 parts at(row, 16-byte piece) bytes into hi and lo
    template <typename At>
    __device__ __forceinline__ void store(__half *hi, __half *lo, int r, const int (&e)[2], At at) const
    {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int j = row(i);
            const float s = pow2(-(N == 2 ? e[i] : j ? e[1] : e[0]));
            uint2 h, l;
            split2(mul2(make_float2(x[i].x, x[i].y), make_float2(s, s)), h.x, l.x);
            split2(mul2(make_float2(x[i].z, x[i].w), make_float2(s, s)), h.y, l.y);
            const uint32_t to = at(r + j, lane() >> 1) + ((lane() & 1) << 3);
            *reinterpret_cast<uint2 *>(reinterpret_cast<char *>(hi) + to) = h;
            *reinterpret_cast<uint2 *>(reinterpret_cast<char *>(lo) + to) = l;
        }
    }
};

// The kernel on the 5th-generation tensor cores (linear_prompt_tc.cu).  states: every
// segment's own state, but a sequence's last one's.
cudaError_t launch_linear_prompt_tc(const PromptArgs &p, int Dk, bool states, cudaStream_t st);

}  // namespace zq
