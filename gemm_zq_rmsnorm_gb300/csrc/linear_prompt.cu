// linear_prompt.cu -- linear attention with a decay for each head over prompts
// (MIInfer README, "Status": recurrent layers with a state of [heads][128][128]).
//
// A CTA owns DVT columns of one head and walks through a segment of a sequence.
// Each compute warp holds 16 of the columns, as the transposed state [16][Dk] in
// MMA accumulators, whose layout is that of the MMA's second operand: the product
// with the queries takes the state from registers.  Four more warps load and
// convert the next chunk meanwhile.
#include <atomic>

#include "linear_prompt.cuh"

namespace zq {
namespace {

constexpr int C = kChunk;
constexpr int kLoaders = 4;        // warps that load
constexpr int kSlots = 152;        // CTAs that the plan cuts long sequences for
constexpr int kMaxCut = 512;       // sequences of a call up to which they are cut

// Segments: every sequence in pieces of `length` tokens, at least one.
struct Plan {
    int length;        // tokens, a multiple of C; 0: sequences are not cut
    int segments;      // at most, over all sequences
};

Plan plan_of(int T, int B, int Hv, int Dv)
{
    const int ctas = Hv * ((Dv + 127) / 128);
    const int n = kSlots / ctas;
    if (B > kMaxCut || n < 2 || T <= 2 * C) return {0, B};
    const int length = ((T + n - 1) / n + C - 1) / C * C;
    if (length >= T) return {0, B};
    return {length, T / length + B};
}

// ---------------------------------------------------------------- shared memory of a stage
template <int DK, int DVT>
struct Stage {
    __half q[2][C * DK], k[2][C * DK], v[2][C * DVT];   // hi, lo; rows with swizzled 16-byte pieces
    Factors f;
    int eq[C], ekv[C];
};

// P in 16 x 16 blocks on and below the diagonal, block (r, c) at r (r + 1) / 2 + c
struct Weights {
    __half p[2][10 * 256];
};

template <int DK, int DVT>
struct Smem {
    Stage<DK, DVT> stage[2];
    Weights p[2];
    Segment seg;
};

// byte offset of 16-byte piece `c` of row r in a tile of rows of D values
template <int D>
__device__ __forceinline__ uint32_t piece(int r, int c)
{
    return r * (D * 2) + ((c ^ (r & 7)) << 4);
}
// the same in a block of 16 rows of 16
__device__ __forceinline__ uint32_t block_piece(int r, int c) { return r * 32 + ((c ^ ((r >> 2) & 1)) << 4); }

template <int ID_THREADS>
__device__ __forceinline__ void bar_sync(int id)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(ID_THREADS) : "memory");
}
template <int ID_THREADS>
__device__ __forceinline__ void bar_arrive(int id)
{
    asm volatile("bar.arrive %0, %1;" ::"r"(id), "n"(ID_THREADS) : "memory");
}
// named barriers; pairs alternate with the chunks, so that a warp which is a chunk ahead meets another one
enum { kFull = 1, kEmpty = 3, kLoad = 5, kCompute = 7 };

// ---------------------------------------------------------------- loaders
template <int DK, int DVT, bool STATES>
__device__ __forceinline__ void load_chunks(const PromptArgs &p, Smem<DK, DVT> &sm, int h, int col0, int chunks)
{
    constexpr int THREADS = (DVT / 16 + kLoaders) * 32;
    constexpr int DEPTH = 4;   // steps of two rows on their way
    const LinearAttnArgs &a = p.a;
    const int w = (threadIdx.x >> 5) - DVT / 16, lane = threadIdx.x & 31;
    const int hk = h / (a.Hv / a.Hk);
    for (int c = 0; c < chunks; ++c) {
        Stage<DK, DVT> &s = sm.stage[c & 1];
        const long long row = sm.seg.row0 + c * C;
        const int n = sm.seg.row1 - (int)row;      // rows that there are
        const float *q = a.q + row * a.q_stride + (long long)hk * DK, *k = a.k + row * a.k_stride + (long long)hk * DK;
        const float *v = a.v + row * a.v_stride + (long long)h * p.Dv + col0;
        const float *g = a.g ? a.g + row * a.g_stride + h : nullptr;
        Rows<DK> qr[DEPTH], kr[DEPTH];
        Rows<DVT> vr[DEPTH];
        float gr[DEPTH];
        float g2[2] = {0.0f, 0.0f};   // of the warp that makes the factors
        // rows 2 (w + 4 j), 2 (w + 4 j) + 1 for j = 0 .. 7; those of j + 1 are on their way while j's are converted
        auto fetch = [&](int j, int b) {
            const int r = 2 * (w + kLoaders * j);
            if (!STATES) qr[b].load(q, a.q_stride, r, n);
            kr[b].load(k, a.k_stride, r, n);
            vr[b].load(v, a.v_stride, r, n);
            gr[b] = g && r + (lane & 1) < n ? g[(r + (lane & 1)) * a.g_stride] : 0.0f;
        };
#pragma unroll
        for (int j = 0; j < DEPTH - 1; ++j) fetch(j, j);
        if (w == 0 && g) {
            if (2 * lane < n) g2[0] = g[2 * lane * a.g_stride];
            if (2 * lane + 1 < n) g2[1] = g[(2 * lane + 1) * a.g_stride];
        }
        if (c >= 2) bar_sync<THREADS>(kEmpty + (c & 1));
#pragma unroll
        for (int j = 0; j < C / (2 * kLoaders); ++j) {
            if (j + DEPTH - 1 < C / (2 * kLoaders)) fetch(j + DEPTH - 1, (j + DEPTH - 1) % DEPTH);
            const int r = 2 * (w + kLoaders * j), b = j % DEPTH;
            const unsigned nan = __ballot_sync(0xffffffffu, gr[b] != gr[b]);
            uint32_t mk[2], mv[2], mq[2] = {0u, 0u};
            kr[b].largest(mk);
            vr[b].largest(mv);
            if (!STATES) qr[b].largest(mq);
            int ek[2], ev[2], eq[2], kfill[2], vfill[2];
            const int qfill[2] = {0, 0};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                // what is not finite makes the token's key NaN, and so its own row, all later ones and the state; its
                // value must not meet the zero weights of earlier rows
                const bool bad = mk[i] >= 0x7f800000u || mv[i] >= 0x7f800000u || (nan >> i & 1);
                ek[i] = row_exponent(mk[i]);
                ev[i] = row_exponent(mv[i]);
                eq[i] = mq[i] >= 0x7f800000u ? 0 : row_exponent(mq[i]);
                kfill[i] = bad ? 2 : 0;
                vfill[i] = bad ? 1 : 0;
                if (bad) ek[i] = ev[i] = 0;
                if (lane == i) {
                    s.ekv[r + i] = !bad && (mk[i] == 0u || mv[i] == 0u) ? INT_MIN : ek[i] + ev[i];
                    s.eq[r + i] = eq[i];
                }
            }
            if (!STATES) qr[b].store(s.q[0], s.q[1], r, eq, qfill, piece<DK>);
            kr[b].store(s.k[0], s.k[1], r, ek, kfill, piece<DK>);
            vr[b].store(s.v[0], s.v[1], r, ev, vfill, piece<DVT>);
        }
        if (w == 0) {
            bar_sync<kLoaders * 32>(kLoad + (c & 1));
            make_factors(s.f, g2, {s.ekv[2 * lane], s.ekv[2 * lane + 1]}, {s.eq[2 * lane], s.eq[2 * lane + 1]}, a.scale);
        } else {
            bar_arrive<kLoaders * 32>(kLoad + (c & 1));
        }
        bar_arrive<THREADS>(kFull + (c & 1));
    }
}

// ---------------------------------------------------------------- compute warps
template <int DK, int DVT>
__device__ __forceinline__ void scores(const Stage<DK, DVT> &s, Weights &pw, int w)
{
    // blocks (r, c) of 16 x 16, c <= r, dealt to the warps
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint32_t q0 = smem_u32(s.q[0]), q1 = smem_u32(s.q[1]), k0 = smem_u32(s.k[0]), k1 = smem_u32(s.k[1]);
    for (int i = w; i < 10; i += DVT / 16) {
        const int r = i >= 6 ? 3 : i >= 3 ? 2 : i >= 1 ? 1 : 0, c = i - r * (r + 1) / 2;
        float acc[2][4] = {};
        const int ar = 16 * r + (lane & 15), ac = lane >> 4;
        const int br = 16 * c + (lane & 7) + ((lane >> 4) << 3), bc = (lane >> 3) & 1;
#pragma unroll
        for (int kk = 0; kk < DK / 16; ++kk) {
            uint32_t ah[4], al[4], bh[4], bl[4];
            const uint32_t ap = piece<DK>(ar, 2 * kk + ac), bp = piece<DK>(br, 2 * kk + bc);
            ldsm4(ah, q0 + ap);
            ldsm4(bh, k0 + bp);
            ldsm4(al, q1 + ap);
            ldsm4(bl, k1 + bp);
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                mma16<ZQ_F16>(acc[n], ah[0], ah[1], ah[2], ah[3], bh[2 * n], bh[2 * n + 1]);
                mma16<ZQ_F16>(acc[n], ah[0], ah[1], ah[2], ah[3], bl[2 * n], bl[2 * n + 1]);
                mma16<ZQ_F16>(acc[n], al[0], al[1], al[2], al[3], bh[2 * n], bh[2 * n + 1]);
            }
        }
        char *p0 = reinterpret_cast<char *>(pw.p[0] + i * 256), *p1 = reinterpret_cast<char *>(pw.p[1] + i * 256);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int tr = 16 * r + g + 8 * half;
            const float mh = s.f.mh[tr], ml = s.f.ml[tr];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const int sc = 16 * c + 8 * n + 2 * t;
                const float2 uh = *reinterpret_cast<const float2 *>(&s.f.uh[sc]), ul = *reinterpret_cast<const float2 *>(&s.f.ul[sc]);
                const float x = sc <= tr ? acc[n][2 * half] * exp2_fast((uh.x - mh) + (ul.x - ml)) : 0.0f;
                const float y = sc + 1 <= tr ? acc[n][2 * half + 1] * exp2_fast((uh.y - mh) + (ul.y - ml)) : 0.0f;
                uint32_t hi, lo;
                split2(x, y, hi, lo);
                const uint32_t at = block_piece(g + 8 * half, n) + 4 * t;
                *reinterpret_cast<uint32_t *>(p0 + at) = hi;
                *reinterpret_cast<uint32_t *>(p1 + at) = lo;
            }
        }
    }
}

template <int DK, int DVT, bool STATES>
__global__ void __launch_bounds__((DVT / 16 + kLoaders) * 32, 1)
linear_prompt_kernel(const __grid_constant__ PromptArgs p)
{
    constexpr int NW = DVT / 16, THREADS = (NW + kLoaders) * 32, N8 = DK / 8;
    extern __shared__ char raw[];
    Smem<DK, DVT> &sm = *reinterpret_cast<Smem<DK, DVT> *>((reinterpret_cast<uintptr_t>(raw) + 127) & ~(uintptr_t)127);
    const LinearAttnArgs &a = p.a;
    pdl_wait();   // the projection's rows, the starts and the states come from earlier kernels
    pdl_launch_dependents();
    const int tiles = p.Dv / DVT;
    const int tile = blockIdx.x % tiles, item = blockIdx.x / tiles;
    const int h = item % a.Hv, at = item / a.Hv;
    if (threadIdx.x < 32) {
        const Segment s = find_segment(p, at);
        if (threadIdx.x == 0) sm.seg = s;
    }
    __syncthreads();
    const int seq = sm.seg.seq;
    if (seq < 0 || (STATES && sm.seg.last)) return;
    const int chunks = (sm.seg.row1 - sm.seg.row0 + C - 1) / C;
    const int w = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int col0 = tile * DVT;
    if (w >= NW) {
        load_chunks<DK, DVT, STATES>(p, sm, h, col0, chunks);
        return;
    }

    const int g = lane >> 2, t = lane & 3;
    // S^T: rows 16 w + g and + 8, columns 8 j + 2 t and + 1
    float S[N8][4];
    const int slot = a.slots[seq];
    const bool kept = slot >= 0 && slot < a.n;
    const int dv = col0 + 16 * w + g;
    const bool cut = p.length != 0 && (sm.seg.seg > 0 || !sm.seg.last);   // the sequence has several segments
    float *local = p.local + ((long long)at * a.Hv + h) * DK * p.Dv;
    float *pool = a.state + ((long long)(kept ? slot : 0) * a.Hv + h) * DK * p.Dv;
    const bool zeros = STATES || (!cut && (!kept || (a.fresh && a.fresh[seq] != 0)));
    auto value = [&](float *of, int j, int e) { return of + (8 * j + 2 * t + (e & 1)) * p.Dv + dv + 8 * (e >> 1); };
#pragma unroll
    for (int j = 0; j < N8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) S[j][e] = zeros ? 0.0f : *value(cut ? local : pool, j, e);
    long long G = 0;

    for (int c = 0; c < chunks; ++c) {
        const Stage<DK, DVT> &s = sm.stage[c & 1];
        Weights &pw = sm.p[c & 1];
        bar_sync<THREADS>(kFull + (c & 1));
        if constexpr (!STATES) {
            scores<DK, DVT>(s, pw, w);
            // exponents of the state's rows
            uint32_t m0 = 0, m1 = 0;
#pragma unroll
            for (int j = 0; j < N8; ++j) {
                m0 = max(m0, max(__float_as_uint(S[j][0]) & 0x7fffffffu, __float_as_uint(S[j][1]) & 0x7fffffffu));
                m1 = max(m1, max(__float_as_uint(S[j][2]) & 0x7fffffffu, __float_as_uint(S[j][3]) & 0x7fffffffu));
            }
#pragma unroll
            for (int d = 1; d < 4; d <<= 1) {
                m0 = max(m0, __shfl_xor_sync(0xffffffffu, m0, d));
                m1 = max(m1, __shfl_xor_sync(0xffffffffu, m1, d));
            }
            const int e0 = m0 >= 0x7f800000u ? 0 : row_exponent(m0), e1 = m1 >= 0x7f800000u ? 0 : row_exponent(m1);
            const float s0 = pow2(-e0), s1 = pow2(-e1);
            float o[4][2][4] = {};
            const uint32_t q0 = smem_u32(s.q[0]), q1 = smem_u32(s.q[1]);
#pragma unroll
            for (int kk = 0; kk < DK / 16; ++kk) {
                uint32_t bh[2][2], bl[2][2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    split2(S[2 * kk + i][0] * s0, S[2 * kk + i][1] * s0, bh[0][i], bl[0][i]);
                    split2(S[2 * kk + i][2] * s1, S[2 * kk + i][3] * s1, bh[1][i], bl[1][i]);
                }
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    uint32_t ah[4], al[4];
                    const uint32_t ap = piece<DK>(16 * m + (lane & 15), 2 * kk + (lane >> 4));
                    ldsm4(ah, q0 + ap);
                    ldsm4(al, q1 + ap);
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        mma16<ZQ_F16>(o[m][n], ah[0], ah[1], ah[2], ah[3], bh[n][0], bh[n][1]);
                        mma16<ZQ_F16>(o[m][n], ah[0], ah[1], ah[2], ah[3], bl[n][0], bl[n][1]);
                        mma16<ZQ_F16>(o[m][n], al[0], al[1], al[2], al[3], bh[n][0], bh[n][1]);
                    }
                }
            }
            // the exponents of this thread's columns 2 t, 2 t + 1 (and + 8): the lanes 4 (2 t) and 4 (2 t + 1) have them
            float x[2][2];
            x[0][0] = pow2(__shfl_sync(0xffffffffu, e0, 8 * t));
            x[0][1] = pow2(__shfl_sync(0xffffffffu, e0, 8 * t + 4));
            x[1][0] = pow2(__shfl_sync(0xffffffffu, e1, 8 * t));
            x[1][1] = pow2(__shfl_sync(0xffffffffu, e1, 8 * t + 4));
            bar_sync<NW * 32>(kCompute);   // the weights are there, and nobody reads those of two chunks ago

            uint32_t vh[4][4], vl[4][4];   // the warp's values as second operands: 16 tokens x 16 columns
            const uint32_t v0 = smem_u32(s.v[0]), v1 = smem_u32(s.v[1]);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                const uint32_t vp = piece<DVT>(16 * kk + (lane & 15), 2 * w + (lane >> 4));
                ldsm4t(vh[kk], v0 + vp);
                ldsm4t(vl[kk], v1 + vp);
            }
            const uint32_t p0 = smem_u32(pw.p[0]), p1 = smem_u32(pw.p[1]);
            const int rows = sm.seg.row1 - sm.seg.row0 - c * C;
            float *out = a.out + (long long)(sm.seg.row0 + c * C) * a.out_stride + (long long)h * p.Dv + col0 + 16 * w + 2 * t;
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                float acc[2][4] = {};
#pragma unroll
                for (int kk = 0; kk <= m; ++kk) {
                    uint32_t ah[4], al[4];
                    const uint32_t pp = (m * (m + 1) / 2 + kk) * 512 + block_piece(lane & 15, lane >> 4);
                    ldsm4(ah, p0 + pp);
                    ldsm4(al, p1 + pp);
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        mma16<ZQ_F16>(acc[n], ah[0], ah[1], ah[2], ah[3], vh[kk][2 * n], vh[kk][2 * n + 1]);
                        mma16<ZQ_F16>(acc[n], ah[0], ah[1], ah[2], ah[3], vl[kk][2 * n], vl[kk][2 * n + 1]);
                        mma16<ZQ_F16>(acc[n], al[0], al[1], al[2], al[3], vh[kk][2 * n], vh[kk][2 * n + 1]);
                    }
                }
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int tr = 16 * m + g + 8 * half;
                    const float f1 = s.f.f1[tr], f2 = s.f.f2[tr];
                    if (tr < rows)
#pragma unroll
                        for (int n = 0; n < 2; ++n)
                            *reinterpret_cast<float2 *>(out + tr * a.out_stride + 8 * n) =
                                make_float2(__fmaf_rn(f1, acc[n][2 * half], f2 * (o[m][n][2 * half] * x[n][0])),
                                            __fmaf_rn(f1, acc[n][2 * half + 1], f2 * (o[m][n][2 * half + 1] * x[n][1])));
                }
            }
        }

        // the state: S^T = keep S^T + add sum_s (w_s v_s) k_s^T
        {
            uint32_t ah[4][4], al[4][4];
            const uint32_t v0 = smem_u32(s.v[0]), v1 = smem_u32(s.v[1]);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                uint32_t xh[4], xl[4];
                const uint32_t vp = piece<DVT>(16 * kk + (lane & 7) + ((lane >> 4) << 3), 2 * w + ((lane >> 3) & 1));
                ldsm4t(xh, v0 + vp);
                ldsm4t(xl, v1 + vp);
                const float2 wa = *reinterpret_cast<const float2 *>(&s.f.w[16 * kk + 2 * t]);
                const float2 wb = *reinterpret_cast<const float2 *>(&s.f.w[16 * kk + 2 * t + 8]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 hi = __half22float2(*reinterpret_cast<const __half2 *>(&xh[i]));
                    const float2 lo = __half22float2(*reinterpret_cast<const __half2 *>(&xl[i]));
                    const float2 f = i < 2 ? wa : wb;
                    split2((hi.x + lo.x) * f.x, (hi.y + lo.y) * f.y, ah[kk][i], al[kk][i]);
                }
            }
            const uint32_t k0 = smem_u32(s.k[0]), k1 = smem_u32(s.k[1]);
            const float keep = s.f.keep, add = s.f.add;
#pragma unroll
            for (int jj = 0; jj < DK / 16; ++jj) {
                float acc[2][4] = {};
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    uint32_t bh[4], bl[4];
                    const uint32_t kp = piece<DK>(16 * kk + (lane & 15), 2 * jj + (lane >> 4));
                    ldsm4t(bh, k0 + kp);
                    ldsm4t(bl, k1 + kp);
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        mma16<ZQ_F16>(acc[n], ah[kk][0], ah[kk][1], ah[kk][2], ah[kk][3], bh[2 * n], bh[2 * n + 1]);
                        mma16<ZQ_F16>(acc[n], ah[kk][0], ah[kk][1], ah[kk][2], ah[kk][3], bl[2 * n], bl[2 * n + 1]);
                        mma16<ZQ_F16>(acc[n], al[kk][0], al[kk][1], al[kk][2], al[kk][3], bh[2 * n], bh[2 * n + 1]);
                    }
                }
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) S[2 * jj + n][e] = __fmaf_rn(add, acc[n][e], keep * S[2 * jj + n][e]);
            }
            G = clamp_units(G + s.f.G);
        }
        if (c + 2 < chunks) bar_arrive<THREADS>(kEmpty + (c & 1));
    }

    if (STATES || (kept && sm.seg.last))
#pragma unroll
        for (int j = 0; j < N8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) *value(STATES ? local : pool, j, e) = S[j][e];
    if (STATES && threadIdx.x == 0 && tile == 0) p.decay[(long long)at * a.Hv + h] = G;
}

// The states that the segments of cut sequences start from, in the place of their
// own: first(i + 1) = exp(G_i) first(i) + own(i).  A thread has four values of the
// state; grid: values / 1024, heads, sequences.
__global__ void __launch_bounds__(256) linear_join_kernel(const __grid_constant__ PromptArgs p, int Dk)
{
    pdl_wait();
    pdl_launch_dependents();
    const LinearAttnArgs &a = p.a;
    __shared__ int base_s;
    const int b = blockIdx.z, h = blockIdx.y;
    const int n = segments_of(p, b);
    if (n < 2) return;
    if (threadIdx.x < 32) {   // segments of the sequences before this one
        int sum = 0;
        for (int i = threadIdx.x; i < b; i += 32) sum += segments_of(p, i);
        sum = __reduce_add_sync(0xffffffffu, sum);
        if (threadIdx.x == 0) base_s = sum;
    }
    __syncthreads();
    const int base = base_s;
    const long long size = (long long)p.Dv * Dk, at = 4 * (blockIdx.x * 256 + threadIdx.x);
    const int slot = a.slots[b];
    float4 first = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (slot >= 0 && slot < a.n && !(a.fresh && a.fresh[b] != 0))
        first = *reinterpret_cast<const float4 *>(a.state + ((long long)slot * a.Hv + h) * size + at);
    auto own = [&](int i) { return reinterpret_cast<float4 *>(p.local + ((long long)(base + i) * a.Hv + h) * size + at); };
    float4 mine = *own(0);
    for (int i = 0; i < n; ++i) {
        const float4 next = i + 2 < n ? *own(i + 1) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);   // the last has none
        *own(i) = first;
        if (i + 1 < n) {
            const float f = exp2_units(p.decay[(long long)(base + i) * a.Hv + h], 0);
            first = make_float4(__fmaf_rn(f, first.x, mine.x), __fmaf_rn(f, first.y, mine.y),
                                __fmaf_rn(f, first.z, mine.z), __fmaf_rn(f, first.w, mine.w));
            mine = next;
        }
    }
}

template <int DK, int DVT, bool STATES>
cudaError_t launch_kernel(const PromptArgs &p, cudaStream_t st)
{
    static std::atomic<bool> ready[64];
    auto *kernel = linear_prompt_kernel<DK, DVT, STATES>;
    constexpr int smem = sizeof(Smem<DK, DVT>) + 128;
    static_assert(smem <= 227 * 1024, "a CTA's shared memory");
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (!ready[dev & 63].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        ready[dev & 63].store(true, std::memory_order_release);
    }
    const long long ctas = (long long)p.segments * p.a.Hv * (p.Dv / DVT);
    return launch_pdl(kernel, dim3((unsigned)ctas), dim3((DVT / 16 + kLoaders) * 32), smem, st, p);
}

template <int DK, int DVT>
cudaError_t launch_shape(const PromptArgs &p, cudaStream_t st)
{
    auto run = [&](bool states) {
        if constexpr (DVT == 128) return launch_linear_prompt_tc(p, DK, states, st);
        else return states ? launch_kernel<DK, DVT, true>(p, st) : launch_kernel<DK, DVT, false>(p, st);
    };
    if (p.length) {
        cudaError_t e = run(true);
        if (e != cudaSuccess) return e;
        e = launch_pdl(linear_join_kernel, dim3(DK * p.Dv / 1024, p.a.Hv, p.a.B), dim3(256), 0, st, p, DK);
        if (e != cudaSuccess) return e;
    }
    return run(false);
}

size_t state_bytes(const Plan &plan, int Hv, int Dk, int Dv) { return (size_t)plan.segments * Hv * Dk * Dv * 4; }

}  // namespace

size_t linear_attn_workspace(int T, int B, int Hv, int Dk, int Dv)
{
    const Plan plan = plan_of(T, B, Hv, Dv);
    return plan.length ? state_bytes(plan, Hv, Dk, Dv) + (size_t)plan.segments * Hv * 8 : 0;
}

cudaError_t launch_linear_attn(const LinearAttnArgs &a, int Dk, int Dv, void *workspace, cudaStream_t st)
{
    const Plan plan = plan_of(a.T, a.B, a.Hv, Dv);
    PromptArgs p{};
    p.a = a;
    p.Dv = Dv;
    p.length = plan.length;
    p.segments = plan.segments;
    p.local = static_cast<float *>(workspace);
    if (plan.length) p.decay = reinterpret_cast<long long *>(static_cast<char *>(workspace) + state_bytes(plan, a.Hv, Dk, Dv));
    if (Dk == 64) return Dv == 64 ? launch_shape<64, 64>(p, st) : launch_shape<64, 128>(p, st);
    return Dv == 64 ? launch_shape<128, 64>(p, st) : launch_shape<128, 128>(p, st);
}

}  // namespace zq
