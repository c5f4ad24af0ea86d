// linear_prompt_tc.cu -- linear attention with a decay for each head over prompts,
// on the 5th-generation tensor cores.
//
// A CTA owns 128 columns of one head and walks through a segment of a sequence in
// chunks of 64 tokens.  Everything is transposed, so that a column of the head is a
// lane of tensor memory and of the warps that work on it:
//   U  [128][Dk] = V~ K      (V~ = w_s v_s, 128 x 64, in tensor memory; K in shared)
//   O1 [128][64] = S^T Q^T   (S^T, 128 x Dk, in tensor memory; Q in shared)
//   O2 [128][64] = V^T P^T   (V^T, 128 x 64, in tensor memory; P in shared)
// each as three products of binary16 parts, the small ones first.  The state itself
// stays in the registers of eight warps (two threads for a column), which add U to
// it, split it for the next chunk and put O1 and O2 together.
//
// Warps: 0 issues the MMAs; 1..3 compute the scores and weights P (mma.sync: 64 x 64
// on and below the diagonal is too small a tile); 4..7 convert queries and keys;
// 8..11 values, a lane for a column (128-byte loads), and the chunk's factors;
// 12..19 the state.  Keys and queries are two stages deep, P too; the key tile serves
// the scores as rows and U as columns (the same bytes, a descriptor of the other
// order).
//
// Every wait is bounded: after one has run out no MMA is issued any more, the
// others return at once and the kernel ends (its results are invalid).
#include <atomic>

#include "linear_prompt.cuh"
#include "zq_tc_common.cuh"

namespace zq {
namespace {

constexpr int C = kChunk;
constexpr int kWarpP = 1, kWarpL = 4, kWarpV = 8, kWarpE = 12, kWarps = 20;   // first warp of each role; 0 issues
constexpr int kThreads = kWarps * 32;
// tensor memory columns
constexpr int kO1 = 0, kO2 = 64, kU = 128, kSh = 256, kSl = 320, kVh = 384, kVl = 416, kWh = 448, kWl = 480;

template <int DK>
struct Smem {
    __half q[2][2][C * DK], k[2][2][C * DK];   // [stage][part]: rows in tiles of 64 columns, 128-byte swizzle
    __half p[2][2][C * C];                     // [stage][part], rows of 64 tokens
    Factors f[4];
    uint32_t vmax[4][C];                       // largest magnitudes of the values of 32 columns
    float vscale[C];                           // 2^-e of the values' rows
    float wscale[C];                           // that times w
    int ek[2][C], eq[2][C];
    uint32_t smax[2][128];
    uint64_t qk_full[2], qk_empty[2], p_full[2], p_empty[2], fact[4], v_full, s_full, o_full, o_empty, u_full, u_empty;
    uint32_t tmem;
    int abort, any_bad;
    Segment seg;
};

// byte offset of 16-byte piece c of row r of a tile of rows of D values
template <int D>
__device__ __forceinline__ uint32_t tile_piece(int r, int c)
{
    return (c >> 3) * (C * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}

// B from columns: bit 16 of the instruction descriptor
__host__ __device__ constexpr uint32_t idesc_b_columns(uint32_t M, uint32_t N) { return idesc_f16_f32(M, N) | 1u << 16; }

template <int DK, bool STATES>
__global__ void __launch_bounds__(kThreads, 1) linear_prompt_tc_kernel(const __grid_constant__ PromptArgs p)
{
    extern __shared__ char raw[];
    Smem<DK> &sm = *reinterpret_cast<Smem<DK> *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    const LinearAttnArgs &a = p.a;
    const int w = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    volatile int *abort_flag = &sm.abort;
    unsigned int *status = p.status;
    auto wait = [&](uint64_t &bar, int parity) {   // by the whole warp
        wait_fast(&bar, (uint32_t)(parity & 1), abort_flag, status);
        __syncwarp();
    };
    auto arrive = [&](uint64_t &bar) {   // one arrival of the warp
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar);
    };

    if (w == 0) tmem_alloc(&sm.tmem, 512);
    if (threadIdx.x == 32) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.qk_full[i], 4);
            mbar_init(&sm.qk_empty[i], STATES ? 1 : 1 + 3);
            mbar_init(&sm.p_full[i], 3);
            mbar_init(&sm.p_empty[i], 1);
        }
        for (int i = 0; i < 4; ++i) mbar_init(&sm.fact[i], 1);
        mbar_init(&sm.v_full, 4);
        mbar_init(&sm.s_full, 8);
        mbar_init(&sm.o_full, 1);
        mbar_init(&sm.o_empty, 8);
        mbar_init(&sm.u_full, 1);
        mbar_init(&sm.u_empty, 8);
        sm.abort = 0;
        fence_mbar_init();
    }
    if (!STATES)   // P above the diagonal's blocks stays zero
        for (int i = threadIdx.x; i < (int)sizeof(sm.p) / 16; i += kThreads)
            reinterpret_cast<uint4 *>(sm.p)[i] = make_uint4(0u, 0u, 0u, 0u);
    fence_async_smem();
    pdl_wait();   // the projection's rows, the starts and the states come from earlier kernels
    const int tiles = p.Dv / 128;
    const int tile = blockIdx.x % tiles, item = blockIdx.x / tiles;
    const int h = item % a.Hv, at = item / a.Hv, col0 = tile * 128;
    if (w == 4) {
        const Segment s = find_segment(p, at);
        if (lane == 0) sm.seg = s;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // the next kernel's CTAs may come now: this one has its tensor memory already
    pdl_launch_dependents();
    const uint32_t tmem = sm.tmem;
    const Segment seg = sm.seg;
    const int chunks = seg.seq < 0 || (STATES && seg.last) ? 0 : (seg.row1 - seg.row0 + C - 1) / C;
    const bool any = seg.seq >= 0 && !(STATES && seg.last);
    const int hk = h / (a.Hv / a.Hk);

    if (w == 0) {
        // ------------------------------------------------------------ MMAs
        constexpr uint32_t id_u = idesc_b_columns(128, DK), id_o = idesc_f16_f32(128, C);
        const bool leader = elect_one();
        for (int c = 0; c < chunks; ++c) {
            const int st = c & 1, ph = c >> 1;
            wait(sm.qk_full[st], ph);
            wait(sm.v_full, c);
            if (c) wait(sm.u_empty, c - 1);
            tc_fence_after();
            const uint32_t kh = smem_u32(sm.k[st][0]), kl = smem_u32(sm.k[st][1]);
            if (!*abort_flag && leader) {
#pragma unroll
                for (int i = 0; i < 3; ++i) {   // lo hi, hi lo, hi hi
                    const uint32_t av = tmem + (i == 0 ? kWl : kWh), b = i == 1 ? kl : kh;
#pragma unroll
                    for (int kk = 0; kk < C / 16; ++kk)
                        mma_f16_ta(tmem + kU, av + 8 * kk, smem_desc(b + kk * 2048, C * 128, 1024, kLayoutSw128), id_u,
                                   i || kk);
                }
                mma_commit(&sm.u_full);
                if (STATES) mma_commit(&sm.qk_empty[st]);
            }
            __syncwarp();
            if (STATES) continue;
            wait(sm.s_full, c);
            if (c) wait(sm.o_empty, c - 1);
            tc_fence_after();
            const uint32_t qh = smem_u32(sm.q[st][0]), ql = smem_u32(sm.q[st][1]);
            if (!*abort_flag && leader) {
#pragma unroll
                for (int i = 0; i < 3; ++i) {
                    const uint32_t as = tmem + (i == 0 ? kSl : kSh), b = i == 1 ? ql : qh;
#pragma unroll
                    for (int kk = 0; kk < DK / 16; ++kk)
                        mma_f16_ta(tmem + kO1, as + 8 * kk,
                                   smem_desc(b + (kk >> 2) * (C * 128) + (kk & 3) * 32, 16, 1024, kLayoutSw128), id_o,
                                   i || kk);
                }
            }
            __syncwarp();
            wait(sm.p_full[st], ph);
            tc_fence_after();
            const uint32_t p0 = smem_u32(sm.p[st][0]), p1 = smem_u32(sm.p[st][1]);
            if (!*abort_flag && leader) {
#pragma unroll
                for (int i = 0; i < 3; ++i) {
                    const uint32_t av = tmem + (i == 0 ? kVl : kVh), b = i == 1 ? p1 : p0;
#pragma unroll
                    for (int kk = 0; kk < C / 16; ++kk)
                        mma_f16_ta(tmem + kO2, av + 8 * kk, smem_desc(b + kk * 32, 16, 1024, kLayoutSw128), id_o, i || kk);
                }
                mma_commit(&sm.o_full);
                mma_commit(&sm.qk_empty[st]);
                mma_commit(&sm.p_empty[st]);
            }
            __syncwarp();
        }
    } else if (w < kWarpL) {
        // ------------------------------------------------------------ scores and weights
        if (!STATES) {
            const int g = lane >> 2, t = lane & 3, wp = w - kWarpP;
            for (int c = 0; c < chunks; ++c) {
                const int st = c & 1, ph = c >> 1;
                wait(sm.qk_full[st], ph);
                const uint32_t q0 = smem_u32(sm.q[st][0]), q1 = smem_u32(sm.q[st][1]), k0 = smem_u32(sm.k[st][0]),
                               k1 = smem_u32(sm.k[st][1]);
                // blocks (r, c) of 16 x 16, c <= r: a row of four, a row of three, a row of two and one
                const int first = wp ? 1 + 3 * wp : 0, count = wp ? 3 : 4;
                float acc[4][2][4];
                auto block = [&](int i, int &r, int &cc) {
                    i += first;
                    r = i < 4 ? 3 : i < 7 ? 2 : i < 9 ? 1 : 0;
                    cc = i < 4 ? 3 - i : i < 7 ? 6 - i : i < 9 ? 8 - i : 0;
                };
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (i >= count) break;
                    int r, cc;
                    block(i, r, cc);
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[i][n][e] = 0.0f;
                    float small[2][4] = {};   // the products of a low part, apart: the accumulator cuts off
                    const int ar = 16 * r + (lane & 15), br = 16 * cc + (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
                    for (int kk = 0; kk < DK / 16; ++kk) {
                        uint32_t ah[4], al[4], bh[4], bl[4];
                        const uint32_t ap = tile_piece<DK>(ar, 2 * kk + (lane >> 4)),
                                       bp = tile_piece<DK>(br, 2 * kk + ((lane >> 3) & 1));
                        ldsm4(ah, q0 + ap);
                        ldsm4(bh, k0 + bp);
                        ldsm4(al, q1 + ap);
                        ldsm4(bl, k1 + bp);
#pragma unroll
                        for (int n = 0; n < 2; ++n) {
                            mma16<ZQ_F16>(acc[i][n], ah[0], ah[1], ah[2], ah[3], bh[2 * n], bh[2 * n + 1]);
                            mma16<ZQ_F16>(small[n], ah[0], ah[1], ah[2], ah[3], bl[2 * n], bl[2 * n + 1]);
                            mma16<ZQ_F16>(small[n], al[0], al[1], al[2], al[3], bh[2 * n], bh[2 * n + 1]);
                        }
                    }
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[i][n][e] += small[n][e];
                }
                arrive(sm.qk_empty[st]);
                wait(sm.fact[c & 3], c >> 2);
                if (c >= 2) wait(sm.p_empty[st], ph - 1);
                const Factors &f = sm.f[c & 3];
                char *p0 = reinterpret_cast<char *>(sm.p[st][0]), *p1 = reinterpret_cast<char *>(sm.p[st][1]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (i >= count) break;
                    int r, cc;
                    block(i, r, cc);
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const int tr = 16 * r + g + 8 * half;
                        const float mh = f.mh[tr], ml = f.ml[tr];
#pragma unroll
                        for (int n = 0; n < 2; ++n) {
                            const int sc = 16 * cc + 8 * n + 2 * t;
                            const float2 uh = *reinterpret_cast<const float2 *>(&f.uh[sc]),
                                         ul = *reinterpret_cast<const float2 *>(&f.ul[sc]);
                            const float x = sc <= tr ? acc[i][n][2 * half] * exp2_fast((uh.x - mh) + (ul.x - ml)) : 0.0f;
                            const float y =
                                sc + 1 <= tr ? acc[i][n][2 * half + 1] * exp2_fast((uh.y - mh) + (ul.y - ml)) : 0.0f;
                            uint32_t hi, lo;
                            split2(x, y, hi, lo);
                            const uint32_t to = tile_piece<C>(tr, 2 * cc + n) + 4 * t;
                            *reinterpret_cast<uint32_t *>(p0 + to) = hi;
                            *reinterpret_cast<uint32_t *>(p1 + to) = lo;
                        }
                    }
                }
                fence_async_smem();
                arrive(sm.p_full[st]);
            }
        }
    } else if (w < kWarpV) {
        // ------------------------------------------------------------ queries and keys
        constexpr int STEPS = C / 8, DEPTH = 3;   // two rows of each a step
        const int wl = w - kWarpL;
        const int none[2] = {0, 0};
        for (int c = 0; c < chunks; ++c) {
            const int st = c & 1;
            const long long row = seg.row0 + c * C;
            const int n = seg.row1 - (int)row;
            const float *q = a.q + row * a.q_stride + (long long)hk * DK, *k = a.k + row * a.k_stride + (long long)hk * DK;
            Rows<DK> qr[DEPTH], kr[DEPTH];
            auto fetch = [&](int j) {
                const int r = 2 * (wl + 4 * j);
                if (!STATES) qr[j % DEPTH].load(q, a.q_stride, r, n);
                kr[j % DEPTH].load(k, a.k_stride, r, n);
            };
#pragma unroll
            for (int j = 0; j < DEPTH - 1; ++j) fetch(j);
            if (c >= 2) wait(sm.qk_empty[st], (c >> 1) - 1);
#pragma unroll
            for (int j = 0; j < STEPS; ++j) {
                if (j + DEPTH - 1 < STEPS) fetch(j + DEPTH - 1);
                const int r = 2 * (wl + 4 * j);
                auto convert = [&](const Rows<DK> &x, __half(&dst)[2][C * DK], int *exponents) {
                    uint32_t m[2];
                    x.largest(m);
                    const int e[2] = {row_exponent(m[0]), row_exponent(m[1])};
                    // a row of zeros is told apart; an infinity or NaN gives parts that are NaN, and so a row of NaN
                    if (lane < 2) exponents[r + lane] = (lane ? m[1] : m[0]) ? (lane ? e[1] : e[0]) : INT_MIN;
                    x.store(dst[0], dst[1], r, e, none, tile_piece<DK>);
                };
                if (!STATES) convert(qr[j % DEPTH], sm.q[st], sm.eq[st]);
                convert(kr[j % DEPTH], sm.k[st], sm.ek[st]);
            }
            fence_async_smem();
            arrive(sm.qk_full[st]);
        }
    } else if (w < kWarpE) {
        // ------------------------------------------------------------ values and factors
        const int quarter = w & 3, column = 32 * quarter + lane;   // tensor memory lanes of this warp
        const uint32_t lanes = tmem + ((uint32_t)(32 * quarter) << 16);
        const bool maker = quarter == 3;
        for (int c = 0; c < chunks; ++c) {
            const long long row = seg.row0 + c * C;
            const int n = seg.row1 - (int)row;
            const float *v = a.v + row * a.v_stride + (long long)h * p.Dv + col0 + column;
            float x[C];
#pragma unroll
            for (int s = 0; s < C; ++s) x[s] = s < n ? v[s * a.v_stride] : 0.0f;
            float g[2] = {0.0f, 0.0f};
            if (maker && a.g)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (2 * lane + i < n) g[i] = a.g[(row + 2 * lane + i) * a.g_stride + h];
#pragma unroll
            for (int s = 0; s < C; ++s) {
                const uint32_t m = __reduce_max_sync(0xffffffffu, magnitude(x[s]));
                if (lane == (s & 31)) sm.vmax[quarter][s] = m;
            }
            named_bar(1, 128);
            int ev[2] = {0, 0};
            bool bad[2] = {false, false}, zero[2] = {false, false};
            if (maker) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int s = 2 * lane + i;
                    const uint32_t m = max(max(sm.vmax[0][s], sm.vmax[1][s]), max(sm.vmax[2][s], sm.vmax[3][s]));
                    ev[i] = row_exponent(m);
                    zero[i] = m == 0u;
                    // a token whose value or decay is not finite: its weights become NaN, and so its own row, all
                    // later ones and the state; the value itself must not meet the zero weights of earlier rows
                    bad[i] = m >= 0x7f800000u || g[i] != g[i];
                    sm.vscale[s] = bad[i] ? 0.0f : pow2(-ev[i]);
                }
                const int some = __any_sync(0xffffffffu, bad[0] || bad[1]);
                if (lane == 0) sm.any_bad = some;
            }
            named_bar(1, 128);
            if (sm.any_bad)
#pragma unroll
                for (int s = 0; s < C; ++s) x[s] = sm.vscale[s] == 0.0f ? 0.0f : x[s];
            if (maker) {
                wait(sm.qk_full[c & 1], c >> 1);
                Factors &f = sm.f[c & 3];
                int ekv[2], eq[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int s = 2 * lane + i, ek = sm.ek[c & 1][s];
                    ekv[i] = !bad[i] && (zero[i] || ek == INT_MIN) ? INT_MIN : (bad[i] ? 0 : ev[i]) + max(ek, -126);
                    eq[i] = STATES ? 0 : max(sm.eq[c & 1][s], -126);
                }
                make_factors(f, g, ekv, eq, a.scale);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int s = 2 * lane + i;
                    if (bad[i]) f.uh[s] = __int_as_float(0x7fc00000);
                    sm.wscale[s] = bad[i] ? __int_as_float(0x7fc00000) : f.w[s] * pow2(-ev[i]);
                }
                arrive(sm.fact[c & 3]);
            }
            // the last chunk's MMAs have read what is written now
            if (c) wait(STATES ? sm.u_full : sm.o_full, c - 1);
            tc_fence_after();
            auto parts = [&](const float *scale, int hi, int lo) {
#pragma unroll
                for (int b = 0; b < C / 16; ++b) {
                    uint32_t ph[8], pl[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 f = *reinterpret_cast<const float2 *>(scale + 16 * b + 2 * i);
                        split2(x[16 * b + 2 * i] * f.x, x[16 * b + 2 * i + 1] * f.y, ph[i], pl[i]);
                    }
                    tmem_st8(lanes + hi + 8 * b, ph);
                    tmem_st8(lanes + lo + 8 * b, pl);
                }
            };
            if (!STATES) parts(sm.vscale, kVh, kVl);
            named_bar(1, 128);
            parts(sm.wscale, kWh, kWl);
            tmem_wait_st();
            tc_fence_before();
            arrive(sm.v_full);
        }
    } else {
        // ------------------------------------------------------------ state and output
        const int quarter = w & 3, half = (w - kWarpE) >> 2, column = 32 * quarter + lane;
        const uint32_t lanes = tmem + ((uint32_t)(32 * quarter) << 16);
        constexpr int N = DK / 2;   // values of the state of a thread: rows half * N ..
        const bool cut = p.length != 0 && (seg.seg > 0 || !seg.last);
        const int slot = any ? a.slots[seg.seq] : -1;
        const bool kept = slot >= 0 && slot < a.n;
        const long long place = (long long)half * N * p.Dv + col0 + column;
        float *local = p.local + ((long long)at * a.Hv + h) * DK * p.Dv + place;
        float *pool = a.state + ((long long)(kept ? slot : 0) * a.Hv + h) * DK * p.Dv + place;
        const bool zeros = !any || STATES || (!cut && (!kept || (a.fresh && a.fresh[seg.seq] != 0)));
        float S[N];
#pragma unroll
        for (int i = 0; i < N; ++i) S[i] = zeros ? 0.0f : (cut ? local : pool)[(long long)i * p.Dv];
        long long G = 0;
        int exponent = 0;
        // the state's parts for the next product with the queries
        auto publish = [&]() {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < N; ++i) m = max(m, magnitude(S[i]));
            sm.smax[half][column] = m;
            named_bar(2, 256);
            m = max(m, sm.smax[half ^ 1][column]);
            exponent = row_exponent(m);
            const float s = pow2(-exponent);
#pragma unroll
            for (int b = 0; b < N / 16; ++b) {
                uint32_t ph[8], pl[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) split2(S[16 * b + 2 * i] * s, S[16 * b + 2 * i + 1] * s, ph[i], pl[i]);
                tmem_st8(lanes + kSh + half * (N / 2) + 8 * b, ph);
                tmem_st8(lanes + kSl + half * (N / 2) + 8 * b, pl);
            }
            tmem_wait_st();
            tc_fence_before();
            named_bar(2, 256);   // the maxima are read before the next ones are written
            arrive(sm.s_full);
        };
        if (!STATES && chunks) publish();
        for (int c = 0; c < chunks; ++c) {
            const Factors &f = sm.f[c & 3];
            wait(sm.fact[c & 3], c >> 2);
            wait(sm.u_full, c);
            tc_fence_after();
            const float keep = f.keep, add = f.add;
#pragma unroll
            for (int b = 0; b < N / 16; ++b) {
                uint32_t u[16];
                tmem_ld16(lanes + kU + half * N + 16 * b, u);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) S[16 * b + i] = __fmaf_rn(add, __uint_as_float(u[i]), keep * S[16 * b + i]);
            }
            G = clamp_units(G + f.G);
            tc_fence_before();
            arrive(sm.u_empty);
            if (STATES) continue;
            wait(sm.o_full, c);
            tc_fence_after();
            const float xs = pow2(exponent);
            if (c + 1 < chunks) publish();
            const int n = seg.row1 - seg.row0 - c * C;
            float *out = a.out + (long long)(seg.row0 + c * C + 32 * half) * a.out_stride + (long long)h * p.Dv + col0 + column;
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                uint32_t o1[8], o2[8];
                tmem_ld8(lanes + kO1 + 32 * half + 8 * b, o1);
                tmem_ld8(lanes + kO2 + 32 * half + 8 * b, o2);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int t = 32 * half + 8 * b + i;
                    const float y = __fmaf_rn(f.f1[t], __uint_as_float(o2[i]), f.f2[t] * (__uint_as_float(o1[i]) * xs));
                    if (t < n) out[(8 * b + i) * a.out_stride] = y;
                }
            }
            tc_fence_before();
            arrive(sm.o_empty);
        }
        if (any && (STATES || (kept && seg.last))) {
#pragma unroll
            for (int i = 0; i < N; ++i) (STATES ? local : pool)[(long long)i * p.Dv] = S[i];
        }
        if (STATES && any && tile == 0 && w == kWarpE && lane == 0) p.decay[(long long)at * a.Hv + h] = G;
    }
    tc_fence_before();
    __syncthreads();
    if (w == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int DK, bool STATES>
cudaError_t launch(const PromptArgs &p, cudaStream_t st)
{
    static std::atomic<bool> ready[64];
    auto *kernel = linear_prompt_tc_kernel<DK, STATES>;
    constexpr int smem = sizeof(Smem<DK>) + 1024;
    static_assert(smem <= 227 * 1024, "a CTA's shared memory");
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (!ready[dev & 63].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        ready[dev & 63].store(true, std::memory_order_release);
    }
    const long long ctas = (long long)p.segments * p.a.Hv * (p.Dv / 128);
    PromptArgs args = p;
    args.status = device_status_word();
    return launch_pdl(kernel, dim3((unsigned)ctas), dim3(kThreads), smem, st, args);
}

}  // namespace

cudaError_t launch_linear_prompt_tc(const PromptArgs &p, int Dk, bool states, cudaStream_t st)
{
    if (Dk == 64) return states ? launch<64, true>(p, st) : launch<64, false>(p, st);
    return states ? launch<128, true>(p, st) : launch<128, false>(p, st);
}

}  // namespace zq
