// linear_prompt_tc.cu -- linear attention with a decay for each head over prompts,
// on the 5th-generation tensor cores.
//
// A CTA owns 128 columns of one head (64 of a head of 64) and walks through a
// segment of a sequence in chunks of 64 tokens.  Everything is transposed, so that a column of the head is a
// lane of tensor memory and of the warps that work on it:
//   U  [128][Dk] = V~ K      (V~ = w_s v_s, 128 x 64, in tensor memory; K in shared)
//   O1 [128][64] = S^T Q^T   (S^T, 128 x Dk, in tensor memory; Q in shared)
//   O2 [128][64] = V^T P^T   (V^T, 128 x 64, in tensor memory; P in shared)
// and the scores Q K^T in U's place, each as three products of binary16 parts, the
// small ones first.  The state itself stays in the registers of sixteen warps (four
// threads for a column), which add U to it, split it for the next chunk and put O1 and
// O2 together.
//
// Warps: 0, 1 and 5 weigh scores, 0 makes the chunk's weights and the state's factors as
// well, 1 those of the output's rows, 1 and 5 find the sizes of the values' rows; 2 issues the MMAs; 3, 4 and 6..11 convert queries and keys;
// 12..15 values for the output, a lane for a column; 16..31 the state and the values
// weighted for it.  Keys and queries are two stages deep; the key tile serves the scores
// as rows and U as columns (the same bytes, a descriptor of the other order).  Every
// barrier is one that its waiters cannot be two phases behind: where they could, there
// are two, for even and odd chunks.
//
// What bounds it is instructions and the steps that wait for one another, not memory:
// a chunk of 128 x 128 takes about 6800 cycles (issue slots 60 % busy, tensor pipe a
// third, HBM as well).  4096 tokens of 48 heads 129 us (floor by bytes 40, by products
// 42), 16384 of 8 heads 113, 24 prompts of up to 1500 tokens with 32 heads of 128 x 64
// 187, one of 37 tokens 6.4.  Keeping exponents beside the registers (see Factors) is 1 to
// 3 % of that.  All 512 columns of tensor memory are in use, so U and the
// scores share theirs; mma.sync beside these MMAs slowed both (214 us), and values
// unrolled over a whole chunk, or waits in every warp, lose to the instruction cache and
// the issue slots.
//
// Every wait is bounded: after one has run out no MMA is issued any more, the
// others return at once and the kernel ends (its results are invalid), when the copies
// and MMAs on their way have come in.
#include <atomic>
#include <cmath>

#include "linear_prompt.cuh"
#include "zq_tc_common.cuh"

namespace zq {
namespace {

constexpr int C = kChunk;
// the warps' parts; a warp can reach the tensor memory lanes 32 (its number mod 4) .. only, which is why 5 weighs scores
constexpr int kWarpM = 2, kWarpV = 12, kWarpE = 16, kWarps = 32, LW = 8;
__device__ __forceinline__ bool weighs(int w) { return w == 0 || w == 1 || w == 5; }
constexpr int kLoadRows = C / LW;  // rows of a chunk of a warp that converts
constexpr int kThreads = kWarps * 32;
// tensor memory columns
constexpr int kO1 = 0, kO2 = 64, kU = 128, kSh = 256, kSl = 320, kVh = 384, kVl = 416, kWh = 448, kWl = 480;
constexpr int kU2 = 0;   // a second U where there is no output
constexpr int kEmpty = -(1 << 30);   // exponent of a column of the state that is zero
static_assert(kVl - kVh == kWl - kWh, "low parts behind high ones");

template <int DK, int DV>
struct Smem {
    __half q[2][2][C * DK], k[2][2][C * DK];   // [stage][part]: rows in tiles of 64 columns, 128-byte swizzle
    __half p[2][C * C];                        // [part], rows of 64 tokens
    float v[2][C * DV];                        // [chunk's parity]: values as they come
    struct alignas(16) Chunk : Factors {       // read four values at a time
        alignas(16) float vscale[C], wscale[C];   // 2^-e of the values' rows, and that times w
        int some_bad;
    } f[4];
    alignas(16) uint32_t mq[2][C], mk[2][C], mv[2][C];   // bits of the rows' largest magnitudes
    uint32_t smax[4][128];
    uint64_t qk_full[2], qk_empty[2], values[2], sizes[2], w_full[2], fact[4];
    uint64_t scores, scores_read, p_full, v_full, s_full, o_full, o_empty, u_full, u_empty[2];
    uint64_t drained;
    uint32_t tmem;
    int abort;
    unsigned int wait_us;   // the waits' limit (behind `abort`)
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

__device__ __forceinline__ void tmem_ld4(uint32_t taddr, uint32_t (&r)[4])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(taddr));
}

__device__ __forceinline__ void tmem_st4(uint32_t taddr, const uint32_t (&r)[4])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
                 : "memory");
}

// The warp waits for a phase.  Many waiting warps share the issue slots (and the
// instruction cache) with the ones that work, so the loop is as short as it can be,
// and of every group of warps one waits here while the others sleep in a named
// barrier; the limit and the others' failure are looked at after 8 probes and then every
// 64 (of which each lets the warp sleep for a while by itself).
__device__ __noinline__ void wait_long(uint64_t *bar, int parity, volatile int *abort_flag, unsigned int *status)
{
    uint64_t since = 0;
    for (uint32_t turns = 1;; turns = 8) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\tmov.u32 n, %3;\n\t"
            "AGAIN:\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t@p bra DONE;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t@p bra DONE;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t@p bra DONE;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t@p bra DONE;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t@p bra DONE;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t@p bra DONE;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t@p bra DONE;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t@p bra DONE;\n\t"
            "sub.u32 n, n, 1;\n\tsetp.ne.u32 q, n, 0;\n\t"
            "@q bra AGAIN;\n\t"
            "DONE:\n\tselp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(smem_u32(bar)), "r"((uint32_t)(parity & 1)), "r"(turns)
            : "memory");
        if (__all_sync(0xffffffffu, done) || __any_sync(0xffffffffu, *abort_flag)) return;
        const uint64_t now = global_ns();
        if (!since) since = now;
        if (now - since > 1000ull * *reinterpret_cast<volatile unsigned int *>(abort_flag + 1)) {
            flag_timeout(status);
            *abort_flag = 1;
        }
    }
}

__device__ __forceinline__ void wait_phase(uint64_t *bar, int parity, volatile int *abort_flag, unsigned int *status)
{
    if (!__all_sync(0xffffffffu, mbar_try_wait(bar, (uint32_t)(parity & 1)))) wait_long(bar, parity, abort_flag, status);
}

// B from columns: bit 16 of the instruction descriptor
__host__ __device__ constexpr uint32_t idesc_b_columns(uint32_t M, uint32_t N) { return idesc_f16_f32(M, N) | 1u << 16; }

// 32 columns of the scores, from tensor memory: weighted, as parts to P.  The warp has
// the rows 32 quarter .., a lane each; columns 32 side ...  All of them are taken before
// the first is weighted, since the chunk's U waits for their place.
template <int DK, int DV>
__device__ __noinline__ void weigh_scores(Smem<DK, DV> &sm, const Factors &f, uint32_t tmem, int quarter, int side)
{
    const int lane = threadIdx.x & 31, tr = 32 * quarter + lane;
    uint32_t s[2][16];
    tmem_ld16(tmem + ((uint32_t)(32 * quarter) << 16) + kU + 32 * side, s[0]);
    tmem_ld16(tmem + ((uint32_t)(32 * quarter) << 16) + kU + 32 * side + 16, s[1]);
    const float m = -f.m[tr];
    tmem_wait_ld();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.scores_read);
#pragma unroll
    for (int piece = 0; piece < 4; ++piece) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            const int sc = 32 * side + 8 * piece + 2 * i;
            const float4 uh = *reinterpret_cast<const float4 *>(&f.uh[sc]), ul = *reinterpret_cast<const float4 *>(&f.ul[sc]);
            auto two = [&](int e, float2 h, float2 l, uint32_t &phi, uint32_t &plo) {
                const float2 x = add2(add2(h, make_float2(m, m)), l);
                const uint32_t *y0 = &s[piece >> 1][8 * (piece & 1) + 2 * i + e];
                float2 y = mul2(make_float2(__uint_as_float(y0[0]), __uint_as_float(y0[1])),
                                make_float2(exp2_fast(x.x), exp2_fast(x.y)));
                y = mul2(y, make_float2(pow2(-kRoom), pow2(-kRoom)));
                if (side == quarter) y = make_float2(sc + e <= tr ? y.x : 0.0f, sc + e + 1 <= tr ? y.y : 0.0f);
                split2(y, phi, plo);
            };
            two(0, make_float2(uh.x, uh.y), make_float2(ul.x, ul.y), hi[i], lo[i]);
            two(2, make_float2(uh.z, uh.w), make_float2(ul.z, ul.w), hi[i + 1], lo[i + 1]);
        }
        const uint32_t to = tile_piece<C>(tr, 4 * side + piece);
        *reinterpret_cast<uint4 *>(reinterpret_cast<char *>(sm.p[0]) + to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4 *>(reinterpret_cast<char *>(sm.p[1]) + to) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
}

// the largest magnitude of three, NaN if one is
__device__ __forceinline__ float largest3(float a, float b, float c)
{
    float d;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Bits of the largest magnitudes of 32 values' rows of a chunk, by a warp, a lane each
// (every lane starts at another piece of its row, so that the lanes' banks differ).
template <int DK, int DV>
__device__ __forceinline__ void value_sizes(Smem<DK, DV> &sm, int c, int first)
{
    const int lane = threadIdx.x & 31;
    const float4 *row = reinterpret_cast<const float4 *>(sm.v[c & 1] + (first + lane) * DV);
    float m[2] = {0.0f, 0.0f};
#pragma unroll 8
    for (int i = 0; i < DV / 4; ++i) {
        const float4 x = row[(i + lane) & (DV / 4 - 1)];
        m[0] = largest3(m[0], x.x, x.y);
        m[1] = largest3(m[1], x.z, x.w);
    }
    sm.mv[c & 1][first + lane] = __float_as_uint(largest3(m[0], m[1], 0.0f));
}

// Eight tokens' values of the lane's column, scaled, as parts to tensor memory.
template <int DK, int DV>
__device__ __forceinline__ void value_parts(const Smem<DK, DV> &sm, const typename Smem<DK, DV>::Chunk &f, const float *scale, int c,
                                            int first, int column, uint32_t to)
{
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = sm.v[c & 1][(first + i) * DV + column];
    if (f.some_bad)
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = f.vscale[first + i] == 0.0f ? 0.0f : x[i];
    uint32_t ph[4], pl[4];
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        const float4 y = *reinterpret_cast<const float4 *>(scale + first + 2 * i);
        split2(mul2(make_float2(x[2 * i], x[2 * i + 1]), make_float2(y.x, y.y)), ph[i], pl[i]);
        split2(mul2(make_float2(x[2 * i + 2], x[2 * i + 3]), make_float2(y.z, y.w)), ph[i + 1], pl[i + 1]);
    }
    tmem_st4(to, ph);
    tmem_st4(to + (kVl - kVh), pl);
}

// Sixteen rows of the output where fp32 does not hold the rows' factors or their
// products with the state's exponent, while the output itself may be a number like any
// other (a state of 2^100 after decays of 2^-150; a query of 2^-100 for a state of 2^120).
// Both of a row's terms count from the larger one, and the power of two comes last.
// Where the factors are numbers the result is the same, bit for bit.
//
// A chunk needs it when its factors say so (`wide`), a warp when its state's exponent is
// above 20 (values of 2^31 and more).
__device__ __noinline__ void far_outputs(const Factors &f, int first, uint32_t o1_at, uint32_t o2_at, char *out, int os, int n,
                                         int exponent)
{
#pragma unroll 1
    for (int b = 0; b < 16; b += 4) {
        uint32_t o1[4], o2[4];
        tmem_ld4(o1_at + b, o1);
        tmem_ld4(o2_at + b, o2);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = first + b + i, x = f.n[t] + (int)f.m[t] + kRoom, e = f.n[t] + exponent;
            const float part = f.part[t], state = __uint_as_float(o1[i]);
            const int base = state == 0.0f ? x : max(x, e);
            const float y = __fmaf_rn(times_pow2(part, x - base), __uint_as_float(o2[i]), times_pow2(part * state, min(0, e - base)));
            if (b + i < n) *reinterpret_cast<float *>(out + (long long)(b + i) * os) = ldexpf(y, base);
        }
    }
}

template <int DK, int DV, bool STATES>
__global__ void __launch_bounds__(kThreads, 1)
linear_prompt_tc_kernel(const __grid_constant__ PromptArgs p, const __grid_constant__ CUtensorMap map_q,
                        const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v)
{
    constexpr int QUARTERS = DV / 32;   // of the tensor memory's lanes that are in use
    extern __shared__ char raw[];
    // (an offset, not a rounded address: the compiler goes on seeing shared memory)
    Smem<DK, DV> &sm = *reinterpret_cast<Smem<DK, DV> *>(raw + (-smem_u32(raw) & 1023u));
    const LinearAttnArgs &a = p.a;
    const int w = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    volatile int *abort_flag = &sm.abort;
    unsigned int *status = p.status;
    auto wait = [&](uint64_t &bar, int parity) { wait_phase(&bar, parity, abort_flag, status); };
    // of a group of warps one waits, the others in the group's named barrier
    auto sync = [&](int group) {
        named_bar(group == kWarpV ? 1 : group == kWarpE ? 2 : 3, group == kWarpV ? 128 : group == kWarpE ? 128 * QUARTERS : 32 * LW);
    };
    auto arrive = [&](uint64_t &bar) {   // one arrival of the warp
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar);
    };

    if (w == kWarpM) tmem_alloc(&sm.tmem, 512);
    if (threadIdx.x == 32) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.qk_full[i], LW + (a.withhold_rows == i + 1));
            mbar_init(&sm.qk_empty[i], 1);
            mbar_init(&sm.sizes[i], 2);
            mbar_init(&sm.w_full[i], 4 * QUARTERS);
        }
        for (int i = 0; i < 4; ++i) mbar_init(&sm.fact[i], 1);
        for (int i = 0; i < 2; ++i) mbar_init(&sm.values[i], 1 + (a.withhold_values == i + 1));
        mbar_init(&sm.p_full, 3);
        mbar_init(&sm.scores, 1);
        mbar_init(&sm.scores_read, 3);
        mbar_init(&sm.v_full, QUARTERS);
        mbar_init(&sm.s_full, 4 * QUARTERS);
        mbar_init(&sm.o_full, 1);
        mbar_init(&sm.o_empty, 4 * QUARTERS);
        mbar_init(&sm.u_full, 1);
        mbar_init(&sm.u_empty[0], 4 * QUARTERS);
        mbar_init(&sm.u_empty[1], 4 * QUARTERS);
        mbar_init(&sm.drained, 1);
        sm.abort = 0;
        sm.wait_us = a.wait_us ? a.wait_us : (unsigned int)(kWaitLimitNs / 1000);
        fence_mbar_init();
    }
    if (!STATES)   // P above the diagonal's blocks stays zero
        for (int i = threadIdx.x; i < (int)sizeof(sm.p) / 16; i += kThreads)
            reinterpret_cast<uint4 *>(sm.p)[i] = make_uint4(0u, 0u, 0u, 0u);
    fence_async_smem();
    pdl_wait();   // the projection's rows, the starts and the states come from earlier kernels
    const int tiles = p.Dv / DV;
    const int tile = blockIdx.x % tiles, item = blockIdx.x / tiles;
    const int h = item % a.Hv, at = item / a.Hv, col0 = tile * DV;
    if (w == 3) {
        const Segment s = find_segment(p, at, STATES);
        if (lane == 0) sm.seg = s;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // the next kernel's CTAs may come now: this one has its tensor memory already
    pdl_launch_dependents();
    const uint32_t tmem = sm.tmem;
    const Segment seg = sm.seg;
    const bool any = seg.seq >= 0;
    const int chunks = any ? (seg.row1 - seg.row0 + C - 1) / C : 0;
    const int hk = h / (a.Hv / a.Hk);

    if (w == kWarpM) {
        // ------------------------------------------------------------ MMAs
        constexpr uint32_t id_u = idesc_b_columns(128, DK), id_o = idesc_f16_f32(128, C);
        const bool leader = elect_one();
        // Descriptors as their low word (address, offset between 64-column tiles) and a constant high one, so that an MMA
        // takes an addition or two: with the issue slots shared by eight warps every instruction between two MMAs counts.
        constexpr uint32_t high = 1024 >> 4 | 1u << 14 | kLayoutSw128 << 29;
        auto low = [](const void *tile) { return smem_u32(tile) >> 4 | (uint32_t)(C * 128 >> 4) << 16; };
        auto desc = [](uint32_t lo) { return (uint64_t)high << 32 | lo; };
        auto rows_at = [](int kk) { return (uint32_t)(((kk >> 2) * (C * 128) + (kk & 3) * 32) >> 4); };   // columns 16 kk ..
        constexpr uint32_t part = C * DK * 2 >> 4, stage = 2 * part, ppart = C * C * 2 >> 4;
        const uint32_t q0 = low(sm.q[0][0]), k0 = low(sm.k[0][0]), p0 = low(sm.p[0]);
        auto scores = [&](int c) {   // Q K^T in U's place; lanes 64 .. hold the product of whatever lies behind the queries
            const int st = c & 1;
            wait(sm.qk_full[st], c >> 1);
            if (c) wait(sm.u_empty[0], c - 1);
            tc_fence_after();
            if (!*abort_flag && leader) {
#pragma unroll
                for (int i = 0; i < 3; ++i) {   // lo hi, hi lo, hi hi
                    const uint32_t x = q0 + st * stage + (i == 0 ? part : 0), y = k0 + st * stage + (i == 1 ? part : 0);
#pragma unroll
                    for (int kk = 0; kk < DK / 16; ++kk)
                        mma_f16(tmem + kU, desc(x + rows_at(kk)), desc(y + rows_at(kk)), id_o, i || kk);
                }
                mma_commit(&sm.scores);
            }
            __syncwarp();
        };
        if (!STATES && chunks) scores(0);
        for (int c = 0; c < chunks; ++c) {
            const int st = c & 1;
            if (!STATES) {
                wait(sm.scores_read, c);
            } else {
                wait(sm.qk_full[st], c >> 1);
                if (c >= 2) wait(sm.u_empty[st], (c >> 1) - 1);
            }
            wait(sm.w_full[st], c >> 1);
            tc_fence_after();
            if (!*abort_flag && leader) {
#pragma unroll
                for (int i = 0; i < 3; ++i) {
                    const uint32_t av = tmem + (i == 0 ? kWl : kWh), b = k0 + st * stage + (i == 1 ? part : 0);
#pragma unroll
                    for (int kk = 0; kk < C / 16; ++kk)
                        mma_f16_ta(tmem + (STATES && st ? kU2 : kU), av + 8 * kk, desc(b + (kk * 2048 >> 4)), id_u, i || kk);
                }
                mma_commit(&sm.u_full);
                if (STATES) mma_commit(&sm.qk_empty[st]);
            }
            __syncwarp();
            if (STATES) continue;
            wait(sm.s_full, c);
            if (c) wait(sm.o_empty, c - 1);
            tc_fence_after();
            if (!*abort_flag && leader) {
#pragma unroll
                for (int i = 0; i < 3; ++i) {
                    const uint32_t as = tmem + (i == 0 ? kSl : kSh), b = q0 + st * stage + (i == 1 ? part : 0);
#pragma unroll
                    for (int kk = 0; kk < DK / 16; ++kk)
                        mma_f16_ta(tmem + kO1, as + 8 * kk, desc(b + rows_at(kk)), id_o, i || kk);
                }
                mma_commit(&sm.qk_empty[st]);
            }
            __syncwarp();
            wait(sm.v_full, c);
            wait(sm.p_full, c);
            tc_fence_after();
            if (!*abort_flag && leader) {
#pragma unroll
                for (int i = 0; i < 3; ++i) {
                    const uint32_t av = tmem + (i == 0 ? kVl : kVh), b = p0 + (i == 1 ? ppart : 0);
#pragma unroll
                    for (int kk = 0; kk < C / 16; ++kk) mma_f16_ta(tmem + kO2, av + 8 * kk, desc(b + rows_at(kk)), id_o, i || kk);
                }
                mma_commit(&sm.o_full);
            }
            __syncwarp();
            if (c + 1 < chunks) scores(c + 1);
        }
    } else if (weighs(w)) {
        // ------------------------------------------------------------ a chunk's factors (warp 0) and the scores' weights
        // warp 0 has the rows 0 .. 31 (32 columns), the others the rows 32 .. 63, half of the columns each
        const int quarter = w & 3, side = w == 5;
        float next[2], g[2];   // decays of the chunk after the next and of the next
        long long G[2];        // and their sums
        long long counts = kNoScale;
        auto decays = [&](int c) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const long long row = (long long)seg.row0 + c * C + 2 * lane + i;
                next[i] = a.g && row < seg.row1 ? a.g[row * a.g_stride + h] : 0.0f;
            }
        };
        if (w == 0 && chunks) decays(0);
        auto sums = [&](int c) {
            g[0] = next[0], g[1] = next[1];
            decays(c + 1);
            sum_decays(g, G);
        };
        auto factors = [&](int c) {
            const int st = c & 1, n = seg.row1 - seg.row0 - c * C;
            wait(sm.qk_full[st], c >> 1);
            wait(sm.sizes[st], c >> 1);
            typename Smem<DK, DV>::Chunk &f = sm.f[c & 3];
            int ekv[2], ev[2];
            float weight[2];
            bool bad[2], odd[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int s = 2 * lane + i;
                const uint32_t mk = sm.mk[st][s], mv = sm.mv[st][s];
                ev[i] = row_exponent(mv);
                // a token whose value is not finite, or whose decay is none or infinity: its weights become NaN, and so
                // its own row, all later ones and the state; the value itself must not meet the zero weights of earlier
                // rows.  (One of the key does the same by the key's parts.)
                bad[i] = s < n && (mv >= 0x7f800000u || !(g[i] < __int_as_float(0x7f800000)));
                odd[i] = mv >= 0x7f800000u || bad[i];   // (the rows behind the last are somebody else's)
                ekv[i] = !bad[i] && (s >= n || mk == 0u || mv == 0u) ? INT_MIN : ev[i] + row_exponent(mk);
            }
            make_weights<!STATES>(f, G, ekv, weight, counts);
            const float nan = __int_as_float(0x7fc00000);
            float vscale[2], wscale[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int s = 2 * lane + i;
                const float x = pow2(-ev[i]);
                if (bad[i]) f.uh[s] = nan;
                vscale[i] = bad[i] || s >= n ? 0.0f : x;
                wscale[i] = s >= n ? 0.0f : bad[i] ? nan : weight[i] * x;
            }
            store2(f.vscale + 2 * lane, vscale[0], vscale[1]);
            store2(f.wscale + 2 * lane, wscale[0], wscale[1]);
            const int some = __any_sync(0xffffffffu, odd[0] || odd[1]);
            if (lane == 0) f.some_bad = some;
            arrive(sm.fact[c & 3]);
        };
        for (int c = -1; c < chunks; ++c) {   // the sizes and the factors are a chunk ahead
            if (w && c + 1 < chunks) {
                wait(sm.values[(c + 1) & 1], (c + 1) >> 1);
                value_sizes(sm, c + 1, 32 * side);
                arrive(sm.sizes[(c + 1) & 1]);
            }
            if (w == 0 && c + 1 < chunks) sums(c + 1);   // (while the scores are on their way)
            if (!STATES && c >= 0) {
                if (w) wait(sm.fact[c & 3], c >> 2);
                // (what the output alone needs: its warps come to it by way of p_full)
                if (w == 1) make_factors(sm.f[c & 3], sm.mq[c & 1], p.scale, p.scale_exponent);
                if (c) wait(sm.o_full, c - 1);   // the last weights have been read
                wait(sm.scores, c);
                tc_fence_after();
                weigh_scores<DK, DV>(sm, sm.f[c & 3], tmem, quarter, side);
                fence_async_smem();
                arrive(sm.p_full);
            }
            if (w == 0 && c + 1 < chunks) factors(c + 1);
        }
    } else if (w < kWarpV) {
        // ------------------------------------------------------------ rows: parts of queries and keys, factors
        // warp wl has the rows kLoadRows wl .. of a chunk, in steps of two: the next two are on their way while two are
        // converted (from L2, where they come with the values)
        constexpr int STEPS = kLoadRows / 2;
        static_assert(STEPS % 2 == 0, "two steps a turn of the loop");
        const int wl = w < 5 ? w - 3 : w - 4;
        struct Step {
            Rows<DK> q, k;
        } step[2];
        const int rows = chunks ? seg.row1 - seg.row0 : 0;
        const float *qp = a.q + seg.row0 * a.q_stride + (long long)hk * DK, *kp = a.k + seg.row0 * a.k_stride + (long long)hk * DK;
        const int qs = 4 * (int)a.q_stride, ks = 4 * (int)a.k_stride;
        auto read = [&](Step &x, int i) {   // step i of the segment
            const int r = i / STEPS * C + kLoadRows * wl + 2 * (i % STEPS);
            if (!STATES) x.q.load(qp, qs, r, rows);
            x.k.load(kp, ks, r, rows);
        };
        read(step[0], 0);
        for (int c = 0; c < chunks; ++c) {
            const int st = c & 1;
            if (c >= 2 && wl == 0) wait(sm.qk_empty[st], (c >> 1) - 1);
            sync(0);
            auto convert = [&](const Step &x, int j) {
                const int r = kLoadRows * wl + 2 * j;
                uint32_t mq[2], mk[2];
                if (!STATES) x.q.template largest<false>(mq[0], mq[1]);
                x.k.template largest<false>(mk[0], mk[1]);
                // an infinity or NaN gives parts that are NaN
                if (!STATES)
                    x.q.store(sm.q[st][0], sm.q[st][1], r, {row_exponent(mq[0]), row_exponent(mq[1])}, tile_piece<DK>);
                x.k.store(sm.k[st][0], sm.k[st][1], r, {row_exponent(mk[0]), row_exponent(mk[1])}, tile_piece<DK>);
                if (lane < 2) {
                    if (!STATES) sm.mq[st][r + lane] = lane ? mq[1] : mq[0];
                    sm.mk[st][r + lane] = lane ? mk[1] : mk[0];
                }
            };
#pragma unroll 1
            for (int j = 0; j < STEPS; j += 2) {
                read(step[1], c * STEPS + j + 1);
                convert(step[0], j);
                read(step[0], c * STEPS + j + 2);
                convert(step[1], j + 1);
            }
            fence_async_smem();
            arrive(sm.qk_full[st]);
        }
    } else if (w < kWarpE) {
        // ------------------------------------------------------------ values
        const int quarter = w & 3, column = 32 * quarter + lane;   // tensor memory lanes of this warp
        const uint32_t lanes = tmem + ((uint32_t)(32 * quarter) << 16);
        const bool mine = quarter < QUARTERS;
        int asked = 0;
        auto request = [&](int c) {   // the values of a chunk, its queries and keys as far as L2
            if (c < chunks && w == kWarpV && !__any_sync(0xffffffffu, *abort_flag)) {
                asked = c + 1;
                if (lane == 0) {
                    if (!STATES) tma_prefetch_2d(&map_q, hk * DK, seg.row0 + c * C);
                    tma_prefetch_2d(&map_k, hk * DK, seg.row0 + c * C);
                    mbar_arrive_expect_tx(&sm.values[c & 1], C * DV * 4);
                    tma_load_2d(sm.v[c & 1], &map_v, h * p.Dv + col0, seg.row0 + c * C, &sm.values[c & 1]);
                    if (c + 1 < chunks) tma_prefetch_2d(&map_v, h * p.Dv + col0, seg.row0 + (c + 1) * C);
                }
                __syncwarp();
            }
        };
        request(0);
        request(1);
        for (int c = 0; c < chunks; ++c) {
            if (!STATES) {
                if (w == kWarpV) {
                    wait(sm.values[c & 1], c >> 1);
                    wait(sm.fact[c & 3], c >> 2);
                    if (c) wait(sm.o_full, c - 1);   // the last chunk's MMAs have read what is written now
                }
                sync(kWarpV);
                tc_fence_after();
                if (mine) {
#pragma unroll 1
                    for (int b = 0; b < C / 8; ++b) value_parts(sm, sm.f[c & 3], sm.f[c & 3].vscale, c, 8 * b, column, lanes + kVh + 4 * b);
                    tmem_wait_st();
                    tc_fence_before();
                    arrive(sm.v_full);
                }
                sync(kWarpV);   // the values are read before the next ones come, by the state's warps as well
            }
            if (w == kWarpV) wait(sm.w_full[c & 1], c >> 1);
            request(c + 2);
        }
        // copies still on their way when a wait has run out
        for (int i = max(0, asked - 2); i < asked; ++i) mbar_wait_for(&sm.values[i & 1], (i >> 1) & 1, nullptr, 1000000ull);
    } else {
        // ------------------------------------------------------------ state and output
        const int quarter = w & 3, part = (w - kWarpE) >> 2, column = 32 * quarter + lane;
        const uint32_t lanes = tmem + ((uint32_t)(32 * quarter) << 16);
        constexpr int N = DK / 4;   // values of the state of a thread: rows part * N ..
        const bool cut = p.length != 0 && seg.count > 1;
        // (starts that decrease could make more segments than there is room for)
        const int start = min(seg.place - seg.seg + seg.count, p.segments) - 1;   // where `few` keeps what the sequence starts from
        const int slot = any ? a.slots[seg.seq] : -1;
        const bool kept = slot >= 0 && slot < a.n;
        const long long place = (long long)part * N * p.Dv + col0 + column, size = (long long)DK * p.Dv;
        auto local = [&](int number) { return p.local + ((long long)number * a.Hv + h) * size + place; };
        float *pool = a.state + ((long long)(kept ? slot : 0) * a.Hv + h) * size + place;
        const bool mine = any && quarter < QUARTERS;
        const int last = mine ? chunks : 0;
        const bool zeros = !kept || (a.fresh && a.fresh[seg.seq] != 0);
        float S[N];
#pragma unroll
        for (int i = 0; i < N; ++i) S[i] = 0.0f;
        // The registers hold S / 2^exponent, the exponent kept while the column's largest magnitude stays within
        // 2^8 .. 2^15, set anew for 2^11 .. 2^12 when it leaves.  (STATES: all of them count in the factors' `scale`.)
        int exponent = 0;
        // 2^units of a head's decays as two factors, since a large state may stay a number below what fp32 holds of it
        auto factors_of = [](long long units, float &rest) {
            const int n = whole(units), first = max(-126, min(126, n));
            rest = n < -252 ? 0.0f : pow2(min(126, n - first));
            return exp2_fast(broken(units)) * pow2(first);
        };
        if (STATES) {
            // what the sequence starts from, before its last segment replaces it
            if (mine && p.few && seg.seg == 0)
#pragma unroll 4
                for (int i = 0; i < N; ++i)
                    local(start)[(long long)i * p.Dv] = zeros ? 0.0f : pool[(long long)i * p.Dv];
        } else if (mine && (cut || !zeros)) {
            const float *from = !cut ? pool : local(p.few ? start : seg.place);
#pragma unroll
            for (int i = 0; i < N; ++i) S[i] = from[(long long)i * p.Dv];
            for (int j = cut && p.few ? seg.place - seg.seg : seg.place; j < seg.place; ++j) {
                float rest;
                const float f = factors_of(p.decay[(long long)j * a.Hv + h], rest);
                const float *own = local(j);
                if (rest != 1.0f)
#pragma unroll
                    for (int i = 0; i < N; ++i) S[i] *= rest;
#pragma unroll
                for (int i = 0; i < N; ++i) S[i] = __fmaf_rn(f, S[i], own[(long long)i * p.Dv]);
            }
        }
        long long G = 0;
        auto limit = [](int to) { return max(-126, min(126, to)); };
        // the state's parts for the next product with the queries; between: what has to be over before they are written
        auto publish = [&](auto between) {
            float most = 0.0f;
#pragma unroll
            for (int i = 0; i < N; ++i) most = fmaxf(most, fabsf(S[i]));   // (a NaN needs no scale)
            sm.smax[part][column] = __float_as_uint(most);
            between();
            sync(kWarpE);
            tc_fence_after();
            const uint32_t m = max(max(sm.smax[0][column], sm.smax[1][column]), max(sm.smax[2][column], sm.smax[3][column]));
            if (__any_sync(0xffffffffu, m < 0x43800000u || m >= 0x47000000u)) {
                const int to = max(exponent - 126, limit(exponent + exponent_of(m) - 11));
                const float s = pow2(m == 0u ? 0 : exponent - to);
#pragma unroll
                for (int i = 0; i < N; ++i) S[i] *= s;
                exponent = m == 0u ? kEmpty : to;
            }
#pragma unroll
            for (int b = 0; b < N / 16; ++b) {
                uint32_t ph[8], pl[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) split2(make_float2(S[16 * b + 2 * i], S[16 * b + 2 * i + 1]), ph[i], pl[i]);
                tmem_st8(lanes + kSh + part * (N / 2) + 8 * b, ph);
                tmem_st8(lanes + kSl + part * (N / 2) + 8 * b, pl);
            }
            tmem_wait_st();
            tc_fence_before();
            arrive(sm.s_full);
        };
        // the values weighted for the state, sixteen tokens a warp
        auto weighted = [&](int c) {
            if (w == kWarpE) {
                wait(sm.values[c & 1], c >> 1);
                wait(sm.fact[c & 3], c >> 2);
            }
            sync(kWarpE);
            tc_fence_after();
#pragma unroll 1
            for (int b = 0; b < 2; ++b)
                value_parts(sm, sm.f[c & 3], sm.f[c & 3].wscale, c, 16 * part + 8 * b, column, lanes + kWh + 8 * part + 4 * b);
            tmem_wait_st();
            tc_fence_before();
            arrive(sm.w_full[c & 1]);
        };
        if (!STATES && last) publish([] {});
        if (last) weighted(0);
        for (int c = 0; c < last; ++c) {
            const Factors &f = sm.f[c & 3];
            if (w == kWarpE) wait(sm.u_full, c);
            sync(kWarpE);   // (the maxima of the last chunk have been read, too)
            tc_fence_after();
            if (STATES && c + 1 < chunks) weighted(c + 1);
            const int was = exponent;              // of the state that O1 was made with
            float keep, add;
            if (STATES) {
                keep = f.keep;
                add = f.add;
            } else {
                const Factors::Update update = f.update;
                keep = update.keep;
                int n = update.low - exponent;
                // Out of its scale the state's exponent goes with the decay, or as far as the sums need.  No farther, since a
                // column of values that are zero keeps its state (as far as 2^-210 of the sums).
                if (__any_sync(0xffffffffu, (unsigned)-n > update.range)) {
                    const bool empty = exponent == kEmpty;
                    const int grow = f.grow, reach = f.reach, from = exponent + grow;
                    exponent = limit(empty ? reach + 22 : max(from, reach - 84));
                    n = max(-127, min(127, reach - exponent)) - kReach;
                    keep = empty ? 0.0f : times_pow2(update.gpart, from - exponent);
                }
                add = update.gpart * pow2(n + kReach);           // (pow2(-127) is 0)
            }
#pragma unroll
            for (int b = 0; b < N / 16; ++b) {
                uint32_t u[16];
                tmem_ld16(lanes + (STATES && (c & 1) ? kU2 : kU) + part * N + 16 * b, u);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                    float *x = &S[16 * b + i];
                    const float2 y = fma2(make_float2(add, add), make_float2(__uint_as_float(u[i]), __uint_as_float(u[i + 1])),
                                          mul2(make_float2(keep, keep), make_float2(x[0], x[1])));
                    x[0] = y.x;
                    x[1] = y.y;
                }
            }
            if (STATES) G = clamp_units(G + f.G);
            tc_fence_before();
            arrive(sm.u_empty[STATES ? c & 1 : 0]);
            if (STATES) continue;
            if (c + 1 < chunks) {
                weighted(c + 1);
                // the queries' product with the last parts is done, and so is their place
                publish([&] {
                    if (w == kWarpE) wait(sm.qk_empty[c & 1], c >> 1);
                });
            }
            if (w == kWarpE) wait(sm.o_full, c);
            sync(kWarpE);
            tc_fence_after();
            const int n = seg.row1 - seg.row0 - c * C - 16 * part;
            char *out = reinterpret_cast<char *>(a.out + (seg.row0 + c * C + 16 * part) * a.out_stride + (long long)h * p.Dv +
                                                 col0 + column);
            const int os = 4 * (int)a.out_stride;
            const bool far = __any_sync(0xffffffffu, f.wide || was > 20);
            const float xs = pow2(max(-127, was));
            if (far) far_outputs(f, 16 * part, lanes + kO1 + 16 * part, lanes + kO2 + 16 * part, out, os, n, was);
#pragma unroll 1
            for (int b = far ? 2 : 0; b < 2; ++b) {
                uint32_t o1[8], o2[8];
                tmem_ld8(lanes + kO1 + 16 * part + 8 * b, o1);
                tmem_ld8(lanes + kO2 + 16 * part + 8 * b, o2);
                tmem_wait_ld();
                float y[8];
#pragma unroll
                for (int i = 0; i < 8; i += 4) {
                    const float4 f1 = *reinterpret_cast<const float4 *>(&f.f1[16 * part + 8 * b + i]),
                                 f2 = *reinterpret_cast<const float4 *>(&f.f2[16 * part + 8 * b + i]);
                    auto two = [&](int j, float u0, float u1, float v0, float v1) {
                        const float2 state = mul2(make_float2(__uint_as_float(o1[j]), __uint_as_float(o1[j + 1])), make_float2(xs, xs));
                        const float2 r = fma2(make_float2(u0, u1), make_float2(__uint_as_float(o2[j]), __uint_as_float(o2[j + 1])),
                                              mul2(make_float2(v0, v1), state));
                        y[j] = r.x;
                        y[j + 1] = r.y;
                    };
                    two(i, f1.x, f1.y, f2.x, f2.y);
                    two(i + 2, f1.z, f1.w, f2.z, f2.w);
                }
                if (8 * b + 8 <= n) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) *reinterpret_cast<float *>(out + (long long)(8 * b + i) * os) = y[i];
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (8 * b + i < n) *reinterpret_cast<float *>(out + (long long)(8 * b + i) * os) = y[i];
                }
            }
            tc_fence_before();
            arrive(sm.o_empty);
        }
        if (mine && (STATES || (kept && seg.last))) {
            float rest = 1.0f;
            const float f = STATES ? factors_of(sm.f[(chunks - 1) & 3].scale, rest) : pow2(max(-127, exponent));
#pragma unroll
            for (int i = 0; i < N; ++i) (STATES ? local(seg.place) : pool)[(long long)i * p.Dv] = S[i] * f * rest;
        }
        if (STATES && any && tile == 0 && w == kWarpE && lane == 0) p.decay[(long long)seg.place * a.Hv + h] = G;
    }
    tc_fence_before();
    __syncthreads();
    if (w == kWarpM) {
        if (*abort_flag) {   // MMAs still on their way when a wait has run out
            if (elect_one()) mma_commit(&sm.drained);
            __syncwarp();
            mbar_wait_for(&sm.drained, 0, nullptr, 1000000ull);
        }
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int DK, int DV, bool STATES>
cudaError_t launch(const PromptArgs &p, cudaStream_t st)
{
    static std::atomic<bool> ready[64];
    auto *kernel = linear_prompt_tc_kernel<DK, DV, STATES>;
    constexpr int smem = sizeof(Smem<DK, DV>) + 1024;
    static_assert(smem <= 227 * 1024, "a CTA's shared memory");
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (!ready[dev & 63].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        ready[dev & 63].store(true, std::memory_order_release);
    }
    // segments that are not the last of their sequence are full ones
    const long long ctas = (long long)(STATES ? p.a.T / p.length : p.segments) * p.a.Hv * (p.Dv / DV);
    PromptArgs args = p;
    args.status = device_status_word();
    args.scale = std::frexp(p.a.scale, &args.scale_exponent);
    const LinearAttnArgs &a = p.a;
    CUtensorMap map[3];
    auto rows = [&](int i, const float *x, int heads, int D, long long stride, int box) {
        const uint64_t cols = (uint64_t)heads * D;
        return make_tmap_rows_f32(&map[i], x, cols, a.T, a.T > 1 ? (uint64_t)stride : cols, box, C);
    };
    if ((e = rows(0, a.q, a.Hk, DK, a.q_stride, DK)) != cudaSuccess || (e = rows(1, a.k, a.Hk, DK, a.k_stride, DK)) != cudaSuccess ||
        (e = rows(2, a.v, a.Hv, p.Dv, a.v_stride, DV)) != cudaSuccess)
        return e;
    return launch_pdl(kernel, dim3((unsigned)ctas), dim3(kThreads), smem, st, args, map[0], map[1], map[2]);
}

template <int DK, int DV>
cudaError_t launch_either(const PromptArgs &p, bool states, cudaStream_t st)
{
    return states ? launch<DK, DV, true>(p, st) : launch<DK, DV, false>(p, st);
}

}  // namespace

cudaError_t launch_linear_prompt_tc(const PromptArgs &p, int Dk, bool states, cudaStream_t st)
{
    if (Dk == 64) return p.Dv == 64 ? launch_either<64, 64>(p, states, st) : launch_either<64, 128>(p, states, st);
    return p.Dv == 64 ? launch_either<128, 64>(p, states, st) : launch_either<128, 128>(p, states, st);
}

}  // namespace zq
