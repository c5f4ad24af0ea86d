// head_norm_rope.cu -- RMSNorm of query and key heads, rotation by position
// and the write into the paged cache, in one pass (MIInfer README, "Status":
// the heads' RMS norms in one launch ahead of the cached attention).
//
// A warp owns one token and `chunk` of its Hq + 2 Hk head rows.  Lane l holds
// the D / 32 neighbouring values l * D / 32 .. of a row, so a row is one
// coalesced access, its sum of squares five shuffles, and the partner value of
// the split pairing (p, p + rot / 2) one shuffle per value from a fixed lane.
// A lane's angles belong to its token and columns, not to the head: they are
// computed once per warp and used for all of its rows.
//
// The angle: table entry x position modulo 2^64 is the phase in turns (the
// integer product wraps exactly where the angle does, and is right to 2^-32 turns),
// its top 32 bits as a signed fraction, rounded to fp32 (2^-26 turns at most), give
// sincospi an argument in [-1, 1]: no range reduction and no fp64, which is slow
// on this GPU.
//
// HBM bound for long prompts: 4 D (2 Hq + 2 Hk) + 2 es D Hk bytes per token;
// launch bound for a few tokens.  Measured in a graph: 4096 tokens of 48 + 8 + 8
// heads of 128 to an f16 cache 43.0 us, 5.9 TB/s (0.86 of the measured copy rate);
// 777 tokens of 24 + 4 + 4 heads of 256 to an e4m3 cache 11.0 us, 4.2 TB/s (latency:
// one round of 19 warps an SM with two rows each on their way are 38 KB, less than
// the copy rate wants, between a warp's start and end; issue slots 39 % busy);
// 61 tokens 3.3 us, one token 2.5 us.
#include <atomic>

#include "zq_async.cuh"
#include "zq_internal.cuh"
#include "zq_kv.cuh"

namespace zq {
namespace {

constexpr int kThreads = 128;   // four warps per CTA
constexpr int kBatch = 2;       // rows of a warp in flight together (four cost 256-wide rows a third of their warps)

template <int E>
__device__ __forceinline__ void load_row(const float *p, float (&x)[E])
{
    if constexpr (E == 2) {
        const float2 f = *reinterpret_cast<const float2 *>(p);
        x[0] = f.x;
        x[1] = f.y;
    } else {
#pragma unroll
        for (int v = 0; v < E / 4; ++v) {
            const float4 f = reinterpret_cast<const float4 *>(p)[v];
            x[4 * v] = f.x;
            x[4 * v + 1] = f.y;
            x[4 * v + 2] = f.z;
            x[4 * v + 3] = f.w;
        }
    }
}

template <int E>
__device__ __forceinline__ void store_row(float *p, const float (&x)[E])
{
    if constexpr (E == 2) {
        *reinterpret_cast<float2 *>(p) = make_float2(x[0], x[1]);
    } else {
#pragma unroll
        for (int v = 0; v < E / 4; ++v)
            reinterpret_cast<float4 *>(p)[v] = make_float4(x[4 * v], x[4 * v + 1], x[4 * v + 2], x[4 * v + 3]);
    }
}

// x times 1 / scale rounded to the cache type, E neighbouring values
template <int TYPE, int E>
__device__ __forceinline__ void store_cache(void *dst, const float (&x)[E], float inverse)
{
    float y[E];
#pragma unroll
    for (int e = 0; e < E; ++e) y[e] = x[e] * inverse;
    if constexpr (TYPE == ZQ_E4M3) {
        if constexpr (E == 2) {
            *static_cast<uint16_t *>(dst) = (uint16_t)kv_pack2<TYPE>(y[0], y[1]);
        } else {
#pragma unroll
            for (int v = 0; v < E / 4; ++v)
                static_cast<uint32_t *>(dst)[v] =
                    kv_pack2<TYPE>(y[4 * v], y[4 * v + 1]) | kv_pack2<TYPE>(y[4 * v + 2], y[4 * v + 3]) << 16;
        }
    } else if constexpr (E == 2) {
        *static_cast<uint32_t *>(dst) = kv_pack2<TYPE>(y[0], y[1]);
    } else if constexpr (E == 4) {
        *static_cast<uint2 *>(dst) = make_uint2(kv_pack2<TYPE>(y[0], y[1]), kv_pack2<TYPE>(y[2], y[3]));
    } else {
        *static_cast<uint4 *>(dst) = make_uint4(kv_pack2<TYPE>(y[0], y[1]), kv_pack2<TYPE>(y[2], y[3]),
                                                kv_pack2<TYPE>(y[4], y[5]), kv_pack2<TYPE>(y[6], y[7]));
    }
}

template <int D, int TYPE, bool INTER>
__global__ void __launch_bounds__(kThreads) head_norm_rope_kernel(const __grid_constant__ HeadNormRopeArgs a)
{
    constexpr int E = D / 32;
    pdl_wait();   // q/k/v, positions and slots come from earlier kernels
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    // (a shuffle tells the compiler that the whole warp has the value: token, rows and addresses are then computed
    // once a warp, in uniform registers)
    const int w = blockIdx.x * (kThreads / 32) + __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    const int t = w / a.chunks;
    if (t >= a.T) return;
    const int keys = a.Hq, values = a.Hq + a.Hk, rows = a.Hq + 2 * a.Hk;   // rows: queries, keys, values
    const int r0 = (w - t * a.chunks) * a.chunk, r1 = min(rows, r0 + a.chunk);
    const int col = lane * E;

    const float *q = a.q + (long long)t * a.q_stride + col;
    const float *k = a.k + (long long)t * a.k_stride + col, *v = a.v + (long long)t * a.v_stride + col;
    auto src = [&](int r) {
        return r < keys ? q + r * D : r < values ? k + (r - keys) * D : v + (r - values) * D;
    };
    float x[kBatch][E];
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
        if (r0 + u < r1) load_row(src(r0 + u), x[u]);

    const bool qk = r0 < values;   // this warp has rows to norm and rotate
    float gq[E], gk[E], cs[E], sn[E];
    int partner = lane;
    const bool turned = qk && col < a.rot;
    const int slot = __shfl_sync(0xffffffffu, a.slots[t], 0);
    if (qk) {
        if (a.gamma_q) load_row(a.gamma_q + col, gq);
        if (a.gamma_k) load_row(a.gamma_k + col, gk);
    }
    if (qk && a.rot) {
        const int half = a.rot >> 1;
        const bool second = !INTER && col >= half;
        if (!INTER && turned) partner = second ? lane - half / E : lane + half / E;
        // the positions are read beside the entries that choose between them
        const int at0 = a.pos[t];
        const int at1 = a.axes > 1 ? a.pos[(long long)a.T + t] : at0;
        const int at2 = a.axes > 2 ? a.pos[2LL * a.T + t] : at1;
        auto angle = [&](int pair, float &s, float &c) {
            const uint64_t entry = a.table[pair];
            const int ax = (int)(entry & 3u);
            const int64_t at = ax == 0 ? at0 : ax == 1 ? at1 : at2;
            const uint64_t turns = (entry & ~(uint64_t)3) * (uint64_t)at;
            // top 32 bits as a signed fraction of a turn, times two: the argument in half turns
            sincospif((float)(int32_t)(turns >> 32) * 0x1p-31f, &s, &c);
        };
        auto pair_of = [&](int e) { return INTER ? (col + e) >> 1 : col + e - (second ? half : 0); };
        if (a.rot <= 64) {   // at most one pair a lane: each angle once, passed on (an 8 times smaller share of
                             // 256-wide rows with 64 turned values than an angle for every value)
            float s, c;
            angle(min(lane, half - 1), s, c);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                sn[e] = __shfl_sync(0xffffffffu, s, pair_of(e) & 31);
                cs[e] = __shfl_sync(0xffffffffu, c, pair_of(e) & 31);
            }
        } else if (turned) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                if (INTER && (e & 1)) {   // the pair's first value has the angle already
                    cs[e] = cs[e - 1];
                    sn[e] = sn[e - 1];
                } else {
                    angle(pair_of(e), sn[e], cs[e]);
                }
            }
        }
        // the first of a pair takes -sin of its partner
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (INTER ? !(e & 1) : !second) sn[e] = -sn[e];
    }
    __syncwarp();
    const bool keep = slot >= 0 && slot < a.nslots;
    // the token's place in the cache, at key head 0; a head further is a page's rows further
    const long long place =
        keep ? ((((long long)(slot >> a.page_shift) * a.Hk) << a.page_shift) + (slot & ((1 << a.page_shift) - 1))) * D : 0;
    char *kc = static_cast<char *>(a.kc) + (place + col) * KvBytes<TYPE>::value;
    char *vc = static_cast<char *>(a.vc) + (place + col) * KvBytes<TYPE>::value;
    const long long head = ((long long)D << a.page_shift) * KvBytes<TYPE>::value;
    float *out = a.q_out + (long long)t * a.q_out_stride + col;
    const float k_inverse = 1.0f / a.k_scale, v_inverse = 1.0f / a.v_scale;

    auto row = [&](int r, float(&x)[E]) {
        float y[E];
#pragma unroll
        for (int e = 0; e < E; ++e) y[e] = x[e];
        if (r + kBatch < r1) load_row(src(r + kBatch), x);   // the row kBatch further on takes its place
        if (r >= values) {
            if (keep) store_cache<TYPE, E>(vc + (r - values) * head, y, v_inverse);
            return;
        }
        const bool is_q = r < keys;
        if (is_q ? a.gamma_q != nullptr : a.gamma_k != nullptr) {
            float ss = 0.0f;
#pragma unroll
            for (int e = 0; e < E; ++e) ss = __fmaf_rn(y[e], y[e], ss);
            ss = warp_sum(ss);
            const float rms = rsqrtf(__fmaf_rn(ss, 1.0f / D, a.eps));
#pragma unroll
            for (int e = 0; e < E; ++e) y[e] = y[e] * rms * (is_q ? gq[e] : gk[e]);
        }
        if (a.rot) {
            float z[E];
#pragma unroll
            for (int e = 0; e < E; ++e) z[e] = INTER ? y[e ^ 1] : __shfl_sync(0xffffffffu, y[e], partner);
#pragma unroll
            for (int e = 0; e < E; ++e) y[e] = turned ? __fmaf_rn(y[e], cs[e], z[e] * sn[e]) : y[e];
        }
        if (is_q) store_row(out + r * D, y);
        else if (keep) store_cache<TYPE, E>(kc + (r - keys) * head, y, k_inverse);
    };
    int r = r0;
    for (; r + kBatch <= r1; r += kBatch)
#pragma unroll
        for (int u = 0; u < kBatch; ++u) row(r + u, x[u]);
#pragma unroll
    for (int u = 0; u < kBatch - 1; ++u)
        if (r + u < r1) row(r + u, x[u]);
}

// Rows of a warp: a warp's start (slot, positions, angles, gamma) costs about as
// much as two rows, and a second round of warps as much as the first, so as few
// rows as let all warps run at the same time, between 2 and 16 (1 for a few
// tokens, where latency counts).  777 tokens of 32 rows of 256: 8 rows, one
// round, 11.1 us; 4 rows, two rounds, 12.6; 16 rows 13.7.  500 of 64 rows of 128: 7 rows
// 8.2 us, 4 9.1, 16 10.2.  Rows of up to 128 want 16 warps an SM and no more while a
// warp has up to ten rows (200 tokens of 64 rows: 6 rows 4.7 us, 3 rows and all the
// SM holds 5.2); rows of 256 all of it (400 tokens of 32 rows: 4 rows 6.0, 6 7.2).
template <int D, int TYPE, bool INTER>
cudaError_t launch_kernel(const HeadNormRopeArgs &args, cudaStream_t st)
{
    static std::atomic<int> held;   // CTAs that an SM holds, the same on every device of the architecture
    auto *kernel = head_norm_rope_kernel<D, TYPE, INTER>;
    int per_sm = held.load(std::memory_order_relaxed);
    if (!per_sm) {
        const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, kThreads, 0);
        if (e != cudaSuccess) return e;
        if (per_sm < 1) per_sm = 1;
        held.store(per_sm, std::memory_order_relaxed);
    }
    HeadNormRopeArgs a = args;
    const long long rows = a.Hq + 2LL * a.Hk, sms = num_sms();
    auto chunk_of = [&](long long warps) {   // rows of a warp when so many share the rows
        const long long chunks = warps / a.T < 1 ? 1 : warps / a.T;
        return (rows + chunks - 1) / chunks;
    };
    long long chunk = chunk_of(16 * sms);
    if (D == 256 || chunk > 10) chunk = chunk_of(sms * per_sm * (kThreads / 32));
    const long long least = a.T * rows <= 8 * sms ? 1 : 2;
    chunk = chunk < least ? least : chunk > 16 ? 16 : chunk;
    a.chunk = (int)chunk;
    a.chunks = (int)((rows + chunk - 1) / chunk);
    const long long warps = (long long)a.T * a.chunks;
    return launch_pdl(kernel, dim3((unsigned)((warps + kThreads / 32 - 1) / (kThreads / 32))), dim3(kThreads), 0, st, a);
}

template <int D, int TYPE>
cudaError_t launch_one(const HeadNormRopeArgs &a, cudaStream_t st)
{
    return a.interleaved ? launch_kernel<D, TYPE, true>(a, st) : launch_kernel<D, TYPE, false>(a, st);
}

template <int D>
cudaError_t launch_type(const HeadNormRopeArgs &a, int type, cudaStream_t st)
{
    switch (type) {
    case ZQ_F16: return launch_one<D, ZQ_F16>(a, st);
    case ZQ_BF16: return launch_one<D, ZQ_BF16>(a, st);
    default: return launch_one<D, ZQ_E4M3>(a, st);
    }
}

}  // namespace

cudaError_t launch_head_norm_rope(const HeadNormRopeArgs &a, int D, int type, cudaStream_t st)
{
    switch (D) {
    case 64: return launch_type<64>(a, type, st);
    case 128: return launch_type<128>(a, type, st);
    default: return launch_type<256>(a, type, st);
    }
}

}  // namespace zq
