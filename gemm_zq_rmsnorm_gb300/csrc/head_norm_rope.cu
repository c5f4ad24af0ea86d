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
// integer product wraps exactly where the angle does), its top 32 bits as a
// signed fraction give sincospi an argument in [-1, 1): no range reduction
// and no fp64, whose rate on this GPU is 1/64 of fp32.
//
// HBM bound for long prompts: 4 D (2 Hq + 2 Hk) + 2 es D Hk bytes per token;
// launch bound for a few tokens.
#include "zq_async.cuh"
#include "zq_internal.cuh"
#include "zq_kv.cuh"

namespace zq {
namespace {

constexpr int kThreads = 128;   // four warps per CTA
constexpr int kBatch = 4;       // rows whose loads are in flight together

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

// x / scale rounded to the cache type, E neighbouring values
template <int TYPE, int E>
__device__ __forceinline__ void store_cache(void *dst, const float (&x)[E], float scale)
{
    float y[E];
#pragma unroll
    for (int e = 0; e < E; ++e) y[e] = scale == 1.0f ? x[e] : __fdiv_rn(x[e], scale);
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

template <int D, int TYPE>
__global__ void __launch_bounds__(kThreads) head_norm_rope_kernel(const __grid_constant__ HeadNormRopeArgs a)
{
    constexpr int E = D / 32;
    pdl_wait();   // q/k/v, positions and slots come from earlier kernels
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const long long w = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int t = (int)(w / a.chunks);
    if (t >= a.T) return;
    const int rows = a.Hq + 2 * a.Hk;
    const int r0 = (int)(w - (long long)t * a.chunks) * a.chunk;
    const int r1 = min(rows, r0 + a.chunk);
    const int col = lane * E;

    auto src = [&](int r) {
        if (r < a.Hq) return a.q + (long long)t * a.q_stride + (long long)r * D + col;
        if (r < a.Hq + a.Hk) return a.k + (long long)t * a.k_stride + (long long)(r - a.Hq) * D + col;
        return a.v + (long long)t * a.v_stride + (long long)(r - a.Hq - a.Hk) * D + col;
    };

    float x[kBatch][E];
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
        if (r0 + u < r1) load_row(src(r0 + u), x[u]);

    const bool qk = r0 < a.Hq + a.Hk;   // this warp has rows to norm and rotate
    float gq[E], gk[E], cs[E], sn[E];
    int partner = lane;
    const bool turned = qk && col < a.rot;
    if (qk) {
        if (a.gamma_q) load_row(a.gamma_q + col, gq);
        if (a.gamma_k) load_row(a.gamma_k + col, gk);
    }
    if (turned) {
        const int half = a.rot >> 1;
        const bool second = !a.interleaved && col >= half;
        if (!a.interleaved) partner = second ? lane - half / E : lane + half / E;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int p = a.interleaved ? (col + e) >> 1 : col + e - (second ? half : 0);
            const uint64_t entry = a.table[p];
            const int ax = min((int)(entry & 3u), a.axes - 1);
            const int64_t at = a.pos[(long long)ax * a.T + t];
            const uint64_t turns = (entry & ~(uint64_t)3) * (uint64_t)at;
            // top 32 bits as a signed fraction of a turn, times two: the argument in half turns
            sincospif((float)(int32_t)(turns >> 32) * 0x1p-31f, &sn[e], &cs[e]);
            // the first of a pair takes -sin of its partner
            if (a.interleaved ? !(e & 1) : !second) sn[e] = -sn[e];
        }
    }
    const long long slot = a.slots[t];
    const bool keep = slot >= 0 && slot < a.nslots;
    const int page = 1 << a.page_shift;
    const long long cache_page = keep ? slot >> a.page_shift : 0;
    const long long cache_off = keep ? slot & (page - 1) : 0;

    for (int rb = r0; rb < r1; rb += kBatch) {
        if (rb != r0) {
#pragma unroll
            for (int u = 0; u < kBatch; ++u)
                if (rb + u < r1) load_row(src(rb + u), x[u]);
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int r = rb + u;
            if (r >= r1) break;
            const bool is_q = r < a.Hq, is_v = r >= a.Hq + a.Hk;
            if (!is_v) {
                if (is_q ? a.gamma_q != nullptr : a.gamma_k != nullptr) {
                    float ss = 0.0f;
#pragma unroll
                    for (int e = 0; e < E; ++e) ss = __fmaf_rn(x[u][e], x[u][e], ss);
                    ss = warp_sum(ss);
                    const float rms = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(ss * (1.0f / D), a.eps)));
#pragma unroll
                    for (int e = 0; e < E; ++e) x[u][e] = x[u][e] * rms * (is_q ? gq[e] : gk[e]);
                }
                if (a.rot) {
                    float y[E];
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        const float other = __shfl_sync(0xffffffffu, x[u][e], partner);
                        y[e] = a.interleaved ? x[u][e ^ 1] : other;
                    }
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        if (turned) y[e] = __fmaf_rn(x[u][e], cs[e], y[e] * sn[e]);
                        else y[e] = x[u][e];
#pragma unroll
                    for (int e = 0; e < E; ++e) x[u][e] = y[e];
                }
            }
            if (is_q) {
                store_row(a.q_out + (long long)t * a.q_out_stride + (long long)r * D + col, x[u]);
            } else if (keep) {
                const int h = r - a.Hq - (is_v ? a.Hk : 0);
                const long long row = ((cache_page * a.Hk + h) << a.page_shift) + cache_off;
                char *dst = static_cast<char *>(is_v ? a.vc : a.kc) + (row * D + col) * KvBytes<TYPE>::value;
                store_cache<TYPE, E>(dst, x[u], is_v ? a.v_scale : a.k_scale);
            }
        }
    }
}

template <int D>
cudaError_t launch_type(const HeadNormRopeArgs &a, int type, dim3 grid, cudaStream_t st)
{
    switch (type) {
    case ZQ_F16: return launch_pdl(head_norm_rope_kernel<D, ZQ_F16>, grid, dim3(kThreads), 0, st, a);
    case ZQ_BF16: return launch_pdl(head_norm_rope_kernel<D, ZQ_BF16>, grid, dim3(kThreads), 0, st, a);
    default: return launch_pdl(head_norm_rope_kernel<D, ZQ_E4M3>, grid, dim3(kThreads), 0, st, a);
    }
}

}  // namespace

cudaError_t launch_head_norm_rope(const HeadNormRopeArgs &args, int D, int type, cudaStream_t st)
{
    HeadNormRopeArgs a = args;
    const long long rows = a.Hq + 2LL * a.Hk;
    // Enough warps for every SM first (one row each, latency counts), then up
    // to eight rows a warp, which share the warp's angles.
    long long chunk = a.T * rows / ((long long)num_sms() * 32);
    a.chunk = (int)(chunk < 1 ? 1 : chunk > 8 ? 8 : chunk);
    a.chunks = (int)((rows + a.chunk - 1) / a.chunk);
    const long long warps = (long long)a.T * a.chunks;
    const dim3 grid((unsigned)((warps + kThreads / 32 - 1) / (kThreads / 32)));
    switch (D) {
    case 64: return launch_type<64>(a, type, grid, st);
    case 128: return launch_type<128>(a, type, grid, st);
    default: return launch_type<256>(a, type, grid, st);
    }
}

}  // namespace zq
