// lora.cu -- low-rank adapters of many requests beside a shared projection:
//   y[t] = base[t] + scale_a B_a (A_a x_t),  a = ids[t],
// on the Q8_1 activations the shared projection reads (ZINC docs "ROCm
// backend": Q8 activations packed once and reused by the projections).
//
// Two kernels, one after the other: h_t = A_a x_t split over K, then the
// expansion of h by B_a onto base.  Bound: HBM, the adapters once, and base and
// y (8 B N bytes), which dominate; a few tokens are launch bound.
//
// Tokens come in tiles of 32.  Each warp finds the distinct adapters of its tile
// itself (one match of the lanes' ids) and takes the members of one after the
// other as the columns of its MMAs, eight at a time, so a prompt's tokens share
// each adapter row and a decode batch reads each of its adapters once a tile; no
// sorting pass, no plan to keep, any mixture of both.
//
// First kernel: m16n8k16 with adapter rows as the 16-row operand and tokens as
// the columns.  The order of K inside a step is free, so lane 4g + c loads 8
// neighbouring values of rows g and g + 8, and of token g's codes, which are
// fragments as they stand.  Codes are whole numbers of at most 8 bits, exact in
// binary16 and bf16: a Q8_1 block's products are summed by the tensor core and
// scaled by the block's d in fp32.  Warps split the blocks of a CTA's K range
// and add up in a fixed tree, the CTAs of a cluster add up their ranges in order
// through distributed shared memory, the second kernel the clusters'.
//
// Second kernel: rows of B_a are the 16-row operand, tokens the columns; h is
// two 16-bit parts (binary16 after scaling the token's row to [1, 2), 2^-22 of
// its largest value; bf16 2^-17).  The rows of two MMAs are dealt so that a
// lane holds four neighbouring outputs of its tokens: base and y move as 16-byte
// pieces.
#include "zq_async.cuh"
#include "zq_cluster.cuh"
#include "zq_internal.cuh"
#include "zq_kv.cuh"

namespace zq {
namespace {

constexpr int kTokens = 32;      // tokens of a tile: a warp's lanes, and four MMAs' columns
constexpr int kQ = kTokens / 8;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kDownRows = 32;    // rows of A a CTA of the first kernel takes at most
constexpr int kCluster = 8;      // CTAs of a cluster at most, which add up their K ranges
constexpr int kParts = 4;        // sums the second kernel is left with at most
constexpr int kCols = 32 * kWarps;   // outputs of a CTA of the second kernel
constexpr unsigned kAll = 0xffffffffu;

template <int TYPE>
__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1)
{
    if constexpr (TYPE == ZQ_BF16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same onto zero
template <int TYPE>
__device__ __forceinline__ void mma16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1)
{
    if constexpr (TYPE == ZQ_BF16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%10,%10,%10,%10};"
                     : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%10,%10,%10,%10};"
                     : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// Four int8 codes to two pairs of the MMA's type, exactly: binary16 1024 + (q
// + 128) has the byte in its low bits.
template <int TYPE>
__device__ __forceinline__ void codes4(uint32_t w, uint32_t &lo, uint32_t &hi)
{
    const uint32_t u = w ^ 0x80808080u, off = 0x64806480u;   // 1152, twice
    const uint32_t p0 = __byte_perm(u, 0x64646464u, 0x4140), p1 = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 k = *reinterpret_cast<const __half2 *>(&off);
    const __half2 h0 = __hsub2(*reinterpret_cast<const __half2 *>(&p0), k);
    const __half2 h1 = __hsub2(*reinterpret_cast<const __half2 *>(&p1), k);
    if constexpr (TYPE == ZQ_F16) {
        lo = *reinterpret_cast<const uint32_t *>(&h0);
        hi = *reinterpret_cast<const uint32_t *>(&h1);
    } else {
        const float2 f0 = __half22float2(h0), f1 = __half22float2(h1);
        lo = kv_pack2<ZQ_BF16>(f0.x, f0.y);
        hi = kv_pack2<ZQ_BF16>(f1.x, f1.y);
    }
}

// A tile's tokens by adapter, found by each warp for itself.
struct Tile {
    int id;           // adapter of token `lane`, -1: none (or past the last token)
    uint32_t lead;    // tokens that are the first of their adapter

    __device__ __forceinline__ void open(const LoraArgs &a, int tile)
    {
        const int lane = threadIdx.x & 31, t = tile * kTokens + lane;
        id = t < a.B ? a.ids[t] : -1;
        if (id < 0 || id >= a.n) id = -1;
        const uint32_t same = __match_any_sync(kAll, id);   // by every lane, adapter or none
        lead = __ballot_sync(kAll, id >= 0 && __ffs((int)same) - 1 == lane);
    }
    // Tokens of the j-th adapter, and the adapter; 0: there are no more.
    __device__ __forceinline__ uint32_t members(int j, int &adapter) const
    {
        uint32_t m = lead;
        for (int i = 0; i < j && m; ++i) m &= m - 1;
        if (m == 0) return 0;
        adapter = __shfl_sync(kAll, id, __ffs((int)m) - 1);
        return __ballot_sync(kAll, id == adapter);
    }
};

// h[part][t][r] = sum over the part's K of A[a][r][k] x[t][k].  Grid: (tiles
// and groups of RR rows, adapters of a tile at the same time, K ranges); the
// ranges of a cluster are added up through distributed shared memory into one
// part.
template <int RR, int TYPE>
__global__ void __launch_bounds__(kThreads, 2) lora_down_kernel(const __grid_constant__ LoraArgs a)
{
    constexpr int kRows = RR < 16 ? 1 : RR / 16;   // 16-row operands
    __shared__ float red[kWarps / 2][kRows][kQ][4][32];
    __shared__ uint8_t list_s[kWarps][kTokens];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    pdl_wait();   // codes and ids come from earlier kernels
    pdl_launch_dependents();
    const int halves = a.R / RR, row0 = (int)blockIdx.x % halves * RR;
    const size_t tok0 = (size_t)(blockIdx.x / halves) * kTokens;
    Tile tile;
    tile.open(a, blockIdx.x / halves);
    const int blocks = a.K >> 5;
    const int b0 = min(blocks, (int)blockIdx.z * a.per_split), b1 = min(blocks, b0 + a.per_split);
    const int rank = blockIdx.z % a.cluster;
    float *h = a.h + (size_t)(blockIdx.z / a.cluster) * a.B * a.R + row0;

    for (int j = blockIdx.y;; j += gridDim.y) {
        int adapter;
        const uint32_t mask = tile.members(j, adapter);   // the same in all CTAs of the cluster
        if (mask == 0) return;
        const int members = __popc(mask);
        __syncwarp();
        if (mask >> lane & 1) list_s[warp][__popc(mask & ((1u << lane) - 1))] = (uint8_t)lane;
        __syncwarp();
        const int nq = (members + 7) / 8;   // MMAs' columns in use
        const char *A = a.A + (((size_t)adapter * a.R + row0 + g) * a.K + 8 * c) * 2;
        const size_t step = (size_t)8 * a.K * 2;   // eight rows on
        const int8_t *x[kQ];
        const uint16_t *d[kQ];
#pragma unroll
        for (int q = 0; q < kQ; ++q) {   // columns past the last member repeat it, unused
            const size_t t = tok0 + list_s[warp][min(members - 1, 8 * q + g)];
            x[q] = a.qs + t * a.K + 8 * c;
            d[q] = a.d + t * blocks;
        }
        float sum[kRows][kQ][4] = {};
        // the next block's values are on their way while this one's are used
        struct Block {
            uint4 w[kRows][2];
            uint2 codes[kQ];
            uint16_t d[kQ];
        };
        auto fetch = [&](int b, Block &f) {
            b = min(b, blocks - 1);   // past the end: read, not used
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                f.w[r][0] = __ldg(reinterpret_cast<const uint4 *>(A + 2 * r * step + 64 * (size_t)b));
                if (RR >= 16) f.w[r][1] = __ldg(reinterpret_cast<const uint4 *>(A + (2 * r + 1) * step + 64 * (size_t)b));
                else f.w[r][1] = make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int q = 0; q < kQ; ++q)
                if (q < nq) {
                    f.codes[q] = __ldg(reinterpret_cast<const uint2 *>(x[q] + 32 * b));
                    f.d[q] = __ldg(d[q] + b);
                }
        };
        auto use = [&](const Block &f) {
#pragma unroll
            for (int q = 0; q < kQ; ++q) {
                if (q >= nq) break;
                const float dq = h2f(f.d[q]);
                const float d0 = __shfl_sync(kAll, dq, 8 * c), d1 = __shfl_sync(kAll, dq, 8 * c + 4);
                uint32_t k0, k1, k2, k3;
                codes4<TYPE>(f.codes[q].x, k0, k1);
                codes4<TYPE>(f.codes[q].y, k2, k3);
#pragma unroll
                for (int r = 0; r < kRows; ++r) {
                    float p[4];
                    mma16_first<TYPE>(p, f.w[r][0].x, f.w[r][1].x, f.w[r][0].y, f.w[r][1].y, k0, k1);
                    mma16<TYPE>(p, f.w[r][0].z, f.w[r][1].z, f.w[r][0].w, f.w[r][1].w, k2, k3);
                    sum[r][q][0] += d0 * p[0];
                    sum[r][q][1] += d1 * p[1];
                    sum[r][q][2] += d0 * p[2];
                    sum[r][q][3] += d1 * p[3];
                }
            }
        };
        Block even, odd;
        if (b0 + warp < b1) fetch(b0 + warp, even);
        for (int b = b0 + warp; b < b1; b += 2 * kWarps) {
            fetch(b + kWarps, odd);
            use(even);
            fetch(b + 2 * kWarps, even);
            if (b + kWarps < b1) use(odd);
        }
        // the warps' sums, as a tree: the upper half hands over, the lower half adds
#pragma unroll
        for (int half = kWarps / 2; half >= 1; half >>= 1) {
            __syncthreads();
            if (warp >= half && warp < 2 * half) {
#pragma unroll
                for (int r = 0; r < kRows; ++r)
#pragma unroll
                    for (int q = 0; q < kQ; ++q)
                        if (q < nq)
#pragma unroll
                            for (int e = 0; e < 4; ++e) red[warp - half][r][q][e][lane] = sum[r][q][e];
            }
            __syncthreads();
            if (warp < half) {
#pragma unroll
                for (int r = 0; r < kRows; ++r)
#pragma unroll
                    for (int q = 0; q < kQ; ++q)
                        if (q < nq)
#pragma unroll
                            for (int e = 0; e < 4; ++e) sum[r][q][e] += red[warp][r][q][e][lane];
            }
        }
        if (warp == 0) {
#pragma unroll
            for (int r = 0; r < kRows; ++r)
#pragma unroll
                for (int q = 0; q < kQ; ++q)
                    if (q < nq)
#pragma unroll
                        for (int e = 0; e < 4; ++e) red[0][r][q][e][lane] = sum[r][q][e];
        }
        // each CTA of the cluster adds up its share of the values, in the order of the ranges
        __syncwarp();
        if (a.cluster > 1) cluster_sync();
        else __syncthreads();
        constexpr int kValues = kRows * kQ * 4 * 32;
        const int share = kValues / a.cluster;
        const uint32_t local = smem_u32(&red[0][0][0][0][0]);
        for (int i = rank * share + threadIdx.x; i < (rank + 1) * share; i += kThreads) {
            const int l = i & 31, e = i >> 5 & 3, q = i >> 7 & (kQ - 1), r = i / (kQ * 128);
            const int m = 8 * q + 2 * (l & 3) + (e & 1), row = 16 * r + 8 * (e >> 1) + (l >> 2);
            if (m < members && row < RR) {
                float v = 0.0f;
                for (int k = 0; k < a.cluster; ++k) v += ld_cluster_f32(cluster_addr(local + 4 * i, k));
                h[(tok0 + list_s[warp][m]) * a.R + row] = v;
            }
        }
        __syncwarp();
        if (a.cluster > 1) cluster_sync();   // the sums have been read
    }
}

// y[t] = base[t] + scale_a B_a h_t for the CTA's kCols outputs.  Grid: (tiles,
// column blocks, adapters of a tile at the same time).
template <int R, int TYPE>
__global__ void __launch_bounds__(kThreads) lora_up_kernel(const __grid_constant__ LoraArgs a)
{
    constexpr int kSteps = R < 16 ? 1 : R / 16;
    constexpr int kRun = R < 32 ? R / 4 : 8;   // neighbouring values of R that a lane's fragment takes
    __shared__ uint8_t list_s[kWarps][kTokens];
    __shared__ float back_s[kTokens];          // 2^e of a token's scaling
    __shared__ uint2 hi_s[kQ][kSteps][32], lo_s[kQ][kSteps][32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    const size_t tok0 = (size_t)blockIdx.x * kTokens;
    const int warp0 = blockIdx.y * kCols + 32 * warp;   // a whole warp has outputs, or none
    const int n0 = warp0 + 4 * g;                       // this lane's four outputs
    const bool vec = a.vec && warp0 + 32 <= a.N;        // they are all there, and aligned
    // The first kernel lets this one start only when all before it is complete:
    // ids, base and weights may be read ahead of the wait, h may not.
    Tile tile;
    tile.open(a, blockIdx.x);
    bool waited = false;

    for (int j = blockIdx.z;; j += gridDim.z) {
        int adapter;
        const uint32_t mask = tile.members(j, adapter);
        if (mask == 0) break;
        const int members = __popc(mask), groups = (members + 7) / 8;
        __syncthreads();   // the previous adapter's fragments have been used
        if (mask >> lane & 1) list_s[warp][__popc(mask & ((1u << lane) - 1))] = (uint8_t)lane;
        __syncwarp();
        uint32_t w[2][kSteps][4];   // fragments of rows n0 + 2i (upper) and n0 + 2i + 1 (lower)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const char *row = a.Bm + ((size_t)adapter * a.N + min(a.N - 1, n0 + i)) * R * 2 + kRun * 2 * c;
            if constexpr (R == 8) {
                w[i >> 1][0][i & 1] = __ldg(reinterpret_cast<const uint32_t *>(row));
                w[i >> 1][0][2 + (i & 1)] = 0;
            } else if constexpr (R == 16) {
                const uint2 f = __ldg(reinterpret_cast<const uint2 *>(row));
                w[i >> 1][0][i & 1] = f.x;
                w[i >> 1][0][2 + (i & 1)] = f.y;
            } else {
#pragma unroll
                for (int s = 0; s < kSteps / 2; ++s) {
                    const uint4 f = __ldg(reinterpret_cast<const uint4 *>(row + 64 * s));
                    w[i >> 1][2 * s][i & 1] = f.x;
                    w[i >> 1][2 * s][2 + (i & 1)] = f.y;
                    w[i >> 1][2 * s + 1][i & 1] = f.z;
                    w[i >> 1][2 * s + 1][2 + (i & 1)] = f.w;
                }
            }
        }
        float4 v[kQ][2];        // base of the members 8q + 2c, 8q + 2c + 1
#pragma unroll
        for (int q = 0; q < kQ; ++q)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int m = 8 * q + 2 * c + e;
                v[q][e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (a.base && m < members) {
                    const float *p = a.base + (tok0 + list_s[warp][m]) * a.base_stride + n0;
                    if (vec) {
                        v[q][e] = *reinterpret_cast<const float4 *>(p);
                    } else {
                        if (n0 < a.N) v[q][e].x = p[0];
                        if (n0 + 1 < a.N) v[q][e].y = p[1];
                        if (n0 + 2 < a.N) v[q][e].z = p[2];
                        if (n0 + 3 < a.N) v[q][e].w = p[3];
                    }
                }
            }
        if (!waited) {
            pdl_wait();
            pdl_launch_dependents();
            waited = true;
        }
        // h of the members: its parts in order, times the adapter's scale, as two 16-bit parts in the order of
        // the fragments; R / 4 neighbouring threads have a token, four values each
        const float scale = a.scales ? a.scales[adapter] : 1.0f;
        const int items = groups * 8 * (R / 4);
        for (int i = tid; i < (items + 31) / 32 * 32; i += kThreads) {
            const int m = i / (R / 4), r = i % (R / 4) * 4;
            float4 f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (m < members) {
                const float *h = a.h + (tok0 + list_s[warp][m]) * R + r;
#pragma unroll
                for (int s = 0; s < kParts; ++s)
                    if (s < a.parts) {
                        const float4 p = *reinterpret_cast<const float4 *>(h + (size_t)s * a.B * R);
                        f.x += p.x;
                        f.y += p.y;
                        f.z += p.z;
                        f.w += p.w;
                    }
            }
            float x[4] = {scale * f.x, scale * f.y, scale * f.z, scale * f.w};
            if (TYPE == ZQ_F16) {   // binary16 parts need the row near 1
                float amax = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
#pragma unroll
                for (int off = 1; off < R / 4; off <<= 1) amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, off));
                const int e = min(max((int)(__float_as_uint(amax) >> 23) - 127, -126), 126);
                const float down = __int_as_float((127 - e) << 23);
#pragma unroll
                for (int k = 0; k < 4; ++k) x[k] *= down;
                if (r == 0 && i < items) back_s[m] = __int_as_float((127 + e) << 23);
            }
            uint32_t hi[2], lo[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                hi[k] = kv_pack2<TYPE>(x[2 * k], x[2 * k + 1]);
                float2 y;
                if constexpr (TYPE == ZQ_BF16)
                    y = make_float2(__uint_as_float(hi[k] << 16), __uint_as_float(hi[k] & 0xffff0000u));
                else y = __half22float2(*reinterpret_cast<const __half2 *>(&hi[k]));
                lo[k] = kv_pack2<TYPE>(x[2 * k] - y.x, x[2 * k + 1] - y.y);
            }
            if (i < items) {
                const int q = m >> 3, l = (m & 7) * 4;
                if constexpr (R == 8) {   // two lanes' pairs; their second registers are zeros
                    hi_s[q][0][l + r / 2] = make_uint2(hi[0], 0);
                    hi_s[q][0][l + r / 2 + 1] = make_uint2(hi[1], 0);
                    lo_s[q][0][l + r / 2] = make_uint2(lo[0], 0);
                    lo_s[q][0][l + r / 2 + 1] = make_uint2(lo[1], 0);
                } else {                  // one lane's values of a step
                    const int s = R == 16 ? 0 : 2 * (r / 32) + (r >> 2 & 1);
                    const int to = l + (R == 16 ? r / 4 : (r & 31) >> 3);
                    hi_s[q][s][to] = make_uint2(hi[0], hi[1]);
                    lo_s[q][s][to] = make_uint2(lo[0], lo[1]);
                }
            }
        }
        __syncthreads();
        if (warp0 >= a.N) continue;
#pragma unroll
        for (int q = 0; q < kQ; ++q) {
            if (q >= groups) break;
            float p[2][4];
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                const uint2 hi = hi_s[q][s][lane], lo = lo_s[q][s][lane];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (s == 0) mma16_first<TYPE>(p[i], w[i][s][0], w[i][s][1], w[i][s][2], w[i][s][3], lo.x, lo.y);
                    else mma16<TYPE>(p[i], w[i][s][0], w[i][s][1], w[i][s][2], w[i][s][3], lo.x, lo.y);
                    mma16<TYPE>(p[i], w[i][s][0], w[i][s][1], w[i][s][2], w[i][s][3], hi.x, hi.y);
                }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int m = 8 * q + 2 * c + e;
                if (m < members) {
                    const float f = TYPE == ZQ_F16 ? back_s[m] : 1.0f;
                    float *to = a.y + (tok0 + list_s[warp][m]) * a.y_stride + n0;
                    const float4 y = make_float4(v[q][e].x + p[0][e] * f, v[q][e].y + p[0][2 + e] * f,
                                                 v[q][e].z + p[1][e] * f, v[q][e].w + p[1][2 + e] * f);
                    if (vec) {
                        *reinterpret_cast<float4 *>(to) = y;
                    } else {
                        if (n0 < a.N) to[0] = y.x;
                        if (n0 + 1 < a.N) to[1] = y.y;
                        if (n0 + 2 < a.N) to[2] = y.z;
                        if (n0 + 3 < a.N) to[3] = y.w;
                    }
                }
            }
            __syncwarp();
        }
    }
    if (!waited) {
        pdl_wait();
        pdl_launch_dependents();
    }
    // tokens without an adapter
    if (blockIdx.z == 0 && a.base != a.y) {
        const int col = blockIdx.y * kCols + tid;
        for (int i = 0; i < kTokens && tok0 + i < (size_t)a.B; ++i)
            if (__shfl_sync(kAll, tile.id, i) < 0 && col < a.N)
                a.y[(tok0 + i) * a.y_stride + col] = a.base ? a.base[(tok0 + i) * a.base_stride + col] : 0.0f;
    }
}

template <int R, int TYPE>
cudaError_t launch_rank(const LoraArgs &a, dim3 down, dim3 up, cudaStream_t st)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = down;
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 1;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = (unsigned)a.cluster;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    cudaError_t e = cudaLaunchKernelEx(&cfg, lora_down_kernel<(R < kDownRows ? R : kDownRows), TYPE>, a);
    if (e != cudaSuccess) return e;
    return launch_pdl(lora_up_kernel<R, TYPE>, up, dim3(kThreads), 0, st, a);
}

template <int TYPE>
cudaError_t launch_type(const LoraArgs &a, dim3 down, dim3 up, cudaStream_t st)
{
    switch (a.R) {
    case 8: return launch_rank<8, TYPE>(a, down, up, st);
    case 16: return launch_rank<16, TYPE>(a, down, up, st);
    case 32: return launch_rank<32, TYPE>(a, down, up, st);
    default: return launch_rank<64, TYPE>(a, down, up, st);
    }
}

// How K is cut: clusters of up to eight ranges of two blocks a warp or more,
// and up to four clusters where K is long and the tiles leave SMs idle.
struct Cut {
    int tiles, cluster, parts, per_split;
};
Cut cut_k(int B, int K, int R)
{
    const int blocks = K / 32, halves = R > kDownRows ? R / kDownRows : 1;
    const int wanted = (blocks + 2 * kWarps - 1) / (2 * kWarps);
    Cut c{(B + kTokens - 1) / kTokens, 1, 1, 0};
    while (c.cluster < kCluster && c.cluster < wanted) c.cluster *= 2;
    const int room = 2 * num_sms() / (c.tiles * halves * kCluster);
    while (c.parts < kParts && c.parts * 2 * kCluster <= wanted && c.parts * 2 <= room) c.parts *= 2;
    c.per_split = (blocks + c.cluster * c.parts - 1) / (c.cluster * c.parts);
    return c;
}

}  // namespace

size_t lora_workspace(int B, int K, int R) { return (size_t)cut_k(B, K, R).parts * B * R * sizeof(float); }

cudaError_t launch_lora(const LoraArgs &args, int type, cudaStream_t st)
{
    LoraArgs a = args;
    const Cut cut = cut_k(a.B, a.K, a.R);
    a.cluster = cut.cluster;
    a.parts = cut.parts;
    a.per_split = cut.per_split;
    const int splits = cut.cluster * cut.parts, halves = a.R > kDownRows ? a.R / kDownRows : 1;
    const int cols = (a.N + kCols - 1) / kCols;
    // adapters of a tile taken at the same time: as many as there can be, while
    // the grid is not several times the GPU already (a CTA takes the others in turn)
    auto at_once = [&](long long others) {
        const int most = min(a.n, min(a.B, kTokens));
        const long long n = 8LL * num_sms() / others;
        return (unsigned)(n < 1 ? 1 : n > most ? most : n);
    };
    const dim3 down(cut.tiles * halves, at_once((long long)cut.tiles * halves * splits), splits);
    const dim3 up(cut.tiles, cols, at_once((long long)cut.tiles * cols));
    return type == ZQ_BF16 ? launch_type<ZQ_BF16>(a, down, up, st) : launch_type<ZQ_F16>(a, down, up, st);
}

}  // namespace zq
