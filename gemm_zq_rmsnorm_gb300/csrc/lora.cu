// lora.cu -- low-rank adapters of many requests beside a shared projection:
//   y[t] = base[t] + scale_a B_a (A_a x_t),  a = ids[t],
// on the Q8_1 activations the shared projection reads (ZINC docs "ROCm
// backend": Q8 activations packed once and reused by the projections).
//
// Two kernels, one after the other: h_t = A_a x_t split over K, then the
// expansion of h by B_a onto base.  Bound: HBM, the adapters once, and base and
// y (8 B N bytes), which dominate; a few tokens are launch bound.
//
// Tokens come in tiles of 64.  A CTA finds the distinct adapters of its tile
// itself (64 ids: one match per warp) and takes the members of one after the
// other as the columns of its MMAs, eight at a time, so a prompt's tokens share
// each adapter row and a decode batch reads each of its adapters once; no sorting
// pass, no plan to keep, any mixture of both.
//
// First kernel: m16n8k16 with adapter rows as the 16-row operand and tokens as
// the columns.  The order of K inside a step is free, so lane 4g + c loads 8
// neighbouring values of rows g and g + 8, and of token g's codes, which are
// fragments as they stand.  Codes are whole numbers of at most 8 bits, exact in
// binary16 and bf16: a Q8_1 block's products are summed by the tensor core and
// scaled by the block's d in fp32.  Warps split the blocks of a CTA's K range
// and add up in a fixed tree; K ranges are summed in order by the second kernel.
//
// Second kernel: rows of B_a are the 16-row operand, tokens the columns; h is
// two 16-bit parts (binary16 after scaling the token's row to [1, 2), 2^-22 of
// its largest value; bf16 2^-17).  The rows of two MMAs are dealt so that a
// lane holds four neighbouring outputs of its tokens: base and y move as 16-byte
// pieces.
#include "zq_async.cuh"
#include "zq_internal.cuh"
#include "zq_kv.cuh"

namespace zq {
namespace {

constexpr int kTokens = 64;      // tokens of a tile
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kGroup = 32;       // members a pass of the first kernel takes: four MMAs' columns
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

// The tile's tokens by adapter, in shared memory; every thread of the CTA.
struct Tile {
    int id[kTokens];              // adapter of a token, -1: none (or past the last token)
    uint32_t lead[2], member[2];  // tokens first of their adapter; tokens of the adapter at hand
    int list[kTokens];            // the latter, in order
};

__device__ __forceinline__ void tile_open(Tile &s, const LoraArgs &a, int tile)
{
    const int tid = threadIdx.x;
    int id = -1;
    if (tid < kTokens) {
        const int t = tile * kTokens + tid;
        if (t < a.B) id = a.ids[t];
        if (id < 0 || id >= a.n) id = -1;
        s.id[tid] = id;
    }
    __syncthreads();
    if (tid < kTokens) {
        const uint32_t same = __match_any_sync(kAll, id);   // by every lane, adapter or none
        bool lead = id >= 0 && __ffs((int)same) - 1 == (tid & 31);
        if (tid >= 32) {
            for (int j = 0; j < 32; ++j) lead = lead && s.id[j] != id;
        }
        const uint32_t m = __ballot_sync(kAll, lead);
        if ((tid & 31) == 0) s.lead[tid >> 5] = m;
    }
    __syncthreads();
}

// Members of the tile's j-th adapter into s.list: their number (0: no such
// adapter), the adapter in `adapter`.
__device__ __forceinline__ int tile_members(Tile &s, int j, int &adapter)
{
    uint64_t lead = (uint64_t)s.lead[1] << 32 | s.lead[0];
    for (int i = 0; i < j; ++i) lead &= lead - 1;
    if (lead == 0) return 0;
    adapter = s.id[__ffsll((long long)lead) - 1];
    const int tid = threadIdx.x;
    __syncthreads();   // the previous list has been read
    uint32_t m = 0;
    if (tid < kTokens) {
        m = __ballot_sync(kAll, s.id[tid] == adapter);
        if ((tid & 31) == 0) s.member[tid >> 5] = m;
    }
    __syncthreads();
    if (tid < kTokens && s.id[tid] == adapter)
        s.list[__popc(m & ((1u << (tid & 31)) - 1)) + (tid >= 32 ? __popc(s.member[0]) : 0)] = tid;
    __syncthreads();
    return __popc(s.member[0]) + __popc(s.member[1]);
}

// h[split][t][r] = sum over the split's K of A[a][r][k] x[t][k].  Grid: (tiles,
// adapters of a tile at the same time, splits).
template <int R, int TYPE>
__global__ void __launch_bounds__(kThreads) lora_down_kernel(const __grid_constant__ LoraArgs a)
{
    constexpr int kRows = R < 16 ? 1 : R / 16;   // 16-row operands
    __shared__ Tile tile;
    __shared__ float red[kWarps / 2][kRows][kGroup / 8][4][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    pdl_wait();   // codes and ids come from earlier kernels
    pdl_launch_dependents();
    tile_open(tile, a, blockIdx.x);
    const int blocks = a.K >> 5;
    const int b0 = blockIdx.z * a.per_split, b1 = min(blocks, b0 + a.per_split);
    const size_t tok0 = (size_t)blockIdx.x * kTokens;

    for (int j = blockIdx.y;; j += gridDim.y) {
        int adapter;
        const int members = tile_members(tile, j, adapter);
        if (members == 0) return;
        const char *A = a.A + (size_t)adapter * R * a.K * 2 + 16 * c;
        for (int m0 = 0; m0 < members; m0 += kGroup) {
            const int nq = min(kGroup, members - m0 + 7) / 8;   // MMAs' columns in use
            const int8_t *x[kGroup / 8];
            const uint16_t *d[kGroup / 8];
#pragma unroll
            for (int q = 0; q < kGroup / 8; ++q) {   // columns past the last member repeat it, unused
                const size_t t = tok0 + tile.list[min(members - 1, m0 + 8 * q + g)];
                x[q] = a.qs + t * a.K + 8 * c;
                d[q] = a.d + t * blocks;
            }
            float sum[kRows][kGroup / 8][4] = {};
#pragma unroll 2
            for (int b = b0 + warp; b < b1; b += kWarps) {
                uint4 w[kRows][2];
#pragma unroll
                for (int r = 0; r < kRows; ++r) {
                    w[r][0] = ld_cached_u4(A + ((size_t)(16 * r + g) * a.K + 32 * b) * 2);
                    w[r][1] = R >= 16 ? ld_cached_u4(A + ((size_t)(16 * r + 8 + g) * a.K + 32 * b) * 2)
                                      : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int q = 0; q < kGroup / 8; ++q) {
                    if (q >= nq) break;
                    const uint2 codes = __ldg(reinterpret_cast<const uint2 *>(x[q] + 32 * b));
                    const float dq = h2f(__ldg(d[q] + b));
                    const float d0 = __shfl_sync(kAll, dq, 8 * c), d1 = __shfl_sync(kAll, dq, 8 * c + 4);
                    uint32_t k0, k1, k2, k3;
                    codes4<TYPE>(codes.x, k0, k1);
                    codes4<TYPE>(codes.y, k2, k3);
#pragma unroll
                    for (int r = 0; r < kRows; ++r) {
                        float p[4] = {};
                        mma16<TYPE>(p, w[r][0].x, w[r][1].x, w[r][0].y, w[r][1].y, k0, k1);
                        mma16<TYPE>(p, w[r][0].z, w[r][1].z, w[r][0].w, w[r][1].w, k2, k3);
                        sum[r][q][0] += d0 * p[0];
                        sum[r][q][1] += d1 * p[1];
                        sum[r][q][2] += d0 * p[2];
                        sum[r][q][3] += d1 * p[3];
                    }
                }
            }
            // the warps' sums, as a tree: the upper half hands over, the lower half adds
#pragma unroll
            for (int half = kWarps / 2; half >= 1; half >>= 1) {
                __syncthreads();
                if (warp >= half && warp < 2 * half) {
#pragma unroll
                    for (int r = 0; r < kRows; ++r)
#pragma unroll
                        for (int q = 0; q < kGroup / 8; ++q)
#pragma unroll
                            for (int e = 0; e < 4; ++e) red[warp - half][r][q][e][lane] = sum[r][q][e];
                }
                __syncthreads();
                if (warp < half) {
#pragma unroll
                    for (int r = 0; r < kRows; ++r)
#pragma unroll
                        for (int q = 0; q < kGroup / 8; ++q)
#pragma unroll
                            for (int e = 0; e < 4; ++e) sum[r][q][e] += red[warp][r][q][e][lane];
                }
            }
            if (warp == 0) {
                float *h = a.h + (size_t)blockIdx.z * a.B * R;
#pragma unroll
                for (int q = 0; q < kGroup / 8; ++q)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int m = m0 + 8 * q + 2 * c + (e & 1);
                        if (m >= members) continue;
                        float *to = h + (tok0 + tile.list[m]) * R + g;
#pragma unroll
                        for (int r = 0; r < kRows; ++r)
                            if (e < 2 || R >= 16) to[16 * r + 8 * (e >> 1)] = sum[r][q][e];
                    }
            }
        }
    }
}

// y[t] = base[t] + scale_a B_a h_t for the CTA's kCols outputs.  Grid: (tiles,
// column blocks, adapters of a tile at the same time).
template <int R, int TYPE>
__global__ void __launch_bounds__(kThreads) lora_up_kernel(const __grid_constant__ LoraArgs a)
{
    constexpr int kSteps = R < 16 ? 1 : R / 16;
    constexpr int kRun = R < 32 ? R / 4 : 8;   // neighbouring values of R that a lane's fragment takes
    __shared__ Tile tile;
    __shared__ float h_s[kTokens][R + 1];
    __shared__ float back_s[kTokens];          // 2^e of a token's scaling
    __shared__ uint2 hi_s[kTokens / 8][kSteps][32], lo_s[kTokens / 8][kSteps][32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    const size_t tok0 = (size_t)blockIdx.x * kTokens;
    const int n0 = blockIdx.y * kCols + 32 * warp + 4 * g;   // this lane's four outputs
    // The first kernel lets this one start only when all before it is complete:
    // ids, base and weights may be read ahead of the wait, h may not.
    tile_open(tile, a, blockIdx.x);
    bool waited = false;

    for (int j = blockIdx.z;; j += gridDim.z) {
        int adapter;
        const int members = tile_members(tile, j, adapter);
        if (members == 0) break;
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
                    const uint4 f = ld_cached_u4(row + 64 * s);
                    w[i >> 1][2 * s][i & 1] = f.x;
                    w[i >> 1][2 * s][2 + (i & 1)] = f.y;
                    w[i >> 1][2 * s + 1][i & 1] = f.z;
                    w[i >> 1][2 * s + 1][2 + (i & 1)] = f.w;
                }
            }
        }
        if (!waited) {
            pdl_wait();
            pdl_launch_dependents();
            waited = true;
        }
        // h of the members: the splits in order, times the adapter's scale
        const float scale = a.scales ? a.scales[adapter] : 1.0f;
        for (int i = tid; i < members * R; i += kThreads) {
            const float *h = a.h + (tok0 + tile.list[i / R]) * R + i % R;
            float v = 0.0f;
#pragma unroll 8
            for (int s = 0; s < a.splits; ++s) v += h[(size_t)s * a.B * R];
            h_s[i / R][i % R] = scale * v;
        }
        __syncthreads();
        if (TYPE == ZQ_F16) {   // binary16 parts need the row near 1
            for (int m = tid; m < members; m += kThreads) {
                float amax = 0.0f;
#pragma unroll
                for (int r = 0; r < R; ++r) amax = fmaxf(amax, fabsf(h_s[m][r]));
                const int e = min(max((int)(__float_as_uint(amax) >> 23) - 127, -126), 126);
                back_s[m] = __int_as_float((127 + e) << 23);
                const float down = __int_as_float((127 - e) << 23);
#pragma unroll
                for (int r = 0; r < R; ++r) h_s[m][r] *= down;
            }
            __syncthreads();
        }
        const int groups = (members + 7) / 8;
        for (int i = tid; i < groups * kSteps * 32; i += kThreads) {   // fragments: column g of a group
            const int l = i & 31, s = i / 32 % kSteps, q = i / 32 / kSteps, m = 8 * q + (l >> 2);
            uint32_t hi[2], lo[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                // a lane's values of step s: kRun neighbours of each 32, four of them a step
                const int r = R < 16 ? 2 * (l & 3) : R < 32 ? 4 * (l & 3) + 2 * k
                                                            : 32 * (s / 2) + 8 * (l & 3) + 4 * (s & 1) + 2 * k;
                const bool in = m < members && (R >= 16 || k == 0);
                const float x = in ? h_s[m][r] : 0.0f, y = in ? h_s[m][r + 1] : 0.0f;
                hi[k] = kv_pack2<TYPE>(x, y);
                float2 f;
                if constexpr (TYPE == ZQ_BF16)
                    f = make_float2(__uint_as_float(hi[k] << 16), __uint_as_float(hi[k] & 0xffff0000u));
                else f = __half22float2(*reinterpret_cast<const __half2 *>(&hi[k]));
                lo[k] = kv_pack2<TYPE>(x - f.x, y - f.y);
            }
            hi_s[q][s][l] = make_uint2(hi[0], hi[1]);
            lo_s[q][s][l] = make_uint2(lo[0], lo[1]);
        }
        __syncthreads();
        if ((int)blockIdx.y * kCols + 32 * warp < a.N) {   // by whole warps: the MMAs take every lane
            const int left = a.N - n0;   // outputs of this lane, none when it is past the last
            for (int q = 0; q < groups; ++q) {
                float p[2][4] = {};
#pragma unroll
                for (int s = 0; s < kSteps; ++s) {
                    const uint2 hi = hi_s[q][s][lane], lo = lo_s[q][s][lane];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        mma16<TYPE>(p[i], w[i][s][0], w[i][s][1], w[i][s][2], w[i][s][3], lo.x, lo.y);
                        mma16<TYPE>(p[i], w[i][s][0], w[i][s][1], w[i][s][2], w[i][s][3], hi.x, hi.y);
                    }
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int m = 8 * q + 2 * c + e;
                    if (m >= members) continue;
                    const float f = TYPE == ZQ_F16 ? back_s[m] : 1.0f;
                    const size_t t = tok0 + tile.list[m];
                    float v[4] = {p[0][e] * f, p[0][2 + e] * f, p[1][e] * f, p[1][2 + e] * f};
                    const float *from = a.base ? a.base + t * a.base_stride + n0 : nullptr;
                    float *to = a.y + t * a.y_stride + n0;
                    if (a.vec && left >= 4) {
                        if (from) {
                            const float4 b = *reinterpret_cast<const float4 *>(from);
                            v[0] += b.x;
                            v[1] += b.y;
                            v[2] += b.z;
                            v[3] += b.w;
                        }
                        *reinterpret_cast<float4 *>(to) = make_float4(v[0], v[1], v[2], v[3]);
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (i < left) to[i] = v[i] + (from ? from[i] : 0.0f);
                    }
                }
            }
        }
    }
    if (!waited) {
        pdl_wait();
        pdl_launch_dependents();
    }
    // tokens without an adapter
    if (blockIdx.z == 0 && a.base != a.y) {
        const int col = blockIdx.y * kCols + tid;
        if (col < a.N)
            for (int i = 0; i < kTokens && tok0 + i < (size_t)a.B; ++i)
                if (tile.id[i] < 0)
                    a.y[(tok0 + i) * a.y_stride + col] = a.base ? a.base[(tok0 + i) * a.base_stride + col] : 0.0f;
    }
}

template <int R, int TYPE>
cudaError_t launch_rank(const LoraArgs &a, dim3 down, dim3 up, cudaStream_t st)
{
    cudaError_t e = launch_pdl(lora_down_kernel<R, TYPE>, down, dim3(kThreads), 0, st, a);
    if (e != cudaSuccess) return e;
    return launch_pdl(lora_up_kernel<R, TYPE>, up, dim3(kThreads), 0, st, a);
}

template <int TYPE>
cudaError_t launch_type(const LoraArgs &a, int R, dim3 down, dim3 up, cudaStream_t st)
{
    switch (R) {
    case 8: return launch_rank<8, TYPE>(a, down, up, st);
    case 16: return launch_rank<16, TYPE>(a, down, up, st);
    case 32: return launch_rank<32, TYPE>(a, down, up, st);
    default: return launch_rank<64, TYPE>(a, down, up, st);
    }
}

// Blocks of K in a split: four a warp, or fewer splits when the tiles alone
// fill the GPU.
int blocks_per_split(int B, int K)
{
    const int blocks = K / 32, tiles = (B + kTokens - 1) / kTokens;
    const int most = (2 * num_sms() + tiles - 1) / tiles;
    const int splits = (blocks + 4 * kWarps - 1) / (4 * kWarps);
    const int use = splits < most ? splits : most;
    return (blocks + use - 1) / use;
}

}  // namespace

size_t lora_workspace(int B, int K, int R)
{
    const int per = blocks_per_split(B, K);
    return (size_t)((K / 32 + per - 1) / per) * B * R * sizeof(float);
}

cudaError_t launch_lora(const LoraArgs &args, int R, int type, cudaStream_t st)
{
    LoraArgs a = args;
    a.per_split = blocks_per_split(a.B, a.K);
    a.splits = (a.K / 32 + a.per_split - 1) / a.per_split;
    const int tiles = (a.B + kTokens - 1) / kTokens, cols = (a.N + kCols - 1) / kCols;
    // adapters of a tile taken at the same time: as many as there can be, while
    // the grid is not several times the GPU already (a CTA takes the others in turn)
    int most = a.B < kTokens ? a.B : kTokens;
    if (a.n < most) most = a.n;
    const long long room = 8LL * num_sms();
    long long down = room / ((long long)tiles * a.splits), up = room / ((long long)tiles * cols);
    down = down < 1 ? 1 : down > most ? most : down;
    up = up < 1 ? 1 : up > most ? most : up;
    const dim3 gd(tiles, (unsigned)down, a.splits), gu(tiles, cols, (unsigned)up);
    return type == ZQ_BF16 ? launch_type<ZQ_BF16>(a, R, gd, gu, st) : launch_type<ZQ_F16>(a, R, gd, gu, st);
}

}  // namespace zq
