// lora.cu -- low-rank adapters of many requests beside a shared projection:
//   y[t] = base[t] + scale_a B_a (A_a x_t),  a = ids[t],
// on the Q8_1 activations the shared projection reads (ZINC docs "ROCm
// backend": Q8 activations packed once and reused by the projections).
//
// Two kernels, one after the other: h_t = A_a x_t split over K, then the
// expansion of h by B_a onto base.  Bound: HBM, the adapters once, and base and
// y (8 B N bytes); a few tokens are launch bound.  Measured in a graph: one token,
// 1024 -> 2048, 7.0 us; 56 tokens of 12 adapters, 5120 -> 17408, R = 16, bf16:
// 12.0 us (16.7 MB: 2.5 us at the copy rate; two launches in a row and their chains of
// dependent loads are the rest); 512 tokens of 4 adapters, 17408 -> 5120, R = 64,
// f16: 25.3 us (42 MB, 6.2 us; the first kernel's two thirds are 54 MB of 32- and 64-byte
// pieces from L2, as each 32 tokens read their adapter again, at 6.7 TB/s, and a
// second turn where a tile has three units); 4096 tokens of 4 adapters in runs,
// 5120 -> 17408, R = 16, bf16: 113 to 117 us, 5.2 TB/s.
//
// Tokens come in tiles of 64.  A CTA sorts its tile's tokens by adapter itself
// (64 ids: a scan of comparisons) and takes them sixteen at a time as the rows of
// its MMAs, so a prompt's tokens share each adapter row and a decode batch reads
// each of its adapters once a tile; no sorting pass, no plan to keep, any
// mixture of both.
//
// First kernel: m16n8k16 with tokens as the rows and eight adapter rows as the
// columns.  The order of K inside a step is free, so lane 4g + c loads 8
// neighbouring values of adapter row g, two steps' fragments as they stand (as
// the 16-row operand they would have to be moved together from two loads), and
// 8 codes of tokens g and g + 8.  Codes are whole numbers of at most 8 bits, exact
// in binary16 and bf16: a Q8_1 block's products are summed by the tensor core and
// scaled by the block's d in fp32.  The warps split the blocks of a CTA's K
// range; their sums are added up in order, so are those of a cluster's CTAs,
// through distributed shared memory, and by the second kernel the clusters'.
//
// Second kernel: tokens are the rows, outputs the columns; h is three bf16 parts
// (2^-24), or two binary16 ones after scaling the token's row to [1, 2) (2^-22 of
// its largest value).  The outputs are dealt to the MMAs' columns so that a lane holds
// four neighbouring ones of its tokens: base and y move as 16-byte pieces.
#include "zq_async.cuh"
#include "zq_cluster.cuh"
#include "zq_internal.cuh"
#include "zq_kv.cuh"
#include "zq_mma.cuh"

namespace zq {
namespace {

constexpr int kTokens = 64;      // tokens of a tile
constexpr int kGroup = 16;       // tokens of a group: an MMA's rows
constexpr int kQ = 2;            // groups a unit has at most
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kDownRows = 32;    // rows of A a CTA of the first kernel takes at most
constexpr int kCluster = 8;      // CTAs of a cluster at most, which add up their K ranges
constexpr int kParts = 4;        // sums the second kernel is left with at most
// outputs that a warp of the second kernel works on at a time, in 16 (at R = 64 registers allow two an SM
// with one: 512 tokens 25.2 us the call, 33.0 with two and half the warps)
__host__ __device__ constexpr int up_pieces(int R) { return R == 64 ? 1 : 2; }
constexpr int kNone = 255;
constexpr int kLong = 6;         // tasks of a warp of the second kernel from which on it asks L2 for those ahead
constexpr unsigned kAll = 0xffffffffu;

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

__device__ __forceinline__ void prefetch_l2(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// A tile's tokens by adapter: each adapter's tokens in groups of sixteen (an
// MMA's rows), its groups in units of up to two.
struct Tile {
    int id[kTokens];               // adapter of a token, -1: none (or past the last token)
    int seen[kTokens];             // tokens of its adapter | those before it << 8 | the first one << 16
    int base[kTokens];             // first group of a token's adapter, at the adapter's first token
    int half, groups, units;       // groups | units << 16 of the lower 32 tokens; in all
    int adapter[kTokens];          // of a group
    uint32_t tok[kTokens][kGroup / 4];   // tokens of a group's rows, a byte each, kNone: no more
    uint8_t unit[kTokens], unit_groups[kTokens];   // first group of a unit, number of its groups

    __device__ __forceinline__ int token(int group, int row) const
    {
        return reinterpret_cast<const uint8_t *>(tok[group])[row];
    }
};

// By all kThreads threads: four of them compare a token's adapter with the
// tile's, then the lower 64 have a token each.
__device__ __forceinline__ void tile_open(Tile &s, const LoraArgs &a, int tile)
{
    const int t = threadIdx.x, lane = t & 31;
    if (t < kTokens) {
        const int at = tile * kTokens + t;
        int id = at < a.B ? a.ids[at] : -1;
        if (id < 0 || id >= a.n) id = -1;
        s.id[t] = id;
#pragma unroll
        for (int i = 0; i < kGroup / 4; ++i) s.tok[t][i] = 0xffffffffu;
    }
    __syncthreads();
    {
        const int me = t / 4, j0 = t % 4 * 16, mine = s.id[me];
        int total = 0, before = 0, first = kTokens;
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
            const int4 o = *reinterpret_cast<const int4 *>(s.id + j0 + j);
            const int v[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const bool same = v[k] == mine;
                total += same;
                before += same && j0 + j + k < me;
                if (same) first = min(first, j0 + j + k);
            }
        }
#pragma unroll
        for (int off = 1; off <= 2; off <<= 1) {
            total += __shfl_xor_sync(kAll, total, off);
            before += __shfl_xor_sync(kAll, before, off);
            first = min(first, __shfl_xor_sync(kAll, first, off));
        }
        if (t % 4 == 0) s.seen[me] = total | before << 8 | first << 16;
    }
    __syncthreads();
    int id = -1, before = 0, first = 0, own = 0, incl = 0;
    if (t < kTokens) {
        id = s.id[t];
        before = s.seen[t] >> 8 & 0xff;
        first = s.seen[t] >> 16;
        if (id >= 0 && before == 0) {
            const int groups = ((s.seen[t] & 0xff) + kGroup - 1) / kGroup;
            own = groups | (groups + kQ - 1) / kQ << 16;
        }
        incl = own;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int up = __shfl_up_sync(kAll, incl, off);
            if (lane >= off) incl += up;
        }
        if (t == 31) s.half = incl;
    }
    __syncthreads();
    if (t < kTokens) {
        if (t >= 32) incl += s.half;
        if (t == kTokens - 1) {
            s.groups = incl & 0xffff;
            s.units = incl >> 16;
        }
        const int at = (incl - own) & 0xffff, unit = (incl - own) >> 16, n = own & 0xffff;
        s.base[t] = at;
        for (int i = 0; i < n; ++i) s.adapter[at + i] = id;
        for (int i = 0; i < own >> 16; ++i) {
            s.unit[unit + i] = (uint8_t)(at + kQ * i);
            s.unit_groups[unit + i] = (uint8_t)min(kQ, n - kQ * i);
        }
    }
    __syncthreads();
    if (t < kTokens && id >= 0)
        reinterpret_cast<uint8_t *>(s.tok[s.base[first] + before / kGroup])[before % kGroup] = (uint8_t)t;
    __syncthreads();
}

// h[part][t][r] = sum over the part's K of A[a][r][k] x[t][k].  Grid: (tiles
// and groups of RR rows, units of a tile at the same time, K ranges); the
// ranges of a cluster are added up through distributed shared memory into one
// part.
template <int RR, int TYPE>
__global__ void __launch_bounds__(kThreads, 2) lora_down_kernel(const __grid_constant__ LoraArgs a)
{
    constexpr int kCols = RR / 8;   // MMAs' columns: rows of A
    constexpr int kValues = kCols * kQ * 4 * 32;
    __shared__ float part_s[kWarps][kCols][kQ][4][32];   // the warps' sums
    __shared__ float sum_s[kValues];                     // the CTA's
    __shared__ __align__(16) Tile tile;
    // (a shuffle tells the compiler that the whole warp has the value)
    const int warp = __shfl_sync(kAll, threadIdx.x >> 5, 0), lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    pdl_wait();   // codes and ids come from earlier kernels
    pdl_launch_dependents();
    const int halves = a.R / RR, row0 = (int)blockIdx.x % halves * RR;
    const size_t tok0 = (size_t)(blockIdx.x / halves) * kTokens;
    tile_open(tile, a, blockIdx.x / halves);
    const int blocks = a.K >> 5;
    const int b0 = min(blocks, (int)blockIdx.z * a.per_split), b1 = min(blocks, b0 + a.per_split);
    const int rank = blockIdx.z % a.cluster;
    float *h = a.h + (size_t)(blockIdx.z / a.cluster) * a.B * a.R + row0;

    for (int u = blockIdx.y, units = __shfl_sync(kAll, tile.units, 0); u < units; u += gridDim.y) {   // the same in all CTAs of the cluster
        const int group0 = __shfl_sync(kAll, tile.unit[u], 0), nq = __shfl_sync(kAll, tile.unit_groups[u], 0);
        const int adapter = __shfl_sync(kAll, tile.adapter[group0], 0);
        const int chunk = (b1 - b0 + kWarps - 1) / kWarps, first = b0 + warp * chunk;
        const int last = min(b1, first + chunk);   // this warp's blocks: first .. last - 1
        const char *A[kCols];
        const int8_t *x[kQ][2];
        const uint16_t *d[kQ][2];          // of block first + c
#pragma unroll
        for (int r = 0; r < kCols; ++r)
            A[r] = a.A + (((size_t)adapter * a.R + row0 + 8 * r + g) * a.K + 32 * (size_t)first + 8 * c) * 2;
#pragma unroll
        for (int q = 0; q < kQ; ++q)
#pragma unroll
            for (int e = 0; e < 2; ++e) {   // rows without a token repeat the first, unused
                const int of = q < nq ? tile.token(group0 + q, g + 8 * e) : kNone;
                const size_t t = tok0 + (of == kNone ? tile.token(group0, 0) : of);
                x[q][e] = a.qs + t * a.K + 32 * (size_t)first + 8 * c;
                d[q][e] = a.d + t * blocks + first + c;
            }
        float sum[kCols][kQ][4] = {};
        // the next block's values are on their way while this one's are used
        struct Block {
            uint4 w[kCols];
            uint2 codes[kQ][2];
        };
        auto fetch = [&](Block &f) {   // and on to the block after it
#pragma unroll
            for (int r = 0; r < kCols; ++r) {
                f.w[r] = __ldg(reinterpret_cast<const uint4 *>(A[r]));
                A[r] += 64;
            }
#pragma unroll
            for (int q = 0; q < kQ; ++q)
                if (q < nq)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        f.codes[q][e] = __ldg(reinterpret_cast<const uint2 *>(x[q][e]));
                        x[q][e] += 32;
                    }
        };
        // the d of four blocks, one a lane of the four that share a token: a load of its own for each
        // block is a third of the L1's work (the call: 200 tokens, 5120 -> 17408, R = 16, 27.1 -> 25.5 us;
        // 512 tokens, R = 64, 33.3 -> 33.0)
        uint32_t dn[kQ][2], dv[kQ][2];
        auto fetch_d = [&](int b) {
#pragma unroll
            for (int q = 0; q < kQ; ++q)
                if (q < nq)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        dn[q][e] = b + c < last ? __ldg(d[q][e]) : 0;
                        d[q][e] += 4;
                    }
        };
        auto use = [&](const Block &f, int j) {
#pragma unroll
            for (int q = 0; q < kQ; ++q) {
                if (q >= nq) break;
                const float d0 = h2f((uint16_t)__shfl_sync(kAll, dv[q][0], (lane & ~3) + j));
                const float d1 = h2f((uint16_t)__shfl_sync(kAll, dv[q][1], (lane & ~3) + j));
                uint32_t k[2][4];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    codes4<TYPE>(f.codes[q][e].x, k[e][0], k[e][1]);
                    codes4<TYPE>(f.codes[q][e].y, k[e][2], k[e][3]);
                }
#pragma unroll
                for (int r = 0; r < kCols; ++r) {
                    float p[4];
                    mma16_first<TYPE>(p, k[0][0], k[1][0], k[0][1], k[1][1], f.w[r].x, f.w[r].y);
                    mma16<TYPE>(p, k[0][2], k[1][2], k[0][3], k[1][3], f.w[r].z, f.w[r].w);
                    sum[r][q][0] += d0 * p[0];
                    sum[r][q][1] += d0 * p[1];
                    sum[r][q][2] += d1 * p[2];
                    sum[r][q][3] += d1 * p[3];
                }
            }
        };
        Block even, odd;
        if (first < last) {
            fetch_d(first);
            fetch(even);
        }
        for (int b = first; b < last; b += 4) {
#pragma unroll
            for (int q = 0; q < kQ; ++q)
#pragma unroll
                for (int e = 0; e < 2; ++e) dv[q][e] = dn[q][e];
            if (b + 4 < last) fetch_d(b + 4);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (b + j >= last) break;
                if (b + j + 1 < last) fetch(j & 1 ? even : odd);
                use(j & 1 ? odd : even, j);
            }
        }
        // the warps' sums, in order
#pragma unroll
        for (int r = 0; r < kCols; ++r)
#pragma unroll
            for (int q = 0; q < kQ; ++q)
                if (q < nq)
#pragma unroll
                    for (int e = 0; e < 4; ++e) part_s[warp][r][q][e][lane] = sum[r][q][e];
        __syncthreads();
        for (int i = threadIdx.x; i < kValues; i += kThreads) {
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) v += (&part_s[w][0][0][0][0])[i];
            sum_s[i] = v;
        }
        // each CTA of the cluster adds up its share of the values, in the order of the ranges
        __syncwarp();
        if (a.cluster > 1) cluster_sync();
        else __syncthreads();
        const int share = kValues / a.cluster;
        const uint32_t local = smem_u32(sum_s);
        for (int i = rank * share + threadIdx.x; i < (rank + 1) * share; i += kThreads) {
            const int l = i & 31, e = i >> 5 & 3, q = i >> 7 & (kQ - 1), r = i / (kQ * 128);
            const int of = q < nq ? tile.token(group0 + q, (l >> 2) + 8 * (e >> 1)) : kNone;
            if (of != kNone) {
                float v = 0.0f;
                for (int k = 0; k < a.cluster; ++k) v += ld_cluster_f32(cluster_addr(local + 4 * i, k));
                h[(tok0 + of) * a.R + 8 * r + 2 * (l & 3) + (e & 1)] = v;
            }
        }
        __syncwarp();
        if (a.cluster > 1) cluster_sync();   // the sums have been read
    }
}

// y[t] = base[t] + scale_a B_a h_t.  Grid: (tiles, column ranges of a.blocks
// blocks of 16 or 32 outputs).  A task is one block for one group of sixteen tokens; a warp
// takes neighbouring tasks of one block after the other, the next one's values
// on their way while it works on one.
// VEC: rows of base and y are 16-byte aligned and N is a multiple of four, so
// four outputs move at once (values alone cost the 17408-wide decode batch half
// as much again).
template <int R, int TYPE, bool VEC>
__global__ void __launch_bounds__(kThreads, 2) lora_up_kernel(const __grid_constant__ LoraArgs a)
{
    constexpr int kSteps = R < 16 ? 1 : R / 16;
    constexpr int kP = up_pieces(R), kBlock = 16 * kP;
    constexpr int kRun = R < 32 ? R / 4 : 8;   // neighbouring values of R that a lane's fragment takes
    constexpr int kHParts = TYPE == ZQ_BF16 ? 3 : 2;   // 16-bit parts of h
    constexpr int kUpGroups = R < 32 ? 16 : R == 64 && TYPE == ZQ_BF16 ? 4 : 8;   // groups whose h is in shared memory
    __shared__ __align__(16) Tile tile;
    __shared__ uint4 h_s[kUpGroups][kSteps][kHParts][32];   // fragments of h, the upper parts first
    __shared__ float back_s[kUpGroups][kGroup];       // 2^e of a member's scaling
    __shared__ const float *from_s[kTokens];          // rows of base and y
    __shared__ float *to_s[kTokens];
    const int tid = threadIdx.x, warp = __shfl_sync(kAll, tid >> 5, 0), lane = tid & 31, g = lane >> 2, c = lane & 3;
    const size_t tok0 = (size_t)blockIdx.x * kTokens;
    const int block0 = blockIdx.y * a.blocks, blocks = min(a.blocks, (a.N + kBlock - 1) / kBlock - block0);
    // ids, base and h are outputs of kernels before this one, and their grouping chooses the weights: nothing is read
    // ahead of the wait.  (The first kernel lets this one start only when all before it is complete, but a grid sees
    // their writes only after a wait of its own.  Read ahead, ids and base saved 1.1 us of one token's call, 0.4
    // of 56 tokens', nothing of 512.)
    if (tid < kTokens) {
        from_s[tid] = a.base + (a.base ? (tok0 + tid) * a.base_stride : 0);
        to_s[tid] = a.y + (tok0 + tid) * a.y_stride;
    }
    pdl_wait();
    pdl_launch_dependents();
    tile_open(tile, a, blockIdx.x);

    // The columns of MMA (p, i) are outputs 16 p + 4 (col / 2) + 2 i + col % 2 of
    // the block, so that lane 4g + c ends with outputs 16 p + 4c .. 4c + 3.
    struct Task {
        uint32_t w[kP][2][kSteps][2];
        float4 v[2][kP];            // base of rows g, g + 8
    };
    auto fetch = [&](int group, int col0, bool weights, Task &f) {
        if (weights) {
            const char *row0 = a.Bm + (size_t)__shfl_sync(kAll, tile.adapter[group], 0) * a.N * R * 2 + kRun * 2 * c;
#pragma unroll
            for (int p = 0; p < kP; ++p)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int n = col0 + 16 * p + 4 * (g >> 1) + 2 * i + (g & 1);
                    const char *row = row0 + (uint32_t)min(a.N - 1, n) * (R * 2);
                    if constexpr (R == 8) {
                        f.w[p][i][0][0] = __ldg(reinterpret_cast<const uint32_t *>(row));
                        f.w[p][i][0][1] = 0;
                    } else if constexpr (R == 16) {
                        const uint2 x = __ldg(reinterpret_cast<const uint2 *>(row));
                        f.w[p][i][0][0] = x.x;
                        f.w[p][i][0][1] = x.y;
                    } else {
#pragma unroll
                        for (int s = 0; s < kSteps / 2; ++s) {
                            const uint4 x = __ldg(reinterpret_cast<const uint4 *>(row + 64 * s));
                            f.w[p][i][2 * s][0] = x.x;
                            f.w[p][i][2 * s][1] = x.y;
                            f.w[p][i][2 * s + 1][0] = x.z;
                            f.w[p][i][2 * s + 1][1] = x.w;
                        }
                    }
                }
        }
        // a row without a token reads the group's first, a column past the last the last: neither is stored
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int t = tile.token(group, g + 8 * e);
            const float *from = from_s[t == kNone ? tile.token(group, 0) : t];
#pragma unroll
            for (int p = 0; p < kP; ++p) {
                const int n = col0 + 16 * p + 4 * c;
                if (!a.base) {
                    f.v[e][p] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                } else if constexpr (VEC) {
                    f.v[e][p] = *reinterpret_cast<const float4 *>(from + min(n, a.N - 4));
                } else {
                    const int last = a.N - 1;
                    f.v[e][p] = make_float4(from[min(n, last)], from[min(n + 1, last)], from[min(n + 2, last)],
                                            from[min(n + 3, last)]);
                }
            }
        }
    };

    const int groups = __shfl_sync(kAll, tile.groups, 0);
    for (int g0 = 0; g0 < groups; g0 += kUpGroups) {
        const int n = min(kUpGroups, groups - g0);
        // this warp's tasks, block by block
        const int t0 = warp * blocks * n / kWarps, t1 = (warp + 1) * blocks * n / kWarps;
        int block = t0 / n, group = t0 - block * n;
        auto col_of = [&](int block) { return (block0 + block) * kBlock; };
        // The lines of the task after the next to L2, base's rows and a new block's weights: a warp with
        // many tasks waits for HBM at each (4096 tokens, R = 16: 140.8 us the call, 125.7 so; 512: 24.9,
        // 22.6), one with few loses more on the way (512 tokens, R = 64, 4 or 5 tasks: 25.2, 26.5)
        int far = t1 - t0 < kLong ? t1 : t0, far_block = block, far_group = group;
        auto step_far = [&]() {
            ++far;
            if (++far_group == n) {
                far_group = 0;
                ++far_block;
            }
        };
        auto ahead = [&]() {
            if (far >= t1) return;
            const int t = tile.token(g0 + far_group, lane & 15), col0 = col_of(far_block);
            if (a.base && lane < kGroup && t != kNone) prefetch_l2(from_s[t] + col0);
            if (far_group == 0) {
                const char *w = a.Bm + ((size_t)tile.adapter[g0] * a.N + col0) * R * 2;
                const int bytes = min(kBlock, a.N - col0) * R * 2;
                if (128 * lane < bytes) prefetch_l2(w + 128 * lane);   // 4 KB at most
            }
            step_far();
        };
        static_assert(kBlock * R * 2 <= 32 * 128, "a lane a line");
        step_far();
        step_far();
        Task even, odd;
        if (t0 < t1) fetch(g0 + group, col_of(block), true, even);
        // h of the groups' members: its parts in order, times the adapter's scale, as 16-bit parts in the
        // fragments' order; R / 4 neighbouring threads have a member, four values each
        constexpr int kAhead = 4;
        const int items = n * kGroup * (R / 4);
        for (int i0 = tid; i0 < items; i0 += kAhead * kThreads) {   // whole warps: items is a multiple of 32
            float4 read[kAhead];
            float scales[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int i = i0 + k * kThreads, m = i / (R / 4), grp = min(m / kGroup, n - 1);
                const int of = i < items ? tile.token(g0 + grp, m % kGroup) : kNone;
                read[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                scales[k] = 1.0f;
                if (of == kNone) continue;
                if (a.scales) scales[k] = a.scales[tile.adapter[g0 + grp]];
                const float *h = a.h + (tok0 + of) * R + i % (R / 4) * 4;
                read[k] = *reinterpret_cast<const float4 *>(h);
#pragma unroll 1
                for (int s = 1; s < a.parts; ++s) {
                    const float4 p = *reinterpret_cast<const float4 *>(h + (size_t)s * a.B * R);
                    read[k].x += p.x;
                    read[k].y += p.y;
                    read[k].z += p.z;
                    read[k].w += p.w;
                }
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int i = i0 + k * kThreads;
                if (i >= items) break;
                const int m = i / (R / 4), r = i % (R / 4) * 4, grp = m / kGroup, row = m % kGroup;
                const float4 f = read[k];
                const float scale = scales[k];
                float x[4] = {scale * f.x, scale * f.y, scale * f.z, scale * f.w};
                float up = 1.0f;
                if constexpr (TYPE == ZQ_F16) {   // binary16 parts need the row near 1
                    float amax = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
#pragma unroll
                    for (int off = 1; off < R / 4; off <<= 1) amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, off));
                    const int e = min(max((int)(__float_as_uint(amax) >> 23) - 127, -126), 126);
                    const float down = __int_as_float((127 - e) << 23);
                    up = __int_as_float((127 + e) << 23);
#pragma unroll
                    for (int j = 0; j < 4; ++j) x[j] *= down;
                }
                if (r == 0) back_s[grp][row] = up;
                const int s = R <= 16 ? 0 : 2 * (r / 32) + (r >> 2 & 1), l = row % 8 * 4;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    // register row / 8 (+ 2 for a step's upper eight) of the lane that has these values
                    const int at = R == 8 ? 4 * (l + r / 2 + j) + row / 8
                                          : 4 * (l + (R == 16 ? r / 4 : (r & 31) >> 3)) + row / 8 + 2 * j;
                    float x0 = x[2 * j], x1 = x[2 * j + 1];
#pragma unroll
                    for (int p = 0; p < kHParts; ++p) {
                        const uint32_t w = kv_pack2<TYPE>(x0, x1);
                        reinterpret_cast<uint32_t *>(h_s[grp][s][p])[at] = w;
                        float2 y;
                        if constexpr (TYPE == ZQ_BF16)
                            y = make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
                        else y = __half22float2(*reinterpret_cast<const __half2 *>(&w));
                        x0 -= y.x;
                        x1 -= y.y;
                    }
                }
            }
        }
        __syncthreads();
        // One task, the one after it (the block's next group, or the next block's first) on its way.
        auto work = [&](bool more, const Task &now, Task &next) {
            const int here = group, col0 = col_of(block);
            const int adapter = __shfl_sync(kAll, tile.adapter[g0 + group], 0);
            bool weights = false;
            ahead();
            if (++group == n) {
                group = 0;
                ++block;
                weights = true;
            }
            if (more) {
                weights |= __shfl_sync(kAll, tile.adapter[g0 + group], 0) != adapter;
                if (!weights) {
#pragma unroll
                    for (int p = 0; p < kP; ++p)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
#pragma unroll
                            for (int s = 0; s < kSteps; ++s)
#pragma unroll
                                for (int k = 0; k < 2; ++k) next.w[p][i][s][k] = now.w[p][i][s][k];
                }
                fetch(g0 + group, col_of(block), weights, next);
            }
            float y[kP][2][4];
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                // the lower parts first
#pragma unroll
                for (int part = kHParts - 1; part >= 0; --part) {
                    const uint4 f = h_s[here][s][part][lane];
#pragma unroll
                    for (int p = 0; p < kP; ++p)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint32_t(&w)[2] = now.w[p][i][s];
                            const bool onto_zero = s == 0 && part == kHParts - 1;
                            if constexpr (R == 8) {
                                if (onto_zero) mma8_first<TYPE>(y[p][i], f.x, f.y, w[0]);
                                else mma8<TYPE>(y[p][i], f.x, f.y, w[0]);
                            } else {
                                if (onto_zero) mma16_first<TYPE>(y[p][i], f.x, f.y, f.z, f.w, w[0], w[1]);
                                else mma16<TYPE>(y[p][i], f.x, f.y, f.z, f.w, w[0], w[1]);
                            }
                        }
                }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int t = tile.token(g0 + here, g + 8 * e);
                if (t != kNone) {
                    const float f = TYPE == ZQ_F16 ? back_s[here][g + 8 * e] : 1.0f;
                    float *to = to_s[t];
#pragma unroll
                    for (int p = 0; p < kP; ++p) {
                        const int n = col0 + 16 * p + 4 * c;
                        const float4 v = now.v[e][p];
                        const float4 r = make_float4(v.x + y[p][0][2 * e] * f, v.y + y[p][0][2 * e + 1] * f,
                                                     v.z + y[p][1][2 * e] * f, v.w + y[p][1][2 * e + 1] * f);
                        if constexpr (VEC) {
                            if (n < a.N) *reinterpret_cast<float4 *>(to + n) = r;
                        } else {
                            if (n < a.N) to[n] = r.x;
                            if (n + 1 < a.N) to[n + 1] = r.y;
                            if (n + 2 < a.N) to[n + 2] = r.z;
                            if (n + 3 < a.N) to[n + 3] = r.w;
                        }
                    }
                }
            }
            __syncwarp();
        };
        for (int task = t0; task < t1; task += 2) {
            work(task + 1 < t1, even, odd);
            if (task + 1 < t1) work(task + 2 < t1, odd, even);
        }
        __syncthreads();   // the fragments have been used
    }
    // tokens without an adapter
    if (a.base != a.y) {
        const int n0 = block0 * kBlock, n1 = min(a.N, n0 + blocks * kBlock);
        for (int i = warp; i < kTokens && tok0 + i < (size_t)a.B; i += kWarps) {
            if (tile.id[i] >= 0) continue;
            for (int col = n0 + lane; col < n1; col += 32)
                a.y[(tok0 + i) * a.y_stride + col] = a.base ? a.base[(tok0 + i) * a.base_stride + col] : 0.0f;
        }
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
    return a.vec ? launch_pdl(lora_up_kernel<R, TYPE, true>, up, dim3(kThreads), 0, st, a)
                 : launch_pdl(lora_up_kernel<R, TYPE, false>, up, dim3(kThreads), 0, st, a);
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
    void set(int K, int p)
    {
        parts = p;
        per_split = (K / 32 + cluster * parts - 1) / (cluster * parts);
    }
};
Cut cut_k(int B, int K, int R)
{
    const int blocks = K / 32, halves = R > kDownRows ? R / kDownRows : 1;
    const int wanted = (blocks + 2 * kWarps - 1) / (2 * kWarps);
    Cut c{(B + kTokens - 1) / kTokens, 1, 1, 0};
    while (c.cluster < kCluster && c.cluster < wanted) c.cluster *= 2;
    const int room = 2 * num_sms() / ((B + kGroup * kQ - 1) / (kGroup * kQ) * halves * kCluster);
    int parts = 1;
    while (parts < kParts && parts * 2 * kCluster <= wanted && parts * 2 <= room) parts *= 2;
    c.set(K, parts);
    return c;
}

}  // namespace

size_t lora_workspace(int B, int K, int R) { return (size_t)cut_k(B, K, R).parts * B * R * sizeof(float); }

cudaError_t launch_lora(const LoraArgs &args, int type, cudaStream_t st)
{
    LoraArgs a = args;
    const int halves = a.R > kDownRows ? a.R / kDownRows : 1;
    // units that a tile can have
    const int most = min(a.n, min(a.B, kTokens)) + (a.B > kGroup * kQ ? 1 : 0);
    Cut cut = cut_k(a.B, a.K, a.R);
    auto taken = [&] { return (long long)cut.tiles * halves * cut.cluster * cut.parts; };   // CTAs of a unit, over all tiles
    // no more parts of K than leave an SM to each CTA with all units taken at the same time (17408
    // wide, 16 tokens of 4 adapters of R = 64: 11.1 us, 14.5 with four parts; 56 tokens of 12 of R = 16:
    // 10.7, 15.6)
    while (cut.parts > 1 && taken() * most > num_sms()) cut.set(a.K, cut.parts / 2);
    // Smaller clusters where not all units fit at the same time, as long as a warp has few blocks: a
    // turn costs about as much as five (5120 wide, 12 adapters, mixed: 200 tokens 17.3 -> 14.9 us, 1024 46.9 ->
    // 38.9; 4 in runs, a tile's two or three units: 512 23.0 -> 23.8; 17408 wide they would lose: 200 tokens 19.8,
    // 25.0)
    while (cut.cluster > 1 && taken() * most > 2 * num_sms() &&
           a.K / 32 <= 5 * kWarps * (cut.cluster / 2) * cut.parts) {
        cut.cluster /= 2;
        cut.set(a.K, cut.parts);
    }
    a.cluster = cut.cluster;
    a.parts = cut.parts;
    a.per_split = cut.per_split;
    // units of a tile taken at the same time: as many as there can be, in a grid
    // that the GPU holds at once (a CTA takes the others in turn: starting one
    // costs more than two blocks' worth of its work)
    const long long room = 2LL * num_sms() / taken();
    const dim3 down(cut.tiles * halves, (unsigned)(room < 1 ? 1 : room > most ? most : room), cut.cluster * cut.parts);
    // column blocks of a CTA of the second kernel: as many CTAs as the GPU holds
    // at once, two an SM, each of which prepares its tile's h once (with one an
    // SM 512 tokens at R = 64 take 31.5 us, 25.2 so; 56 tokens at R = 16 11.9, 11.3)
    const int width = 16 * up_pieces(a.R);
    const long long cols = (a.N + width - 1) / width, ctas = 2LL * num_sms();
    const long long want = (cols * cut.tiles + ctas - 1) / ctas;
    a.blocks = (int)(want < 1 ? 1 : want > 64 ? 64 : want);
    const dim3 up(cut.tiles, (unsigned)((cols + a.blocks - 1) / a.blocks));
    return type == ZQ_BF16 ? launch_type<ZQ_BF16>(a, down, up, st) : launch_type<ZQ_F16>(a, down, up, st);
}

}  // namespace zq
