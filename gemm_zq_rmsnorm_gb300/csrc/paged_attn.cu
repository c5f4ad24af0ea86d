// paged_attn.cu -- attention of one new token per sequence over a paged
// key-value cache, split over the cache's length and joined (MIInfer README,
// "Status": cached single-query attention).
//
//   s_j = scale q.k_j,  o = sum_j exp(s_j) v_j / sum_j exp(s_j),
// in one pass: each warp keeps the running maximum m, the sum l and the
// unnormalised output of its tokens; two such pieces of a row join as
//   m = max(m1, m2), l = l1 2^(m1-m) + l2 2^(m2-m), o alike (base 2).
//
// Bound: HBM, 2 D Hk es bytes per token against 4 D Hq operations.  With G =
// Hq / Hk query heads on a key head the FP32 units would take G times the
// products' time of one head (at G = 6 about the whole HBM time), so the
// products run on the tensor cores through mma.sync: 16 tokens are the 16-row
// operand and the query heads the 8-column one, so G <= 8 heads cost one pass.
// (tcgen05 takes 64 or 128 rows from shared memory through a descriptor and
// returns through tensor memory; at 8 columns the tensor pipe is a third busy at
// most, and the warp-level form needs no hand-over between warps.)
// Measured, kernel pairs in a graph: 48 sequences of 1 to 12000 rows, 48 query
// and 8 key heads of 128, bf16: 127 us, 5.9 TB/s (0.88 of the measured copy
// rate); one sequence of 131071, 24 and 4 heads of 256, bf16: 95 us, 5.7 TB/s; 64
// sequences of 8000 to 24000, e4m3: 285 to 289 us, 6.1 TB/s.  What is left of the
// 16-bit cases is their end: the SMs of some GPCs get 10 % less of the bandwidth, and
// the shares are equal.  200 windows of up to 1024 rows, 64-wide heads, e4m3: 40.7 us,
// 3.5 TB/s: neither the issue slots (59 %) nor HBM are full, the chains of a 4 KB
// tile and of 1600 row blocks' ends are the rest.
// One sequence of 1000: 9.9 us, a chain of latencies (lengths, table, keys, two
// joins) over two launches.  With Q8_1 codes written as well or alone: the same but for
// the windows, 46.0 and 44.3 us.  Registers are spilled at 128-wide bf16 (104 bytes of
// stores) and f16 (48), and at 256-wide (76 to 192).
//
// Work: every (sequence, key head) has ceil(len / 32) tiles of 32 tokens (at
// least one, so that an empty row is written too); all tiles of the call form
// one line, cut into equal contiguous ranges for the warps, whatever the
// lengths.  A warp writes the rows it covers whole; open pieces join
// in the CTA through shared memory, and those that cross CTAs in a second
// kernel that reads at most two pieces per CTA, in order: no atomics, the same
// result every time.
//
// Loads: one lane of a warp copies the keys, or the values, of a tile (two
// pages' halves when pages have 16 tokens; half a tile of 512-byte rows) by TMA
// into the warp's own ring, which needs no other warp.  (With cp.async of 16
// bytes a lane the same loop stopped at 4.4 TB/s whatever the depth of the ring.)
// The box is [segment of 128 bytes][token], 128-byte swizzled.  Fragments of 16-bit
// rows come by ldmatrix, keys as they lie and values transposed; put together
// from 16-byte loads they cost two register moves a product (141 us for 128).
// 8-bit rows are loaded in 16-byte chunks (the order of the head's columns in a
// K-step and of the output rows is free) and converted in pairs, the values' bytes
// paired by token first; every access falls on all banks.
// Rows past the end, before the window or on a page outside the cache never
// meet a product: their scores are replaced by -infinity and their value words
// by zeros, whatever the cache holds there (infinities, NaN).  An infinite key
// of a row that is attended to makes the score it stands for: -infinity weighs
// nothing.
//
// Precision: q is split exactly into parts of the cache's 16-bit type (three
// bf16 parts; two binary16 parts after scaling the row to [1, 2), 2^-22 of its
// largest value), every product is exact, sums are fp32; e4m3 values are binary16
// values.  p in [0, 1] goes to the value product in as many parts: three of bf16,
// 2^-24 of p (two, 2^-17, would be 2 to 3 % faster), or two of binary16, which
// take 2^15 p, because their smallest step is 2^-24: 2^-22 of p, or 2^-40 where
// that is more, so that rows far below a dominant one (an attention sink, whose
// value is often near zero) count; the output carries the 2^15 until its piece
// is written.  l sums the unrounded p.
#include <float.h>
#include <math.h>

#include <atomic>

#include "zq_async.cuh"
#include "zq_internal.cuh"
#include "zq_kv.cuh"
#include "zq_mma.cuh"
#include "zq_tc.cuh"
#include "zq_tc_common.cuh"

namespace zq {
namespace {

constexpr int kMaxWarps = 16;
constexpr int kPlanners = 256;  // threads that add up the line of tiles
constexpr int kJoinThreads = 256;
constexpr int kHalf = 16;       // tokens of an MMA
constexpr int kTile = 32;       // tokens of a step: two MMAs' worth, so that a warp has independent chains
constexpr int kHeads = 8;       // query heads of a pass: the MMA's columns
constexpr int kBlockCost = 1;   // what a row block costs besides its tiles, in tiles (with 6, those windows took 10 % longer)
constexpr float kLn2 = 0.6931471805599453f;
constexpr unsigned kAll = 0xffffffffu;

template <int D, int TYPE>
struct Cfg {
    // As many warps as the registers of their fragments allow (q and the output take D / 2 to D / 1.3 of a
    // lane's): 200 windows of 1024 at D = 64 took 45.8 us with 12, 43.9 with 16
    static constexpr int kWarps = D == 64 ? 16 : D <= 128 ? 12 : 8;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kBytes = KvBytes<TYPE>::value;
    static constexpr int kRow = D * kBytes;             // bytes of a token's head
    // an item of the ring: the keys, or the values, of a tile, or of half a tile of 512-byte rows
    static constexpr int kItem = kRow > 256 ? kHalf : kTile;
    static constexpr int kItems = kTile / kItem;        // of keys (and of values) in a tile
    static constexpr int kSlot = kItem * kRow;
    // ring slots of a warp: as many as fit beside nothing else, eight at most
    static constexpr int kFit = 196608 / (kWarps * kSlot);
    static constexpr int kSlots = kFit > 8 ? 8 : kFit;
    static constexpr int kRing = kWarps * kSlot * kSlots;
    static constexpr int kMerge = kWarps * kHeads * D * 4;   // the warps' open pieces, after the ring is done
    static constexpr int kSmem = (kRing > kMerge ? kRing : kMerge) + 1024;   // aligned to the swizzle's 1024 bytes
    static constexpr int kSplits = TYPE == ZQ_BF16 ? 3 : 2;  // parts of q and of the weights
    static constexpr float kWeightUp = TYPE == ZQ_BF16 ? 1.0f : 0x1p15f;   // of the weights in the value product
    static constexpr float kWeightDown = 1.0f / kWeightUp;
    static constexpr int kSeg = kRow < 128 ? kRow : 128;          // bytes of a segment of a row
    static constexpr int kSegs = kRow / kSeg;
    static constexpr int kKBytes = kSeg / 4;            // a lane's keys of a segment: two chunks, or one
    static constexpr int kKRun = kKBytes / kBytes;
    static constexpr int kVBytes = kSeg / 8;            // a lane's values of a segment: a chunk, or half of one
    static constexpr int kVRun = kVBytes / kBytes;
};

// A piece of a row block in the workspace: kHeads rows of D, then m and l.
__host__ __device__ constexpr size_t piece_floats(int D) { return (size_t)kHeads * D + 2 * kHeads; }

// What a CTA leaves open: `a` continues a row block of an earlier CTA
// (1: goes on, 2: ends here), `b` one that begins here and goes on.
struct Meta {
    int a, b, seq, head, heads;
};

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 8 x 8 transpose of 16-bit values across the warp
__device__ __forceinline__ uint32_t transpose8(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// Four 8 x 8 matrices of 16-bit values, rows of 16 bytes at the lanes'
// addresses (lanes 8i .. 8i + 7: matrix i); TRANS: transposed
template <bool TRANS>
__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t &r0, uint32_t &r1, uint32_t &r2, uint32_t &r3)
{
    if constexpr (TRANS)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
                     : "r"(addr)
                     : "memory");
    else
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
                     : "r"(addr)
                     : "memory");
}

// four e4m3 values to binary16 (exact): the lower two, the upper two
__device__ __forceinline__ void e4m3_f16(uint32_t w, uint32_t &lo, uint32_t &hi)
{
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

// The MMA's 16-bit type: bf16 for a bf16 cache, else binary16.
template <int TYPE>
__device__ __forceinline__ uint32_t pack16(float lo, float hi)
{
    return kv_pack2<TYPE == ZQ_BF16 ? ZQ_BF16 : ZQ_F16>(lo, hi);
}
template <int TYPE>
__device__ __forceinline__ float2 unpack16(uint32_t w)
{
    if constexpr (TYPE == ZQ_BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    else return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}

// Byte of 16-byte chunk `chunk` of token row `row` in a segment as TMA left it:
// rows of 128 bytes, 128-byte swizzle, or of 64 bytes, 64-byte swizzle.
template <int SEG>
__device__ __forceinline__ int swizzled(int row, int chunk)
{
    return row * SEG + ((chunk ^ (SEG == 128 ? row & 7 : row >> 1 & 3)) << 4);
}

// Q8_1 codes of a block of 32 outputs held by lanes that differ in the bits of
// `group` (shuffle masks), N neighbouring values each: the steps of q8_1_pack.
// `at` is the block-ordered index of this lane's first value; `first` marks the
// lane that writes the block's scales.
template <int N, int M0, int M1, int M2>
__device__ __forceinline__ void q8_block(const zq_q8_1 &o, size_t at, const float (&v)[N], bool store, bool first)
{
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) amax = fmaxf(amax, fabsf(v[i]));
    if (M0) amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, M0));
    if (M1) amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, M1));
    if (M2) amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, M2));
    const float d = __fdiv_rn(amax, 127.0f);
    const float id = d != 0.0f ? __fdiv_rn(1.0f, d) : 0.0f;
    int sum = 0;
    uint32_t word[N / 4];
#pragma unroll
    for (int w = 0; w < N / 4; ++w) {
        word[w] = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float q = roundf(__fmul_rn(v[4 * w + i], id));
            q = fminf(fmaxf(q, -127.0f), 127.0f);
            const int qi = (int)q;
            sum += qi;
            word[w] |= (uint32_t)(qi & 0xFF) << (8 * i);
        }
    }
    if (M0) sum += __shfl_xor_sync(kAll, sum, M0);
    if (M1) sum += __shfl_xor_sync(kAll, sum, M1);
    if (M2) sum += __shfl_xor_sync(kAll, sum, M2);
    if (!store) return;
#pragma unroll
    for (int w = 0; w < N / 4; ++w) reinterpret_cast<uint32_t *>(o.qs + at)[w] = word[w];
    if (first) {
        o.d[at >> 5] = __half_as_ushort(__float2half_rn(d));
        o.s[at >> 5] = __half_as_ushort(__float2half_rn(__fmul_rn(d, (float)sum)));
    }
}

// The same for the lanes with one c and g = 0 .. 7, each with the values 8k + g
// of the block that begins at `at`.
__device__ __forceinline__ void q8_block_strided(const zq_q8_1 &o, size_t at, const float (&v)[4], int g, bool store)
{
    float amax = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
#pragma unroll
    for (int off = 4; off <= 16; off <<= 1) amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, off));
    const float d = __fdiv_rn(amax, 127.0f);
    const float id = d != 0.0f ? __fdiv_rn(1.0f, d) : 0.0f;
    int sum = 0, q[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        q[k] = (int)fminf(fmaxf(roundf(__fmul_rn(v[k], id)), -127.0f), 127.0f);
        sum += q[k];
    }
#pragma unroll
    for (int off = 4; off <= 16; off <<= 1) sum += __shfl_xor_sync(kAll, sum, off);
    if (!store) return;
#pragma unroll
    for (int k = 0; k < 4; ++k) o.qs[at + 8 * k + g] = (int8_t)q[k];
    if (g == 0) {
        o.d[at >> 5] = __half_as_ushort(__float2half_rn(d));
        o.s[at >> 5] = __half_as_ushort(__float2half_rn(__fmul_rn(d, (float)sum)));
    }
}

// Factor of a finished row: v_scale / l; an empty row (l = 0) is zeros.
__device__ __forceinline__ float row_factor(float l, float v_scale) { return l == 0.0f ? 0.0f : __fdiv_rn(v_scale, l); }

__device__ __forceinline__ float row_lse(float m, float l)
{
    return l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
}

__device__ __forceinline__ int seq_len(const PagedAttnArgs &a, int b)
{
    return min(max(a.lens[b], 0), a.width << a.page_shift);
}
__device__ __forceinline__ int seq_first(const PagedAttnArgs &a, int len)
{
    return a.window > 0 && len > a.window ? len - a.window : 0;
}
// tiles of a sequence with rows [lo, len): at least one
__device__ __forceinline__ int seq_tiles(int lo, int len)
{
    return max(1, (len + kTile - 1) / kTile - lo / kTile);
}

// A place on the line of tiles: sequence, key head, pass (a group of up to
// eight of its query heads), tile.
struct Walk {
    int b, kh, pass, t, t0, tend, lo, len;
    __device__ __forceinline__ void sequence(const PagedAttnArgs &a, int seq)
    {
        b = seq;
        len = __shfl_sync(kAll, seq_len(a, seq), 0);
        lo = seq_first(a, len);
        t0 = lo / kTile;
        tend = t0 + seq_tiles(lo, len);
        t = t0;
    }
    // from the end of a row block to the next one
    __device__ __forceinline__ void next_block(const PagedAttnArgs &a)
    {
        t = t0;
        if (++pass < a.passes) return;
        pass = 0;
        if (++kh < a.Hk) return;
        kh = 0;
        if (++b < a.B) sequence(a, b);
    }
    // its query heads: the first one, and how many
    __device__ __forceinline__ int head(const PagedAttnArgs &a) const { return kh * a.G + pass * a.per_pass; }
    __device__ __forceinline__ int heads(const PagedAttnArgs &a) const
    {
        return min(a.per_pass, a.G - pass * a.per_pass);
    }
};

template <int D, int TYPE>
__global__ void __launch_bounds__(Cfg<D, TYPE>::kThreads, 1)
paged_attn_kernel(const __grid_constant__ PagedAttnArgs a, const __grid_constant__ CUtensorMap map_k,
                  const __grid_constant__ CUtensorMap map_v)
{
    using C = Cfg<D, TYPE>;
    constexpr int kWarps = C::kWarps;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    __shared__ uint64_t full_s[kWarps][8];     // a ring slot's copy has landed
    __shared__ long long before_s[kPlanners];  // the line ahead of each planner's sequences
    __shared__ long long total_s[kPlanners / 32];
    __shared__ int head_s[kWarps];             // an ending piece in the workspace
    __shared__ Meta open_s[kWarps];            // the warp's last piece (b = 1: begins in the warp, 2: before)
    __shared__ float m_s[kWarps][kHeads], l_s[kWarps][kHeads];

    // (a shuffle tells the compiler that the whole warp has the value: what follows from it is kept and
    // computed once a warp, in uniform registers)
    const int tid = threadIdx.x, warp = __shfl_sync(kAll, tid >> 5, 0), lane = tid & 31, g = lane >> 2, c = lane & 3;
    const int vheads = a.passes * a.Hk;
    if (lane == 0) {
        for (int i = 0; i < C::kSlots; ++i) mbar_init(&full_s[warp][i], 1);
        fence_mbar_init();
        prefetch_tmap(&map_k);
        prefetch_tmap(&map_v);
    }
    __syncwarp();   // a warp's barriers are its own
    pdl_wait();   // queries, cache, table and lengths come from earlier kernels
    pdl_launch_dependents();

    // ---- the line: every row block is kBlockCost places and its tiles.  `total`
    // places; the CTAs that take part share them, their warps one after the
    // other: this warp's are [u0, u0 + left), from place `rem` of sequence `at.b` on
    auto places = [&](int b) {
        const int len = seq_len(a, b);
        return (long long)(seq_tiles(seq_first(a, len), len) + kBlockCost) * vheads;
    };
    const long long gw = (long long)blockIdx.x * kWarps + warp;
    Meta *meta = reinterpret_cast<Meta *>(a.meta);
    long long total, u0 = 0, left = 0, rem = 0;
    int ctas;
    Walk at;
    auto share = [&]() {   // false: this CTA takes no part
        ctas = (int)min((long long)gridDim.x, (total + kWarps - 1) / kWarps);
        if (blockIdx.x >= ctas) return false;
        const uint32_t nw = ctas * kWarps;
        long long q, r;    // the first r warps have a place more
        if (total >> 32) {
            q = total / nw;
            r = total - q * nw;
        } else {
            q = (uint32_t)total / nw;
            r = (uint32_t)total - (uint32_t)q * nw;
        }
        u0 = gw * q + min(gw, r);
        left = q + (gw < r ? 1 : 0);
        return true;
    };
    // Few row blocks of few tiles have a CTA each and a warp a tile, so that the second kernel finds nothing open
    // (one sequence of 300, 128-wide heads: 9.7 us, 10.8 on the line; 8 of 250, 64-wide 7.7, 9.8)
    bool own = false;
    if (a.B <= 32) {       // every warp by itself: lane b has sequence b
        const long long line = lane < a.B ? places(lane) : 0;
        const bool few = __all_sync(kAll, line <= (kWarps + kBlockCost) * vheads);   // at most kWarps tiles in each
        own = __shfl_sync(kAll, few && a.B * vheads <= (int)gridDim.x, 0);   // (a shuffle as above)
        const long long mine = own && lane < a.B ? kWarps * vheads : line;
        long long incl = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long up = __shfl_up_sync(kAll, incl, off);
            if (lane >= off) incl += up;
        }
        total = __shfl_sync(kAll, incl, 31);
        if (!share()) {
            if (tid == 0) meta[blockIdx.x] = Meta{0, 0, 0, 0, 0};
            return;
        }
        const int b = min(__popc(__ballot_sync(kAll, incl <= u0)), a.B - 1);
        rem = u0 - __shfl_sync(kAll, incl - mine, b);
        if (left > 0) at.sequence(a, b);
    } else {               // planner t adds up sequences t * per ..
        const int per = (a.B + kPlanners - 1) / kPlanners;
        long long mine = 0, incl = 0;
        if (tid < kPlanners) {
            for (int b = tid * per; b < min(a.B, (tid + 1) * per); ++b) mine += places(b);
            incl = mine;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const long long up = __shfl_up_sync(kAll, incl, off);
                if (lane >= off) incl += up;
            }
            if (lane == 31) total_s[warp] = incl;
        }
        __syncthreads();
        long long base = 0;
        total = 0;
#pragma unroll
        for (int w = 0; w < kPlanners / 32; ++w) {
            if (w == warp) base = total;
            total += total_s[w];
        }
        if (tid < kPlanners) before_s[tid] = base + incl - mine;
        if (!share()) {
            if (tid == 0) meta[blockIdx.x] = Meta{0, 0, 0, 0, 0};
            return;
        }
        __syncthreads();
        if (left > 0) {
            int i = 0;
#pragma unroll
            for (int step = kPlanners / 2; step >= 1; step >>= 1)
                if ((i + step) * per < a.B && before_s[i + step] <= u0) i += step;
            i = __shfl_sync(kAll, i, 0);
            rem = u0 - __shfl_sync(kAll, before_s[i], 0);
            at.sequence(a, i * per);
            while (rem >= (long long)(at.tend - at.t0 + kBlockCost) * vheads) {
                rem -= (long long)(at.tend - at.t0 + kBlockCost) * vheads;
                at.sequence(a, at.b + 1);
            }
        }
    }
    if (left > 0) {        // key head, pass and tile
        const int tiles = at.tend - at.t0, n = own ? kWarps : tiles + kBlockCost;
        const int vh = rem >> 32 ? (int)(rem / n) : (int)((uint32_t)rem / (uint32_t)n);
        const int r = (int)(rem - (long long)vh * n);
        at.kh = vh / a.passes;
        at.pass = vh - at.kh * a.passes;
        at.t = at.t0 + (own ? r : max(0, r - kBlockCost));
        left -= own ? r >= tiles : max(0, kBlockCost - r);
    }

    // ---- the ring: the items of a tile are keys, keys, values, values, 16 tokens each
    uint8_t *ring = smem + (size_t)warp * C::kSlots * C::kSlot;
    uint64_t *full = full_s[warp];
    Walk ld = at;
    long long ld_left = left;
    int ld_item = 0, ld_slot = 0;
    uint32_t loaded = 0;    // two bits of a slot, its halves: the page is in the cache, so a copy was asked for
    uint32_t flying = 0;    // bit of a slot: the copy has not been waited for yet
    int pid[2] = {-1, -1};
    const int page_mask = (1 << a.page_shift) - 1;
    // an item lies as its boxes came: [segment][row], of 32 rows or twice of 16
    const int seg_stride = (C::kItem > kHalf ? a.box : kHalf) * C::kSeg;
    const int half_stride = a.box == kTile ? kHalf * C::kSeg : kHalf * C::kRow;

    // the next item into the ring, by the whole warp after it has read what the slot held
    auto issue = [&]() {
        if (ld_left > 0) {
            const int tok = ld.t * kTile;
            if (ld_item == 0) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {   // a page holds both halves, or one each; the table ends at len
                    const int row = tok + kHalf * i, col = row >> a.page_shift;
                    pid[i] = row < ld.len ? a.table[(size_t)ld.b * a.width + col] : -1;
                    pid[i] = __shfl_sync(kAll, (unsigned)pid[i] < (unsigned)a.pages ? pid[i] : -1, 0);
                }
                if (a.box == kTile) pid[1] = pid[0];
            }
            const CUtensorMap *map = ld_item < C::kItems ? &map_k : &map_v;
            const int first = ld_item % C::kItems;   // half of the tile the item begins with
            uint8_t *dst = ring + ld_slot * C::kSlot;
            uint32_t ok = 0;
#pragma unroll
            for (int i = 0; i < C::kItem / kHalf; ++i) ok |= (uint32_t)(pid[first + i] >= 0) << i;
            loaded = (loaded & ~(3u << 2 * ld_slot)) | ok << 2 * ld_slot;
            flying |= (uint32_t)(ok != 0) << ld_slot;
            __syncwarp();
            if (ok && lane == 0) {
                mbar_arrive_expect_tx(&full[ld_slot], (ok == 3 ? 2 : 1) * kHalf * C::kRow);
                if (C::kItem > kHalf && a.box == kTile) {
                    tma_load_5d(dst, map, 0, tok & page_mask, 0, ld.kh, pid[0], &full[ld_slot]);
                } else {
#pragma unroll
                    for (int i = 0; i < C::kItem / kHalf; ++i)
                        if (ok >> i & 1)
                            tma_load_5d(dst + i * kHalf * C::kRow, map, 0, (tok + kHalf * (first + i)) & page_mask, 0,
                                        ld.kh, pid[first + i], &full[ld_slot]);
                }
            }
            if (++ld_item == 2 * C::kItems) {
                ld_item = 0;
                --ld_left;
                if (++ld.t == ld.tend) {
                    ld_left -= kBlockCost;
                    ld.next_block(a);
                }
            }
        } else {
            loaded &= ~(3u << 2 * ld_slot);
        }
        if (++ld_slot == C::kSlots) ld_slot = 0;
    };
    // Wait for the slot's copy; the bits of its halves.  After an expired wait
    // (the status word says so) no further copy is asked for or waited for.
    uint32_t parity = 0;    // bit of a slot: the phase to wait for
    bool failed = false;
    auto landed = [&](int slot) {
        const uint32_t has = loaded >> 2 * slot & 3;
        if (has && !failed) {
            if (__all_sync(kAll, mbar_wait(&full[slot], parity >> slot & 1, a.status))) {
                parity ^= 1u << slot;
                flying &= ~(1u << slot);
            } else {
                failed = true;
                ld_left = 0;
            }
        }
        return has;
    };
#pragma unroll 1
    for (int i = 0; i < C::kSlots; ++i) issue();

    // 16-bit rows: a lane's row of the matrices that make a fragment, k-step (or 16 columns) 0 of a segment
    const uint32_t ring_a = smem_u32(ring);
    const int lane_k = ((lane & 15) << 7) + (((lane >> 4) ^ (lane & 7)) << 4);
    const int lane_v = (((lane & 7) + (lane >> 4 << 3)) << 7) + (((lane >> 3 & 1) ^ (lane & 7)) << 4);

    int slot = 0;
    float o[D / 16][4];
    float m0 = 0, m1 = 0, l0 = 0, l1 = 0;
    int has_head = 0;
    Meta open{0, 0, 0, 0, 0};
    float *head_piece = a.pieces + ((size_t)2 * gridDim.x + (size_t)gw) * piece_floats(D);

    // the output as it stands, without the weights' scale, eight rows of D
    auto put_rows = [&](float *to) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float *row = to + (2 * c + e) * D;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                if constexpr (TYPE == ZQ_E4M3) {
                    constexpr int kPairs = C::kVRun / 2;
                    *reinterpret_cast<float2 *>(row + (8 * (i / kPairs) + g) * C::kVRun + 2 * (i % kPairs)) =
                        make_float2(o[i][e] * C::kWeightDown, o[i][2 + e] * C::kWeightDown);
                } else {
                    row[16 * i + g] = o[i][e] * C::kWeightDown;
                    row[16 * i + 8 + g] = o[i][2 + e] * C::kWeightDown;
                }
            }
        }
    };

    while (left > 0) {
        const int n = (int)min(left, (long long)(at.tend - at.t));
        const bool starts = at.t == at.t0, ends = at.t + n == at.tend;
        const int heads = at.heads(a), head0 = at.head(a);

        // queries of head g, in the columns' order of the key chunks
        uint32_t qf[C::kSplits][D / 16][2];
        float scale0, scale1;
        {
            float x[D / 4];
            const float *qr = a.q + (long long)at.b * a.q_stride + (long long)(head0 + min(g, heads - 1)) * D;
            if constexpr (TYPE == ZQ_E4M3) {   // the columns of the lane's chunks
#pragma unroll
                for (int s = 0; s < D / (4 * C::kKRun); ++s)
#pragma unroll
                    for (int i = 0; i < C::kKRun / 4; ++i) {
                        const float4 f = *reinterpret_cast<const float4 *>(qr + (4 * s + c) * C::kKRun + 4 * i);
                        float *y = x + s * C::kKRun + 4 * i;
                        y[0] = f.x, y[1] = f.y, y[2] = f.z, y[3] = f.w;
                    }
            } else {                           // 2c, 2c + 1 of every eight columns
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    const float2 f = *reinterpret_cast<const float2 *>(qr + 8 * i + 2 * c);
                    x[2 * i] = f.x;
                    x[2 * i + 1] = f.y;
                }
            }
            float back = 1.0f;
            if constexpr (TYPE != ZQ_BF16) {
                float amax = 0.0f;
#pragma unroll
                for (int i = 0; i < D / 4; ++i) amax = fmaxf(amax, fabsf(x[i]));
                amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, 1));
                amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, 2));
                const int e = min(max((int)(__float_as_uint(amax) >> 23) - 127, -126), 126);
                const float down = __int_as_float((127 - e) << 23);
                back = __int_as_float((127 + e) << 23);
#pragma unroll
                for (int i = 0; i < D / 4; ++i) x[i] *= down;
            }
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                float lo = x[2 * i], hi = x[2 * i + 1];
#pragma unroll
                for (int p = 0; p < C::kSplits; ++p) {
                    const uint32_t w = pack16<TYPE>(lo, hi);
                    qf[p][i / 2][i % 2] = w;
                    const float2 f = unpack16<TYPE>(w);
                    lo -= f.x;
                    hi -= f.y;
                }
            }
            // positive and finite: times 0 a masked -infinity, times infinity a score of 0 would be NaN
            back = fminf(fmaxf(a.qk_scale * back, __uint_as_float(1)), FLT_MAX);
            scale0 = __shfl_sync(kAll, back, 8 * c);
            scale1 = __shfl_sync(kAll, back, 8 * c + 4);
        }
#pragma unroll
        for (int i = 0; i < D / 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
        m0 = m1 = -INFINITY;
        l0 = l1 = 0.0f;

#pragma unroll 1
        for (int i = 0; i < n; ++i) {
            // scores: two S^T [16 tokens x 8 heads], an accumulator for each part of q
            float sc[2][4];
            bool ok[2];
            uint32_t has = 0;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (C::kItems == 2 || h == 0) has = landed(slot);
                ok[h] = has >> (C::kItems == 2 ? 0 : h) & 1;
                const int from = slot * C::kSlot + (C::kItems == 2 ? 0 : h * half_stride);
                float acc[C::kSplits][4];
                auto product = [&](int k, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
                    for (int p = 0; p < C::kSplits; ++p) {
                        if (k == 0) mma16_first<TYPE>(acc[p], a0, a1, a2, a3, qf[p][k][0], qf[p][k][1]);
                        else mma16<TYPE>(acc[p], a0, a1, a2, a3, qf[p][k][0], qf[p][k][1]);
                    }
                };
                if constexpr (TYPE == ZQ_E4M3) {
#pragma unroll
                    for (int s = 0; s < C::kSegs; ++s)
#pragma unroll
                        for (int u = 0; u < C::kKBytes / 16; ++u) {
                            const int chunk = C::kKBytes / 16 * c + u;
                            const uint8_t *src = ring + from + s * seg_stride;
                            const uint4 ra = *reinterpret_cast<const uint4 *>(src + swizzled<C::kSeg>(g, chunk));
                            const uint4 rb = *reinterpret_cast<const uint4 *>(src + swizzled<C::kSeg>(g + 8, chunk));
                            const uint32_t wa[4] = {ra.x, ra.y, ra.z, ra.w}, wb[4] = {rb.x, rb.y, rb.z, rb.w};
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                uint32_t a0, a1, a2, a3;
                                e4m3_f16(wa[j], a0, a2);
                                e4m3_f16(wb[j], a1, a3);
                                product((s * (C::kKBytes / 16) + u) * 4 + j, a0, a1, a2, a3);
                            }
                        }
                } else {
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        uint32_t a0, a1, a2, a3;
                        ldmatrix4<false>(ring_a + from + k / 4 * seg_stride + (lane_k ^ (k % 4 << 5)), a0, a1, a2, a3);
                        product(k, a0, a1, a2, a3);
                    }
                }
                if (C::kItems == 2 || h == 1) {
                    issue();
                    if (++slot == C::kSlots) slot = 0;
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {   // the small parts first
                    float v = acc[C::kSplits - 1][e];
#pragma unroll
                    for (int p = C::kSplits - 2; p >= 0; --p) v += acc[p][e];
                    // an infinite key makes the first part's score infinite, and the lower ones' NaN where those parts
                    // are zeros or of the other sign (e4m3 has no infinities)
                    if constexpr (TYPE != ZQ_E4M3) v = fabsf(acc[0][e]) == INFINITY ? acc[0][e] : v;
                    sc[h][e] = v;
                }
            }
            const int tok = (at.t + i) * kTile;
            const bool whole = ok[0] && ok[1] && tok >= at.lo && tok + kTile <= at.len;
            if (!whole) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int row = tok + kHalf * h + g + 8 * (e >> 1);
                        if (!(ok[h] && row >= at.lo && row < at.len)) sc[h][e] = -INFINITY;
                    }
            }

            // running maximum over the tile's tokens, per head (columns 2c, 2c + 1)
            float x0 = fmaxf(fmaxf(sc[0][0], sc[0][2]), fmaxf(sc[1][0], sc[1][2]));
            float x1 = fmaxf(fmaxf(sc[0][1], sc[0][3]), fmaxf(sc[1][1], sc[1][3]));
#pragma unroll
            for (int off = 4; off <= 16; off <<= 1) {
                x0 = fmaxf(x0, __shfl_xor_sync(kAll, x0, off));
                x1 = fmaxf(x1, __shfl_xor_sync(kAll, x1, off));
            }
            x0 = fmaxf(x0 * scale0, m0);   // the scales are positive
            x1 = fmaxf(x1 * scale1, m1);
            // nothing seen yet: subtract 0, not the -infinity
            const float u0m = x0 == -INFINITY ? 0.0f : x0, u1m = x1 == -INFINITY ? 0.0f : x1;
            const float f0 = ex2(m0 - u0m), f1 = ex2(m1 - u1m);
            m0 = x0;
            m1 = x1;
            l0 *= f0;
            l1 *= f1;
            uint32_t bp[2][C::kSplits][2];   // weights of 16 tokens x 8 heads, their parts
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float p0 = ex2(__fmaf_rn(sc[h][0], scale0, -u0m)), p1 = ex2(__fmaf_rn(sc[h][1], scale1, -u1m));
                const float p2 = ex2(__fmaf_rn(sc[h][2], scale0, -u0m)), p3 = ex2(__fmaf_rn(sc[h][3], scale1, -u1m));
                l0 += p0 + p2;
                l1 += p1 + p3;
                float r[4] = {p0 * C::kWeightUp, p1 * C::kWeightUp, p2 * C::kWeightUp, p3 * C::kWeightUp};
#pragma unroll
                for (int p = 0; p < C::kSplits; ++p) {
                    const uint32_t w0 = pack16<TYPE>(r[0], r[1]), w1 = pack16<TYPE>(r[2], r[3]);
                    const float2 f0 = unpack16<TYPE>(w0), f1 = unpack16<TYPE>(w1);
                    bp[h][p][0] = transpose8(w0);
                    bp[h][p][1] = transpose8(w1);
                    r[0] -= f0.x;
                    r[1] -= f0.y;
                    r[2] -= f1.x;
                    r[3] -= f1.y;
                }
            }

            // O^T [16 columns x 8 heads] += V^T p: rows g and g + 8 of a product are two neighbouring columns.
            // A tile's products start from zero and are added to the scaled output outside the tensor core,
            // whose accumulator truncates: summed there, hundreds of tiles of one sign lose 1e-5.
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (C::kItems == 2 || h == 0) landed(slot);
                const int from = slot * C::kSlot + (C::kItems == 2 ? 0 : h * half_stride);
                auto product = [&](float(&to)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
                    float y[4];
                    mma16_first<TYPE>(y, a0, a1, a2, a3, bp[h][C::kSplits - 1][0], bp[h][C::kSplits - 1][1]);
#pragma unroll
                    for (int p = C::kSplits - 2; p >= 0; --p) mma16<TYPE>(y, a0, a1, a2, a3, bp[h][p][0], bp[h][p][1]);
                    if (h == 0) {
                        to[0] = to[0] * f0 + y[0];
                        to[1] = to[1] * f1 + y[1];
                        to[2] = to[2] * f0 + y[2];
                        to[3] = to[3] * f1 + y[3];
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e) to[e] += y[e];
                    }
                };
                // row r of 2c, 2c + 1, 2c + 8, 2c + 9 of the half is attended to (asked only where some are not)
                auto in = [&](int r) {
                    const int row = tok + kHalf * h + 2 * c + (r & 1) + 8 * (r >> 1);
                    return ok[h] && row >= at.lo && row < at.len;
                };
                if constexpr (TYPE == ZQ_E4M3) {
#pragma unroll
                    for (int s = 0; s < C::kSegs; ++s) {
                        uint32_t w[4][C::kVBytes / 4];
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const int row = 2 * c + (r & 1) + 8 * (r >> 1);
                            const uint8_t *src = ring + from + s * seg_stride;
                            if constexpr (C::kVBytes == 16) {
                                const uint4 f = *reinterpret_cast<const uint4 *>(src + swizzled<C::kSeg>(row, g));
                                w[r][0] = f.x, w[r][1] = f.y, w[r][2] = f.z, w[r][3] = f.w;
                            } else {
                                const uint2 f = *reinterpret_cast<const uint2 *>(
                                    src + swizzled<C::kSeg>(row, g >> 1) + 8 * (g & 1));
                                w[r][0] = f.x, w[r][1] = f.y;
                            }
                        }
                        if (!whole) {
#pragma unroll
                            for (int r = 0; r < 4; ++r)
#pragma unroll
                                for (int j = 0; j < C::kVBytes / 4; ++j) w[r][j] = in(r) ? w[r][j] : 0;
                        }
#pragma unroll
                        for (int j = 0; j < C::kVRun / 2; ++j) {
                            uint32_t a0, a1, a2, a3;   // two columns of tokens 2c, 2c + 1, and of 2c + 8, 2c + 9
                            const int sel = j & 1 ? 0x7362 : 0x5140;
                            e4m3_f16(__byte_perm(w[0][j / 2], w[1][j / 2], sel), a0, a1);
                            e4m3_f16(__byte_perm(w[2][j / 2], w[3][j / 2], sel), a2, a3);
                            product(o[s * (C::kVRun / 2) + j], a0, a1, a2, a3);
                        }
                    }
                } else {
                    uint32_t keep0 = ~0u, keep1 = ~0u;
                    if (!whole) {
                        keep0 = (in(0) ? 0xffffu : 0) | (in(1) ? 0xffff0000u : 0);
                        keep1 = (in(2) ? 0xffffu : 0) | (in(3) ? 0xffff0000u : 0);
                    }
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        uint32_t a0, a1, a2, a3;
                        ldmatrix4<true>(ring_a + from + k / 4 * seg_stride + (lane_v ^ (k % 4 << 5)), a0, a1, a2, a3);
                        if (!whole) {
                            a0 &= keep0;
                            a1 &= keep0;
                            a2 &= keep1;
                            a3 &= keep1;
                        }
                        product(o[k], a0, a1, a2, a3);
                    }
                }
                if (C::kItems == 2 || h == 1) {
                    issue();
                    if (++slot == C::kSlots) slot = 0;
                }
            }
        }
#pragma unroll
        for (int off = 4; off <= 16; off <<= 1) {
            l0 += __shfl_xor_sync(kAll, l0, off);
            l1 += __shfl_xor_sync(kAll, l1, off);
        }
        left -= n;

        if (starts && ends) {   // the whole row block: finish it
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int h = 2 * c + e;
                const bool store = h < heads;
                const float l = e ? l1 : l0, f = row_factor(l, a.v_scale);
                float *row = a.out + (long long)at.b * a.out_stride + (long long)(head0 + h) * D;
                const size_t code0 = ((size_t)at.b * a.Hq + head0 + h) * D;
                if constexpr (TYPE == ZQ_E4M3) {
#pragma unroll
                    for (int s = 0; s < C::kSegs; ++s) {
                        float y[C::kVRun];
#pragma unroll
                        for (int j = 0; j < C::kVRun / 2; ++j) {
                            y[2 * j] = o[s * (C::kVRun / 2) + j][e] * C::kWeightDown * f;
                            y[2 * j + 1] = o[s * (C::kVRun / 2) + j][2 + e] * C::kWeightDown * f;
                        }
                        const int d0 = (8 * s + g) * C::kVRun;
                        if (store && a.out) {
#pragma unroll
                            for (int q = 0; q < C::kVRun / 4; ++q)
                                reinterpret_cast<float4 *>(row + d0)[q] =
                                    make_float4(y[4 * q], y[4 * q + 1], y[4 * q + 2], y[4 * q + 3]);
                        }
                        if (a.q8.qs)
                            q8_block<C::kVRun, 4, C::kVRun == 8 ? 8 : 0, 0>(a.q8, code0 + d0, y, store,
                                                                           (d0 & 31) == 0);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < D / 16; i += 2) {
                        const float y[4] = {o[i][e] * C::kWeightDown * f, o[i][2 + e] * C::kWeightDown * f,
                                            o[i + 1][e] * C::kWeightDown * f, o[i + 1][2 + e] * C::kWeightDown * f};
                        if (store && a.out) {
#pragma unroll
                            for (int k = 0; k < 4; ++k) row[16 * i + 8 * k + g] = y[k];
                        }
                        if (a.q8.qs) q8_block_strided(a.q8, code0 + 16 * i, y, g, store);
                    }
                }
                if (store && a.lse && g == 0) a.lse[(size_t)at.b * a.Hq + head0 + h] = row_lse(e ? m1 : m0, l);
            }
            left -= kBlockCost;
            at.next_block(a);
        } else if (ends) {      // began in an earlier warp: to the workspace
            has_head = 1;
            put_rows(head_piece);
            if (g == 0) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    head_piece[kHeads * D + 2 * c + e] = e ? m1 : m0;
                    head_piece[kHeads * D + kHeads + 2 * c + e] = e ? l1 : l0;
                }
            }
            left -= kBlockCost;
            at.next_block(a);
        } else {                // goes on in the next warp: the last one here
            open = Meta{0, starts ? 1 : 2, at.b, head0, heads};
        }
    }
    if (failed) {   // copies still in flight land before the ring's place is used again
        for (int i = 0; i < C::kSlots; ++i)
            if (flying >> i & 1) mbar_wait_for(&full[i], parity >> i & 1, nullptr, 1000000ull);
    }
    __syncthreads();   // every warp's ring is done: its place holds the open pieces now
    float *pieces_s = reinterpret_cast<float *>(smem);
    if (open.b) {
        put_rows(pieces_s + (size_t)warp * kHeads * D);
        if (g == 0) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                m_s[warp][2 * c + e] = e ? m1 : m0;
                l_s[warp][2 * c + e] = e ? l1 : l0;
            }
        }
    }
    if (lane == 0) {
        head_s[warp] = has_head;
        open_s[warp] = open;
    }
    __syncthreads();

    // ---- join the CTA's pieces, one warp for each head of a run: the open pieces of
    // warps w0 .. w1 - 1 of one row block and, when it ends here, the ending one of
    // warp w1.  Bits of a warp: an ending piece, an open one, one that begins in it.
    const bool there = lane < kWarps;
    const uint32_t ending = __ballot_sync(kAll, there && head_s[there ? lane : 0]);
    const uint32_t opened = __ballot_sync(kAll, there && open_s[there ? lane : 0].b);
    const uint32_t begun = __ballot_sync(kAll, there && open_s[there ? lane : 0].b == 1);
    const int ends_here = __popc(ending);
    // run r < ends_here ends with the r-th ending piece; after them there may be one that goes on
    const uint32_t after = ending ? ~0u << (31 - __clz((int)ending)) : ~0u;
    const int runs = ends_here + ((opened & after) != 0);
    auto run_of = [&](int r, int &w0, int &w1, bool &begins) {
        uint32_t e = ending, from = ~0u;
        for (int i = 0; i < r; ++i) {
            from = ~0u << (__ffs((int)e) - 1);
            e &= e - 1;
        }
        w1 = e ? __ffs((int)e) - 1 : kWarps;
        const uint32_t o = opened & from & ((1u << w1) - 1);
        w0 = o ? __ffs((int)o) - 1 : w1;
        begins = o && (begun >> w0 & 1);
    };
    if (tid == 0) {
        Meta info{0, 0, 0, 0, 0};   // what this CTA leaves to the second kernel
        int w0, w1;
        bool begins;
        if (runs) {
            run_of(0, w0, w1, begins);
            const int a_state = begins ? 0 : ends_here ? 2 : 1;
            run_of(runs - 1, w0, w1, begins);
            if (runs > ends_here && begins) info = open_s[w0];
            info.a = a_state;
        }
        meta[blockIdx.x] = info;
    }
    // An item is a head of a run; all of its run's ending piece comes from the workspace at once.  (The next item's
    // on its way as well costs the main loop more than it gives: 200 windows 40.8 us, 43.1 so.)
    struct Item {
        int h, w0, w1;
        bool begins, ends;
        float pm, pl;
        float4 tail[(D + 127) / 128];
    };
    auto item = [&](int i, Item &x) {
        const int r = i / a.per_pass;
        x.h = i - r * a.per_pass;
        run_of(r, x.w0, x.w1, x.begins);
        x.ends = r < ends_here;
        x.pm = -INFINITY;
        x.pl = 0.0f;
        if (!x.ends) return;
        const float *tail = a.pieces + ((size_t)2 * gridDim.x + (size_t)blockIdx.x * kWarps + x.w1) * piece_floats(D);
        if (lane == 31) {
            x.pm = tail[kHeads * D + x.h];
            x.pl = tail[kHeads * D + kHeads + x.h];
        }
#pragma unroll
        for (int d0 = 0; d0 < D; d0 += 128)
            x.tail[d0 / 128] = *reinterpret_cast<const float4 *>(tail + x.h * D + d0 + (D < 128 ? 4 * lane % D : 4 * lane));
    };
    auto join = [&](const Item &x) {
        const int h = x.h;
        if (x.begins && h >= open_s[x.w0].heads) return;
        // lane w has the maximum, the sum and then the weight of warp w's piece, lane 31 the ending one's
        const uint32_t pieces = opened & ((1u << x.w1) - 1) & (~0u << x.w0);   // (a call of few tiles leaves gaps)
        float pm = x.pm, pl = x.pl;
        if (pieces >> lane & 1) {
            pm = m_s[lane][h];
            pl = l_s[lane][h];
        }
        float m = pm;
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, off));
        const float f = ex2(pm - (m == -INFINITY ? 0.0f : m));
        const float l = warp_sum((pieces >> lane & 1) || (x.ends && lane == 31) ? f * pl : 0.0f);
#pragma unroll
        for (int d0 = 0; d0 < D; d0 += 128) {
            const int d = d0 + 4 * lane;
            const bool in = d < D;
            float y[4] = {};
            auto add = [&](const float4 &v, float f) {
                y[0] += f * v.x;
                y[1] += f * v.y;
                y[2] += f * v.z;
                y[3] += f * v.w;
            };
#pragma unroll 4
            for (int w = x.w0; w < x.w1; ++w) {
                const float fw = __shfl_sync(kAll, f, w);
                if (pieces >> w & 1)
                    add(*reinterpret_cast<const float4 *>(pieces_s + ((size_t)w * kHeads + h) * D + (in ? d : 0)), fw);
            }
            const float ft = __shfl_sync(kAll, f, 31);
            if (x.ends) add(x.tail[d0 / 128], ft);
            if (x.begins && x.ends) {
                const float g = row_factor(l, a.v_scale);
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] *= g;
                const int seq = open_s[x.w0].seq, head = open_s[x.w0].head + h;
                if (in && a.out)
                    *reinterpret_cast<float4 *>(a.out + (long long)seq * a.out_stride + (long long)head * D +
                                                d) = make_float4(y[0], y[1], y[2], y[3]);
                if (a.q8.qs)
                    q8_block<4, 1, 2, 4>(a.q8, ((size_t)seq * a.Hq + head) * D + d, y, in, (d & 31) == 0);
                if (d == 0 && a.lse) a.lse[(size_t)seq * a.Hq + head] = row_lse(m, l);
            } else if (in) {
                float *to = a.pieces + (size_t)(2 * blockIdx.x + (x.begins ? 1 : 0)) * piece_floats(D);
                *reinterpret_cast<float4 *>(to + h * D + d) = make_float4(y[0], y[1], y[2], y[3]);
                if (d == 0) {
                    to[kHeads * D + h] = m;
                    to[kHeads * D + kHeads + h] = l;
                }
            }
        }
    };
    const int items = runs * a.per_pass;
    for (int i = warp; i < items; i += kWarps) {
        Item x;
        item(i, x);
        join(x);
    }
}

// Row blocks that cross CTAs: block (c, h) joins head h of the one that begins
// in CTA c of the first kernel, from that CTA's piece and those of the CTAs
// that follow, to the one where it ends.  Warp w takes pieces w, w + 8, ...,
// lane j the weight of its j-th, so that nothing but the last step waits for
// another warp: this kernel is a chain of latencies (with a pass over all
// pieces' maxima and two more barriers it took 0.3 us more).
template <int D>
__global__ void __launch_bounds__(kJoinThreads) paged_attn_join_kernel(const __grid_constant__ PagedAttnArgs a, int ctas)
{
    constexpr int kWarps = kJoinThreads / 32, kChunks = (D + 127) / 128, kAhead = 4;
    static_assert(kWarps * 32 >= kMaxAttnCtas, "a warp's lanes hold the weights of its pieces");
    __shared__ float m_s[kWarps], l_s[kWarps];
    __shared__ float4 y_s[kWarps][D / 4];
    pdl_wait();
    pdl_launch_dependents();
    const int warp = __shfl_sync(kAll, threadIdx.x >> 5, 0), lane = threadIdx.x & 31, first = blockIdx.x, h = blockIdx.y;
    const Meta *meta = reinterpret_cast<const Meta *>(a.meta);
    const Meta mine = meta[first];
    // the CTA where it ends, 32 of those that follow at a time
    int at = first + 1;
    int state = at + lane < ctas ? meta[at + lane].a : 0;
    if (!mine.b || h >= mine.heads) return;
    uint32_t found = __ballot_sync(kAll, state == 2);
    while (!found && at + 32 < ctas) {
        at += 32;
        state = at + lane < ctas ? meta[at + lane].a : 0;
        found = __ballot_sync(kAll, state == 2);
    }
    const int n = (found ? at + __ffs((int)found) - 1 : ctas - 1) - first + 1;

    // piece i: the beginning in its CTA's second place, the others in their first
    auto piece = [&](int i) { return a.pieces + (size_t)(2 * (first + i) + (i == 0)) * piece_floats(D); };
    const int count = n > warp ? (n - warp + kWarps - 1) / kWarps : 0;   // this warp's pieces
    float pm = -INFINITY, pl = 0.0f;
    if (lane < count) {
        pm = piece(warp + kWarps * lane)[kHeads * D + h];
        pl = piece(warp + kWarps * lane)[kHeads * D + kHeads + h];
    }
    const int col = D < 128 ? 4 * (lane % (D / 4)) : 4 * lane;   // (64-wide rows: half the lanes repeat the other)
    auto row = [&](int j) { return piece(warp + kWarps * j) + h * D + col; };
    float4 v[kAhead][kChunks];   // the first pieces' values come beside their m and l
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
        if (j < count)
#pragma unroll
            for (int k = 0; k < kChunks; ++k) v[j][k] = *reinterpret_cast<const float4 *>(row(j) + 128 * k);
    float4 y[kChunks];
#pragma unroll
    for (int k = 0; k < kChunks; ++k) y[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float m = pm;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, off));
    const float f = ex2(pm - (m == -INFINITY ? 0.0f : m));
    const float l = warp_sum(lane < count ? f * pl : 0.0f);
    auto add = [&](float fj, const float4(&v)[kChunks]) {
#pragma unroll
        for (int k = 0; k < kChunks; ++k) {
            y[k].x += fj * v[k].x;
            y[k].y += fj * v[k].y;
            y[k].z += fj * v[k].z;
            y[k].w += fj * v[k].w;
        }
    };
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
        if (j < count) add(__shfl_sync(kAll, f, j), v[j]);
#pragma unroll 4
    for (int j = kAhead; j < count; ++j) {
        float4 x[kChunks];
#pragma unroll
        for (int k = 0; k < kChunks; ++k) x[k] = *reinterpret_cast<const float4 *>(row(j) + 128 * k);
        add(__shfl_sync(kAll, f, j), x);
    }
#pragma unroll
    for (int k = 0; k < kChunks; ++k) y_s[warp][col / 4 + 32 * k] = y[k];
    if (lane == 0) {
        m_s[warp] = m;
        l_s[warp] = l;
    }
    __syncthreads();
    if (warp) return;
    // the warps' sums
    const int nw = min(n, kWarps);
    float all = -INFINITY, sum = 0.0f;
    for (int w = 0; w < nw; ++w) all = fmaxf(all, m_s[w]);
    const float u = all == -INFINITY ? 0.0f : all;
#pragma unroll
    for (int k = 0; k < kChunks; ++k) y[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int w = 0; w < nw; ++w) {
        const float fw = ex2(m_s[w] - u);
        sum += fw * l_s[w];
#pragma unroll
        for (int k = 0; k < kChunks; ++k) {
            const float4 v = y_s[w][col / 4 + 32 * k];
            y[k].x += fw * v.x;
            y[k].y += fw * v.y;
            y[k].z += fw * v.z;
            y[k].w += fw * v.w;
        }
    }
    const float factor = row_factor(sum, a.v_scale);
    const int head = mine.head + h;
    const bool store = D >= 128 || lane < D / 4;
#pragma unroll
    for (int k = 0; k < kChunks; ++k) {
        const float v[4] = {y[k].x * factor, y[k].y * factor, y[k].z * factor, y[k].w * factor};
        const int d = col + 128 * k;
        if (store && a.out)
            *reinterpret_cast<float4 *>(a.out + (long long)mine.seq * a.out_stride + (long long)head * D + d) =
                make_float4(v[0], v[1], v[2], v[3]);
        if (a.q8.qs)
            q8_block<4, 1, 2, 4>(a.q8, ((size_t)mine.seq * a.Hq + head) * D + d, v, store, (d & 31) == 0);
    }
    if (lane == 0 && a.lse) a.lse[(size_t)mine.seq * a.Hq + head] = row_lse(all, sum);
}

template <int D, int TYPE>
cudaError_t launch_one(const PagedAttnArgs &a, int ctas, cudaStream_t st)
{
    using C = Cfg<D, TYPE>;
    static std::atomic<bool> set[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!set[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(paged_attn_kernel<D, TYPE>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
        if (e != cudaSuccess) return e;
        set[dev].store(true, std::memory_order_release);
    }
    // [page][key head][segment][row][bytes of a segment]; a box is all segments of 16 or 32 rows
    const uint64_t page = (uint64_t)1 << a.page_shift;
    const uint64_t dims[5] = {C::kSeg, page, C::kSegs, (uint64_t)a.Hk, (uint64_t)a.pages};
    const uint64_t strides[4] = {C::kRow, C::kSeg, page * C::kRow, page * C::kRow * a.Hk};
    const uint32_t box[5] = {C::kSeg, (uint32_t)(C::kItem > kHalf ? a.box : kHalf), C::kSegs, 1, 1};
    const CUtensorMapSwizzle sw = C::kSeg == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
    CUtensorMap mk, mv;
    if ((e = make_tmap_u8(&mk, 5, a.k, dims, strides, box, sw)) != cudaSuccess) return e;
    if ((e = make_tmap_u8(&mv, 5, a.v, dims, strides, box, sw)) != cudaSuccess) return e;
    e = launch_pdl(paged_attn_kernel<D, TYPE>, dim3(ctas), dim3(C::kThreads), C::kSmem, st, a, mk, mv);
    if (e != cudaSuccess) return e;
    return launch_pdl(paged_attn_join_kernel<D>, dim3(ctas, a.per_pass), dim3(kJoinThreads), 0, st, a, ctas);
}

template <int D>
cudaError_t launch_type(const PagedAttnArgs &a, int type, int ctas, cudaStream_t st)
{
    switch (type) {
    case ZQ_F16: return launch_one<D, ZQ_F16>(a, ctas, st);
    case ZQ_BF16: return launch_one<D, ZQ_BF16>(a, ctas, st);
    default: return launch_one<D, ZQ_E4M3>(a, ctas, st);
    }
}

int attn_ctas()
{
    const int n = num_sms();
    return n < kMaxAttnCtas ? n : kMaxAttnCtas;
}

size_t pad256(size_t n) { return (n + 255) & ~(size_t)255; }

}  // namespace

// Pieces: two per CTA, one per warp; then the CTAs' records.
size_t paged_attn_workspace(int D)
{
    const size_t n = (size_t)attn_ctas();
    return pad256(n * (2 + kMaxWarps) * piece_floats(D) * sizeof(float)) + pad256(n * sizeof(Meta));
}

cudaError_t launch_paged_attn(const PagedAttnArgs &args, int D, int type, void *workspace, cudaStream_t st)
{
    PagedAttnArgs a = args;
    const int ctas = attn_ctas();
    a.G = a.Hq / a.Hk;
    a.passes = (a.G + kHeads - 1) / kHeads;
    a.per_pass = (a.G + a.passes - 1) / a.passes;
    a.box = a.page_shift > 4 ? kTile : kHalf;   // rows of a page that one copy brings
    a.status = device_status_word();
    a.pieces = static_cast<float *>(workspace);
    a.meta = static_cast<char *>(workspace) + pad256((size_t)ctas * (2 + kMaxWarps) * piece_floats(D) * sizeof(float));
    switch (D) {
    case 64: return launch_type<64>(a, type, ctas, st);
    case 128: return launch_type<128>(a, type, ctas, st);
    default: return launch_type<256>(a, type, ctas, st);
    }
}

}  // namespace zq
