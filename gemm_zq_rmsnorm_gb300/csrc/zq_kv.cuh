// zq_kv.cuh -- launch descriptions of the attention-side and adapter
// operators, and the rounding of fp32 values to their types.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "zq.h"

namespace zq {

template <int TYPE> struct KvBytes { static constexpr int value = TYPE == ZQ_E4M3 ? 1 : 2; };

// Two fp32 values to two stored ones, `lo` at the lower address: nearest even;
// e4m3 saturates, NaN stays NaN.
template <int TYPE>
__device__ __forceinline__ uint32_t kv_pack2(float lo, float hi)
{
    uint32_t r;
    if constexpr (TYPE == ZQ_F16) {
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    } else if constexpr (TYPE == ZQ_BF16) {
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    } else {
        uint16_t h;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h) : "f"(hi), "f"(lo));
        r = h;
    }
    return r;
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// log2 of the page size (host; page is a power of two)
inline int page_shift(int page)
{
    int s = 0;
    while ((1 << s) < page) ++s;
    return s;
}

struct HeadNormRopeArgs {
    const float *q, *k, *v;
    long long q_stride, k_stride, v_stride;
    int T, Hq, Hk;
    const float *gamma_q, *gamma_k;
    float eps;
    const uint64_t *table;
    int rot, interleaved;
    const int32_t *pos;
    int axes;
    void *kc, *vc;
    int page_shift;
    long long nslots;
    float k_scale, v_scale;
    const int32_t *slots;
    float *q_out;
    long long q_out_stride;
    int chunk, chunks;   // rows per warp, warps per token (set by the launcher)
};
cudaError_t launch_head_norm_rope(const HeadNormRopeArgs &a, int D, int type, cudaStream_t st);

constexpr int kMaxAttnCtas = 256;   // more SMs than any GPU of this architecture has
struct PagedAttnArgs {
    const float *q;
    long long q_stride;
    int B, Hq, Hk;
    const char *k, *v;
    int pages, page_shift;
    const int32_t *table;
    int width;
    const int32_t *lens;
    int window;
    float qk_scale;   // scale * k_scale * log2 e
    float v_scale;
    float *out;       // may be null
    long long out_stride;
    float *lse;       // may be null
    zq_q8_1 q8;       // qs may be null
    // set by the launcher
    int G, passes, per_pass;   // query heads of a key head, in passes of up to eight
    float *pieces;
    void *meta;
    int box;
    unsigned int *status;
};
size_t paged_attn_workspace(int D);
cudaError_t launch_paged_attn(const PagedAttnArgs &a, int D, int type, void *workspace, cudaStream_t st);

struct LoraArgs {
    const int8_t *qs;       // activations of B tokens x K
    const uint16_t *d;
    int B, K, R;
    const int32_t *ids;
    int n;                  // adapters
    const char *A, *Bm;
    const float *scales;    // may be null
    int N;
    const float *base;      // may be null, or y
    long long base_stride;
    float *y;
    long long y_stride;
    int vec;                // base and y rows are 16-byte pieces
    float *h;               // workspace [parts][B][R]
    int cluster, parts, per_split, blocks;   // set by the launcher
};
size_t lora_workspace(int B, int K, int R);
cudaError_t launch_lora(const LoraArgs &a, int type, cudaStream_t st);

}  // namespace zq
