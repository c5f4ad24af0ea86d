// linear_prompt.cu -- linear attention with a decay for each head over prompts: the
// cut of long sequences into segments and the join of their states.
//
// A CTA walks through a sequence chunk after chunk, so a few long sequences of a few
// heads would leave most of the GPU idle.  Then every sequence is cut into segments:
// a first kernel finds what each but the last adds to the state (42 of 129 us at 4096
// tokens of 48 heads), a second one makes the states that many segments start from,
// and the third does the rest.
#include "linear_prompt.cuh"

namespace zq {
namespace {

constexpr int C = kChunk;
constexpr int kSlots = 152;        // CTAs that the plan cuts long sequences for
constexpr int kMaxCut = 512;       // sequences of a call up to which they are cut (more fill the GPU by themselves)
// Segments of a sequence up to which no kernel joins their states: each makes its own
// start from those before it (4096 tokens of 48 heads, three segments, 134.2 us against
// 138.0; of 19 segments the last would read a megabyte first).
constexpr int kFew = 4;

// Segments: every sequence in pieces of `length` tokens, at least one.
struct Plan {
    int length;        // tokens, a multiple of C; 0: sequences are not cut
    int segments;      // at most, over all sequences
    bool few;          // of one sequence
};

Plan plan_of(int T, int B, int Hv, int Dv)
{
    const int ctas = Hv * ((Dv + 127) / 128);
    const int n = kSlots / ctas;
    if (B > kMaxCut || n < 2 || T <= 2 * C) return {0, B, false};
    const int length = ((T + n - 1) / n + C - 1) / C * C;
    if (length >= T) return {0, B, false};
    return {length, T / length + B, n <= kFew};
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
    int n = segments_of(p, b);
    if (n < 2) return;
    if (threadIdx.x < 32) {   // segments of the sequences before this one
        int sum = 0;
        for (int i = threadIdx.x; i < b; i += 32) sum += segments_of(p, i);
        sum = __reduce_add_sync(0xffffffffu, sum);
        if (threadIdx.x == 0) base_s = sum;
    }
    __syncthreads();
    const int base = base_s;
    n = within_room(p, base, n);
    if (n < 1) return;
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
            const long long f = p.decay[(long long)(base + i) * a.Hv + h];
            first = make_float4(decayed(first.x, f, mine.x), decayed(first.y, f, mine.y), decayed(first.z, f, mine.z),
                                decayed(first.w, f, mine.w));
            mine = next;
        }
    }
}

cudaError_t launch_shape(const PromptArgs &p, int Dk, cudaStream_t st)
{
    if (p.length) {
        cudaError_t e = launch_linear_prompt_tc(p, Dk, true, st);
        if (e != cudaSuccess) return e;
        if (!p.few) {
            e = launch_pdl(linear_join_kernel, dim3(Dk * p.Dv / 1024, p.a.Hv, p.a.B), dim3(256), 0, st, p, Dk);
            if (e != cudaSuccess) return e;
        }
    }
    return launch_linear_prompt_tc(p, Dk, false, st);
}

size_t state_bytes(const Plan &plan, int Hv, int Dk, int Dv) { return (size_t)plan.segments * Hv * Dk * Dv * 4; }

}  // namespace

void linear_segments(const LinearAttnArgs &a, int Dv, int32_t *out)
{
    const Plan plan = plan_of(a.T, a.B, a.Hv, Dv);
    PromptArgs p{};
    p.a = a;
    p.length = plan.length;
    p.segments = plan.segments;
    out[0] = plan.length;
    out[1] = plan.segments;
    int base = 0;
    for (int b = 0; b < a.B; ++b) {
        const int n = plan.length ? segments_of(p, b) : 1;
        out[2 + 2 * b] = base;
        out[3 + 2 * b] = within_room(p, base, n);
        base += n;
    }
}

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
    p.few = plan.few;
    p.local = static_cast<float *>(workspace);
    if (plan.length) p.decay = reinterpret_cast<long long *>(static_cast<char *>(workspace) + state_bytes(plan, a.Hv, Dk, Dv));
    return launch_shape(p, Dk, st);
}

}  // namespace zq
