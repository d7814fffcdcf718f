// pkv_scored.cu -- decode attention that also adds every cached token's softmax weight
// to an accumulator, summed over the query heads of a KV head:
//
//     p[h][t] = softmax_t(scale * q[b][h] . K_t),   out[b][h] = sum_t p[h][t] V_t,
//     acc_out[b][g][t] = acc[b][g][t] + sum_{h in group g} p[h][t],   t < seq_lens[b].
//
// A weight is known only when the whole sequence's maximum and sum are, so the work is
// two launches.  The first is the grid kernel of pkv_step.cuh over every page, which
// also stores the scores (log2 domain, FP32, the four heads of a token side by side)
// and, from the unit that merges a (sequence, KV head), log2 of each head's sum.  The
// second turns scores into weights and adds them, one (KV head, token) per thread.  It
// re-reads 128 bytes per token where a second pass over the keys would read 1024 (BF16
// pages) or 544 (FP8), and no atomics are involved: the sum has one order.
#include "pkv_step.cuh"

namespace pkv {
namespace {

struct ScoredPages {
    static constexpr bool kIdentity = true, kSortable = true, kLateWait = false, kPublish = false, kLoops = false;
    float *scores;  // [B][8][tokens][4]
    float *lse;     // [B][32] log2 of the sum of 2^score
    int tokens;     // per (sequence, KV head): 16 * max_blocks

    struct EmitOf {
        float *row;  // the (sequence, KV head)'s scores
        struct Emit {
            float *page;
            __device__ __forceinline__ void operator()(int t, int h, float x0, float x1) const
            {
                *reinterpret_cast<float2 *>(page + t * kGroup + h) = make_float2(x0, x1);
            }
        };
        __device__ __forceinline__ Emit operator()(int j) const { return {row + (size_t)j * (kPage * kGroup)}; }
    };

    __device__ __forceinline__ float *row(int b, int g) const
    {
        return scores + ((size_t)b * kHkv + g) * tokens * kGroup;
    }
    __device__ __forceinline__ WholeSequence list(int, int L) const { return {L}; }
    __device__ __forceinline__ EmitOf emit(int b, int g) const { return {row(b, g)}; }
    // A unit that was not computed (a bad page id): its tokens weigh nothing.
    __device__ __forceinline__ void skipped(int b, int g, int j0, int jn) const
    {
        float4 *p = reinterpret_cast<float4 *>(row(b, g)) + (size_t)j0 * kPage;
        for (int t = threadIdx.x; t < jn * kPage; t += kThreads)
            p[t] = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    }
    __device__ __forceinline__ void norm(int b, int h, float M, float l) const
    {
        lse[b * kHq + h] = l > 0.f ? M + log2f(l) : INFINITY;  // nothing computed: every weight is 0
    }
};

constexpr int kAccThreads = 256;
constexpr int kAccTokens = 4 * kAccThreads;  // tokens per CTA, so that long tables make few empty CTAs

__global__ void __launch_bounds__(kAccThreads)
accumulate_kernel(const float4 *__restrict__ scores, const float *__restrict__ lse, const int32_t *__restrict__ seq_lens,
                  int max_blocks, const float *acc, float *acc_out, int64_t acc_stride)
{
    const int g = blockIdx.y, b = blockIdx.z, t0 = blockIdx.x * kAccTokens;
    const int L = seq_lens[b];
    grid_dependency_wait();
    allow_dependent_launch();
    if (L < 1 || L > max_blocks * kPage || t0 >= L)
        return;
    const float4 n = *reinterpret_cast<const float4 *>(lse + b * kHq + g * kGroup);
    const size_t row = (size_t)b * kHkv + g;
    const float4 *x = scores + row * ((size_t)max_blocks * kPage);
#pragma unroll
    for (int i = 0; i < kAccTokens / kAccThreads; ++i) {
        const int t = t0 + i * kAccThreads + threadIdx.x;
        if (t < L) {
            const float4 s = __ldcg(x + t);
            const float w = (ex2_approx(s.x - n.x) + ex2_approx(s.y - n.y)) + (ex2_approx(s.z - n.z) + ex2_approx(s.w - n.w));
            acc_out[row * acc_stride + t] = acc[row * acc_stride + t] + w;
        }
    }
}

struct ScoredWorkspace {
    size_t attention, scores, lse;
    size_t total() const { return attention + scores + lse; }
};

ScoredWorkspace scored_workspace(int B, int max_blocks, int max_chunks)
{
    ScoredWorkspace w;
    w.attention = align256(workspace_layout(B, max_chunks).total());
    w.scores = align256((size_t)B * kHq * max_blocks * kPage * sizeof(float));
    w.lse = align256((size_t)B * kHq * sizeof(float));
    return w;
}

bool scored_args_ok(int B, int max_blocks, int pages_per_chunk)
{
    return B >= 1 && B <= 65535 && max_blocks >= 1 && max_blocks <= (1 << 20) && pages_per_chunk >= 0 &&
           pages_per_chunk <= kMaxPagesPerChunk;
}

}  // namespace
}  // namespace pkv

extern "C" size_t pkv_decode_scored_workspace_bytes(int B, int max_blocks, int pages_per_chunk)
{
    using namespace pkv;
    if (!scored_args_ok(B, max_blocks, pages_per_chunk))
        return 0;
    const int ppc = pages_per_chunk ? pages_per_chunk : default_chunk(B, max_blocks, 2);
    return scored_workspace(B, max_blocks, (max_blocks + ppc - 1) / ppc).total();
}

extern "C" int pkv_decode_scored(const pkv_pool *pool, const uint16_t *q, const int32_t *bt_dev, int max_blocks,
                                 const int32_t *seq_lens_dev, int B, float scale, const float *acc, float *acc_out,
                                 int64_t acc_stride, int pages_per_chunk, void *workspace, size_t workspace_bytes,
                                 uint16_t *out, int32_t *dev_err_flag, void *cuda_stream, int options)
{
    using namespace pkv;
    if (!pool || !q || !bt_dev || !seq_lens_dev || !acc || !acc_out || !workspace || !out ||
        !scored_args_ok(B, max_blocks, pages_per_chunk))
        return PKV_ERR_INVALID_ARG;
    if (!(scale > 0.f) || !(scale < INFINITY) || acc_stride < (int64_t)max_blocks * kPage)
        return PKV_ERR_INVALID_ARG;
    const uintptr_t align =
        reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out) | reinterpret_cast<uintptr_t>(workspace);
    if ((align & 15u) || ((reinterpret_cast<uintptr_t>(acc) | reinterpret_cast<uintptr_t>(acc_out)) & 3u))
        return PKV_ERR_INVALID_ARG;
    if (workspace_bytes < pkv_decode_scored_workspace_bytes(B, max_blocks, pages_per_chunk))
        return PKV_ERR_WORKSPACE_TOO_SMALL;
    const int ppc = pages_per_chunk ? pages_per_chunk : default_chunk(B, max_blocks, 2);
    const ScoredWorkspace w = scored_workspace(B, max_blocks, (max_blocks + ppc - 1) / ppc);
    char *base = static_cast<char *>(workspace);
    ScoredPages sel;
    sel.scores = reinterpret_cast<float *>(base + w.attention);
    sel.lse = reinterpret_cast<float *>(base + w.attention + w.scores);
    sel.tokens = max_blocks * kPage;
    StepArgs a = {};
    a.q = const_cast<uint16_t *>(q);
    a.bt = bt_dev;
    a.seq_lens = seq_lens_dev;
    a.max_pos = INT_MAX;
    a.scale_log2 = scale * kLog2e;
    a.out = out;
    a.err = dev_err_flag;
    cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
    // Largest units first where there are several waves of them and the library chooses: 64
    // sequences up to 16384 tokens (FP8) 85 us instead of 93; with up to 2048 tokens, two waves,
    // the order costs more than it gives (18.8 us instead of 17.2).
    if (pages_per_chunk == 0 && B <= kMaxSortedBatch && (int64_t)B * kHkv * ((max_blocks + ppc - 1) / ppc) > 4 * 152 * 6)
        options |= PKV_STEP_SORTED;
    if (const int st = launch_fused<false>(pool, a, sel, B, max_blocks, max_blocks, 0, ppc, workspace, s, options);
        st != PKV_OK)
        return st;
    const dim3 grid((max_blocks * kPage + kAccTokens - 1) / kAccTokens, kHkv, B);
    return launch_kernel(accumulate_kernel, grid, dim3(kAccThreads), 0, s, !(options & PKV_STEP_NO_PDL),
                         reinterpret_cast<const float4 *>(sel.scores), static_cast<const float *>(sel.lse), seq_lens_dev,
                         max_blocks, acc, acc_out, acc_stride);
}
