// pkv_scored.cu -- decode attention that also adds every cached token's softmax weight
// to an accumulator, summed over the query heads of a KV head:
//
//     p[h][t] = softmax_t(scale * q[b][h] . K_t),   out[b][h] = sum_t p[h][t] V_t,
//     acc_out[b][g][t] = acc[b][g][t] + sum_{h in group g} p[h][t],   t < seq_lens[b].
//
// A weight is known only when the whole sequence's maximum and sum are.  The grid kernel of
// pkv_step.cuh goes over every page and also stores the scores (log2 domain, FP32, the four heads
// of a token side by side); the unit that finishes a (sequence, KV head) knows each head's maximum M
// and log2 of its sum l and turns the scores into weights, 2^((x - M) - log2 l).  (Not 2^(x - (M +
// log2 l)): that sum's rounding at M would be every weight's, up to 4e-5 of it at an M of 2000.)  For short rows it does so itself, while other units
// stream their pages; a long row would keep one CTA busy behind all others, so there a second
// launch does it, one (KV head, token) per thread.
// Either way 128 bytes per token are re-read where a second pass over the keys would read 1024
// (BF16 pages) or 544 (FP8), no atomics are involved, and the sum has one order.
#include "pkv_step.cuh"

namespace pkv {
namespace {

// acc_out[t] = acc[t] + the four heads' weights of token t, from its scores, the heads' maxima and log2
// of their sums, for t = t0, t0 + STEP, ... < L (t0: a multiple of 32, plus the lane): N of them, all read
// before any is written (acc and acc_out may be one array, so the compiler may not reorder them
// itself).
template <int N, int STEP>
__device__ __forceinline__ void add_weights(const float4 *scores, float4 m, float4 n, const float *acc, float *acc_out, int t0, int L)
{
    float4 s[N];
    float a[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int t = t0 + i * STEP;
        if (t < L) {
            s[i] = __ldcg(scores + t);
            a[i] = acc[t];
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int t = t0 + i * STEP;
        if (t < L)
            acc_out[t] = a[i] + ((ex2_approx((s[i].x - m.x) - n.x) + ex2_approx((s[i].y - m.y) - n.y)) +
                                 (ex2_approx((s[i].z - m.z) - n.z) + ex2_approx((s[i].w - m.w) - n.w)));
    }
    // The scores are not needed again: whole lines that this warp has read (its tokens are 32 in a
    // row) are dropped from L2 instead of being written to memory some time later (64 sequences up
    // to 16384 tokens 83 us instead of 90).
    __syncwarp();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int t = t0 + i * STEP;
        if (t % 32 <= 24 && t + 8 <= L && (reinterpret_cast<uintptr_t>(scores + t) & 127) == 0)
            asm volatile("discard.global.L2 [%0], 128;" ::"l"(scores + t) : "memory");
    }
}

template <bool INLINE>
struct ScoredPages {
    static constexpr bool kIdentity = true, kSortable = true, kLateWait = false, kPublish = false, kLoops = false,
                          kFine = true;
    float *scores;  // [B][8][tokens][4]
    float *logs;    // [B][32] log2 of the sum of 2^(score - maximum)
    float2 *tops;   // [B][32][max_chunks] the attention's partials; the first one's place takes the maximum
    int max_chunks;
    int tokens;     // per (sequence, KV head): 16 * max_blocks
    const float *acc;
    float *acc_out;
    int64_t acc_stride;

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
    __device__ __forceinline__ void finished(int b, int g, int L, float M, float l, float *scratch) const
    {
        const int hl = threadIdx.x >> 5;
        const bool some = l > 0.f;  // nothing computed: every weight is 0
        const float m = some ? M : 0.f, n = some ? log2f(l) : INFINITY;
        if (!INLINE) {
            __syncwarp();  // the warp has merged its head's partials
            if ((threadIdx.x & 31) == 0) {
                const int h = b * kHq + g * kGroup + hl;
                logs[h] = n;
                tops[(size_t)h * max_chunks].x = m;
            }
            return;
        }
        __syncthreads();
        if ((threadIdx.x & 31) == 0) {
            scratch[hl] = m;
            scratch[kGroup + hl] = n;
        }
        __syncthreads();
        const float4 ms = *reinterpret_cast<const float4 *>(scratch);
        const float4 ns = *reinterpret_cast<const float4 *>(scratch + kGroup);
        const float4 *x = reinterpret_cast<const float4 *>(row(b, g));
        const size_t at = ((size_t)b * kHkv + g) * acc_stride;
        for (int t0 = 0; t0 < L; t0 += 8 * kThreads)
            add_weights<8, kThreads>(x, ms, ns, acc + at, acc_out + at, t0 + threadIdx.x, L);
    }
};

constexpr int kAccThreads = 256;
constexpr int kAccTokens = 4 * kAccThreads;  // tokens per CTA, so that long tables make few empty CTAs

__global__ void __launch_bounds__(kAccThreads)
accumulate_kernel(const float4 *__restrict__ scores, const float *__restrict__ logs, const float2 *__restrict__ tops,
                  int max_chunks, const int32_t *__restrict__ seq_lens, int max_blocks, const float *acc, float *acc_out,
                  int64_t acc_stride)
{
    const int g = blockIdx.y, b = blockIdx.z, t0 = blockIdx.x * kAccTokens;
    const int L = seq_lens[b];
    grid_dependency_wait();
    allow_dependent_launch();
    if (L < 1 || L > max_blocks * kPage || t0 >= L)
        return;
    const int h = b * kHq + g * kGroup;
    const float4 n = *reinterpret_cast<const float4 *>(logs + h);
    const float2 *top = tops + (size_t)h * max_chunks;
    const float4 m = make_float4(top[0].x, top[max_chunks].x, top[2 * (size_t)max_chunks].x, top[3 * (size_t)max_chunks].x);
    const size_t row = (size_t)b * kHkv + g;
    const float4 *x = scores + row * ((size_t)max_blocks * kPage);
    add_weights<kAccTokens / kAccThreads, kAccThreads>(x, m, n, acc + row * acc_stride, acc_out + row * acc_stride,
                                                       t0 + threadIdx.x, L);
}

struct ScoredWorkspace {
    size_t attention, scores, logs;
    size_t total() const { return attention + scores + logs; }
};

ScoredWorkspace scored_workspace(int B, int max_blocks, int max_chunks)
{
    ScoredWorkspace w;
    w.attention = align256(workspace_layout(B, max_chunks).total());
    w.scores = align256((size_t)B * kHq * max_blocks * kPage * sizeof(float));
    w.logs = align256((size_t)B * kHq * sizeof(float));
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
    ScoredPages<true> sel;
    sel.scores = reinterpret_cast<float *>(base + w.attention);
    sel.logs = reinterpret_cast<float *>(base + w.attention + w.scores);
    sel.max_chunks = (max_blocks + ppc - 1) / ppc;
    sel.tops = reinterpret_cast<float2 *>(base + workspace_layout(B, sel.max_chunks).ml_offset());
    sel.tokens = max_blocks * kPage;
    sel.acc = acc;
    sel.acc_out = acc_out;
    sel.acc_stride = acc_stride;
    StepArgs a = {};
    a.q = const_cast<uint16_t *>(q);
    a.bt = bt_dev;
    a.seq_lens = seq_lens_dev;
    a.max_pos = INT_MAX;
    a.scale_log2 = scale * kLog2e;
    a.out = out;
    a.err = dev_err_flag;
    cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
    // Largest units first where they are more than the GPU holds and can be long, and the library
    // chooses: 64 sequences up to 16384 tokens (FP8) 83 us instead of 99, 32 up to 16384 69 instead
    // of 75, 160 up to 2048 34 instead of 42; but 64 up to 4096 43 instead of 41, and with units of
    // 64 pages or less 256 up to 1024 39 instead of 36, 8 up to 8192 30 instead of 27.
    if (pages_per_chunk == 0 && B <= kMaxSortedBatch && ppc > 64 &&
        (int64_t)B * kHkv * ((max_blocks + ppc - 1) / ppc) > 152 * 6)
        options |= PKV_STEP_SORTED;
    // in the same launch: rows of 2048 tokens at most, or of 16384 where many units finish at
    // different times (1 sequence of 1024 tokens 5.5 us instead of 6.3, 64 up to 2048 14.8 instead of
    // 16.9; but 8 up to 4096 20 instead of 18, 8 up to 8192 34 instead of 27)
    if (sel.tokens <= (B * kHkv >= 3 * 152 ? 16384 : 2048))
        return launch_fused<false>(pool, a, sel, B, max_blocks, max_blocks, 0, ppc, workspace, s, options);
    const ScoredPages<false> apart = {sel.scores, sel.logs, sel.tops, sel.max_chunks, sel.tokens,
                                      acc,        acc_out,  acc_stride};
    if (const int st = launch_fused<false>(pool, a, apart, B, max_blocks, max_blocks, 0, ppc, workspace, s, options);
        st != PKV_OK)
        return st;
    const dim3 grid((sel.tokens + kAccTokens - 1) / kAccTokens, kHkv, B);
    return launch_kernel(accumulate_kernel, grid, dim3(kAccThreads), 0, s, !(options & PKV_STEP_NO_PDL),
                         reinterpret_cast<const float4 *>(sel.scores), static_cast<const float *>(sel.logs),
                         static_cast<const float2 *>(sel.tops), sel.max_chunks, seq_lens_dev, max_blocks, acc, acc_out, acc_stride);
}
