// pkv_shared.cu -- decode attention for groups of sequences that share a prefix.
#include "pkv_step.cuh"

namespace pkv {
namespace {

// Every page of the sequence, the prefix's through the table row of the group's first
// sequence.
struct SharedPages {
    static constexpr bool kIdentity = false, kSortable = false, kLateWait = false;
    const int32_t *starts, *prefix_pages;
    int groups, max_prefix;

    struct List : WholeSequence {
        int lead, prefix;  // the group's first sequence, its prefix pages (-1: no such group)
        __device__ __forceinline__ int row(int b, int j) const { return j < prefix ? lead : b; }
        __device__ __forceinline__ bool ok() const { return prefix >= 0 && (int64_t)prefix * kPage <= L; }
    };

    __device__ __forceinline__ List list(int b, int L) const
    {
        List x;
        x.L = L;
        x.lead = 0;
        x.prefix = -1;
        for (int i = threadIdx.x & 31; i < groups; i += 32) {
            const int s0 = starts[i], s1 = starts[i + 1], p = prefix_pages[i];
            if (s0 >= 0 && s0 <= b && b < s1 && p >= 0 && p <= max_prefix) {
                x.lead = s0;
                x.prefix = p;
            }
        }
        x.prefix = __reduce_max_sync(kFull, x.prefix);
        x.lead = __reduce_max_sync(kFull, x.lead);
        return x;
    }
    __device__ __forceinline__ EmitNothing emit(int, int) const { return {}; }
    __device__ __forceinline__ void skipped(int, int, int, int) const {}
    __device__ __forceinline__ void norm(int, int, float, float) const {}
};

bool shared_args_ok(int B, int max_blocks, int groups, int max_prefix_pages, int pages_per_chunk,
                    int prefix_pages_per_chunk)
{
    return B >= 1 && B <= 65535 && max_blocks >= 1 && max_blocks <= (1 << 20) && groups >= 1 && groups <= B &&
           max_prefix_pages >= 0 && max_prefix_pages <= max_blocks && pages_per_chunk >= 0 &&
           pages_per_chunk <= kMaxPagesPerChunk && prefix_pages_per_chunk >= 0;
}

}  // namespace
}  // namespace pkv

extern "C" size_t pkv_decode_shared_workspace_bytes(int B, int max_blocks, int groups, int max_prefix_pages,
                                                    int pages_per_chunk, int prefix_pages_per_chunk)
{
    using namespace pkv;
    if (!shared_args_ok(B, max_blocks, groups, max_prefix_pages, pages_per_chunk, prefix_pages_per_chunk))
        return 0;
    const int ppc = pages_per_chunk ? pages_per_chunk : default_chunk(B, max_blocks);
    return workspace_layout(B, (max_blocks + ppc - 1) / ppc).total();
}

extern "C" int pkv_decode_shared(const pkv_pool *pool, const uint16_t *q, const int32_t *bt_dev, int max_blocks,
                                 const int32_t *seq_lens_dev, int B, const int32_t *group_starts_dev,
                                 const int32_t *prefix_pages_dev, int groups, int max_prefix_pages, float scale,
                                 int pages_per_chunk, int prefix_pages_per_chunk, void *workspace,
                                 size_t workspace_bytes, uint16_t *out, int32_t *dev_err_flag, void *cuda_stream,
                                 int options)
{
    using namespace pkv;
    if (!pool || !q || !bt_dev || !seq_lens_dev || !group_starts_dev || !prefix_pages_dev || !workspace || !out ||
        !shared_args_ok(B, max_blocks, groups, max_prefix_pages, pages_per_chunk, prefix_pages_per_chunk))
        return PKV_ERR_INVALID_ARG;
    if (!(scale > 0.f) || !(scale < INFINITY))
        return PKV_ERR_INVALID_ARG;
    const uintptr_t align =
        reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out) | reinterpret_cast<uintptr_t>(workspace);
    if (align & 15u)
        return PKV_ERR_INVALID_ARG;
    if (workspace_bytes < pkv_decode_shared_workspace_bytes(B, max_blocks, groups, max_prefix_pages, pages_per_chunk,
                                                            prefix_pages_per_chunk))
        return PKV_ERR_WORKSPACE_TOO_SMALL;
    const int ppc = pages_per_chunk ? pages_per_chunk : default_chunk(B, max_blocks);
    const SharedPages sel = {group_starts_dev, prefix_pages_dev, groups, max_prefix_pages};
    StepArgs a = {};
    a.q = const_cast<uint16_t *>(q);
    a.bt = bt_dev;
    a.seq_lens = seq_lens_dev;
    a.max_pos = INT_MAX;
    a.scale_log2 = scale * kLog2e;
    a.out = out;
    a.err = dev_err_flag;
    return launch_fused<false>(pool, a, sel, B, max_blocks, max_blocks, 0, ppc, workspace,
                               static_cast<cudaStream_t>(cuda_stream), options);
}
