// pkv_step.cu -- the fused grid kernel of the decode path, one launch per layer.
//
// pkv_decode_step: RoPE + page-slot append of the new token, paged GQA decode
// attention over the sequence's pages, and the log-sum-exp merge of the chunk
// partials, in one launch.  It computes exactly what pkv_append_rope (positions =
// seq_lens - 1, q rotated in place) followed by pkv_decode_attention computes -- the
// samir-vllm README summary ("从零用 C++ 和 CUDA 实现 Llama 3.2 1B 推理引擎", section
// "目前已完成的功能") describes both steps: decode appends one token at its absolute
// RoPE position, then each query head streams its sequence's pages with an FP32
// online softmax -- with the same arithmetic, so the results are bit-identical to
// the two separate calls.  pkv_decode_attention runs the same kernel without the
// append (APPEND = false): the query rows are read as given and no page is written.
//
// Work unit = (sequence b, KV head g, chunk c of pages_per_chunk pages); one CTA per
// unit (grid = KV heads x B x chunks), optionally dispatched largest unit first.
// Per unit:
//  * the 4 query rows of group g are rotated to position L-1 by the unit itself;
//    the rotated rows are written back once, by the unit that finishes (b, g) last;
//  * the sequence's last chunk computes the new token's rotated key and its value,
//    stores them into their page slot in HBM and patches them into the
//    shared-memory copy of the last page, so no unit waits for an append kernel;
//  * chunk partials are merged in-kernel: each unit publishes its partial and
//    takes a ticket from a per-(b, g) counter (one release-acquire atomicAdd, no
//    waiting); the unit drawing the last ticket merges all chunks in chunk order
//    (deterministic) and resets the counter to zero for the next launch.
// Programmatic dependent launch: before griddepcontrol.wait a CTA reads only this
// step's lengths and block tables and starts the TMA copies of those of its pages
// that hold only positions below L - 2 (no kernel of this step or the previous one
// writes them: the previous step's append of this layer wrote position L - 2, this
// step's writes L - 1, and layers never share pages); the pages holding L - 2 or
// L - 1 are copied after the wait, q, k_new, v_new are read after it, and every
// output is written after it.  A CTA lets the next launch begin only after its own
// wait, so at most one earlier kernel can still be running while it copies early.
#include "pkv_step.cuh"

namespace pkv {

int launch_attention_fused(const pkv_pool *pool, const uint16_t *q, const int32_t *bt, int max_blocks,
                           const int32_t *seq_lens, int B, float scale, int pages_per_chunk, void *workspace,
                           uint16_t *out, int32_t *err, cudaStream_t s, int options)
{
    StepArgs a = {};
    a.k_new = nullptr;
    a.v_new = nullptr;
    a.q = const_cast<uint16_t *>(q);  // read only: no append writes the rows back
    a.bt = bt;
    a.seq_lens = seq_lens;
    a.rope = nullptr;
    a.max_pos = INT_MAX;
    a.scale_log2 = scale * kLog2e;
    a.out = out;
    a.err = err;
    return launch_fused<false>(pool, a, AllPages{}, B, max_blocks, max_blocks, 0, pages_per_chunk, workspace, s, options);
}

}  // namespace pkv

extern "C" size_t pkv_decode_step_workspace_bytes(int B, int max_blocks, int pages_per_chunk)
{
    return pkv_decode_workspace_bytes(B, max_blocks, pages_per_chunk);
}

extern "C" int pkv_decode_step(const pkv_pool *pool, const uint16_t *k_new, const uint16_t *v_new, uint16_t *q,
                               const int32_t *bt_dev, int max_blocks, const int32_t *seq_lens_dev, int B,
                               const float *rope_table, int max_pos, float scale, int pages_per_chunk,
                               void *workspace, size_t workspace_bytes, uint16_t *out, int32_t *dev_err_flag,
                               void *cuda_stream, int options)
{
    using namespace pkv;
    if (!pool || !k_new || !v_new || !q || !bt_dev || !seq_lens_dev || !rope_table || !out || !workspace)
        return PKV_ERR_INVALID_ARG;
    if (B < 1 || B > 65535 || max_blocks < 1 || max_blocks > (1 << 20) || max_pos < 1)
        return PKV_ERR_INVALID_ARG;
    if (pages_per_chunk < 1 || pages_per_chunk > kMaxPagesPerChunk || !(scale > 0.f) || !(scale < INFINITY))
        return PKV_ERR_INVALID_ARG;
    const uintptr_t align = reinterpret_cast<uintptr_t>(k_new) | reinterpret_cast<uintptr_t>(v_new) |
                            reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out) |
                            reinterpret_cast<uintptr_t>(rope_table) | reinterpret_cast<uintptr_t>(workspace);
    if (align & 15u)
        return PKV_ERR_INVALID_ARG;
    if (workspace_bytes < pkv_decode_step_workspace_bytes(B, max_blocks, pages_per_chunk))
        return PKV_ERR_WORKSPACE_TOO_SMALL;
    StepArgs a = {};
    a.k_new = k_new;
    a.v_new = v_new;
    a.q = q;
    a.bt = bt_dev;
    a.seq_lens = seq_lens_dev;
    a.rope = reinterpret_cast<const float4 *>(rope_table);
    a.max_pos = max_pos;
    a.scale_log2 = scale * kLog2e;
    a.out = out;
    a.err = dev_err_flag;
    return launch_fused<true>(pool, a, AllPages{}, B, max_blocks, max_blocks, 0, pages_per_chunk, workspace,
                              static_cast<cudaStream_t>(cuda_stream), options);
}

#ifdef PKV_TIMELINE
extern "C" int pkv_timeline_read(uint64_t *stamps, int32_t *meta, int n)
{
    using namespace pkv;
    if (!stamps || !meta || n < 1)
        return PKV_ERR_INVALID_ARG;
    if (n > kTimelineMax)
        n = kTimelineMax;
    if (cudaMemcpyFromSymbol(stamps, g_timeline_stamps, (size_t)n * 5 * sizeof(uint64_t)) != cudaSuccess ||
        cudaMemcpyFromSymbol(meta, g_timeline_meta, (size_t)n * 4 * sizeof(int32_t)) != cudaSuccess)
        return PKV_ERR_CUDA;
    return n;
}
#endif
