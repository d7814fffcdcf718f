// pkv_window.cu -- decode attention over a sliding window and the first tokens, alone
// (pkv_decode_window) and fused with the append (pkv_decode_step_window).
//
//     out[b][h] = sum_t softmax_t(scale * q[b][h] . K_t) V_t   over the t < L with
//                 t < sinks or t >= L - window,                 L = seq_lens[b].
//
// It is the grid kernel of pkv_step.cuh over a list of pages: the pages of the first
// `sinks` tokens, then the pages of the last `window`, cut into chunks like a whole
// sequence.  Pages in between are neither read nor looked up, so their table entries
// may name pages that have been given back.  Every listed page holds a token that is
// attended to, so no page leaves a row of the softmax empty; at most three of a list's
// pages (the last of the first tokens', the window's first, the sequence's last) are
// masked, by a set of 16 token bits.
#include "pkv_step.cuh"

namespace pkv {
namespace {

struct WindowPages {
    static constexpr bool kIdentity = false, kSortable = true, kLateWait = false, kPublish = false, kLoops = false,
                          kFine = false;
    int window, sinks;

    struct List {
        static constexpr bool kWhole = true;
        int L, cut, head;  // tokens below head and from cut on are attended to (head <= cut)
        int nhead, gap;    // pages of the first tokens; pages left out behind them
        __device__ __forceinline__ bool ok() const { return true; }
        __device__ __forceinline__ int count() const { return (L + kPage - 1) / kPage - gap; }
        __device__ __forceinline__ int logical(int i) const { return i < nhead ? i : i + gap; }
        __device__ __forceinline__ int before(int j) const { return j <= nhead ? j : max(nhead, j - gap); }
        __device__ __forceinline__ bool whole(int j) const
        {
            const int t0 = j * kPage;
            return t0 + kPage <= head || (t0 >= cut && t0 + kPage <= L);
        }
        __device__ __forceinline__ TokenSet tokens(int j) const
        {
            const int t0 = j * kPage;
            return {below(head - t0) | (below(L - t0) & ~below(cut - t0))};
        }
        // the tokens of a page below n (any n)
        __device__ __forceinline__ static uint32_t below(int n) { return (1u << min(max(n, 0), kPage)) - 1; }
        __device__ __forceinline__ int first_slot() const { return 0; }
    };

    __device__ __forceinline__ List list(int, int L) const
    {
        List x;
        x.L = L;
        x.cut = max(max(L, 0) - window, 0);
        x.head = min(sinks, x.cut);
        x.nhead = (x.head + kPage - 1) / kPage;
        x.gap = max(x.cut / kPage - x.nhead, 0);
        return x;
    }
    __device__ __forceinline__ EmitNothing emit(int, int) const { return {}; }
    __device__ __forceinline__ void skipped(int, int, int, int) const {}
    __device__ __forceinline__ void finished(int, int, int, float, float, float *) const {}
};

// The most pages a list can have: n tokens in a row touch at most (n + 14) / 16 + 1 pages.
int window_list_pages(int max_blocks, int window, int sinks)
{
    const int64_t n = ((int64_t)sinks + kPage - 1) / kPage + ((int64_t)window + kPage - 2) / kPage + 1;
    return (int)(n < max_blocks ? n : max_blocks);
}

bool window_args_ok(int B, int max_blocks, int window, int sinks, int pages_per_chunk)
{
    return B >= 1 && B <= 65535 && max_blocks >= 1 && max_blocks <= (1 << 20) && window >= 1 && sinks >= 0 &&
           pages_per_chunk >= 0 && pages_per_chunk <= kMaxPagesPerChunk;
}

}  // namespace
}  // namespace pkv

extern "C" size_t pkv_decode_window_workspace_bytes(int B, int max_blocks, int window, int sinks, int pages_per_chunk)
{
    using namespace pkv;
    if (!window_args_ok(B, max_blocks, window, sinks, pages_per_chunk))
        return 0;
    const int list = window_list_pages(max_blocks, window, sinks);
    const int ppc = pages_per_chunk ? pages_per_chunk : default_chunk(B, list, 1);
    return workspace_layout(B, (list + ppc - 1) / ppc).total();
}

namespace {

// Both entry points; k_new, v_new and rope_table are null without the append.
int decode_window(const pkv_pool *pool, const uint16_t *k_new, const uint16_t *v_new, uint16_t *q,
                  const int32_t *bt_dev, int max_blocks, const int32_t *seq_lens_dev, int B, const float *rope_table,
                  int max_pos, float scale, int window, int sinks, int pages_per_chunk, void *workspace,
                  size_t workspace_bytes, uint16_t *out, int32_t *dev_err_flag, void *cuda_stream, int options)
{
    using namespace pkv;
    const bool append = k_new != nullptr;
    if (!pool || !q || !bt_dev || !seq_lens_dev || !out || !window_args_ok(B, max_blocks, window, sinks, pages_per_chunk))
        return PKV_ERR_INVALID_ARG;
    if (!(scale > 0.f) || !(scale < INFINITY))
        return PKV_ERR_INVALID_ARG;
    const uintptr_t align = reinterpret_cast<uintptr_t>(k_new) | reinterpret_cast<uintptr_t>(v_new) |
                            reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out) |
                            reinterpret_cast<uintptr_t>(rope_table) | reinterpret_cast<uintptr_t>(workspace);
    if (align & 15u)
        return PKV_ERR_INVALID_ARG;
    const int list = window_list_pages(max_blocks, window, sinks);
    const int ppc = pages_per_chunk ? pages_per_chunk : default_chunk(B, list, 1);
    if (list > ppc || append) {
        if (!workspace)
            return PKV_ERR_INVALID_ARG;
        if (workspace_bytes < pkv_decode_window_workspace_bytes(B, max_blocks, window, sinks, pages_per_chunk))
            return PKV_ERR_WORKSPACE_TOO_SMALL;
    }
    StepArgs a = {};
    a.k_new = k_new;
    a.v_new = v_new;
    a.q = q;
    a.bt = bt_dev;
    a.seq_lens = seq_lens_dev;
    a.rope = reinterpret_cast<const float4 *>(rope_table);
    a.max_pos = append ? max_pos : INT_MAX;
    a.scale_log2 = scale * kLog2e;
    a.out = out;
    a.err = dev_err_flag;
    const WindowPages sel = {window, sinks};
    cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
    return append ? launch_fused<true>(pool, a, sel, B, max_blocks, list, 0, ppc, workspace, s, options)
                  : launch_fused<false>(pool, a, sel, B, max_blocks, list, 0, ppc, workspace, s, options);
}

}  // namespace

extern "C" int pkv_decode_window(const pkv_pool *pool, const uint16_t *q, const int32_t *bt_dev, int max_blocks,
                                 const int32_t *seq_lens_dev, int B, float scale, int window, int sinks,
                                 int pages_per_chunk, void *workspace, size_t workspace_bytes, uint16_t *out,
                                 int32_t *dev_err_flag, void *cuda_stream, int options)
{
    return decode_window(pool, nullptr, nullptr, const_cast<uint16_t *>(q), bt_dev, max_blocks, seq_lens_dev, B,
                         nullptr, 0, scale, window, sinks, pages_per_chunk, workspace, workspace_bytes, out,
                         dev_err_flag, cuda_stream, options);
}

extern "C" int pkv_decode_step_window(const pkv_pool *pool, const uint16_t *k_new, const uint16_t *v_new, uint16_t *q,
                                      const int32_t *bt_dev, int max_blocks, const int32_t *seq_lens_dev, int B,
                                      const float *rope_table, int max_pos, float scale, int window, int sinks,
                                      int pages_per_chunk, void *workspace, size_t workspace_bytes, uint16_t *out,
                                      int32_t *dev_err_flag, void *cuda_stream, int options)
{
    if (!k_new || !v_new || !rope_table || max_pos < 1)
        return PKV_ERR_INVALID_ARG;
    return decode_window(pool, k_new, v_new, q, bt_dev, max_blocks, seq_lens_dev, B, rope_table, max_pos, scale, window,
                         sinks, pages_per_chunk, workspace, workspace_bytes, out, dev_err_flag, cuda_stream, options);
}
