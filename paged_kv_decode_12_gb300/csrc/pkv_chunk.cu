// pkv_chunk.cu -- causal attention of a step's new tokens over their sequences' pages.
#include <cmath>

#include "pkv_device.cuh"
#include "pkv_fp8.cuh"

namespace pkv {
namespace {

using namespace dev;
using namespace fp8;

constexpr int kMaxRows = 4096;  // sequences of a call

struct ChunkArgs {
    int num_pages;
    const uint16_t *q;
    const int32_t *bt;
    int max_blocks;
    const int32_t *lens, *starts;
    int B, T;
    float scale_log2;
    int window, sinks;
    uint16_t *out;
    int32_t *err;
};

template <bool FP8>
__global__ void __launch_bounds__(kThreads) chunk_token_kernel(const __grid_constant__ CUtensorMap tmap, ChunkArgs a)
{
    constexpr int kStages = 2, kSize = FP8 ? kFp8Unit : kStageBytes;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *stages = smem_raw + (-smem_addr(smem_raw) & 1023u);
    __shared__ uint64_t bars[kWarps][kStages];
    __shared__ float scratch[kWarps][kScratchFloats];
    const int t = blockIdx.x, g = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_dependency_wait();
    allow_dependent_launch();
    if (t == 0 && g == 0) {
        bool bad = threadIdx.x == 0 && a.starts[0] != 0;
        for (int i = threadIdx.x; i < a.B; i += kThreads)
            bad |= a.starts[i] < 0 || a.starts[i + 1] < a.starts[i] || a.starts[i + 1] > a.T;
        if (__syncthreads_or(bad) && threadIdx.x == 0 && a.err)
            atomicOr(a.err, PKV_DEVERR_LENGTH);
    }
    int lo = 0, hi = a.B;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.starts[mid] <= t)
            lo = mid;
        else
            hi = mid;
    }
    const int b = lo, t0 = a.starts[b], t1 = a.starts[b + 1], L = a.lens[b];
    if (t < t0 || t >= t1)
        return;
    uint32_t *out = reinterpret_cast<uint32_t *>(a.out + ((size_t)t * kHq + g * kGroup + warp) * kD) + lane;
    if (L < t1 - t0 || L > a.max_blocks * kPage) {
        *out = 0;
        if (threadIdx.x == 0 && a.err)
            atomicOr(a.err, PKV_DEVERR_LENGTH);
        return;
    }
    const int p = L - (t1 - t0) + (t - t0);
    const int first = a.window ? max(0, p + 1 - a.window) : 0;
    const int sink_pages = min((a.sinks + kPage - 1) / kPage, first / kPage);
    const int n = sink_pages + p / kPage - first / kPage + 1;
    const auto logical = [&](int i) { return i < sink_pages ? i : i - sink_pages + first / kPage; };
    const int nmine = warp < n ? (n - warp + kWarps - 1) / kWarps : 0;
    bool bad = false;
    for (int k = lane; k < nmine; k += 32) {
        const int id = a.bt[(size_t)b * a.max_blocks + logical(warp + k * kWarps)];
        bad |= id < 0 || id >= a.num_pages;
    }
    if (__syncthreads_or(bad)) {
        *out = 0;
        if (threadIdx.x == 0 && a.err)
            atomicOr(a.err, PKV_DEVERR_PAGE_RANGE);
        return;
    }
    init_warp_barriers<kStages>(bars[warp], lane);
    const uint64_t policy = l2_evict_first_policy();
    uint8_t *mine = stages + warp * kStages * kSize;
    const auto load = [&](int k) {
        if (lane == 0) {
            const int id = a.bt[(size_t)b * a.max_blocks + logical(warp + k * kWarps)], s = k % kStages;
            fence_proxy_async_smem();
            if constexpr (FP8) {
                fp8_issue(&tmap, mine + s * kSize, &bars[warp][s], g, id, policy);
            } else {
                mbar_arrive_expect_tx(&bars[warp][s], kSize);
                tma_load_page_head(mine + s * kSize, &tmap, &bars[warp][s], g, id, policy);
            }
        }
        __syncwarp();
    };
    std::conditional_t<FP8, Fp8MmaWarp, MmaWarp> w;
    const uint16_t *q = a.q + ((size_t)t * kHq + g * kGroup) * kD;
    if constexpr (FP8)
        w.init(q, a.scale_log2, lane);
    else
        w.init(q, a.scale_log2, lane, scratch[warp]);
    for (int k = 0; k < min(kStages, nmine); ++k)
        load(k);
    int k = 0;
    for (; k < nmine; ++k) {
        const int s = k % kStages;
        if (!mbar_wait_warp(&bars[warp][s], (uint32_t)((k / kStages) & 1)))
            break;
        const int at = logical(warp + k * kWarps) * kPage;
        uint32_t bits = 0;
        for (int i = 0; i < kPage; ++i)
            if (at + i <= p && (at + i >= first || at + i < a.sinks))
                bits |= 1u << i;
        w.page(mine + s * kSize, TokenSet{bits});
        __syncwarp();
        if (k + kStages < nmine)
            load(k + kStages);
    }
    if (k < nmine) {
        for (int i = k; i < min(nmine, k + kStages); ++i)
            (void)mbar_wait_warp(&bars[warp][i % kStages], (uint32_t)((i / kStages) & 1));
        if (lane == 0 && a.err)
            atomicOr(a.err, PKV_DEVERR_TIMEOUT);
    }
    __syncthreads();
    float *state = reinterpret_cast<float *>(stages);
    w.store_state(state + warp * kStateFloats);
    __syncthreads();
    float M, lsum, o0, o1;
    combine_warps(state, warp, lane, M, lsum, o0, o1);
    *out = finish_pair(o0, o1, lsum);
}

template <bool FP8>
int launch_chunk(const pkv_pool *pool, const ChunkArgs &a, cudaStream_t s, bool pdl)
{
    const CUtensorMap *tmap = pool_tensor_map(pool);
    if (!tmap)
        return PKV_ERR_CUDA;
    constexpr int smem = 1024 + kWarps * 2 * (FP8 ? kFp8Unit : kStageBytes);
    return launch_kernel(chunk_token_kernel<FP8>, dim3(a.T, kHkv), dim3(kThreads), smem, s, pdl, *tmap, a);
}

bool chunk_args_ok(int B, int T) { return B >= 1 && B <= kMaxRows && T >= 1 && T <= INT32_MAX / 16; }

}  // namespace
}  // namespace pkv

extern "C" size_t pkv_chunk_attention_workspace_bytes(int B, int T) { return pkv::chunk_args_ok(B, T) ? 16 : 0; }

extern "C" int pkv_chunk_attention(const pkv_pool *pool, const uint16_t *q, const int32_t *bt_dev, int max_blocks,
                                   const int32_t *seq_lens_dev, const int32_t *starts_dev, int B, int T, float scale,
                                   int window, int sinks, void *workspace, size_t workspace_bytes, uint16_t *out,
                                   int32_t *dev_err_flag, void *cuda_stream, int options)
{
    using namespace pkv;
    if (!pool || !q || !bt_dev || !seq_lens_dev || !starts_dev || !workspace || !out || !chunk_args_ok(B, T))
        return PKV_ERR_INVALID_ARG;
    if (max_blocks < 1 || max_blocks > (1 << 20) || window < 0 || sinks < 0 || (sinks && !window))
        return PKV_ERR_INVALID_ARG;
    if (!(scale > 0.f) || !(scale < INFINITY) || (options & ~(PKV_STEP_NO_PDL | PKV_STEP_TEST_EXPIRE_WAIT)))
        return PKV_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out) | reinterpret_cast<uintptr_t>(workspace)) & 15u)
        return PKV_ERR_INVALID_ARG;
    if (workspace_bytes < pkv_chunk_attention_workspace_bytes(B, T))
        return PKV_ERR_WORKSPACE_TOO_SMALL;
    ChunkArgs a;
    a.num_pages = pool->num_pages;
    a.q = q;
    a.bt = bt_dev;
    a.max_blocks = max_blocks;
    a.lens = seq_lens_dev;
    a.starts = starts_dev;
    a.B = B;
    a.T = T;
    a.scale_log2 = scale * kLog2e;
    const int64_t most = (int64_t)max_blocks * kPage;  // a window of the table's width is none
    a.window = window < most ? window : 0;
    a.sinks = (int)std::min<int64_t>(sinks, most);
    a.out = out;
    a.err = dev_err_flag;
    cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
    const bool pdl = !(options & PKV_STEP_NO_PDL);
    return pool->kv_format == PKV_KV_FP8 ? launch_chunk<true>(pool, a, s, pdl) : launch_chunk<false>(pool, a, s, pdl);
}
